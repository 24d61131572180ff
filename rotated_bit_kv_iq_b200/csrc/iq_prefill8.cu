// Causal attention of a chunk of query tokens over the 8-bit cache.
//
// One CTA per (sequence, block of 8 / G tokens, kv head): its eight query rows share every tile, and its
// warps take the tiles in turn.
#include <algorithm>

#include "iq_attend8.cuh"
#include "iq_prefill8_tc.cuh"

namespace iq {

constexpr int P8_WARPS = 8;

struct Prefill8Args {
  View8 v;
  const void* q;
  int dtype, batch, n_tok, n_q_heads, g_real, n_qblk, max_ctx;
  const int32_t* start;
  const int32_t* n_valid;
  float scale;
  void* out;
};

template <int CODE>
__global__ void __launch_bounds__(P8_WARPS * 32) prefill8_kernel(Prefill8Args a) {
  extern __shared__ __align__(128) uint8_t smem[];  // [warp] tile, then [warp][8][128] sums
  __shared__ float sml[P8_WARPS][A8_ROWS][4];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const int Hkv = a.v.n_kv_heads, G = a.g_real, TQ = A8_ROWS / G;
  const int kvh = blockIdx.x % Hkv, qb = (blockIdx.x / Hkv) % a.n_qblk, b = blockIdx.x / Hkv / a.n_qblk;
  uint32_t err = 0;
  int cnt = a.n_valid ? a.n_valid[b] : a.n_tok;
  if (cnt < 0 || cnt > a.n_tok) {
    err = IQ_DEVERR_CTX;
    cnt = cnt < 0 ? 0 : a.n_tok;
  }
  int start = a.start[b];
  if (start < 0 || start > a.max_ctx - cnt) {
    err = IQ_DEVERR_CTX;
    start = start < 0 ? 0 : a.max_ctx - cnt;
  }
  if (err && a.v.status && threadIdx.x == 0) atomicOr(a.v.status, err);
  const int tok0 = qb * TQ, n_live = min(TQ, cnt - tok0);
  if (n_live <= 0) return;
  const int ctx = start + tok0 + n_live, tok = g / G, h = g % G;
  const bool live = g < TQ * G && tok < n_live;
  uint32_t qa[8][4];
  const float qs = load_q8(a.q, a.dtype, ((size_t)b * a.n_tok + tok0 + tok) * a.n_q_heads + (size_t)kvh * G + h, live, a.scale, qa);
  const int seen = live ? start + tok0 + tok + 1 : 0;  // tokens that row g sees
  Row8 r;
  row8_init(r);
  uint8_t* const t = smem + warp * TILE8_BYTES;
  for (int tile = warp; tile * TILE_TOKENS < ctx; tile += P8_WARPS) {
    uint32_t e = 0;
    const int page = find_page8(a.v, b, (long long)tile * TILE_TOKENS, &e);
    if (page < 0) {
      if (a.v.status && lane == 0) atomicOr(a.v.status, e);
      continue;
    }
    const uint8_t* src = tile_record8(a.v, page, kvh, (int)(((long long)tile * TILE_TOKENS) % a.v.page_size));
    __syncwarp();
    for (int i = lane; i < TILE8_BYTES / 16; i += 32)
      reinterpret_cast<uint4*>(t)[i] = __ldcg(reinterpret_cast<const uint4*>(src) + i);
    __syncwarp();
    const int n_valid = min(TILE_TOKENS, ctx - tile * TILE_TOKENS);
    if (n_valid < TILE_TOKENS) clear_v_rows8(t, n_valid);
    tile8<CODE, false>(t, min(TILE_TOKENS, seen - tile * TILE_TOKENS), qa, qs, r);
  }
  float* const so = reinterpret_cast<float*>(smem + P8_WARPS * TILE8_BYTES);
  row8_store<false>(r, sml[warp], so + warp * A8_ROWS * D);
  __syncthreads();
  for (int x = warp; x < TQ * G; x += P8_WARPS) {
    if (x / G >= n_live) continue;
    float M = -CUDART_INF_F, MO = -CUDART_INF_F;
    for (int w = 0; w < P8_WARPS; ++w) {
      M = fmaxf(M, sml[w][x][0]);
      MO = fmaxf(MO, sml[w][x][1]);
    }
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < P8_WARPS; ++w) {
      L += sml[w][x][2] * (sml[w][x][0] == -CUDART_INF_F ? 0.f : fast_exp2(sml[w][x][0] - M));
      const float f = sml[w][x][1] == -CUDART_INF_F ? 0.f : fast_exp2(sml[w][x][1] - MO);
      const float4 y = *reinterpret_cast<const float4*>(so + (w * A8_ROWS + x) * D + 4 * lane);
      o.x = fmaf(y.x, f, o.x); o.y = fmaf(y.y, f, o.y); o.z = fmaf(y.z, f, o.z); o.w = fmaf(y.w, f, o.w);
    }
    const float f = L > 0.f ? fast_exp2(MO - M) / L : (L == L ? 0.f : L);
    store4(a.out, a.dtype, (((size_t)b * a.n_tok + tok0 + x / G) * a.n_q_heads + (size_t)kvh * G + x % G) * D + 4 * lane,
           make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
  }
}

size_t prefill8_workspace_bytes(int batch, int n_tok, int n_q_heads, int n_kv_heads, int max_ctx) {
  return pt_plan(batch, n_tok, std::min(8, n_q_heads / n_kv_heads), n_kv_heads, max_ctx).bytes;
}

int launch_prefill8(const View8& v, const void* q, int dtype, int batch, int n_tok, int n_q_heads, const int32_t* start,
                    const int32_t* n_valid, int max_ctx, float scale, void* out, void* workspace, void* stream) {
  if (batch == 0 || n_tok == 0) return 0;
  if (dtype != IQ_F32)
    return launch_prefill8_tc(v, q, dtype, batch, n_tok, n_q_heads, start, n_valid, max_ctx, scale, out, workspace, stream);
  Prefill8Args a;
  a.v = v;
  a.q = q;
  a.dtype = dtype;
  a.batch = batch;
  a.n_tok = n_tok;
  a.n_q_heads = n_q_heads;
  a.g_real = n_q_heads / v.n_kv_heads;
  const int tq = A8_ROWS / a.g_real;
  a.n_qblk = (n_tok + tq - 1) / tq;
  a.max_ctx = max_ctx;
  a.start = start;
  a.n_valid = n_valid;
  a.scale = scale;
  a.out = out;
  const size_t smem = P8_WARPS * (TILE8_BYTES + A8_ROWS * D * 4);
  auto fn = v.code == IQ_E4M3 ? prefill8_kernel<IQ_E4M3> : prefill8_kernel<IQ_S8>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return (int)e;
  return (int)launch_pdl(fn, dim3((unsigned)(batch * a.n_qblk * v.n_kv_heads)), dim3(P8_WARPS * 32), smem,
                         (cudaStream_t)stream, a);
}

}  // namespace iq
