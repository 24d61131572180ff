// Decode attention over the 8-bit cache: one query token per sequence.
//
// The work is the list of 32-token tiles of all (sequence, kv head) groups; CTA c of N takes tiles
// [c T / N, (c + 1) T / N), whatever the mix of lengths.  Its warps take the tiles of each group's segment in turn, each
// through a ring of its own of two bulk-copied tile records: twelve warps, three a scheduler, at 168 registers.  On the
// 16-sequence layer: PLACEHOLDER_SERVE us, 105 with eight warps (197 registers); 121 with sixteen (128 registers, which
// do not hold a tile's work) on one ring of 26 records.  A segment that is a whole group is finished at once; the others
// leave a partial (m, mo, l, O), and the last CTA of a group to arrive merges the group's partials in a fixed order, so
// that results do not depend on who is last.  Bound by memory: 257 B for each (token, kv head).
#include <algorithm>

#include "iq_attend8.cuh"

namespace iq {

constexpr int D8_WARPS = 12;
constexpr int D8_THREADS = 32 * D8_WARPS;
constexpr int D8_NB = 2;                                       // tile records in a warp's ring
constexpr int D8_SMEM = D8_WARPS * D8_NB * TILE8_BYTES;        // (at a segment's end: the warps' value sums)
static_assert(D8_WARPS * A8_ROWS * D * 4 <= D8_SMEM, "value sums in the rings' place");

struct Decode8Args {
  View8 v;
  const void* q;
  int dtype, batch, n_q_heads, g_real, max_ctx;
  const int32_t* ctx_len;
  float scale;
  void* out;
  int32_t* counters;  // [batch * Hkv], zero between calls
  float4* part_ml;    // [2 N][8]: m, mo, l
  float* part_o;      // [2 N][8][128]
};

__device__ __forceinline__ int clamp_ctx8(const Decode8Args& a, int b) {
  const int c = a.ctx_len[b];
  return c < 0 ? 0 : (c > a.max_ctx ? a.max_ctx : c);
}

// Final value of one row of the group: lane holds sums of coordinates 4 lane ..
__device__ __forceinline__ void finish_row8(const Decode8Args& a, size_t row, float M, float MO, float L, float4 o) {
  const float f = L > 0.f ? fast_exp2(MO - M) / L : (L == L ? 0.f : L);
  store4(a.out, a.dtype, row * D + 4 * (threadIdx.x & 31), make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
}

template <int CODE, bool FEW>
__global__ void __launch_bounds__(D8_THREADS, 1) decode8_kernel(Decode8Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[D8_WARPS][D8_NB];
  __shared__ float sml[D8_WARPS][A8_ROWS][4];
  __shared__ long long s_scan[D8_WARPS];
  __shared__ int s_start[2];  // the CTA's first sequence, and the tiles before it within all kv heads
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;
  const int Hkv = a.v.n_kv_heads, G = a.g_real, c = blockIdx.x;
  float* const so = reinterpret_cast<float*>(smem);
  if (lane == 0) {
    for (int i = 0; i < D8_NB; ++i) mbar_init(&bars[warp][i], 1);
    mbar_fence_init();
  }
  __syncwarp();
  pdl_wait();

  // ---- plan: total tiles, this CTA's range, the sequence that it starts in
  const int per = (a.batch + D8_THREADS - 1) / D8_THREADS, b0 = tid * per;
  long long mine = 0;
  for (int b = b0; b < min(a.batch, b0 + per); ++b) mine += (clamp_ctx8(a, b) + TILE_TOKENS - 1) / TILE_TOKENS;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < D8_WARPS; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  before *= Hkv;
  total *= Hkv;
  // the CTAs that share the tiles: none without one, and no more than give every warp one
  const int N = (int)min((long long)gridDim.x, max(1ll, (total + D8_WARPS - 1) / D8_WARPS));
  const long long lo = c < N ? c * total / N : total, hi = c < N ? (c + 1) * total / N : total;
  long long acc = before;  // tiles of all groups before sequence b
  for (int b = b0; b < min(a.batch, b0 + per); ++b) {
    const long long nt = (long long)Hkv * ((clamp_ctx8(a, b) + TILE_TOKENS - 1) / TILE_TOKENS);
    if (lo < hi && acc <= lo && lo < acc + nt) {
      s_start[0] = b;
      s_start[1] = (int)(lo - acc);
    }
    acc += nt;
  }
  if (c == 0 && a.v.status)
    for (int b = tid; b < a.batch; b += D8_THREADS)
      if (clamp_ctx8(a, b) != a.ctx_len[b]) atomicOr(a.v.status, IQ_DEVERR_CTX);
  // sequences with nothing to see: zero rows
  for (int b = c; b < a.batch; b += gridDim.x)
    if (clamp_ctx8(a, b) == 0)
      for (int i = tid; i < a.n_q_heads * (D / 4); i += D8_THREADS)
        store4(a.out, a.dtype, (size_t)b * a.n_q_heads * D + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
  __syncthreads();
  if (lo >= hi) return;

  int b = s_start[0];
  int ctx = clamp_ctx8(a, b), nt = (ctx + TILE_TOKENS - 1) / TILE_TOKENS;
  int kvh = s_start[1] / nt, tile0 = s_start[1] % nt;
  long long pos = lo;
  uint32_t used = 0;  // of this warp's ring, so far
  bool ok = true;
  uint8_t* const ring = smem + warp * D8_NB * TILE8_BYTES;
  const int page_tiles = a.v.page_size / TILE_TOKENS;
  while (pos < hi) {
    // ---- one segment: tiles [tile0, tile1) of group (b, kvh)
    const int tile1 = (int)min((long long)nt, tile0 + (hi - pos));
    const int mine = ok && tile1 - tile0 > warp ? (tile1 - tile0 - warp + D8_WARPS - 1) / D8_WARPS : 0;  // this warp's
    auto issue = [&](int j) {  // the warp's j-th tile of the segment; whether it has a page
      const int tile = tile0 + warp + D8_WARPS * j, idx = tile / page_tiles;
      uint64_t* const bar = &bars[warp][(used + j) % D8_NB];
      int page = b;
      if (a.v.block_table) page = idx < a.v.max_pages ? a.v.block_table[(size_t)b * a.v.max_pages + idx] : -1;
      const bool there = page >= 0 && page < a.v.n_pages;
      if (lane == 0) {
        if (there) {
          mbar_arrive_expect_tx(bar, TILE8_BYTES);
          bulk_g2s(ring + (used + j) % D8_NB * TILE8_BYTES,
                   a.v.pool + (((size_t)page * Hkv + kvh) * page_tiles + tile % page_tiles) * (size_t)TILE8_BYTES, TILE8_BYTES, bar);
        } else {
          if (a.v.status) atomicOr(a.v.status, IQ_DEVERR_PAGE);
          mbar_arrive(bar);
        }
      }
      return (uint32_t)there;
    };
    uint32_t have = 0;  // bit j mod NB: the warp's tile j has a page
    for (int j = 0; j < D8_NB && j < mine; ++j) have |= issue(j) << (j % D8_NB);
    uint32_t qa[8][4];
    const int head = FEW ? g & 3 : g;
    const float qs = load_q8(a.q, a.dtype, (size_t)b * a.n_q_heads + (size_t)kvh * G + head, head < G, a.scale, qa);
    Row8 r;
    row8_init(r);
    int j = 0;
    for (; j < mine; ++j) {
      const uint32_t n = used + j;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[warp][n % D8_NB], (n / D8_NB) & 1, a.v.status));
      if (!ok) break;
      uint8_t* const t = ring + n % D8_NB * TILE8_BYTES;
      if ((have >> (j % D8_NB)) & 1) {
        const int n_valid = min(TILE_TOKENS, ctx - (tile0 + warp + D8_WARPS * j) * TILE_TOKENS);
        if (n_valid < TILE_TOKENS) clear_v_rows8(t, n_valid);
        tile8<CODE, FEW>(t, n_valid, qa, qs, r);
      }
      __syncwarp();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // this slot's reads before the next copy into it
      if (j + D8_NB < mine) have = (have & ~(1u << (j % D8_NB))) | issue(j + D8_NB) << (j % D8_NB);
    }
    if (!ok)  // a wait gave up: nothing more is loaded, and no copy is left in flight
      for (int i = j; i < min(mine, j + D8_NB); ++i)
        mbar_wait(&bars[warp][(used + i) % D8_NB], ((used + i) / D8_NB) & 1, nullptr);
    used += mine;
    __syncthreads();  // the rings are used up
    // ---- merge the warps; a whole group is finished, a part of one leaves a partial
    row8_store<FEW>(r, sml[warp], so + warp * A8_ROWS * D);
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == nt;
    const int slot = 2 * c + (pos == lo ? 0 : 1);
    for (int h = warp; h < G; h += D8_WARPS) {
      float M = -CUDART_INF_F, MO = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < D8_WARPS; ++w) {
        M = fmaxf(M, sml[w][h][0]);
        MO = fmaxf(MO, sml[w][h][1]);
      }
      float L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 6
      for (int w = 0; w < D8_WARPS; ++w) {
        L += sml[w][h][2] * (sml[w][h][0] == -CUDART_INF_F ? 0.f : fast_exp2(sml[w][h][0] - M));
        const float f = sml[w][h][1] == -CUDART_INF_F ? 0.f : fast_exp2(sml[w][h][1] - MO);
        const float4 x = *reinterpret_cast<const float4*>(so + (w * A8_ROWS + h) * D + 4 * lane);
        o.x = fmaf(x.x, f, o.x); o.y = fmaf(x.y, f, o.y); o.z = fmaf(x.z, f, o.z); o.w = fmaf(x.w, f, o.w);
      }
      if (whole) {
        finish_row8(a, (size_t)b * a.n_q_heads + (size_t)kvh * G + h, M, MO, L, o);
      } else {
        __stcg(reinterpret_cast<float4*>(a.part_o + ((size_t)slot * A8_ROWS + h) * D) + lane, o);
        if (lane == 0) __stcg(&a.part_ml[slot * A8_ROWS + h], make_float4(M, MO, L, 0.f));
      }
    }
    if (!whole) {
      // contributors: the CTAs whose ranges meet the group's tiles [g0, g1)
      const long long g0 = pos - tile0, g1 = g0 + nt;
      // the CTA of tile x is the last c with c total / N <= x
      auto cta_of = [&](long long x) {
        long long k = x * N / total;
        while ((k + 1) * total / N <= x) ++k;
        while (k * total / N > x) --k;
        return (int)k;
      };
      const int c0 = cta_of(g0), c1 = cta_of(g1 - 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int gi = b * Hkv + kvh;
        const int seen = atomicAdd(&a.counters[gi], 1);
        s_last = seen == c1 - c0;
        if (seen < 0 || seen > c1 - c0) {
          if (a.v.status) atomicOr(a.v.status, IQ_DEVERR_WORKSPACE);
        }
        if (s_last) atomicExch(&a.counters[gi], 0);
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        // slot of contributor k: 2 k + 1 where the group starts inside k's range, 2 k otherwise
        const int extra = g0 > c0 * total / N ? 1 : 0;
        for (int h = warp; h < G; h += D8_WARPS) {
          auto slot_of = [&](int k) { return (2 * k + (k == c0 ? extra : 0)) * A8_ROWS + h; };
          float M = -CUDART_INF_F, MO = -CUDART_INF_F, L = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = c0; k <= c1; k += 12) {  // twelve partials in flight
            float4 ml[12], x[12];
#pragma unroll
            for (int i = 0; i < 12; ++i) {
              ml[i] = make_float4(-CUDART_INF_F, -CUDART_INF_F, 0.f, 0.f);
              x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (k + i <= c1) {
                ml[i] = __ldcg(&a.part_ml[slot_of(k + i)]);
                x[i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (size_t)slot_of(k + i) * D) + lane);
              }
            }
            float m = M, mo = MO;
#pragma unroll
            for (int i = 0; i < 12; ++i) {
              m = fmaxf(m, ml[i].x);
              mo = fmaxf(mo, ml[i].y);
            }
            const float f0 = M == -CUDART_INF_F ? 0.f : fast_exp2(M - m), f1 = MO == -CUDART_INF_F ? 0.f : fast_exp2(MO - mo);
            L = M == -CUDART_INF_F ? L : L * f0;
            o = make_float4(o.x * f1, o.y * f1, o.z * f1, o.w * f1);
            M = m;
            MO = mo;
#pragma unroll
            for (int i = 0; i < 12; ++i) {
              // (a partial that saw nothing holds 0, or the NaN of a query that holds one)
              L += ml[i].x == -CUDART_INF_F ? ml[i].z : ml[i].z * fast_exp2(ml[i].x - M);
              const float f = ml[i].y == -CUDART_INF_F ? 0.f : fast_exp2(ml[i].y - MO);
              o.x = fmaf(x[i].x, f, o.x); o.y = fmaf(x[i].y, f, o.y); o.z = fmaf(x[i].z, f, o.z); o.w = fmaf(x[i].w, f, o.w);
            }
          }
          finish_row8(a, (size_t)b * a.n_q_heads + (size_t)kvh * G + h, M, MO, L, o);
        }
      }
    }
    // sml, s_last and the sums are read before the next segment's copies and sums take their place
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    pos += tile1 - tile0;
    tile0 = 0;
    if (pos < hi && ++kvh == Hkv) {
      kvh = 0;
      do ++b; while (clamp_ctx8(a, b) == 0);
      ctx = clamp_ctx8(a, b);
      nt = (ctx + TILE_TOKENS - 1) / TILE_TOKENS;
    }
  }
}

// CTAs of a call: one per SM, fewer where that leaves warps without a tile.
static int decode8_ctas(int batch, int n_kv_heads, int max_ctx) {
  const long long tiles = (long long)batch * n_kv_heads * ((max_ctx + TILE_TOKENS - 1) / TILE_TOKENS);
  return (int)std::max(1ll, std::min((long long)sm_count(), (tiles + D8_WARPS - 1) / D8_WARPS));
}

static size_t counter8_bytes(int batch, int n_kv_heads) { return ((size_t)batch * n_kv_heads * 4 + 255) & ~(size_t)255; }

size_t decode8_workspace_bytes(int batch, int n_kv_heads, int max_ctx) {
  const size_t slots = 2 * (size_t)decode8_ctas(batch, n_kv_heads, max_ctx);
  return counter8_bytes(batch, n_kv_heads) + slots * A8_ROWS * (sizeof(float4) + D * sizeof(float));
}

int launch_decode8(const View8& v, const void* q, int dtype, int batch, int n_q_heads, const int32_t* ctx_len,
                   int max_ctx, float scale, void* out, void* workspace, void* stream) {
  if (batch == 0) return 0;
  Decode8Args a;
  a.v = v;
  a.q = q;
  a.dtype = dtype;
  a.batch = batch;
  a.n_q_heads = n_q_heads;
  a.g_real = n_q_heads / v.n_kv_heads;
  a.max_ctx = max_ctx;
  a.ctx_len = ctx_len;
  a.scale = scale;
  a.out = out;
  const int n = decode8_ctas(batch, v.n_kv_heads, max_ctx);
  uint8_t* w = (uint8_t*)workspace;
  a.counters = (int32_t*)w;
  w += counter8_bytes(batch, v.n_kv_heads);
  a.part_ml = (float4*)w;
  a.part_o = (float*)(w + 2 * (size_t)n * A8_ROWS * sizeof(float4));
  const bool few = a.g_real <= 4;
  auto fn = v.code == IQ_E4M3 ? (few ? decode8_kernel<IQ_E4M3, true> : decode8_kernel<IQ_E4M3, false>)
                              : (few ? decode8_kernel<IQ_S8, true> : decode8_kernel<IQ_S8, false>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, D8_SMEM);
  if (e != cudaSuccess) return (int)e;
  return (int)launch_pdl(fn, dim3(n), dim3(D8_THREADS), D8_SMEM, (cudaStream_t)stream, a);
}

}  // namespace iq
