// Attention over the 8-bit cache of few query rows: one token of each sequence (decode), or a chunk of float32 tokens in
// blocks of up to eight rows.
//
// The work is the list of 32-token tiles of all (entry, kv head) groups, an entry being a sequence or a block of its query
// tokens; CTA c of N takes an N-th of them, whatever the mix of lengths, a group's first tile counting for more.  Its warps
// take the tiles of each group's segment in turn, each through a ring of its own of two bulk-copied tile records: twelve
// warps, three a scheduler, at 168 registers.  A segment that is a whole group is finished at once; the others leave a
// partial (m, mo, l, O), and the last CTA of a group to arrive merges the group's partials in a fixed order, so that results
// do not depend on who is last.
// Bound by memory, 257 B for each (token, kv head).  A layer of 16 sequences of 2K to 32K tokens, 32 query and 8 kv heads:
// 82-89 us, 82-89% of the copy rate.  (Before groups counted for more than their tiles: 94; 105 with eight warps of 197
// registers; 121 with sixteen, whose 128 registers do not hold a tile's work, on one ring of 26 records.)
#include <algorithm>

#include "iq_attend8.cuh"

namespace iq {

constexpr int D8_WARPS = 12;
constexpr int D8_THREADS = 32 * D8_WARPS;
constexpr int D8_NB = 2;                                       // tile records in a warp's ring
constexpr int D8_UNCUT = 2 * D8_WARPS;                         // tiles of a group that is not cut
// What a group costs beside its tiles (its queries, an empty ring, the warps' merge), in tiles, about 6 us: without it the
// CTAs that get many short groups are the last (the 16-sequence layer: CTAs of 63 to 90 us; with it 62 to 80).  Leads of
// 0, 8, 16, 24, 32, 48, 64: 96, 90, 88, 84, 82, 83, 84 us.  Other shapes, cold caches, leads of 0 / 16 / 32, us a call with
// its events: 128 sequences of 100 to 4096 tokens, 8 kv heads 180 / 136 / 127; 64 of 2048 74 / 73 / 74; 4 of 8192 35 / 33 / 31;
// one of 131072 76 / 73 / 71, of 32768 36 / 33 / 31, of 4096 22.5 / 18.4 / 18.4.  A lead longer than a CTA's share leaves some CTAs
// of a small call without a tile, but has a group cut into fewer pieces to merge: held to half of the share, 22.5 for 4096 tokens.
constexpr int D8_LEAD = 32;
constexpr int D8_SMEM = D8_WARPS * D8_NB * TILE8_BYTES;        // (at a segment's end: the warps' value sums)
static_assert(D8_WARPS * A8_ROWS * D * 4 <= D8_SMEM, "value sums in the rings' place");

struct Decode8Args {
  View8 v;
  const void* q;
  int dtype, batch, n_q_heads, g_real, max_ctx;
  const int32_t* ctx_len;  // decode; or (CHUNK, ctx_len NULL) blocks of tq of a chunk's n_tok tokens, n_blk a sequence:
  int n_tok, tq, n_blk;
  const int32_t* start;
  const int32_t* n_valid;
  float scale;
  void* out;
  int32_t* counters;  // [batch * n_blk * Hkv], zero between calls
  float4* part_ml;    // [2 SMs][8]: m, mo, l
  float* part_o;      // [2 SMs][8][128]
};

// Entry e: a sequence (decode), or a block of a sequence's query tokens.
struct D8Entry {
  int b, tok0, n_live, pos0, ctx;  // its tokens, the first one's position, the keys that the last one sees
};
template <bool CHUNK>
__device__ __forceinline__ D8Entry d8_entry(const Decode8Args& a, int e) {
  D8Entry x;
  if (!CHUNK) {
    const int c = a.ctx_len[e];
    x.b = e;
    x.tok0 = 0;
    x.n_live = 1;
    x.ctx = c < 0 ? 0 : (c > a.max_ctx ? a.max_ctx : c);
    x.pos0 = x.ctx - 1;
  } else {
    x.b = e / a.n_blk;
    x.tok0 = e % a.n_blk * a.tq;
    const int cnt = max(0, min(a.n_tok, a.n_valid ? a.n_valid[x.b] : a.n_tok));
    x.n_live = max(0, min(a.tq, cnt - x.tok0));
    x.pos0 = max(0, min(a.max_ctx - cnt, a.start[x.b])) + x.tok0;
    x.ctx = x.n_live ? x.pos0 + x.n_live : 0;
  }
  return x;
}
template <bool CHUNK>
__device__ __forceinline__ int d8_tiles(const Decode8Args& a, int e) {
  return (d8_entry<CHUNK>(a, e).ctx + TILE_TOKENS - 1) / TILE_TOKENS;
}

// The same with the lead, for the sharing of the work.
__device__ __forceinline__ int d8_cost(int tiles) { return tiles ? tiles + D8_LEAD : 0; }

// Final value of one row of the group: lane holds sums of coordinates 4 lane ..
__device__ __forceinline__ void finish_row8(const Decode8Args& a, size_t row, float M, float MO, float L, float4 o) {
  const float f = L > 0.f ? fast_exp2(MO - M) / L : (L == L ? 0.f : L);
  store4(a.out, a.dtype, row * D + 4 * (threadIdx.x & 31), make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
}

template <int CODE, bool FEW, bool CHUNK>
__global__ void __launch_bounds__(D8_THREADS, 1) decode8_kernel(Decode8Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[D8_WARPS][D8_NB];
  __shared__ float sml[D8_WARPS][A8_ROWS][4];
  __shared__ long long s_scan[D8_WARPS];
  __shared__ int s_most[D8_WARPS], s_live[D8_WARPS];
  __shared__ int s_start[2];  // the CTA's first entry, and the cost before it within all kv heads
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

  // ---- plan: total cost, this CTA's range, the sequence that it starts in.  A group is D8_LEAD places and its tiles.
  const int E = a.batch * a.n_blk, per = (E + D8_THREADS - 1) / D8_THREADS, e0 = min(E, tid * per), e1 = min(E, e0 + per);
  long long mine = 0;
  int most = 0, live = 0;  // tiles of an entry; entries that have any
  for (int e = e0; e < e1; ++e) {
    const int n = d8_tiles<CHUNK>(a, e);
    mine += d8_cost(n);
    most = max(most, n);
    live += n > 0;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  long long incl = mine;
  int incl_live = live;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    const int y = __shfl_up_sync(0xffffffffu, incl_live, o);
    if (lane >= o) {
      incl += x;
      incl_live += y;
    }
  }
  if (lane == 31) {
    s_most[warp] = most;
    s_scan[warp] = incl;
    s_live[warp] = incl_live;
  }
  __syncthreads();
  for (int w = 0; w < D8_WARPS; ++w) most = max(most, s_most[w]);
  // Short groups, of two rounds of the warps at the most, are not cut: each counts one, and there is nothing to merge (a
  // 512-token layer of two kv heads: 9 us a call, 15 cut).
  const bool uncut = most <= D8_UNCUT;
  auto cost = [&](int tiles) { return uncut ? (tiles > 0 ? 1 : 0) : d8_cost(tiles); };
  long long before = uncut ? incl_live - live : incl - mine, total = 0;
  for (int w = 0; w < D8_WARPS; ++w) {
    const long long x = uncut ? s_live[w] : s_scan[w];
    if (w < warp) before += x;
    total += x;
  }
  before *= Hkv;
  total *= Hkv;
  // the CTAs that share the work: none without a tile, and no more than give every warp one
  const int N = (int)min((long long)gridDim.x, max(1ll, uncut ? total : (total + D8_WARPS - 1) / D8_WARPS));
  const long long lo = c < N ? c * total / N : total, hi = c < N ? (c + 1) * total / N : total;
  long long acc = before;  // cost of all groups before entry e
  for (int e = e0; e < e1 && acc <= lo; ++e) {
    const long long n = (long long)Hkv * cost(d8_tiles<CHUNK>(a, e));
    if (lo < hi && lo < acc + n) {
      s_start[0] = e;
      s_start[1] = (int)(lo - acc);
    }
    acc += n;
  }
  if (c == 0 && a.v.status)  // lengths, counts and starts outside their ranges
    for (int b = tid; b < a.batch; b += D8_THREADS) {
      bool bad;
      if (!CHUNK) {
        bad = a.ctx_len[b] < 0 || a.ctx_len[b] > a.max_ctx;
      } else {
        const int cnt = a.n_valid ? a.n_valid[b] : a.n_tok, st = a.start[b];
        bad = cnt < 0 || cnt > a.n_tok || st < 0 || st > a.max_ctx - max(0, min(a.n_tok, cnt));
      }
      if (bad) atomicOr(a.v.status, IQ_DEVERR_CTX);
    }
  // sequences with nothing to see: zero rows
  if (!CHUNK)
    for (int b = c; b < a.batch; b += gridDim.x)
      if (d8_entry<CHUNK>(a, b).ctx == 0)
        for (int i = tid; i < a.n_q_heads * (D / 4); i += D8_THREADS)
          store4(a.out, a.dtype, (size_t)b * a.n_q_heads * D + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
  __syncthreads();
  if (lo >= hi) return;
  int e = s_start[0];
  D8Entry x = d8_entry<CHUNK>(a, e);
  int nt = (x.ctx + TILE_TOKENS - 1) / TILE_TOKENS;                       // the group's tiles
  int kvh = s_start[1] / cost(nt), at = s_start[1] % cost(nt);            // at: where in the group's places the segment starts
  long long pos = lo;
  bool more = true;
  uint32_t used = 0;  // of this warp's ring, so far
  bool ok = true;
  uint8_t* const ring = smem + warp * D8_NB * TILE8_BYTES;
  const int page_tiles = a.v.page_size / TILE_TOKENS;
  auto out_row = [&](int row) {
    return CHUNK ? ((size_t)x.b * a.n_tok + x.tok0 + row / G) * a.n_q_heads + (size_t)kvh * G + row % G
                 : (size_t)x.b * a.n_q_heads + (size_t)kvh * G + row;
  };
  while (more) {
    // ---- one segment: tiles [tile0, tile1) of group (e, kvh)
    const int end = (int)min((long long)cost(nt), at + (hi - pos));
    const int tile0 = uncut ? 0 : max(0, at - D8_LEAD), tile1 = uncut ? nt : end - D8_LEAD;
    if (tile1 <= tile0) break;  // the range ends before the group's first tile
    const int mine = ok && tile1 - tile0 > warp ? (tile1 - tile0 - warp + D8_WARPS - 1) / D8_WARPS : 0;  // this warp's
    auto issue = [&](int j) {  // the warp's j-th tile of the segment; whether it has a page
      const int tile = tile0 + warp + D8_WARPS * j, idx = tile / page_tiles;
      uint64_t* const bar = &bars[warp][(used + j) % D8_NB];
      int page = x.b;
      if (a.v.block_table) page = idx < a.v.max_pages ? a.v.block_table[(size_t)x.b * a.v.max_pages + idx] : -1;
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
    const int rows = CHUNK ? x.n_live * G : G, row = FEW ? g & 3 : g;  // row: token row / G of the block, head row % G of the group
    const float qs = load_q8(a.q, a.dtype, out_row(row), row < rows, a.scale, qa);
    const int seen = !CHUNK ? x.ctx : row < rows ? x.pos0 + row / G + 1 : 0;  // keys
    Row8 r;
    row8_init(r);
    int j = 0;
    for (; j < mine; ++j) {
      const uint32_t n = used + j;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[warp][n % D8_NB], (n / D8_NB) & 1, a.v.status));
      if (!ok) break;
      uint8_t* const t = ring + n % D8_NB * TILE8_BYTES;
      if ((have >> (j % D8_NB)) & 1) {
        const int first = (tile0 + warp + D8_WARPS * j) * TILE_TOKENS;
        if (written8(*reinterpret_cast<const float2*>(t + TILE8_SCALES))) {
          if (x.ctx - first < TILE_TOKENS) clear_v_rows8(t, x.ctx - first);
          tile8<CODE, FEW>(t, seen - first, qa, qs, r);
        } else if (lane == 0 && a.v.status) {
          atomicOr(a.v.status, IQ_DEVERR_PAGE);
        }
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
    for (int h = warp; h < rows; h += D8_WARPS) {
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
        finish_row8(a, out_row(h), M, MO, L, o);
      } else {
        __stcg(reinterpret_cast<float4*>(a.part_o + ((size_t)slot * A8_ROWS + h) * D) + lane, o);
        if (lane == 0) __stcg(&a.part_ml[slot * A8_ROWS + h], make_float4(M, MO, L, 0.f));
      }
    }
    if (!whole) {
      // contributors: the CTAs whose ranges meet the tiles of the group's places [g0, g1)
      const long long g0 = pos - at, g1 = g0 + d8_cost(nt);
      // the CTA of place x is the last c with c total / N <= x
      auto cta_of = [&](long long x) {
        long long k = x * N / total;
        while ((k + 1) * total / N <= x) ++k;
        while (k * total / N > x) --k;
        return (int)k;
      };
      const int c0 = cta_of(g0 + D8_LEAD), c1 = cta_of(g1 - 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const size_t gi = (size_t)e * Hkv + kvh;
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
        for (int h = warp; h < rows; h += D8_WARPS) {
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
          finish_row8(a, out_row(h), M, MO, L, o);
        }
      }
    }
    // sml, s_last and the sums are read before the next segment's copies and sums take their place
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    pos += end - at;
    at = 0;
    more = pos < hi;
    if (more && ++kvh == Hkv) {
      kvh = 0;
      do x = d8_entry<CHUNK>(a, ++e);
      while (x.ctx == 0);
      nt = (x.ctx + TILE_TOKENS - 1) / TILE_TOKENS;
    }
  }
}

// CTAs of a call over `entries` sequences or blocks: one per SM, fewer where that leaves CTAs without a group and warps
// without a tile.
static int decode8_ctas(long long entries, int n_kv_heads, int max_ctx) {
  const long long groups = entries * n_kv_heads, tiles = groups * ((max_ctx + TILE_TOKENS - 1) / TILE_TOKENS);
  return (int)std::max(1ll, std::min((long long)sm_count(), std::max(groups, (tiles + D8_WARPS - 1) / D8_WARPS)));
}

static size_t counter8_bytes(long long entries, int n_kv_heads) { return ((size_t)entries * n_kv_heads * 4 + 255) & ~(size_t)255; }

// Workspace: partials of a CTA on every SM, then the counters: at one place for calls of all sizes, so that none writes
// its partials over the counters of another.
static size_t part8_slots() { return 2 * (size_t)sm_count(); }
static size_t part8_bytes() { return part8_slots() * A8_ROWS * (sizeof(float4) + D * sizeof(float)); }
static size_t workspace8_bytes(long long entries, int n_kv_heads) { return part8_bytes() + counter8_bytes(entries, n_kv_heads); }

static int launch8(Decode8Args& a, int n_q_heads, float scale, const void* q, int dtype, void* out, void* workspace, void* stream) {
  a.q = q;
  a.dtype = dtype;
  a.n_q_heads = n_q_heads;
  a.g_real = n_q_heads / a.v.n_kv_heads;
  a.scale = scale;
  a.out = out;
  const long long entries = (long long)a.batch * a.n_blk;
  const int n = decode8_ctas(entries, a.v.n_kv_heads, a.max_ctx);
  a.part_ml = (float4*)workspace;
  a.part_o = (float*)(a.part_ml + part8_slots() * A8_ROWS);
  a.counters = (int32_t*)((uint8_t*)workspace + part8_bytes());
  const bool few = a.g_real <= 4, e4 = a.v.code == IQ_E4M3;  // (a chunk's blocks have five rows or more)
  auto fn = !a.ctx_len ? (e4 ? decode8_kernel<IQ_E4M3, false, true> : decode8_kernel<IQ_S8, false, true>)
            : few      ? (e4 ? decode8_kernel<IQ_E4M3, true, false> : decode8_kernel<IQ_S8, true, false>)
                       : (e4 ? decode8_kernel<IQ_E4M3, false, false> : decode8_kernel<IQ_S8, false, false>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, D8_SMEM);
  if (e != cudaSuccess) return (int)e;
  return (int)launch_pdl(fn, dim3(n), dim3(D8_THREADS), D8_SMEM, (cudaStream_t)stream, a);
}

size_t decode8_workspace_bytes(int batch, int n_kv_heads) { return workspace8_bytes(batch, n_kv_heads); }

int launch_decode8(const View8& v, const void* q, int dtype, int batch, int n_q_heads, const int32_t* ctx_len,
                   int max_ctx, float scale, void* out, void* workspace, void* stream) {
  if (batch == 0) return 0;
  Decode8Args a = {};
  a.v = v;
  a.batch = batch;
  a.max_ctx = max_ctx;
  a.ctx_len = ctx_len;
  a.n_tok = a.tq = a.n_blk = 1;
  return launch8(a, n_q_heads, scale, q, dtype, out, workspace, stream);
}

// A chunk of query tokens, up to eight rows (tokens x heads) a block: float32 queries, whose products take two terms.
size_t chunk8_workspace_bytes(int batch, int n_tok, int g, int n_kv_heads) {
  return workspace8_bytes((long long)batch * ((n_tok + A8_ROWS / g - 1) / (A8_ROWS / g)), n_kv_heads);
}
int launch_chunk8(const View8& v, const void* q, int dtype, int batch, int n_tok, int n_q_heads, const int32_t* start,
                  const int32_t* n_valid, int max_ctx, float scale, void* out, void* workspace, void* stream) {
  Decode8Args a = {};
  a.v = v;
  a.batch = batch;
  a.max_ctx = max_ctx;
  a.n_tok = n_tok;
  a.tq = A8_ROWS / (n_q_heads / v.n_kv_heads);
  a.n_blk = (n_tok + a.tq - 1) / a.tq;
  a.start = start;
  a.n_valid = n_valid;
  if (max_ctx > D8_UNCUT * TILE_TOKENS) {  // groups may be cut, and this workspace comes as it is
    const cudaError_t e = cudaMemsetAsync((uint8_t*)workspace + part8_bytes(), 0,
                                          counter8_bytes((long long)batch * a.n_blk, v.n_kv_heads), (cudaStream_t)stream);
    if (e != cudaSuccess) return (int)e;
  }
  return launch8(a, n_q_heads, scale, q, dtype, out, workspace, stream);
}

}  // namespace iq
