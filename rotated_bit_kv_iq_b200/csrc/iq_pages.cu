// The block table's operations: extend, free, fork, compact and copy pages, on the device.
//
// Each call is one small planning kernel (a single CTA where the order of a list or of the free pages
// matters: prefix sums, no atomics whose order could show), then copies of page contents that read the
// plan's lists from the workspace, spread over the whole device.  The plans are bound by latency (a pass
// or two over n_pages counts), the copies by memory (each byte read once and written once).
#include <algorithm>

#include "iq_device.cuh"
#include "iq_internal8.h"

namespace iq {

constexpr int PG_THREADS = 1024;
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_PER = IQ_PAGES_MAX_LIST / PG_THREADS;  // list entries per thread

// Workspace: the number of entries to copy; then the lists.
struct PagesWs {
  int32_t* count;
  int32_t* src;    // page copied from
  int32_t* dst;    // page copied to
  int32_t* tiles;  // tile records of each head to copy
  int32_t* remap;  // per page: where it is now, -1 if nobody holds it (compact), or the free pages in order (extend, fork)
};
static size_t list_len(const iq_pages& p) { return std::max((size_t)IQ_PAGES_MAX_LIST, (size_t)p.n_pages); }
size_t pages_workspace_bytes(const iq_pages& p) { return 256 + sizeof(int32_t) * (3 * list_len(p) + p.n_pages); }
static PagesWs carve(const iq_pages& p, void* ws) {
  PagesWs w;
  w.count = (int32_t*)ws;
  w.src = w.count + 64;
  w.dst = w.src + list_len(p);
  w.tiles = w.dst + list_len(p);
  w.remap = w.tiles + list_len(p);
  return w;
}

__device__ __forceinline__ void flag(const iq_pages& p, uint32_t bit) {
  if (p.status_dev) atomicOr(p.status_dev, bit);
}

// Exclusive prefix sum over the block's threads; *total gets the sum.  scratch: PG_WARPS + 1 numbers.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* scratch, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const T own = scratch[lane];
    T s = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    scratch[lane] = s - own;
    if (lane == 31) scratch[PG_WARPS] = s;
  }
  __syncthreads();
  *total = scratch[PG_WARPS];
  return scratch[warp] + incl - x;
}

// For every page with pred(page), in ascending order: put(rank, page).  Returns their number.  Warp w takes
// pages [w S, (w + 1) S), 32 at a time; two passes.
template <typename Pred, typename Put>
__device__ int rank_pages(int n_pages, int* scratch, Pred pred, Put put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = ((n_pages + PG_WARPS - 1) / PG_WARPS + 31) & ~31;
  const int lo = min(n_pages, warp * S), hi = min(n_pages, lo + S);
  int mine = 0;
#pragma unroll 4
  for (int p = lo; p < hi; p += 32) mine += __popc(__ballot_sync(0xffffffffu, p + lane < hi && pred(p + lane)));
  int total;
  int at = block_scan(lane == 0 ? mine : 0, scratch, &total);
  at = __shfl_sync(0xffffffffu, at, 0);
  for (int p = lo; p < hi; p += 32) {
    const bool yes = p + lane < hi && pred(p + lane);
    const uint32_t m = __ballot_sync(0xffffffffu, yes);
    if (yes) put(at + __popc(m & ((1u << lane) - 1u)), p + lane);
    at += __popc(m);
  }
  return total;
}

// Whether ids[0..i) holds id (shared memory).
__device__ __forceinline__ bool listed_before(const int* ids, int i, int id) {
  for (int j = 0; j < i; ++j)
    if (ids[j] == id) return true;
  return false;
}

__global__ void __launch_bounds__(PG_THREADS) pages_extend_kernel(iq_pages p, const int32_t* __restrict__ ids,
                                                                  const int32_t* __restrict__ new_len, int n, PagesWs w) {
  pdl_wait();
  __shared__ int s_id[IQ_PAGES_MAX_LIST];
  __shared__ int s_need[IQ_PAGES_MAX_LIST];
  __shared__ int scratch[PG_WARPS + 1];
  __shared__ long long wide[PG_WARPS + 1];
  const int tid = threadIdx.x;
  for (int i = tid; i < n; i += PG_THREADS) s_id[i] = ids[i];
  __syncthreads();
  int need[PG_PER];
  long long sum = 0;  // (what a long list asks for may pass 32 bits, however few pages there are)
#pragma unroll
  for (int k = 0; k < PG_PER; ++k) {
    const int i = tid * PG_PER + k;
    need[k] = 0;
    if (i >= n) continue;
    const int id = s_id[i], len = new_len[i];
    if (id < 0 || id >= p.max_seqs || listed_before(s_id, i, id)) {
      flag(p, IQ_DEVERR_SEQ);
      need[k] = -1;
    } else if ((long long)len > (long long)p.max_pages_per_seq * p.page_size) {
      flag(p, IQ_DEVERR_NOPAGE);
      need[k] = -1;
    } else {
      const int have = max(0, p.seq_len_dev[id]);
      if (len <= have) need[k] = -1;  // nothing to do
      else need[k] = (len - 1) / p.page_size + 1 - (have == 0 ? 0 : (have - 1) / p.page_size + 1);
    }
    sum += max(0, need[k]);
  }
  long long total;
  long long at = block_scan(sum, wide, &total);
  const int n_free = rank_pages(p.n_pages, scratch, [&](int g) { return p.ref_dev[g] <= 0; },
                                [&](int rank, int g) { if (rank < total) w.remap[rank] = g; });
#pragma unroll
  for (int k = 0; k < PG_PER; ++k) {
    const int i = tid * PG_PER + k;
    if (i >= n) continue;
    int start = -1;  // first free-page rank of this entry; -1: nothing to take
    if (need[k] >= 0) {
      if (at + need[k] > n_free) flag(p, IQ_DEVERR_NOPAGE);
      else start = (int)at;
      at += need[k];
    }
    s_need[i] = start;
  }
  __syncthreads();  // also: the free pages' list is written
  // a warp per entry: pages into the row, then the length
  const int lane = tid & 31;
  for (int i = tid >> 5; i < n; i += PG_WARPS) {
    const int start = s_need[i];
    if (start < 0) continue;
    const int id = s_id[i], have = max(0, p.seq_len_dev[id]), len = new_len[i];
    const int j0 = have == 0 ? 0 : (have - 1) / p.page_size + 1, j1 = (len - 1) / p.page_size + 1;
    for (int j = j0 + lane; j < j1; j += 32) {
      const int g = w.remap[start + j - j0];
      p.block_table_dev[(size_t)id * p.max_pages_per_seq + j] = g;
      p.ref_dev[g] = 1;
    }
    __syncwarp();
    if (lane == 0) p.seq_len_dev[id] = len;
  }
}

// One CTA per entry.
__global__ void __launch_bounds__(128) pages_free_kernel(iq_pages p, const int32_t* __restrict__ ids) {
  pdl_wait();
  const int i = blockIdx.x, id = ids[i];
  bool bad = id < 0 || id >= p.max_seqs;
  for (int j = threadIdx.x; j < i; j += 128) bad |= ids[j] == id;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) flag(p, IQ_DEVERR_SEQ);
    return;
  }
  int32_t* row = p.block_table_dev + (size_t)id * p.max_pages_per_seq;
  for (int j = threadIdx.x; j < p.max_pages_per_seq; j += 128) {
    const int g = row[j];
    if (g < 0) continue;
    if (g >= p.n_pages) flag(p, IQ_DEVERR_PAGE);
    else atomicSub(&p.ref_dev[g], 1);  // counts commute: the order does not show
    row[j] = -1;
  }
  if (threadIdx.x == 0) p.seq_len_dev[id] = 0;
}

__global__ void __launch_bounds__(PG_THREADS) pages_fork_kernel(iq_pages p, const int32_t* __restrict__ parent,
                                                                const int32_t* __restrict__ child, int n, PagesWs w) {
  pdl_wait();
  __shared__ int s_child[IQ_PAGES_MAX_LIST];
  __shared__ int s_len[IQ_PAGES_MAX_LIST];  // the parent's length; -1: refused
  __shared__ int scratch[PG_WARPS + 1];
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < n; i += PG_THREADS) s_child[i] = child[i];
  __syncthreads();
  int need[PG_PER], sum = 0;
#pragma unroll
  for (int k = 0; k < PG_PER; ++k) {
    const int i = tid * PG_PER + k;
    need[k] = 0;
    if (i >= n) continue;
    const int c = s_child[i], q = parent[i];
    int len = -1;
    if (c < 0 || c >= p.max_seqs || q < 0 || q >= p.max_seqs || q == c || p.seq_len_dev[c] != 0 ||
        p.block_table_dev[(size_t)c * p.max_pages_per_seq] >= 0 || listed_before(s_child, i, c)) {
      flag(p, IQ_DEVERR_SEQ);
    } else {
      len = max(0, p.seq_len_dev[q]);
      if ((long long)len > (long long)p.max_pages_per_seq * p.page_size) {
        flag(p, IQ_DEVERR_POSITION);
        len = -1;
      }
    }
    s_len[i] = len;
    need[k] = len > 0 && len % p.page_size ? 1 : 0;
    sum += need[k];
  }
  int total;
  int at = block_scan(sum, scratch, &total);
  const int n_free = rank_pages(p.n_pages, scratch, [&](int g) { return p.ref_dev[g] <= 0; },
                                [&](int rank, int g) { if (rank < total) w.remap[rank] = g; });
  __syncthreads();  // the counts are read, the list is written
#pragma unroll
  for (int k = 0; k < PG_PER; ++k) {
    const int i = tid * PG_PER + k;
    if (i >= n) continue;
    int src = -1, dst = -1, tiles = 0;
    const int len = s_len[i];
    if (len >= 0) {
      if (at + need[k] > n_free) {
        flag(p, IQ_DEVERR_NOPAGE);
        s_len[i] = -1;
      } else if (need[k]) {
        src = p.block_table_dev[(size_t)parent[i] * p.max_pages_per_seq + len / p.page_size];
        dst = w.remap[at];
        tiles = (len % p.page_size + TILE_TOKENS - 1) / TILE_TOKENS;
        p.ref_dev[dst] = 1;
        if (src < 0 || src >= p.n_pages) {
          flag(p, IQ_DEVERR_PAGE);
          tiles = 0;
        }
      }
      at += need[k];
    }
    w.src[i] = src;
    w.dst[i] = dst;
    w.tiles[i] = tiles;
  }
  if (tid == 0) w.count[0] = n;
  __syncthreads();
  for (int i = tid >> 5; i < n; i += PG_WARPS) {
    const int len = s_len[i];
    if (len < 0) continue;
    const int full = len / p.page_size;
    const int32_t* from = p.block_table_dev + (size_t)parent[i] * p.max_pages_per_seq;
    int32_t* to = p.block_table_dev + (size_t)s_child[i] * p.max_pages_per_seq;
    for (int j = lane; j < p.max_pages_per_seq; j += 32) {
      int g = -1;
      if (j < full) {
        g = from[j];
        if (g < 0 || g >= p.n_pages) flag(p, IQ_DEVERR_PAGE);
        else atomicAdd(&p.ref_dev[g], 1);
      } else if (j == full && len % p.page_size) {
        g = w.dst[i];
      }
      to[j] = g;
    }
    if (lane == 0) p.seq_len_dev[s_child[i]] = len;
  }
}

__global__ void __launch_bounds__(PG_THREADS) pages_compact_kernel(iq_pages p, int32_t* n_held, PagesWs w) {
  pdl_wait();
  __shared__ int scratch[PG_WARPS + 1];
  int32_t* const ref = p.ref_dev;
  for (int g = threadIdx.x; g < p.n_pages; g += PG_THREADS) w.remap[g] = ref[g] > 0 ? g : -1;
  const int held = rank_pages(p.n_pages, scratch, [&](int g) { return ref[g] > 0; }, [](int, int) {});
  __syncthreads();
  const int holes = rank_pages(p.n_pages, scratch, [&](int g) { return g < held && ref[g] <= 0; },
                               [&](int k, int g) { w.dst[k] = g; });
  __syncthreads();
  rank_pages(p.n_pages, scratch, [&](int g) { return g >= held && ref[g] > 0; }, [&](int k, int g) { w.src[k] = g; });
  __syncthreads();
  for (int k = threadIdx.x; k < holes; k += PG_THREADS) {
    const int s = w.src[k], d = w.dst[k];
    w.remap[s] = d;
    w.tiles[k] = p.page_size / TILE_TOKENS;
    ref[d] = ref[s];
    ref[s] = 0;
  }
  if (threadIdx.x == 0) {
    w.count[0] = holes;
    if (n_held) *n_held = held;
  }
}

// The tables after a compaction.  An entry of a page that nobody holds stays as it is.
__global__ void __launch_bounds__(256) pages_remap_kernel(iq_pages p, PagesWs w) {
  pdl_wait();
  const size_t n = (size_t)p.max_seqs * p.max_pages_per_seq;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
    const int g = p.block_table_dev[i];
    if (g < 0) continue;
    const int to = g < p.n_pages ? w.remap[g] : -1;
    if (to < 0) flag(p, IQ_DEVERR_PAGE);
    else if (to != g) p.block_table_dev[i] = to;
  }
}

__global__ void __launch_bounds__(PG_THREADS) pages_copy_plan_kernel(iq_pages p, const int32_t* __restrict__ src,
                                                                     const int32_t* __restrict__ dst, int n, PagesWs w) {
  pdl_wait();
  __shared__ int s_src[IQ_PAGES_MAX_LIST];
  __shared__ int s_dst[IQ_PAGES_MAX_LIST];
  for (int i = threadIdx.x; i < n; i += PG_THREADS) {
    s_src[i] = src[i];
    s_dst[i] = dst[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += PG_THREADS) {
    const int s = s_src[i], d = s_dst[i];
    bool bad = s < 0 || s >= p.n_pages || d < 0 || d >= p.n_pages;
    for (int j = 0; j < n && !bad; ++j) bad = (j != i && s_src[j] == d) || (j < i && s_dst[j] == d);
    if (bad) flag(p, IQ_DEVERR_PAGE);
    w.src[i] = s;
    w.dst[i] = d;
    w.tiles[i] = bad || s == d ? 0 : p.page_size / TILE_TOKENS;
  }
  if (threadIdx.x == 0) w.count[0] = n;
}

// The lists' pages in every layer of one pool.  An (entry, layer, head) run of whole tile records is cut into pieces of
// 4 KB, a warp's eight loads of 512 bytes each, all in flight before the first store.  Pages of 8224-byte records, 135 MB
// moved: 45 us (a run of 16 KB a warp, four loads at a time: 58 us).
constexpr int MOVE_PIECE = 256;  // 16-byte words
__global__ void __launch_bounds__(256) pages_move_kernel(uint8_t* pool, int n_layers, int n_heads, int tile_bytes,
                                                         int page_tiles, int n_pages, PagesWs w) {
  pdl_wait();
  const int lane = threadIdx.x & 31, words = page_tiles * (tile_bytes / 16), pieces = (words + MOVE_PIECE - 1) / MOVE_PIECE;
  const long long items = (long long)w.count[0] * n_layers * n_heads * pieces;
  for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5; i < items; i += (long long)gridDim.x * 8) {
    const int piece = (int)(i % pieces);
    const long long j = i / pieces;
    const int head = (int)(j % n_heads), layer = (int)(j / n_heads % n_layers), e = (int)(j / n_heads / n_layers);
    const int n = w.tiles[e] * (tile_bytes / 16), at = piece * MOVE_PIECE + lane;
    if (piece * MOVE_PIECE >= n) continue;
    const size_t base = (size_t)layer * n_pages;
    const uint4* s = reinterpret_cast<const uint4*>(pool) + ((base + w.src[e]) * n_heads + head) * words + at;
    uint4* d = reinterpret_cast<uint4*>(pool) + ((base + w.dst[e]) * n_heads + head) * words + at;
    uint4 x[MOVE_PIECE / 32];
#pragma unroll
    for (int k = 0; k < MOVE_PIECE / 32; ++k)
      if (at + 32 * k < n) x[k] = __ldcs(s + 32 * k);
#pragma unroll
    for (int k = 0; k < MOVE_PIECE / 32; ++k)
      if (at + 32 * k < n) __stcs(d + 32 * k, x[k]);
  }
}

// Nothing: launched plainly, it starts once the kernels before it are complete, so that what follows it on the stream may
// start early.
__global__ void pages_end_kernel() {}

static int finish(const iq_pages& p, const PagePools& pools, const PagesWs& w, cudaStream_t st) {
  for (int i = 0; i < pools.n; ++i)
    launch_pdl(pages_move_kernel, dim3(sm_count() * 8), dim3(256), 0, st, pools.base[i], pools.n_layers[i],
               pools.n_kv_heads[i], pools.tile_bytes[i], (int)(p.page_size / TILE_TOKENS), (int)p.n_pages, w);
  pages_end_kernel<<<1, 32, 0, st>>>();
  return (int)cudaGetLastError();
}

int launch_pages_extend(const iq_pages& p, const int32_t* ids, const int32_t* len, int n, void* ws, void* stream) {
  if (n == 0) return 0;
  const cudaStream_t st = (cudaStream_t)stream;
  launch_pdl(pages_extend_kernel, dim3(1), dim3(PG_THREADS), 0, st, p, ids, len, n, carve(p, ws));
  pages_end_kernel<<<1, 32, 0, st>>>();
  return (int)cudaGetLastError();
}
int launch_pages_free(const iq_pages& p, const int32_t* ids, int n, void* stream) {
  if (n == 0) return 0;
  const cudaStream_t st = (cudaStream_t)stream;
  launch_pdl(pages_free_kernel, dim3(n), dim3(128), 0, st, p, ids);
  pages_end_kernel<<<1, 32, 0, st>>>();
  return (int)cudaGetLastError();
}
int launch_pages_fork(const iq_pages& p, const PagePools& pools, const int32_t* parent, const int32_t* child, int n,
                      void* ws, void* stream) {
  if (n == 0) return 0;
  const PagesWs w = carve(p, ws);
  launch_pdl(pages_fork_kernel, dim3(1), dim3(PG_THREADS), 0, (cudaStream_t)stream, p, parent, child, n, w);
  return finish(p, pools, w, (cudaStream_t)stream);
}
int launch_pages_compact(const iq_pages& p, const PagePools& pools, int32_t* n_held, void* ws, void* stream) {
  const PagesWs w = carve(p, ws);
  const cudaStream_t st = (cudaStream_t)stream;
  launch_pdl(pages_compact_kernel, dim3(1), dim3(PG_THREADS), 0, st, p, n_held, w);
  const size_t entries = (size_t)p.max_seqs * p.max_pages_per_seq;
  launch_pdl(pages_remap_kernel, dim3((unsigned)std::min<size_t>((entries + 255) / 256, (size_t)sm_count() * 8)), dim3(256), 0, st, p, w);
  return finish(p, pools, w, st);
}
int launch_pages_copy(const iq_pages& p, const PagePools& pools, const int32_t* src, const int32_t* dst, int n,
                      void* ws, void* stream) {
  if (n == 0) return 0;
  const PagesWs w = carve(p, ws);
  launch_pdl(pages_copy_plan_kernel, dim3(1), dim3(PG_THREADS), 0, (cudaStream_t)stream, p, src, dst, n, w);
  return finish(p, pools, w, (cudaStream_t)stream);
}

}  // namespace iq
