// Causal attention of a chunk of 16-bit query tokens over the 8-bit cache on the 5th-generation tensor cores.
//
// A block is 256 query rows (256 / G tokens x the G heads of one kv head) as two tiles of 128; it streams the keys in steps
// of 128 (four tile records).  8-bit codes are exact in binary16, so a step's K and V are expanded once for both tiles into
// shared memory, and with S in tensor memory, in half-steps of 64 keys:
//   S = Q K^T       128 x 64 x 128, Q and K in shared memory (both along the coordinates)
//   O += P V        128 x 128 x 64, P in tensor memory (binary16, over S's own columns), V in shared memory as it lies in
//                   the cache: rows of coordinates (N-major operand)
// Each tile has two S buffers: while the softmax is at one half-step's scores the tensor core adds the P of the half-step
// before and makes the scores of the one after.  (One buffer of 128 keys a tile: 334 us on the 2048-token
// chunk, 265 so.  This and the other variants' times are from before ref had its margin, below, which costs 6 us.)
// The block scales stay out of both products: a score is S times (K scale of its 32 keys) times a row factor, and the V
// scale joins the exponent, p' = 2^(s + log2 v - ref); the row's sum takes p' / v.  ref is 8 below the first half-step's
// maximum of s + log2 v, and follows only once the p' of a half-step add up to more than 65504: O is then rescaled in tensor
// memory, rarely.
// p' is one binary16 number, all sums are float32.  A weight is rounded by 2^-11 of itself, as the output is by its own
// type: the error of the fp16 chunk against 64 bits is 2.6e-4 for the 2.1e-4 of the output's rounding alone (two terms, as
// for float32 queries, would double the products P V).  2^8 for the largest p' of the first half-step leaves binary16's normal
// numbers for weights down to 2^-22 of the largest times V scale that the row has met, and its steps of 2^-24 below: a key
// is off by at most 2^-33 of that, 131072 keys by 2^-16.
//
// Work: the list of (block, step) over all blocks is cut into equal runs, one per CTA (one CTA per SM), so that neither
// causal lengths nor ragged batches nor a number of blocks off the number of SMs leave SMs idle.  A block cut by a run's
// end leaves partials, which a second kernel merges in order.
// Roles: warps 0-3 and 4-7 the softmax of the two tiles (thread = row), 8-11 and 12-15 the expansion of K and of V, 16
// and 18 issue the two tiles' MMAs, 17 finds the records and their scales.
//
// Measured (2048 tokens after 6144, 32 query and 8 kv heads, int8): 273 us back to back, 880 TFLOP/s, 53% of cuBLAS's
// bf16 rate; 297 with the caches flushed between calls.  Of a
// step's 4,700 cycles the MMAs take 2,500 (a 64-key score product, fed from shared memory, runs at 64% of the MMA rate: 50
// cycles for 32), the exponentials (MUFU) 2,050, instruction issue 2,100 a scheduler; the rest is latency of the softmax
// warps, two a scheduler.
#pragma once
#include <algorithm>

#include "iq_attend8.cuh"
#include "iq_tcgen05.cuh"

namespace iq {

constexpr int PT_TILE = 128;  // rows of a tile: the MMA's M
constexpr int PT_ROWS = 256;  // rows of a block
constexpr int PT_BN = 128;    // keys of a step
constexpr int PT_THREADS = 640;
// registers a thread: softmax (two warpgroups), expansion (two), MMA issue; the block is launched with 5 * 96.  The
// 2048-token chunk took 265 us so, 273 with 120 / 80 / 80, 269 with 104 / 88 / 96; the MMA warps spill with 64.
constexpr int PT_REG_SOFTMAX = 112, PT_REG_EXPAND = 80, PT_REG_MMA = 96;
static_assert(2 * PT_REG_SOFTMAX + 2 * PT_REG_EXPAND + PT_REG_MMA <= 5 * 96, "the register split");
constexpr int PT_S_COL = 0, PT_O_COL = 256;  // of tile t: 128 columns from PT_S_COL + 128 t, PT_O_COL + 128 t
constexpr float PT_TOP = 65504.f;  // the most that p' of a half-step add up to: binary16's largest number
// log2 of the largest p' of a half-step that sets ref (64 of them are below PT_TOP).  The 2048-token chunk takes 295 us so (cold
// caches) and 290 with 4, which leaves 12 bits until the next rescaling, not 8; but then 131072 keys are off by 2^-12.
constexpr float PT_ABOVE = 8.f;
// log2 of the row's sum beside the first V scale: V scales 2^104 apart leave the sum between 2^-112 and, over T keys,
// 2^98 T, within float32 either way.
constexpr float PT_BASE = -16.f;

struct PtSmem {
  static constexpr int q = 0;                 // [tile] 128 rows x 128 coordinates
  static constexpr int k = 65536;             // [buffer] 128 keys x 128 coordinates
  static constexpr int v = 131072;            // [buffer]
  static constexpr int ks = 196608;           // float [8][4]: K scales of step n mod 8's records
  static constexpr int lv = ks + 128;         // float [8][4]: log2 of the V scales; NaN: the record is not there
  static constexpr int w = lv + 128;          // float [8][4]: 2^(base - log2 of the V scale)
  static constexpr int base = w + 128;        // float [8]: the segment's base, PT_BASE and log2 of its first V scale
  static constexpr int rec = base + 32;       // int [4][4]: step n mod 4's records in the layer; -1: not there
  static constexpr int keys = rec + 64;       // int [4]: the step's keys up to the block's last; 0: the run's end
  static constexpr int scan = keys + 16;      // int64 [20], then the plan: int [4]
  static constexpr int bars = scan + 192;     // uint64 [TB_COUNT]
  static constexpr int misc = bars + 30 * 8;  // uint32 tensor-memory base, int abort
  static constexpr int bytes = misc + 16 + 1024;
};
static_assert(PtSmem::bytes <= 232448, "one CTA's shared memory");

// mbarriers: K and V of step parity expanded / free again; by tile and half-step parity (2 t + b): scores ready, P
// written; by tile: a segment's last O += P V done, the one before it; queries; all MMAs done; records of step n mod 4
// located / taken.
enum { TB_KFULL = 0, TB_KFREE = 2, TB_VFULL = 4, TB_VFREE = 6, TB_SFULL = 8, TB_PFULL = 12, TB_ODONE = 16, TB_OLAST = 18,
       TB_Q = 20, TB_DRAIN = 21, TB_LFULL = 22, TB_LFREE = 26, TB_COUNT = 30 };

struct PtArgs {
  View8 v;
  const void* q;
  int dtype, batch, n_tok, n_q_heads, g_real, tq, n_blk, max_ctx, ctas;
  const int32_t* start;
  const int32_t* n_valid;
  float scale;
  void* out;
  int2* cut;        // [batch][n_blk][Hkv]: the first and last CTA of the block
  float4* part_ml;  // [2 N][256]: (max of scores, max with values' scales, sum)
  float* part_o;    // [2 N][256][128]
};

// Bounded wait (about 1 s) that also ends once another thread has given up; the global timer is read in one of 4096 tries.
__device__ __forceinline__ bool pt_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0 && *abort) return false;
    if ((i & 4095u) == 0) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > 1000000000ull) {
        if (status) atomicOr(status, IQ_DEVERR_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
  }
}

// Entry e = (sequence, block of tokens): where its rows and keys are.
struct PtEntry {
  int b, tok0, n_live, pos0, kv_end, steps;
};
__device__ __forceinline__ PtEntry pt_entry(const PtArgs& a, int e) {
  PtEntry x;
  x.b = e / a.n_blk;
  x.tok0 = (e % a.n_blk) * a.tq;
  int cnt = a.n_valid ? a.n_valid[x.b] : a.n_tok;
  cnt = max(0, min(a.n_tok, cnt));
  const int start = max(0, min(a.max_ctx - cnt, a.start[x.b]));
  x.n_live = max(0, min(a.tq, cnt - x.tok0));
  x.pos0 = start + x.tok0;
  x.kv_end = x.pos0 + x.n_live;
  x.steps = x.n_live ? (x.kv_end + PT_BN - 1) / PT_BN : 0;
  return x;
}

// A CTA's run of (block, step) pairs, one segment (steps [k0, k1) of one block) after another.
struct PtWalk {
  PtEntry x;
  int pos, end;  // within the run
  int e, kvh, k0, k1;
  __device__ __forceinline__ void cut() { k1 = min(x.steps, k0 + (end - pos)); }
  __device__ __forceinline__ bool next(const PtArgs& a) {  // false at the run's end
    pos += k1 - k0;
    if (pos >= end) return false;
    k0 = 0;
    if (++kvh == a.v.n_kv_heads) {
      kvh = 0;
      do x = pt_entry(a, ++e);
      while (x.steps == 0);
    }
    cut();
    return true;
  }
};

// 16 bytes past L1, of which shared memory leaves little.
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
template <int REGS>
__device__ __forceinline__ void set_registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void set_registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }

template <int CODE>
__global__ void __launch_bounds__(PT_THREADS, 1) prefill8_tc_kernel(PtArgs a) {
  using SM = PtSmem;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + SM::bars);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::misc);
  volatile int* const abort = reinterpret_cast<volatile int*>(smem + SM::misc + 4);
  long long* const s_scan = reinterpret_cast<long long*>(smem + SM::scan);
  int* const s_plan = reinterpret_cast<int*>(smem + SM::scan + 20 * 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = a.v.n_kv_heads, G = a.g_real, c = blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < TB_COUNT; ++i) {
      // one arrival a warp (of all 32 lanes' it would be 32 in a row)
      const bool expanded = i == TB_KFULL || i == TB_KFULL + 1 || i == TB_VFULL || i == TB_VFULL + 1;
      const bool written = i >= TB_PFULL && i < TB_PFULL + 4;
      const bool freed = i == TB_KFREE || i == TB_KFREE + 1 || i == TB_VFREE || i == TB_VFREE + 1 || i == TB_DRAIN;  // by both tiles
      const int count = expanded || written ? 4 : i >= TB_LFREE || i == TB_Q ? 8 : freed ? 2 : 1;
      mbar_init(&bars[i], count);
    }
    mbar_fence_init();
    *abort = 0;
  }
  pdl_wait();

  // ---- plan: the total number of steps, this CTA's run, the block that it starts in
  const int E = a.batch * a.n_blk, per = (E + PT_THREADS - 1) / PT_THREADS, e0 = min(E, tid * per), e1 = min(E, e0 + per);
  long long mine = 0;
  for (int e = e0; e < e1; ++e) mine += pt_entry(a, e).steps;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long acc = incl - mine, total = 0;
  for (int w = 0; w < PT_THREADS / 32; ++w) {
    if (w < warp) acc += s_scan[w];
    total += s_scan[w];
  }
  acc *= Hkv;
  total *= Hkv;
  const int N = (int)min((long long)gridDim.x, total);  // the CTAs that share the steps: none without one
  if (c >= N && c) return;
  const long long lo = c * total / max(N, 1), hi = (c + 1) * total / max(N, 1);
  for (int e = e0; e < e1 && acc <= lo; ++e) {
    const long long nt = (long long)Hkv * pt_entry(a, e).steps;
    if (lo < hi && lo < acc + nt) {
      s_plan[0] = e;
      s_plan[1] = (int)(lo - acc);
      break;
    }
    acc += nt;
  }
  if (c == 0 && a.v.status)  // counts and starts outside their ranges
    for (int b = tid; b < a.batch; b += PT_THREADS) {
      const int cnt = a.n_valid ? a.n_valid[b] : a.n_tok, st = a.start[b];
      if (cnt < 0 || cnt > a.n_tok || st < 0 || st > a.max_ctx - max(0, min(a.n_tok, cnt))) atomicOr(a.v.status, IQ_DEVERR_CTX);
    }
  if (lo >= hi) return;
  if (warp == 16) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PtWalk s;
  s.e = s_plan[0];
  s.x = pt_entry(a, s.e);
  s.kvh = s_plan[1] / s.x.steps;
  s.k0 = s_plan[1] % s.x.steps;
  s.pos = 0;
  s.end = (int)(hi - lo);
  s.cut();

  if (warp < 8) {
    // ==== softmax: thread = row r of the block (row r mod 128 of tile t); half-steps of 64 keys
    set_registers_up<PT_REG_SOFTMAX>();
    const int t = warp >> 2, r = 128 * t + 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + PT_S_COL + 128 * t, tO = tmem + lanes + PT_O_COL + 128 * t;
    uint32_t done = 0;  // half-steps of this tile so far
    uint32_t n = 0;     // steps of the run so far
    uint32_t seg = 0;
    bool ok = true;
    do {
      const int tiles = s.x.n_live * G > PT_TILE ? 2 : 1, tok = r / G;
      const bool live = r < a.tq * G && tok < s.x.n_live;
      const size_t row = ((size_t)s.x.b * a.n_tok + s.x.tok0 + tok) * a.n_q_heads + (size_t)s.kvh * G + r % G;
      // queries: scaled by the power of two that brings the row's largest magnitude to [2^14, 2^15)
      float qs = 1.f;
      {
        uint4 u[16];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          u[i] = live ? __ldg(reinterpret_cast<const uint4*>((const uint16_t*)a.q + row * D) + i) : make_uint4(0, 0, 0, 0);
        auto widen = [&](uint32_t x) {
          return a.dtype == IQ_F16 ? half2_floats(x) : make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
        };
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 f0 = widen(u[i].x), f1 = widen(u[i].y), f2 = widen(u[i].z), f3 = widen(u[i].w);
          amax = fmaxf(amax, fmaxf(fmaxf(fmaxf(fabsf(f0.x), fabsf(f0.y)), fmaxf(fabsf(f1.x), fabsf(f1.y))),
                                   fmaxf(fmaxf(fabsf(f2.x), fabsf(f2.y)), fmaxf(fabsf(f3.x), fabsf(f3.y)))));
        }
        int ex = (int)(__float_as_uint(amax) >> 23) - 127;
        ex = max(-100, min(127, ex));
        const float sig = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
        if (live) qs = a.scale * kLog2E8 * __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 f0 = widen(u[i].x), f1 = widen(u[i].y), f2 = widen(u[i].z), f3 = widen(u[i].w);
          *reinterpret_cast<uint4*>(smem + SM::q + 32768 * t + umma_sw128_off(r & 127, 8 * i, PT_TILE)) =
              make_uint4(half2_bits(f0.x * sig, f0.y * sig), half2_bits(f1.x * sig, f1.y * sig),
                         half2_bits(f2.x * sig, f2.y * sig), half2_bits(f3.x * sig, f3.y * sig));
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[TB_Q]);
      float ref = -CUDART_INF_F, l = 0.f;
      if (t < tiles) {
        const int qpos = live ? s.x.pos0 + tok : -1;  // the last key that the row sees
        const int halves = 2 * (s.k1 - s.k0);
        for (int i = 0; i < halves; ++i, ++done) {
          const int buf = done & 1;
          ok = __all_sync(0xffffffffu, ok && pt_wait(&bars[TB_SFULL + 2 * t + buf], (done >> 1) & 1, abort, a.v.status));
          if (!ok) break;
          tc_fence_after();
          uint32_t x[32];
          tmem_ld32(tS + 64 * buf, x);  // under way while the scales are looked up
          const int slot = 2 * ((n + (i >> 1)) & 7) + (i & 1);
          const int lim = qpos - PT_BN * s.k0 - 64 * i;  // keys 0 .. lim of the half-step
          const float2 ks = reinterpret_cast<const float2*>(smem + SM::ks)[slot];
          const float2 lvs = reinterpret_cast<const float2*>(smem + SM::lv)[slot];
          const float2 ws = reinterpret_cast<const float2*>(smem + SM::w)[slot];
          // some key is not seen by some row of the warp, or some record is not there
          const bool some = __any_sync(0xffffffffu, lim < 63) || !(lvs.x == lvs.x) || !(lvs.y == lvs.y);
          auto record = [&](int b) {  // scores of record b, whose load was started; keys that the row does not see: -inf
            tmem_wait_ld(x);
            if (some) {
              const float lv = b ? lvs.y : lvs.x;
              const int last = lv == lv ? lim - 32 * b : -1;
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = k <= last ? x[k] : 0xFF800000u;
            }
          };
          // p' of the half-step under the ref that stands; P waits in registers.  The row's sum, which is
          // needed anyway, tells whether a p' has become too large: no maximum has to be found.
          uint32_t pp[32];
          float add_l, top;
          auto pass = [&](float at) {
            add_l = top = 0.f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (b) tmem_ld32(tS + 64 * buf + 32, x);
              record(b);
              const float lv = b ? lvs.y : lvs.x;
              const bool here = lv == lv;
              // (a row of zeros over a block of zeros: the product may underflow, and 0 times a hidden key's -inf is NaN)
              const float f1 = here ? fmaxf((b ? ks.y : ks.x) * qs, 1.17549435e-38f) : 1.f, add1 = here ? lv - at : 0.f;
              const uint64_t ff = f2(f1, f1), add = f2(add1, add1);
              uint64_t sum[2] = {0, 0};
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float y0, y1;
                f2s(fma2(f2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), ff, add), y0, y1);
                y0 = fast_exp2(y0);
                y1 = fast_exp2(y1);
                sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], f2(y0, y1));
                pp[16 * b + k / 2] = half2_bits(y0, y1);
              }
              float s0, s1;
              f2s(add2(sum[0], sum[1]), s0, s1);
              top += s0 + s1;
              add_l = fmaf(s0 + s1, b ? ws.y : ws.x, add_l);
            }
          };
          // A block's first half-step, and rarely one after it: ref first goes to PT_ABOVE below the half-step's maximum
          bool up = i == 0;
          for (bool first = true;; first = false) {
            if (__any_sync(0xffffffffu, up)) {
              float mo = -CUDART_INF_F;
#pragma unroll 1
              for (int b = 0; b < 2; ++b) {
                if (b) tmem_ld32(tS + 64 * buf + 32, x);
                record(b);
                float m1 = -CUDART_INF_F;
#pragma unroll
                for (int k = 0; k < 32; k += 2) m1 = fmaxf(m1, fmaxf(__uint_as_float(x[k]), __uint_as_float(x[k + 1])));
                const float lv = b ? lvs.y : lvs.x;
                if (m1 > -CUDART_INF_F) mo = fmaxf(mo, lv == lv ? fmaf(m1, (b ? ks.y : ks.x) * qs, lv) : m1);
              }
              // (rows that could wait follow too, since O is gone through anyway: fewer times for the warp in all)
              mo -= PT_ABOVE;
              const float al = mo > ref ? (ref == -CUDART_INF_F ? 0.f : fast_exp2(ref - mo)) : 1.f;
              ref = fmaxf(ref, mo);
              if (i > 0) {
                // O += P V of the half-step before is done: the scores of the next one, or at the end a barrier of its
                // own, are signalled after it
                const bool next = i + 1 < halves;
                ok = __all_sync(0xffffffffu, next ? pt_wait(&bars[TB_SFULL + 2 * t + (buf ^ 1)], ((done + 1) >> 1) & 1, abort, a.v.status)
                                                  : pt_wait(&bars[TB_ODONE + t], seg & 1, abort, a.v.status));
                if (!ok) break;
                tc_fence_after();
                l *= al;
#pragma unroll 1
                for (int b = 0; b < 8; ++b) {
                  uint32_t o[16];
                  tmem_ld16(tO + 16 * b, o);
                  tmem_wait_ld(o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
                  tmem_st16(tO + 16 * b, o);
                }
              }
              first = false;
              tmem_ld32(tS + 64 * buf, x);
            }
            pass(ref == -CUDART_INF_F ? 0.f : ref);
            if (!first) break;
            up = !(top <= PT_TOP) || (ref == -CUDART_INF_F && lim >= 0);
            if (!__any_sync(0xffffffffu, up)) break;
            tmem_ld32(tS + 64 * buf, x);
          }
          if (!ok) break;
          l += add_l;
          // P over the columns of S
#pragma unroll
          for (int b = 0; b < 2; ++b)
            tmem_st16(tS + 64 * buf + 16 * b, *reinterpret_cast<const uint32_t(*)[16]>(pp + 16 * b));
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[TB_PFULL + 2 * t + buf]);
        }
        if (ok) ok = __all_sync(0xffffffffu, pt_wait(&bars[TB_OLAST + t], seg & 1, abort, a.v.status));
        if (!ok) break;
        tc_fence_after();
        const bool whole = s.k0 == 0 && s.k1 == s.x.steps;
        const float base = reinterpret_cast<const float*>(smem + SM::base)[(n + s.k1 - s.k0 - 1) & 7];
        const float inv = l > 0.f ? fast_exp2(base) / l : (l == l ? 0.f : l);
        const size_t prow = (size_t)(2 * c + (s.pos == 0 ? 0 : 1)) * PT_ROWS + r;
        if (!whole) {
          // the sum as its exponent and a number in [1, 2), since sums of segments of other bases are far from it
          const int ex = l > 0.f && l < CUDART_INF_F ? ilogbf(l) : 0;
          a.part_ml[prow] = l == 0.f ? make_float4(-CUDART_INF_F, -CUDART_INF_F, 0.f, 0.f)
                                     : make_float4(ref - base + (float)ex, ref, ldexpf(l, -ex), 0.f);
        }
#pragma unroll 1
        for (int b = 0; b < 8; ++b) {
          uint32_t x[16];
          __syncwarp();
          tmem_ld16(tO + 16 * b, x);
          tmem_wait_ld(x);
          if (live) {
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 y = make_float4(__uint_as_float(x[k]), __uint_as_float(x[k + 1]), __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
              if (whole) store4(a.out, a.dtype, row * D + 16 * b + k, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
              else *reinterpret_cast<float4*>(a.part_o + prow * D + 16 * b + k) = y;
            }
          }
        }
        __syncwarp();
        tc_fence_before();
      } else {  // no row of this tile: no more than a segment ahead of the tile that has rows
        ok = __all_sync(0xffffffffu, ok && pt_wait(&bars[TB_OLAST + t], seg & 1, abort, a.v.status));
        if (!ok) break;
      }
      n += s.k1 - s.k0;
      ++seg;
    } while (s.next(a));
  } else if (warp < 16) {
    // ==== expansion: warps 8-11 K, 12-15 V; eight lanes to a 128-byte row of codes, 16 rows at a time.  The codes of
    // the next step are loaded as this one's leave the registers.
    set_registers_down<PT_REG_EXPAND>();
    const int side = warp >= 12, e = tid & 127;
    // eight lanes that store together take four chunks of a row and the same four of the next one: the rows'
    // swizzles differ in their lowest bit, so that the eight never meet in a bank
    const int p8 = (e & 3) | ((e >> 1) & 4), r16 = ((e >> 2) & 1) | ((e >> 3) & 14);
    const int ch = p8 ^ (r16 & 7);  // the 16 coordinates that this thread's 16 bytes hold
    const uint32_t off0 = (uint32_t)(ch >> 2) * 16384 + r16 * 128 + (((2 * (ch & 3)) ^ (r16 & 7)) << 4), off1 = off0 ^ 16;
    const uint8_t* const codes = a.v.pool + side * TILE8_V + r16 * D + 16 * p8;
    uint8_t* const tiles = smem + (side ? SM::v : SM::k);
    uint64_t* const full = &bars[side ? TB_VFULL : TB_KFULL];
    uint64_t* const freed = &bars[side ? TB_VFREE : TB_KFREE];
    uint4 u[8];
    int4 rec;
    int keys;
    bool ok = true;
    auto where = [&](uint32_t m) {  // step m's records
      ok = ok && pt_wait(&bars[TB_LFULL + (m & 3)], (m >> 2) & 1, abort, a.v.status);
      ok = __all_sync(0xffffffffu, ok);
      rec = reinterpret_cast<const int4*>(smem + SM::rec)[m & 3];
      keys = ok ? reinterpret_cast<const int*>(smem + SM::keys)[m & 3] : 0;
    };
    auto load = [&](int j) {
      const int r = j < 2 ? rec.x : j < 4 ? rec.y : j < 6 ? rec.z : rec.w;
      u[j] = make_uint4(0, 0, 0, 0);
      if (r >= 0 && 16 * j + r16 < keys) u[j] = ld_stream(codes + (size_t)r * TILE8_BYTES + 16 * D * (j & 1));
    };
    where(0);
#pragma unroll
    for (int j = 0; j < 8; ++j) load(j);
    if (lane == 0) mbar_arrive(&bars[TB_LFREE]);
    for (uint32_t n = 0; ok && keys; ++n) {
      where(n + 1);
      if (!ok) break;
      ok = __all_sync(0xffffffffu, pt_wait(&freed[n & 1], ((n >> 1) & 1) ^ 1, abort, a.v.status));
      if (!ok) break;
      uint8_t* const dst = tiles + 32768 * (n & 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint4 x, y;
        codes4_to_half2x2<CODE>(u[j].x, x.x, x.y);
        codes4_to_half2x2<CODE>(u[j].y, x.z, x.w);
        codes4_to_half2x2<CODE>(u[j].z, y.x, y.y);
        codes4_to_half2x2<CODE>(u[j].w, y.z, y.w);
        load(j);
        *reinterpret_cast<uint4*>(dst + off0 + 2048 * j) = x;
        *reinterpret_cast<uint4*>(dst + off1 + 2048 * j) = y;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[n & 1]);
        mbar_arrive(&bars[TB_LFREE + ((n + 1) & 3)]);
      }
    }
  } else {
    set_registers_down<PT_REG_MMA>();
    if (warp == 17) {
      // ==== where the records of each step are, and their scales; lane b < 4: record b
      const int page_tiles = a.v.page_size / TILE_TOKENS;
      float base = 0.f, least = CUDART_INF_F, most = -CUDART_INF_F;  // of the segment's log2 of V scales
      bool based = false;                                            // the segment has had a record
      bool more = true;
      int step = s.k0;
      for (uint32_t n = 0; more; ++n) {
        if (!__all_sync(0xffffffffu, pt_wait(&bars[TB_LFREE + (n & 3)], ((n >> 2) & 1) ^ 1, abort, a.v.status))) break;
        const int at = (PT_BN / TILE_TOKENS) * step + lane, keys = s.x.kv_end - PT_BN * step;
        int rec = -1;
        float2 sc = make_float2(0.f, 0.f);
        if (lane < 4 && TILE_TOKENS * lane < keys) {
          const int idx = at / page_tiles;
          int page = s.x.b;
          if (a.v.block_table) page = idx < a.v.max_pages ? a.v.block_table[(size_t)s.x.b * a.v.max_pages + idx] : -1;
          if (page >= 0 && page < a.v.n_pages) {
            rec = (page * Hkv + s.kvh) * page_tiles + at % page_tiles;
            sc = *reinterpret_cast<const float2*>(a.v.pool + (size_t)rec * TILE8_BYTES + TILE8_SCALES);
            if (!written8(sc)) rec = -1;  // nor are its codes read: they may be NaN
          }
          if (rec < 0 && a.v.status) atomicOr(a.v.status, IQ_DEVERR_PAGE);
        }
        const bool there = rec >= 0;
        // log2 in two parts: exact for a power of two
        const float lv = there ? (float)((int)(__float_as_uint(sc.y) >> 23) - 127) +
                                     log2f(__uint_as_float((__float_as_uint(sc.y) & 0x7FFFFFu) | 0x3F800000u))
                               : __uint_as_float(0x7FC00000u);
        if (step == s.k0) based = false;
        if (const uint32_t m = __ballot_sync(0xffffffffu, there); m && !based) {
          base = __shfl_sync(0xffffffffu, lv, __ffs(m) - 1) + PT_BASE;
          based = true;
        }
        // p' below 2^-126 is 0, and with it the key's share of the row's sum: of scales within 2^104 of each other (a block
        // of zeros has 2^-100) only keys of weights below 2^-30 are lost so
        if (step == s.k0) {
          least = CUDART_INF_F;
          most = -CUDART_INF_F;
        }
        if (there) {
          least = fminf(least, lv);
          most = fmaxf(most, lv);
        }
        float up = most, down = least;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
          down = fminf(down, __shfl_xor_sync(0xffffffffu, down, o));
        }
        if (lane == 0 && up - down > 104.f && a.v.status) atomicOr(a.v.status, IQ_DEVERR_RANGE);
        if (lane < 4) {
          const int i = 4 * (n & 7) + lane;
          reinterpret_cast<float*>(smem + SM::ks)[i] = sc.x;
          reinterpret_cast<float*>(smem + SM::lv)[i] = lv;
          reinterpret_cast<float*>(smem + SM::w)[i] = there ? fast_exp2(base - lv) : 0.f;
          reinterpret_cast<int*>(smem + SM::rec)[4 * (n & 3) + lane] = rec;
          if (lane == 0) {
            reinterpret_cast<float*>(smem + SM::base)[n & 7] = base;
            reinterpret_cast<int*>(smem + SM::keys)[n & 3] = keys;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[TB_LFULL + (n & 3)]);
        if (++step == s.k1) {
          more = s.next(a);
          step = s.k0;
        }
        if (!more) {  // the run's end, for the expansion
          ++n;
          if (!__all_sync(0xffffffffu, pt_wait(&bars[TB_LFREE + (n & 3)], ((n >> 2) & 1) ^ 1, abort, a.v.status))) break;
          if (lane == 0) {
            reinterpret_cast<int*>(smem + SM::keys)[n & 3] = 0;
            mbar_arrive(&bars[TB_LFULL + (n & 3)]);
          }
        }
      }
    } else if (warp == 16 || warp == 18) {
      // ==== MMAs of tile t, a warp for each: what one waits for does not hold up the other, whose MMAs the tensor core
      // has meanwhile.  The tensor core takes its operands' descriptors from uniform registers: a warp runs as one, on
      // counts that are broadcast and in loops without an early end (where a wait has given up the others do too, soon,
      // and what is computed then is nobody's), so that the compiler keeps them there.  With descriptors from one
      // lane's registers an MMA took about 94 cycles to issue, not 52.
      const uint32_t idS = umma_idesc_f16(128, 64), idO = umma_idesc_f16(128, 128) | UMMA_B_MN_MAJOR;
      const int t = __shfl_sync(0xffffffffu, (int)(warp == 18), 0);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sm = __shfl_sync(0xffffffffu, smem_addr(smem), 0);
      const uint32_t tS = tm + PT_S_COL + 128 * t, tO = tm + PT_O_COL + 128 * t;
      const uint64_t dq = umma_sdesc_sw128(sm + SM::q + 32768 * t), dk = umma_sdesc_sw128(sm + SM::k),
                     dv = umma_sdesc_sw128_mn(sm + SM::v, 128);
      uint32_t n = 0, seg = 0, written = 0;  // steps, segments; half-steps of P
      auto wait = [&](int bar, uint32_t parity) {
        pt_wait(&bars[bar], parity & 1, abort, a.v.status);
        __syncwarp();
      };
      // scores of half-step h of step m: 64 keys, 8192 bytes of a buffer's blocks (512 descriptor units); buffers are 32 KB
      // (2048) apart
      auto scores = [&](uint32_t m, int h) {
        umma_f16_k128(tS + 64 * h, dq, dk + 2048 * (m & 1) + 512 * h, idS);
        umma_commit(&bars[TB_SFULL + 2 * t + h]);
      };
      bool more = true;
      do {
        const bool rows = __shfl_sync(0xffffffffu, (int)(s.x.n_live * G > PT_TILE * t), 0);  // of this tile, in the block
        const int steps = __shfl_sync(0xffffffffu, s.k1 - s.k0, 0);
        if (t == 0 && lane == 0) {  // where the block is cut, for the merge
          int2* const cut = a.cut + (size_t)s.e * Hkv + s.kvh;
          if (s.k0 == 0) cut->x = 2 * c + (s.pos == 0 ? 0 : 1);
          if (s.k1 == s.x.steps) cut->y = c;
        }
        wait(TB_Q, seg);
        wait(TB_KFULL + (n & 1), n >> 1);
        tc_fence_after();
        if (elect_one()) {
          if (rows) {
            scores(n, 0);
            scores(n, 1);
          }
          umma_commit(&bars[TB_KFREE + (n & 1)]);
        }
        __syncwarp();
        // a step's half-steps b: O += P V, then the scores of the next step's half b into the columns that P leaves
        for (int i = 0; i < steps; ++i, ++n) {
          const bool last = i + 1 == steps;
          wait(TB_VFULL + (n & 1), n >> 1);
          if (!last) wait(TB_KFULL + ((n + 1) & 1), (n + 1) >> 1);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (rows) {
              wait(TB_PFULL + 2 * t + b, written >> 1);
              ++written;
              tc_fence_after();
            }
            if (elect_one()) {
              if (rows) {
                umma_f16_ts_k64(tO, tS + 64 * b, dv + 2048 * (n & 1) + 512 * b, idO, i + b > 0);
                if (!last) scores(n + 1, b);
              }
              if (last) umma_commit(&bars[(b ? TB_OLAST : TB_ODONE) + t]);
              if (b) {
                umma_commit(&bars[TB_VFREE + (n & 1)]);
                if (!last) umma_commit(&bars[TB_KFREE + ((n + 1) & 1)]);
              }
            }
            __syncwarp();
          }
        }
        ++seg;
        more = __shfl_sync(0xffffffffu, (int)s.next(a), 0);
      } while (more);
      if (elect_one()) umma_commit(&bars[TB_DRAIN]);  // every MMA issued is complete before tensor memory is released
      __syncwarp();
      mbar_wait(&bars[TB_DRAIN], 0, nullptr);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_free(tmem, 512);
}

// Merge of the blocks that were cut: a warp takes four rows at a time, their partials in order.  Bound by the partials'
// reading; four rows' loads in flight a warp (one row's: 24 us for the 2048-token chunk's 147 cut blocks).
constexpr int PTM_WARPS = 8, PTM_ROWS = 4, PTM_TIMES = 2;  // rows of a CTA: their product
static __global__ void __launch_bounds__(32 * PTM_WARPS) prefill8_merge_kernel(PtArgs a) {
  pdl_wait();
  const int Hkv = a.v.n_kv_heads, G = a.g_real;
  const int2 cut = a.cut[blockIdx.x];
  const int e = blockIdx.x / Hkv, kvh = blockIdx.x % Hkv;
  const PtEntry x = pt_entry(a, e);
  const int lane = threadIdx.x & 31, rows = x.n_live * G;
  if (rows == 0) return;
  // (clamped: after a timeout they may not have been written)
  const int first = max(0, min(2 * a.ctas - 1, cut.x)), c0 = first >> 1, c1 = max(c0, min(a.ctas - 1, cut.y));
  if (c0 == c1) return;
#pragma unroll 1
  for (int i = 0; i < PTM_TIMES; ++i) {
    const int r0 = ((blockIdx.y * PTM_TIMES + i) * PTM_WARPS + (threadIdx.x >> 5)) * PTM_ROWS;
    if (r0 >= rows) return;
    float M[PTM_ROWS], MO[PTM_ROWS], L[PTM_ROWS];
    float4 o[PTM_ROWS];
#pragma unroll
    for (int j = 0; j < PTM_ROWS; ++j) {
      M[j] = MO[j] = -CUDART_INF_F;
      L[j] = 0.f;
      o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k = c0; k <= c1; ++k) {
      const size_t slot = (size_t)(k == c0 ? first : 2 * k) * PT_ROWS + r0;
      float4 ml[PTM_ROWS], y[PTM_ROWS];
#pragma unroll
      for (int j = 0; j < PTM_ROWS; ++j) {  // (rows behind the block's last, up to a tile's end, hold neutral partials)
        const bool live = r0 + j < rows;
        ml[j] = live ? a.part_ml[slot + j] : make_float4(0.f, 0.f, 0.f, 0.f);
        y[j] = live ? reinterpret_cast<const float4*>(a.part_o + (slot + j) * D)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < PTM_ROWS; ++j) {
        if (ml[j].z == 0.f) continue;
        const float m = fmaxf(M[j], ml[j].x), mo = fmaxf(MO[j], ml[j].y);
        const float fl = M[j] == -CUDART_INF_F ? 0.f : fast_exp2(M[j] - m), fo = MO[j] == -CUDART_INF_F ? 0.f : fast_exp2(MO[j] - mo);
        const float wl = fast_exp2(ml[j].x - m), wo = fast_exp2(ml[j].y - mo);
        L[j] = L[j] * fl + ml[j].z * wl;
        o[j] = make_float4(o[j].x * fo + y[j].x * wo, o[j].y * fo + y[j].y * wo, o[j].z * fo + y[j].z * wo, o[j].w * fo + y[j].w * wo);
        M[j] = m;
        MO[j] = mo;
      }
    }
#pragma unroll
    for (int j = 0; j < PTM_ROWS; ++j) {
      const int r = r0 + j;
      if (r >= rows) break;
      // (of a long context whose V scales are the smallest the factor itself is below float32's numbers)
      const float f = L[j] > 0.f ? fast_exp2(MO[j] - M[j] + 32.f) / L[j] : (L[j] == L[j] ? 0.f : L[j]), g = 0x1p-32f;
      const size_t row = ((size_t)x.b * a.n_tok + x.tok0 + r / G) * a.n_q_heads + (size_t)kvh * G + r % G;
      store4(a.out, a.dtype, row * D + 4 * lane, make_float4(o[j].x * f * g, o[j].y * f * g, o[j].z * f * g, o[j].w * f * g));
    }
  }
}

struct PtPlan {
  int tq, n_blk, ctas;
  size_t cut_bytes, bytes;
};
inline PtPlan pt_plan(int batch, int n_tok, int g, int n_kv_heads, int max_ctx) {
  PtPlan p;
  p.tq = PT_ROWS / g;
  p.n_blk = (n_tok + p.tq - 1) / p.tq;
  const long long steps = (long long)batch * p.n_blk * n_kv_heads * ((max_ctx + PT_BN - 1) / PT_BN);
  p.ctas = (int)std::max(1ll, std::min((long long)sm_count(), steps));
  p.cut_bytes = ((size_t)batch * p.n_blk * n_kv_heads * sizeof(int2) + 255) & ~(size_t)255;
  p.bytes = p.cut_bytes + 2 * (size_t)p.ctas * PT_ROWS * (sizeof(float4) + D * sizeof(float));
  return p;
}

inline int launch_prefill8_tc(const View8& v, const void* q, int dtype, int batch, int n_tok, int n_q_heads,
                              const int32_t* start, const int32_t* n_valid, int max_ctx, float scale, void* out,
                              void* workspace, void* stream) {
  PtArgs a;
  a.v = v;
  a.q = q;
  a.dtype = dtype;
  a.batch = batch;
  a.n_tok = n_tok;
  a.n_q_heads = n_q_heads;
  a.g_real = n_q_heads / v.n_kv_heads;
  const PtPlan p = pt_plan(batch, n_tok, a.g_real, v.n_kv_heads, max_ctx);
  a.tq = p.tq;
  a.n_blk = p.n_blk;
  a.ctas = p.ctas;
  a.max_ctx = max_ctx;
  a.start = start;
  a.n_valid = n_valid;
  a.scale = scale;
  a.out = out;
  uint8_t* w = (uint8_t*)workspace;
  a.cut = (int2*)w;
  a.part_ml = (float4*)(w + p.cut_bytes);
  a.part_o = (float*)(w + p.cut_bytes + 2 * (size_t)p.ctas * PT_ROWS * sizeof(float4));
  auto fn = v.code == IQ_E4M3 ? prefill8_tc_kernel<IQ_E4M3> : prefill8_tc_kernel<IQ_S8>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, PtSmem::bytes);
  if (e != cudaSuccess) return (int)e;
  e = launch_pdl(fn, dim3(p.ctas), dim3(PT_THREADS), PtSmem::bytes, (cudaStream_t)stream, a);
  if (e != cudaSuccess || p.ctas == 1) return (int)e;
  const int rows = std::min(n_tok, p.tq) * a.g_real, per = PTM_WARPS * PTM_ROWS * PTM_TIMES;
  return (int)launch_pdl(prefill8_merge_kernel, dim3((unsigned)(batch * p.n_blk * v.n_kv_heads), (rows + per - 1) / per),
                         dim3(32 * PTM_WARPS), 0, (cudaStream_t)stream, a);
}

}  // namespace iq
