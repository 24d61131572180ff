// Rotary positions: (x0, x1) -> mscale (x0 cos a - x1 sin a, x0 sin a + x1 cos a), a = position * freq.
//
// One CTA per token: its threads first start the loads of the token's heads, then find the token's
// rotary_dim / 2 sines and cosines once for all heads (the angle in turns, reduced to [-1/2, 1/2] in
// double; sine and cosine of that fraction in float32, whose rounding is at most 2^-26 of a turn, 1e-7 rad:
// float32 outputs are 1.3 times as far from 64 bits as with float64 sines), then turn what they loaded.  A
// thread owns whole pairs, so that a call may work in place.  Bound by memory: every value read once and written once.
// 8192 tokens of 40 heads in 16 bits: 29 us, 91% of the copy rate (48 with the angles before the loads); 16 tokens: 5.6 us,
// latency.
#include <algorithm>

#include "iq_cache8.cuh"

namespace iq {

constexpr int ROPE_THREADS = 256;

template <int DT>
struct RopeVec {  // eight values in 16-byte registers
  uint4 w[DT == IQ_F32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ RopeVec<DT> rope_load(const void* base, long long i) {
  RopeVec<DT> r;
  const uint4* p = reinterpret_cast<const uint4*>((const uint8_t*)base + i * (DT == IQ_F32 ? 4 : 2));
  r.w[0] = p[0];
  if constexpr (DT == IQ_F32) r.w[1] = p[1];
  return r;
}
template <int DT>
__device__ __forceinline__ void rope_store(void* base, long long i, const RopeVec<DT>& r) {
  uint4* p = reinterpret_cast<uint4*>((uint8_t*)base + i * (DT == IQ_F32 ? 4 : 2));
  p[0] = r.w[0];
  if constexpr (DT == IQ_F32) p[1] = r.w[1];
}
template <int DT>
__device__ __forceinline__ void rope_widen(const RopeVec<DT>& r, float f[8]) {
  if constexpr (DT == IQ_F32) {
    const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(u[k]);
  } else {
    const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == IQ_F16) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
        f[2 * k] = a.x;
        f[2 * k + 1] = a.y;
      } else {
        f[2 * k] = __uint_as_float(u[k] << 16);
        f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
      }
    }
  }
}
template <int DT>
__device__ __forceinline__ RopeVec<DT> rope_narrow(const float f[8]) {
  RopeVec<DT> r;
  if constexpr (DT == IQ_F32) {
    r.w[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    r.w[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  } else {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == IQ_F16) {
        const __half2 a = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
        u[k] = *reinterpret_cast<const uint32_t*>(&a);
      } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        u[k] = *reinterpret_cast<const uint32_t*>(&a);
      }
    }
    r.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
  }
  return r;
}
template <int DT>
__device__ __forceinline__ float rope_get(const void* base, long long i) {
  if constexpr (DT == IQ_F32) return ((const float*)base)[i];
  if constexpr (DT == IQ_F16) return __half2float(((const __half*)base)[i]);
  return __uint_as_float((uint32_t)((const uint16_t*)base)[i] << 16);
}
template <int DT>
__device__ __forceinline__ void rope_put(void* base, long long i, float f) {
  if constexpr (DT == IQ_F32) ((float*)base)[i] = f;
  else if constexpr (DT == IQ_F16) ((__half*)base)[i] = __float2half_rn(f);
  else ((__nv_bfloat16*)base)[i] = __float2bfloat16_rn(f);
}

__device__ __forceinline__ void rope_angles(const RopeArgs& a, int n, float2* cs) {
  const double at = a.pos[n];
  for (int i = threadIdx.x; i < a.rd / 2; i += ROPE_THREADS) {
    double t = at * a.freq[i] * 0.15915494309189535;  // 1 / (2 pi): turns
    t -= rint(t);
    float s, c;
    sincospif(2.f * (float)t, &s, &c);
    cs[i] = make_float2(c * a.mscale, (a.inverse ? -s : s) * a.mscale);
  }
}

// LAYOUT interleaved: an item is eight neighbouring coordinates (four pairs).  LAYOUT half (rotary_dim / 2 a
// multiple of 8): an item is eight coordinates of the first half and their partners; behind the rotary part an item
// is eight coordinates to copy.  A thread's items are loaded four at a time, the first four before the angles.
template <int DT, int LAYOUT>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(RopeArgs a) {
  constexpr int U = 4;
  __shared__ float2 cs[D / 2];
  pdl_wait();
  const int n = blockIdx.x, half = a.rd / 2;
  const int turn = LAYOUT == IQ_ROPE_HALF ? half / 8 : D / 8;               // items of a head that turn
  const int items = LAYOUT == IQ_ROPE_HALF ? turn + (D - a.rd) / 8 : turn;  // and all of them
  const int nq = a.heads[0] * items, total = nq + a.heads[1] * items;
  const uint8_t* const xq = (const uint8_t*)a.x[0] + n * a.xs[0] * (DT == IQ_F32 ? 4 : 2);
  const uint8_t* const xk = (const uint8_t*)a.x[1] + n * a.xs[1] * (DT == IQ_F32 ? 4 : 2);
  uint8_t* const yq = (uint8_t*)a.y[0] + n * a.ys[0] * (DT == IQ_F32 ? 4 : 2);
  uint8_t* const yk = (uint8_t*)a.y[1] + n * a.ys[1] * (DT == IQ_F32 ? 4 : 2);
  for (int i0 = threadIdx.x; i0 < total || i0 == threadIdx.x; i0 += U * ROPE_THREADS) {
    RopeVec<DT> u[U], w[LAYOUT == IQ_ROPE_HALF ? U : 1];
    int at[U];  // the item's first coordinate in its head, its head's place added
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j * ROPE_THREADS, k = i >= nq, h = (k ? i - nq : i) / items, it = (k ? i - nq : i) % items;
      at[j] = h * D + (LAYOUT == IQ_ROPE_HALF && it >= turn ? a.rd + 8 * (it - turn) : 8 * it);
      if (i >= total) continue;
      u[j] = rope_load<DT>(k ? xk : xq, at[j]);
      if (LAYOUT == IQ_ROPE_HALF && it < turn) w[LAYOUT == IQ_ROPE_HALF ? j : 0] = rope_load<DT>(k ? xk : xq, at[j] + half);
    }
    if (i0 == threadIdx.x) {
      rope_angles(a, n, cs);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j * ROPE_THREADS;
      if (i >= total) break;
      uint8_t* const y = i >= nq ? yk : yq;
      const int c = at[j] % D;
      if (LAYOUT == IQ_ROPE_HALF) {
        if (c < half) {
          RopeVec<DT>& v = w[LAYOUT == IQ_ROPE_HALF ? j : 0];
          float x0[8], x1[8];
          rope_widen<DT>(u[j], x0);
          rope_widen<DT>(v, x1);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 t = cs[c + k];
            const float p = x0[k] * t.x - x1[k] * t.y, q = x0[k] * t.y + x1[k] * t.x;
            x0[k] = p;
            x1[k] = q;
          }
          u[j] = rope_narrow<DT>(x0);
          rope_store<DT>(y, at[j] + half, rope_narrow<DT>(x1));
        }
      } else if (c < a.rd) {
        float x[8];
        rope_widen<DT>(u[j], x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (c + 2 * k >= a.rd) continue;
          const float2 t = cs[c / 2 + k];
          const float p = x[2 * k] * t.x - x[2 * k + 1] * t.y, q = x[2 * k] * t.y + x[2 * k + 1] * t.x;
          x[2 * k] = p;
          x[2 * k + 1] = q;
        }
        u[j] = rope_narrow<DT>(x);
      }
      rope_store<DT>(y, at[j], u[j]);
    }
  }
}

// Half layout with rotary_dim / 2 not a multiple of 8: the partners are not 16-byte aligned together, so a
// thread takes one pair, or one coordinate to copy, at a time.
template <int DT>
__global__ void __launch_bounds__(ROPE_THREADS) rope_pair_kernel(RopeArgs a) {
  __shared__ float2 cs[D / 2];
  pdl_wait();
  const int n = blockIdx.x, half = a.rd / 2, items = half + D - a.rd;
  rope_angles(a, n, cs);
  __syncthreads();
  for (int i = threadIdx.x; i < (a.heads[0] + a.heads[1]) * items; i += ROPE_THREADS) {
    int h = i / items;
    const int it = i % items;
    const int side = h >= a.heads[0];
    if (side) h -= a.heads[0];
    const long long src = n * a.xs[side] + h * D, dst = n * a.ys[side] + h * D;
    if (it >= half) {
      rope_put<DT>(a.y[side], dst + half + it, rope_get<DT>(a.x[side], src + half + it));
      continue;
    }
    const float x = rope_get<DT>(a.x[side], src + it), y = rope_get<DT>(a.x[side], src + half + it);
    const float2 t = cs[it];
    rope_put<DT>(a.y[side], dst + it, x * t.x - y * t.y);
    rope_put<DT>(a.y[side], dst + half + it, x * t.y + y * t.x);
  }
}

template <int DT>
static int launch_rope_t(const RopeArgs& a, cudaStream_t st) {
  const dim3 grid(a.n_tokens), block(ROPE_THREADS);
  if (a.layout == IQ_ROPE_INTERLEAVED) return (int)launch_pdl(rope_kernel<DT, IQ_ROPE_INTERLEAVED>, grid, block, 0, st, a);
  if (a.rd % 16 == 0) return (int)launch_pdl(rope_kernel<DT, IQ_ROPE_HALF>, grid, block, 0, st, a);
  return (int)launch_pdl(rope_pair_kernel<DT>, grid, block, 0, st, a);
}

int launch_rope(const RopeArgs& a, int dtype, void* stream) {
  if (a.n_tokens == 0 || a.heads[0] + a.heads[1] == 0) return 0;
  const cudaStream_t st = (cudaStream_t)stream;
  return dtype == IQ_F16 ? launch_rope_t<IQ_F16>(a, st) : dtype == IQ_BF16 ? launch_rope_t<IQ_BF16>(a, st) : launch_rope_t<IQ_F32>(a, st);
}

}  // namespace iq
