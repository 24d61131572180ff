// One warp's work on one 32-token tile of the 8-bit cache for up to eight query rows: scores, online
// softmax and value sums on binary16 tensor-core tiles (mma.sync m16n8k16, float32 sums).
//
// Codes are exact in binary16, so the only roundings are those of q and of the probabilities; both are
// taken as two binary16 terms (hi + lo, 22 bits), whose products the tensor core adds in float32.
//   S (heads x tokens) = Q K^T   A = q rows (hi in rows 0-7, lo in rows 8-15), B = K codes
//   O^T (coordinates x heads) += V^T P^T   A = V codes, token pairs side by side, B = P hi, then lo
// The coordinate order within a k-step of S, and the coordinate that a row of O^T stands for, are free:
// they are chosen so that every fragment comes from 16-byte shared-memory loads (lane (g, t) = (lane / 4,
// lane % 4)): K row 8 n + g, chunks 2 t and 2 t + 1; V rows 2 t (+ 1, + 8, + 9), chunk g.  The record's
// chunk swizzle makes these loads free of bank conflicts.
#pragma once
#include <math_constants.h>

#include "iq_cache8.cuh"

namespace iq {

constexpr int A8_ROWS = 8;  // query rows of a warp (the group's heads)
constexpr float kLog2E8 = 1.4426950408889634f;
// log2 of what probabilities and their sums are held times: times V's scale, in binary16, the largest is below 2^15 then, and
// weights 2^-17 of it still have 22 bits in their two terms, whose steps of 2^-24 are 2^-38 of it.
constexpr float A8_ABOVE = 14.f;

__device__ __forceinline__ void hmma8(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// Running softmax of row g (in log2 units) and the warp's value sums.  The values' block scales are
// folded into the probabilities: sums are of p * vs / 2^(mo - m), with a running maximum mo of (score +
// log2 of the block's scale) of its own, so that neither the scores' nor the scales' range matters.
struct Row8 {
  float m, mo, l;  // running maxima; this lane's share of the sum, times 2^14 as o is
  float o[8][4];   // o[i]: coordinates 16 g + 2 i (entries 0, 1) and + 1 (2, 3) of rows 2 t and 2 t + 1
};
__device__ __forceinline__ void row8_init(Row8& r) {
  r.m = r.mo = -CUDART_INF_F;
  r.l = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.o[i][0] = r.o[i][1] = r.o[i][2] = r.o[i][3] = 0.f;
}

// Q fragments of row g from the row's 128 values, of which this lane holds coordinates 32 t .. 32 t + 31
// (read with load4): scaled by the power of two that brings the largest magnitude to [2^14, 2^15), hi and
// lo binary16 terms; returns the factor from S to log2-unit scores, scale * log2(e) / that power.
__device__ __forceinline__ float load_q8(const void* q, int dtype, size_t row, bool live, float scale, uint32_t qa[8][4]) {
  const int t = threadIdx.x & 3;
  float4 x[8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = live ? load4(q, dtype, row * D + 32 * t + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w))));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // exponent of amax clamped, for zeros and infinities, so that both powers below are normal numbers
  int ex = (int)(__float_as_uint(amax) >> 23) - 127;
  ex = max(-100, min(127, ex));
  const float sig = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = x[i].x * sig, b = x[i].y * sig, c = x[i].z * sig, d = x[i].w * sig;
    qa[i][0] = half2_bits(a, b);
    qa[i][2] = half2_bits(c, d);
    const float2 ab = half2_floats(qa[i][0]), cd = half2_floats(qa[i][2]);
    qa[i][1] = half2_bits(a - ab.x, b - ab.y);
    qa[i][3] = half2_bits(c - cd.x, d - cd.y);
  }
  return scale * kLog2E8 * __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
}

// The tile at `tile` (shared memory) into r: row g sees the first `lim` tokens.  The codes of V rows that
// no row sees must be finite (zeroed by the caller).  FEW (at most four heads): rows 4-7 repeat rows 0-3 and carry the
// lo terms of P, so that one product does for both (48 instead of 64 MMAs a tile).
template <int CODE, bool FEW>
__device__ __forceinline__ void tile8(const uint8_t* tile, int lim, const uint32_t qa[8][4], float qs, Row8& r) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float ks = reinterpret_cast<const float*>(tile + TILE8_SCALES)[0] * qs;
  const uint32_t vsb = reinterpret_cast<const uint32_t*>(tile + TILE8_SCALES)[1];
  const float vexp = (float)((int)(vsb >> 23) - 127);                        // scale = 2^vexp * vman
  const float vman = __uint_as_float((vsb & 0x7FFFFFu) | 0x3F800000u);
  float s[8];
  float mx = -CUDART_INF_F;
  float d[4][4];
#pragma unroll
  for (int n = 0; n < 4; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
#pragma unroll
  for (int c = 0; c < 2; ++c) {  // the four token groups side by side: four independent chains of MMAs
    uint4 k[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) k[n] = *reinterpret_cast<const uint4*>(tile + chunk8(8 * n + g, 2 * t + c));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t b0, b1;
        codes4_to_half2x2<CODE>(i == 0 ? k[n].x : i == 1 ? k[n].y : i == 2 ? k[n].z : k[n].w, b0, b1);
        hmma8(d[n], qa[4 * c + i], b0, b1);
      }
  }
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s[2 * n + e] = 8 * n + 2 * t + e < lim ? (d[n][e] + d[n][2 + e]) * ks : -CUDART_INF_F;
      mx = fmaxf(mx, s[2 * n + e]);
    }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const float m = fmaxf(r.m, mx), mo = fmaxf(r.mo, mx + vexp);
  if (__any_sync(0xffffffffu, m > r.m || mo > r.mo)) {
    r.l *= r.m == -CUDART_INF_F ? 0.f : fast_exp2(r.m - m);
    const float f = r.mo == -CUDART_INF_F ? 0.f : fast_exp2(r.mo - mo);
    const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r.o[i][0] *= f0;
      r.o[i][1] *= f1;
      r.o[i][2] *= f0;
      r.o[i][3] *= f1;
    }
    r.m = m;
    r.mo = mo;
  }
  // p * vs / 2^(mo - m), below 2^15
  const float fac = mo == -CUDART_INF_F ? 0.f : fast_exp2(fminf(m + vexp - mo, 126.f)) * vman, at = m - A8_ABOVE;
  uint32_t ph[4], pl[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float p0 = s[2 * n] == -CUDART_INF_F ? 0.f : fast_exp2(s[2 * n] - at);
    const float p1 = s[2 * n + 1] == -CUDART_INF_F ? 0.f : fast_exp2(s[2 * n + 1] - at);
    r.l += p0 + p1;
    const float x0 = p0 * fac, x1 = p1 * fac;
    ph[n] = half2_bits(x0, x1);
    const float2 h = half2_floats(ph[n]);
    pl[n] = half2_bits(x0 - h.x, x1 - h.y);
    if (FEW && g >= 4) ph[n] = pl[n];
  }
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const int t0 = 16 * kk + 2 * t;
    const uint8_t* v = tile + TILE8_V;
    const uint4 u0 = *reinterpret_cast<const uint4*>(v + chunk8(t0, g)), u1 = *reinterpret_cast<const uint4*>(v + chunk8(t0 + 1, g));
    const uint4 u2 = *reinterpret_cast<const uint4*>(v + chunk8(t0 + 8, g)), u3 = *reinterpret_cast<const uint4*>(v + chunk8(t0 + 9, g));
    const uint32_t x0[4] = {u0.x, u0.y, u0.z, u0.w}, x1[4] = {u1.x, u1.y, u1.z, u1.w};
    const uint32_t x2[4] = {u2.x, u2.y, u2.z, u2.w}, x3[4] = {u3.x, u3.y, u3.z, u3.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // coordinates 16 g + 4 w .. + 3
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[4];
        const uint32_t sel = h ? 0x7362u : 0x5140u;  // bytes 2 h, 2 h + 1 of both tokens
        codes4_to_half2x2<CODE>(prmt(x0[w], x1[w], sel), a[0], a[1]);
        codes4_to_half2x2<CODE>(prmt(x2[w], x3[w], sel), a[2], a[3]);
        hmma8(r.o[2 * w + h], a, ph[2 * kk], ph[2 * kk + 1]);
        if (!FEW) hmma8(r.o[2 * w + h], a, pl[2 * kk], pl[2 * kk + 1]);
      }
    }
  }
}

// Zeroes V rows n .. 31 of a tile in shared memory (whole warp).
__device__ __forceinline__ void clear_v_rows8(uint8_t* tile, int n) {
  for (int i = threadIdx.x & 31; i < (TILE_TOKENS - n) * 8; i += 32)
    *reinterpret_cast<uint4*>(tile + TILE8_V + (n + (i >> 3)) * D + 16 * (i & 7)) = make_uint4(0, 0, 0, 0);
  __syncwarp();
}

// The warp's state into shared memory: (m, mo, l) per row, and rows of 128 sums (FEW: of four rows).
template <bool FEW>
__device__ __forceinline__ void row8_store(Row8& r, float (*ml)[4], float* so) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float l = r.l + __shfl_xor_sync(0xffffffffu, r.l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (t == 0) {
    ml[g][0] = r.m;
    ml[g][1] = r.mo;
    ml[g][2] = l;
  }
  if (FEW) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) r.o[i][e] += __shfl_xor_sync(0xffffffffu, r.o[i][e], 2);
    if (t >= 2) return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    *reinterpret_cast<float2*>(so + (2 * t) * D + 16 * g + 2 * i) = make_float2(r.o[i][0], r.o[i][2]);
    *reinterpret_cast<float2*>(so + (2 * t + 1) * D + 16 * g + 2 * i) = make_float2(r.o[i][1], r.o[i][3]);
  }
}

}  // namespace iq
