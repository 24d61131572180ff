// Quantise-and-append into the 8-bit cache, and its read-back.
//
// One warp owns the K or the V half of one tile record (32 tokens of one sequence and kv head) that
// gets new tokens: it finds the largest finite magnitude, hence the block's scale; re-rounds the codes
// of the tokens that were there if the scale grew; writes the new tokens' codes.  Powers of two
// (e4m3) and scales of 8 significant bits (int8) make every quotient below correctly rounded, so that
// the result does not depend on how the tokens were split over calls, apart from that re-rounding.
// Bound by memory, 512 B in and 257 B out for each token and kv head: 32768 tokens of 8 kv heads, bf16 to int8, in 33 to
// 36 us, 87-94% of the copy rate; one token of 16 sequences in 6, a chain of dependent loads.
#include <math_constants.h>

#include <type_traits>

#include "iq_cache8.cuh"

namespace iq {

constexpr int AP8_WARPS = 4;

struct Append8Args {
  View8 v;
  const void *k, *v_new;
  long long ks, vs;  // elements from a token's row to the next
  int batch, n_new, tiles;  // tiles: the most that n_new tokens can touch
  const int32_t* start;
  const int32_t* n_valid;
};

// The scale that a block with largest magnitude amax (float32 bits, finite) asks for.
template <int CODE>
__device__ __forceinline__ float scale_for(uint32_t amax) {
  if constexpr (CODE == IQ_E4M3) {
    // amax <= 448 2^e = 1.75 * 2^(8 + e): e = exponent - 8, one more above a mantissa of 1.75
    int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = amax < 0x00800000u ? -100 : max(-100, min(120, e));
    return __uint_as_float((uint32_t)(e + 127) << 23);
  } else {
    const float s = fmaxf(__fdiv_rn(__uint_as_float(amax), 127.f), 7.888609052210118e-31f);  // 2^-100
    return __uint_as_float((__float_as_uint(s) + 0xFFFFu) & 0xFFFF0000u);
  }
}

// Codes of eight values as two words; NaN -> 0, saturating.
//   e4m3: the product with a power of two is exact, the conversion the one rounding.
//   int8: q = x (1 / s), its remainder x - q s and q + remainder (1 / s), each rounded once, give the correctly rounded
//   quotient (Markstein, 1990: 1 / s correctly rounded, q within one unit in the last place); adding 1.5 2^23 rounds that
//   to the nearest integer, ties to even, in the low byte.  (The compiler's division for each value took 1.7 times as long
//   for the whole call.)
template <int CODE, bool ODD>
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float scale, float inv) {
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = !ODD || fabsf(x[k]) < CUDART_INF_F ? x[k] : 0.f;  // ODD: NaN or infinities among them
  uint32_t o[2];
  if constexpr (CODE == IQ_E4M3) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[k] *= inv;
      if (ODD && fabsf(x[k]) == CUDART_INF_F) y[k] = copysignf(448.f, x[k]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm("{\n .reg .b16 t, u;\n cvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 u, %4, %3;\n mov.b32 %0, {t, u};\n}\n"
          : "=r"(o[h])
          : "f"(y[4 * h]), "f"(y[4 * h + 1]), "f"(y[4 * h + 2]), "f"(y[4 * h + 3]));
  } else {
    uint32_t c[8];
    const uint64_t inv2 = f2(inv, inv), neg2 = f2(-scale, -scale), magic2 = f2(kMagicF, kMagicF);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {  // two values an instruction
      const uint64_t x2 = f2(y[k], y[k + 1]), q = mul2(x2, inv2);
      float a, b;
      f2s(add2(fma2(fma2(q, neg2, x2), inv2, q), magic2), a, b);
      c[k] = __float_as_uint(a);
      c[k + 1] = __float_as_uint(b);
    }
    // (127 scale in an infinity's place would itself be infinite beside float32's largest numbers)
    if (ODD) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (fabsf(x[k]) == CUDART_INF_F) c[k] = x[k] > 0.f ? 127u : (uint32_t)-127;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o[h] = prmt(prmt(c[4 * h], c[4 * h + 1], 0x0040u), prmt(c[4 * h + 2], c[4 * h + 3], 0x0040u), 0x5410u);
  }
  return make_uint2(o[0], o[1]);
}

// Eight values of one row as float32.
template <typename T>
__device__ __forceinline__ void widen8(const uint4& u, float f[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = a.x;
      f[2 * i + 1] = a.y;
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
  const uint32_t a = __float_as_uint(x) & 0x7FFFFFFFu;
  return a < 0x7F800000u ? a : 0u;
}

// Lanes 0-15 take row 2 i, lanes 16-31 row 2 i + 1, eight coordinates each: 16-byte loads (16-bit
// types) of whole 256-byte rows, 8-byte stores.
template <int CODE, typename T>
__global__ void __launch_bounds__(AP8_WARPS * 32) append8_kernel(Append8Args a) {
  pdl_wait();
  const int lane = threadIdx.x & 31, c8 = lane & 15, odd = lane >> 4;
  // unit = ((sequence, tile), side, head), heads fastest: neighbouring warps read neighbouring rows
  long long u = (long long)blockIdx.x * AP8_WARPS + (threadIdx.x >> 5);
  const int head = (int)(u % a.v.n_kv_heads);
  u /= a.v.n_kv_heads;
  const int side = (int)(u & 1);
  u >>= 1;
  const int j = (int)(u % a.tiles), b = (int)(u / a.tiles);
  const T* const x = (const T*)(side ? a.v_new : a.k);
  const long long stride = side ? a.vs : a.ks;
  if (b >= a.batch || !x) return;
  int cnt = a.n_valid ? a.n_valid[b] : a.n_new;
  uint32_t err = 0;
  if (cnt < 0 || cnt > a.n_new) {
    err |= IQ_DEVERR_CTX;
    cnt = cnt < 0 ? 0 : a.n_new;
  }
  const long long start = a.start[b];
  const long long t0 = ((start >> 5) + j) * TILE_TOKENS;  // position of the tile's first slot
  const long long first = max(start, t0), end = min(start + cnt, t0 + TILE_TOKENS);
  int page = -1;
  if (first < end) page = find_page8(a.v, b, t0, &err);
  if (err && a.v.status && lane == 0) atomicOr(a.v.status, err);
  if (page < 0) return;
  uint8_t* const rec = tile_record8(a.v, page, head, (int)(t0 % a.v.page_size));
  uint8_t* const rows = rec + side * TILE8_V;
  float* const sc = reinterpret_cast<float*>(rec + TILE8_SCALES) + side;
  const int lo = (int)(first - t0), hi = (int)(end - t0);  // the new tokens' rows
  const T* const src = x + ((long long)b * a.n_new + (t0 - start)) * stride + head * D + 8 * c8;

  // f(i) of the rows 2 i + odd that are new.
  const bool all = lo == 0 && hi == TILE_TOKENS;
  auto each = [&](auto f) {
    if (all) {
#pragma unroll 8
      for (int i = 0; i < TILE_TOKENS / 2; ++i) f(i);
    } else {
#pragma unroll 1
      for (int i = lo >> 1; 2 * i + odd < hi; ++i)
        if (2 * i + odd >= lo) f(i);
    }
  };
  // Two passes over the rows.  A warp's rows of a 16-bit type, 8 KB, are copied to shared memory, all of them in flight at
  // once; a lane reads back what it copied.  (Loads to registers, and from L1 again, which 40 warps' rows do not fit: 53 us
  // for the 32K prompt.)  First the largest magnitude, of 16-bit types two at a time.
  constexpr bool WIDE = sizeof(T) == 4;
  __shared__ uint4 s_rows[WIDE ? 1 : AP8_WARPS][WIDE ? 1 : TILE_TOKENS * D / 8];
  uint4* const held = s_rows[WIDE ? 0 : threadIdx.x >> 5] + (WIDE ? 0 : lane);
  auto get = [&](int i, float f[8]) {
    if constexpr (WIDE) {
      const float4* const p = reinterpret_cast<const float4*>(src + (2 * i + odd) * stride);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
      widen8<T>(held[32 * i], f);
    }
  };
  uint32_t amax = 0;
  bool odd_values = false;  // a NaN or an infinity
  if constexpr (!WIDE) {
    each([&](int i) { copy16_async(held + 32 * i, src + (2 * i + odd) * stride); });
    asm volatile("cp.async.wait_all;" ::: "memory");
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    auto larger = [](uint32_t x, uint32_t y) {  // of two pairs of magnitudes; NaN wins
      const T2 z = __hmax2_nan(*reinterpret_cast<const T2*>(&x), *reinterpret_cast<const T2*>(&y));
      return *reinterpret_cast<const uint32_t*>(&z);
    };
    uint32_t m = 0;
    each([&](int i) {
      const uint4 u = held[32 * i];
      m = larger(m, larger(larger(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), larger(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
    });
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    constexpr bool half = std::is_same<T, __half>::value;
    odd_values = m >= (half ? 0x7C00u : 0x7F80u);
    amax = half ? __float_as_uint(__half2float(__ushort_as_half((uint16_t)m))) : m << 16;
  }
  if (WIDE || odd_values) {
    amax = 0;
    each([&](int i) {
      float f[8];
      get(i, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        odd_values |= !(fabsf(f[k]) < CUDART_INF_F);
        amax = max(amax, finite_magnitude(f[k]));
      }
    });
    odd_values = __any_sync(0xffffffffu, odd_values);
    amax = __reduce_max_sync(0xffffffffu, amax);
  }
  float scale = scale_for<CODE>(amax);
  float was = lo > 0 ? *sc : 0.f;  // tokens before the new ones: their scale stays or grows
  was = was > 0.f && was < CUDART_INF_F ? was : 0.f;
  const bool grew = lo > 0 && scale > was;
  if (lo > 0 && !grew) scale = was;
  const float inv = 1.f / scale;  // (e4m3: exact, a power of two)
  __syncwarp();
  if (lane == 0) *sc = scale;
  if (grew) {
    for (int r = odd; r < lo; r += 2) {
      uint2* p = reinterpret_cast<uint2*>(rows + chunk8(r, c8 >> 1) + 8 * (c8 & 1));
      const uint2 w = *p;
      uint32_t h[4];
      codes4_to_half2x2<CODE>(w.x, h[0], h[1]);
      codes4_to_half2x2<CODE>(w.y, h[2], h[3]);
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
        f[2 * k] = g.x * was;
        f[2 * k + 1] = g.y * was;
      }
      *p = quantise8<CODE, true>(f, scale, inv);  // (slots that held nothing may be NaN codes)
    }
  }
  auto write = [&](auto odd_c) {
    each([&](int i) {
      float f[8];
      get(i, f);
      *reinterpret_cast<uint2*>(rows + chunk8(2 * i + odd, c8 >> 1) + 8 * (c8 & 1)) =
          quantise8<CODE, decltype(odd_c)::value>(f, scale, inv);
    });
  };
  if (odd_values) write(std::true_type());
  else write(std::false_type());
}

int launch_append8(const View8& v, const void* k, const void* vsrc, int dtype, long long ks, long long vs, int batch, int n_new,
                   const int32_t* start, const int32_t* n_valid, void* stream) {
  if (batch == 0 || n_new == 0) return 0;
  Append8Args a;
  a.v = v;
  a.k = k;
  a.v_new = vsrc;
  a.ks = ks;
  a.vs = vs;
  a.batch = batch;
  a.n_new = n_new;
  a.tiles = (int)(((long long)n_new + 2 * TILE_TOKENS - 2) / TILE_TOKENS);
  a.start = start;
  a.n_valid = n_valid;
  const long long units = (long long)batch * a.tiles * 2 * v.n_kv_heads;
  const long long blocks = (units + AP8_WARPS - 1) / AP8_WARPS;
  if (blocks > 0x7FFFFFFFll) return (int)cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(AP8_WARPS * 32);
  const cudaStream_t st = (cudaStream_t)stream;
  const bool e4 = v.code == IQ_E4M3;
  if (dtype == IQ_F16)
    return (int)(e4 ? launch_pdl(append8_kernel<IQ_E4M3, __half>, grid, block, 0, st, a)
                    : launch_pdl(append8_kernel<IQ_S8, __half>, grid, block, 0, st, a));
  if (dtype == IQ_BF16)
    return (int)(e4 ? launch_pdl(append8_kernel<IQ_E4M3, __nv_bfloat16>, grid, block, 0, st, a)
                    : launch_pdl(append8_kernel<IQ_S8, __nv_bfloat16>, grid, block, 0, st, a));
  return (int)(e4 ? launch_pdl(append8_kernel<IQ_E4M3, float>, grid, block, 0, st, a)
                  : launch_pdl(append8_kernel<IQ_S8, float>, grid, block, 0, st, a));
}

// One thread per (kv head, token, 16-byte chunk): code * scale.
__global__ void export8_kernel(View8 v, int kv, int seq, int t0, int n, float* values) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int tok = (int)(i >> 3), c = (int)(i & 7), head = blockIdx.y;
  if (i >= 8ll * n) return;
  uint32_t err = 0;
  const long long pos = (long long)t0 + tok;
  const int page = find_page8(v, seq, pos, &err);
  float* const out = values + ((size_t)head * n + tok) * D + 16 * c;
  if (page < 0) {
    if (v.status) atomicOr(v.status, err);
    for (int k = 0; k < 16; ++k) out[k] = __uint_as_float(0x7FC00000u);
    return;
  }
  const int slot = (int)(pos % v.page_size);
  const uint8_t* rec = tile_record8(v, page, head, slot);
  const float sc = reinterpret_cast<const float*>(rec + TILE8_SCALES)[kv];
  const uint8_t* p = rec + kv * TILE8_V + chunk8(slot % TILE_TOKENS, c);
  for (int k = 0; k < 16; k += 4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p + k);
    uint32_t x, y;
    if (v.code == IQ_E4M3) codes4_to_half2x2<IQ_E4M3>(w, x, y);
    else codes4_to_half2x2<IQ_S8>(w, x, y);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&y));
    out[k] = f.x * sc; out[k + 1] = f.y * sc; out[k + 2] = g.x * sc; out[k + 3] = g.y * sc;
  }
}

int launch_export8(const View8& v, int kv, int seq, int t0, int n, float* values, void* stream) {
  if (n == 0) return 0;
  const dim3 grid((unsigned)(((long long)n * 8 + 127) / 128), v.n_kv_heads);
  export8_kernel<<<grid, 128, 0, (cudaStream_t)stream>>>(v, kv, seq, t0, n, values);
  return (int)cudaGetLastError();
}

}  // namespace iq
