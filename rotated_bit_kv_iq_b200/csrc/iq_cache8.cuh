// The 8-bit cache: tile-record geometry, code <-> number conversions and value loads shared by the
// append, attention and export kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "iq_device.cuh"
#include "iq_internal8.h"

namespace iq {

__device__ __forceinline__ uint8_t* tile_record8(const View8& v, int page, int head, int slot) {
  return v.pool + (((size_t)page * v.n_kv_heads + head) * (v.page_size / TILE_TOKENS) + slot / TILE_TOKENS) *
                      (size_t)TILE8_BYTES;
}

// Page of position `pos` of sequence b, or -1 (with the status bit it flags in *err): a position
// outside the sequence's pages, or a table entry outside the pool.
__device__ __forceinline__ int find_page8(const View8& v, int b, long long pos, uint32_t* err) {
  const long long idx = pos / v.page_size;
  if (pos < 0 || idx >= v.max_pages) {
    *err |= IQ_DEVERR_POSITION;
    return -1;
  }
  const int page = v.block_table ? v.block_table[(size_t)b * v.max_pages + idx] : b;
  if (page < 0 || page >= v.n_pages) {
    *err |= IQ_DEVERR_PAGE;
    return -1;
  }
  return page;
}

// Whether a record's K and V scales are ones that an append leaves, positive finite numbers: otherwise it holds nothing.
__device__ __forceinline__ bool written8(float2 scales) {
  return __float_as_uint(scales.x) - 1u < 0x7F7FFFFFu && __float_as_uint(scales.y) - 1u < 0x7F7FFFFFu;
}

// Byte offset of 16-byte chunk c of row s within a tile's 4096 K (or V) bytes.
__device__ __forceinline__ int chunk8(int s, int c) { return s * D + ((c ^ (s & 7)) << 4); }

// Two codes (the low 16 bits of x) -> the binary16 numbers that they stand for; exact.
template <int CODE>
__device__ __forceinline__ uint32_t codes2_to_half2(uint32_t x) {
  uint32_t r;
  if constexpr (CODE == IQ_E4M3) {
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(x));
  } else {
    // byte + 128 into the low bits of 1024.0 (0x6400), less 1152
    const uint32_t y = prmt(x ^ 0x8080u, 0x64646464u, 0x4140u);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(0x6480)));
    r = *reinterpret_cast<const uint32_t*>(&h);
  }
  return r;
}
// Four codes -> two registers of two binary16 numbers, in order.
template <int CODE>
__device__ __forceinline__ void codes4_to_half2x2(uint32_t x, uint32_t& a, uint32_t& b) {
  if constexpr (CODE == IQ_E4M3) {
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
        : "=r"(a), "=r"(b)
        : "r"(x));
  } else {
    const uint32_t y = x ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));
    const uint32_t u = prmt(y, 0x64646464u, 0x4140u), w = prmt(y, 0x64646464u, 0x4342u);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), bias);
    const __half2 i = __hsub2(*reinterpret_cast<const __half2*>(&w), bias);
    a = *reinterpret_cast<const uint32_t*>(&h);
    b = *reinterpret_cast<const uint32_t*>(&i);
  }
}

// Four values starting at p (16-byte aligned for float, 8-byte for 16-bit types) as float32.
__device__ __forceinline__ float4 load4(const void* base, int dtype, size_t i) {
  if (dtype == IQ_F32) return *reinterpret_cast<const float4*>((const float*)base + i);
  const uint2 u = *reinterpret_cast<const uint2*>((const uint16_t*)base + i);
  if (dtype == IQ_F16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
// The same four values stored, each rounded once.
__device__ __forceinline__ void store4(void* base, int dtype, size_t i, float4 v) {
  if (dtype == IQ_F32) {
    *reinterpret_cast<float4*>((float*)base + i) = v;
    return;
  }
  uint2 u;
  if (dtype == IQ_F16) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  *reinterpret_cast<uint2*>((uint16_t*)base + i) = u;
}

}  // namespace iq
