// 5th-generation tensor core (tcgen05) primitives for sm_100a: tensor-memory allocation, the
// shared-memory matrix and instruction descriptors of a kind::f16 MMA, the MMA itself, its
// completion signal on an mbarrier, and tensor-memory loads.
//
// Operand layout (K-major, 128-byte swizzle): a tile of R rows and K 16-bit elements is stored
// as K / 64 blocks of R rows x 128 bytes, element (r, k) at
//     (k / 64) * R * 128 + r * 128 + ((((k / 8) % 8) ^ (r % 8)) * 16) + (k % 8) * 2   bytes
// from a 1024-byte aligned base (the hardware applies the XOR on address bits 4-6 from bits
// 7-9).  Groups of 8 rows are 1024 bytes apart (SBO); the MMA over elements 16 s .. 16 s + 15
// starts at byte (s / 4) * R * 128 + (s % 4) * 32.
#pragma once
#include <cstdint>

namespace iq {

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Shared-memory matrix descriptor of the layout above: start address (16-byte units), leading
// offset 1 (unused by this layout), 8-row stride 1024 bytes, descriptor version 1, layout type
// 2 (128-byte swizzle).
__device__ __forceinline__ uint64_t umma_sdesc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Byte offset of element (r, k) (k a multiple of 8: the start of a 16-byte chunk) in an R-row tile.
__host__ __device__ constexpr int umma_sw128_off(int r, int k, int R) {
  return (k >> 6) * R * 128 + r * 128 + ((((k >> 3) & 7) ^ (r & 7)) << 4);
}

// Descriptor of a B operand whose rows of 128 bytes run along N (MN-major, 128-byte swizzle): element (k, n) of a
// tile of R k-rows at (n / 64) * R * 128 + k * 128 + ((((n / 8) % 8) ^ (k % 8)) * 16) + (n % 8) * 2 bytes.
// Leading offset: from one block of 64 n to the next (R * 128 bytes); stride offset: from 8 k to the next 8
// (1024 bytes).  The MMA over k = 16 s .. 16 s + 15 starts at byte 2048 s.
__device__ __forceinline__ uint64_t umma_sdesc_sw128_mn(uint32_t saddr, uint32_t R) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(R * 128 >> 4) << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}
constexpr uint32_t UMMA_B_MN_MAJOR = 1u << 16;  // instruction descriptor bit

// Instruction descriptor of kind::f16 with fp16 A and B (both K-major) and an fp32 accumulator.
__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D (tensor memory) = A B^T (+ D when acc != 0); one thread issues it.
__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}

// Eight MMAs over K = 128 from operands in the layouts above, R = 128 rows (of which B may take a part): the
// descriptors of the first one, and for the rest the constant steps of their start addresses (in 16-byte units), so
// that one thread issues them back to back (72-90 cycles each where it made every descriptor anew, 64 so; 52 for 64 keys
// from a warp that keeps the descriptors in uniform registers).  A and B
// along K (two blocks of 64): steps 2, 4, 6, 1024, 1026, ...; D is overwritten.
__device__ __forceinline__ void umma_f16_k128(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
#define IQ_UMMA_STEP(off) "add.u64 a, %1, " #off ";\n add.u64 b, %2, " #off ";\n tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n "
  asm volatile(
      "{\n .reg .pred f, t;\n .reg .b64 a, b;\n setp.ne.b32 f, 0, 0;\n setp.eq.b32 t, 0, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n " IQ_UMMA_STEP(2) IQ_UMMA_STEP(4) IQ_UMMA_STEP(6)
      IQ_UMMA_STEP(1024) IQ_UMMA_STEP(1026) IQ_UMMA_STEP(1028) IQ_UMMA_STEP(1030) "}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc)
      : "memory");
#undef IQ_UMMA_STEP
}
// Four MMAs over K = 64 with A (M lanes x 64 binary16 numbers, two to a 32-bit column: eight columns a step) in tensor
// memory and B along N (2048 bytes a step); D is added to where acc != 0.
__device__ __forceinline__ void umma_f16_ts_k64(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t acc) {
#define IQ_UMMA_STEP(i) "add.u32 a, %1, 8 * " #i ";\n add.u64 b, %2, 128 * " #i ";\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n "
  asm volatile(
      "{\n .reg .pred p, t;\n .reg .b32 a;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n " IQ_UMMA_STEP(1) IQ_UMMA_STEP(2) IQ_UMMA_STEP(3) "}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
#undef IQ_UMMA_STEP
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// The mbarrier receives one arrival once every MMA this thread has issued so far is complete.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Whole warp: allocate / free `cols` columns (a power of two >= 32) of tensor memory; the base
// address is written to shared memory at `dst`.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

// Whole warp: 16 consecutive 32-bit columns of this thread's lane (the warp's 32 lanes start at
// 32 (warp % 4)); the values are valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
// 32 consecutive columns, likewise.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
// Stores of 16 columns; complete after tmem_wait_st.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// The same, tied to the registers that a load fills, so that the compiler moves no use of them before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]));
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31]));
}

}  // namespace iq
