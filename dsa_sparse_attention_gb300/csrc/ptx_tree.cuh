// ptx_tree.cuh — the PTX wrappers of the dense tree attention beyond those of ptx.cuh.
#pragma once
#include "ptx.cuh"

namespace dsa {

// True in one lane of the (converged) warp.  A role that issues tensor-core work runs its
// loop in the whole warp and issues under this predicate: descriptors then stay in
// uniform registers, where a loop inside a one-lane branch moves each of them there per
// instruction and issues slower than the tensor core runs.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Barrier over `nthreads` threads that also returns whether any of them passed a non-zero value.
__device__ __forceinline__ bool named_bar_any(uint32_t id, uint32_t nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

// As mma_f8f6f4, with A kept in the tensor core's operand buffer: the first of a run of
// MMAs on one A fills it, the following ones use it (the last one hands it back), so A is
// read from shared memory once.
enum class KeepA { kFill, kUse, kLast };
template <KeepA OP>
__device__ __forceinline__ void mma_f8f6f4_keep_a(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                  uint32_t accumulate) {
  if (OP == KeepA::kFill)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4.collector::a::fill "
        "[%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else if (OP == KeepA::kUse)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4.collector::a::use "
        "[%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4.collector::a::lastuse "
        "[%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same with a 64-byte swizzle (rows of 64 bytes, 512-byte aligned atoms of 8 rows).
__device__ __forceinline__ uint64_t make_sdesc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (make_sdesc_sw128(saddr, lbo, sbo) & ~(static_cast<uint64_t>(7) << 61)) | (static_cast<uint64_t>(4) << 61);
}

// And with a 32-byte swizzle.
__device__ __forceinline__ uint64_t make_sdesc_sw32(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (make_sdesc_sw128(saddr, lbo, sbo) & ~(static_cast<uint64_t>(7) << 61)) | (static_cast<uint64_t>(6) << 61);
}

#define DSA_TMEM_LD16(taddr, r)                                                                                      \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "     \
               "[%16];"                                                                                              \
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),      \
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),             \
                 "=r"(r[15])                                                                                         \
               : "r"(taddr)                                                                                          \
               : "memory")
#define DSA_TMEM_ST16(taddr, r)                                                                                      \
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"    \
               "%16};" ::"r"(taddr),                                                                                 \
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),     \
               "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])                      \
               : "memory")

// 16 lanes (from the address's lane) x 32 columns as blocks of 8 columns: thread l gets, of
// block b, lane l / 4 columns 2 (l % 4) and + 1 in r[4b], r[4b + 1], lane l / 4 + 8 in r[4b + 2], r[4b + 3].
#define DSA_TMEM_LD_16X256_X4(taddr, r)                                                                              \
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "    \
               "[%16];"                                                                                              \
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),      \
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),             \
                 "=r"(r[15])                                                                                         \
               : "r"(taddr)                                                                                          \
               : "memory")

#define DSA_TMEM_ST8(taddr, r)                                                                                      \
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),   \
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])                         \
               : "memory")

// Four 8 x 8 matrices of 16-bit values, transposed on the way into shared memory: thread l
// holds of matrix i row l / 4, columns 2 (l % 4) and + 1 in r_i; column c of matrix i goes,
// 16 contiguous bytes, to the address that lane 8 i + c passes.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t saddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}

}  // namespace dsa
