// Further tensor-core forms, those that attention needs beside tc.cuh's: a B
// operand that is M/N-major in shared memory (values as they lie in a cache),
// products into some of the accumulator's lanes only, 16-column loads, an L2
// policy for tiles that are read again.
#pragma once

#include "tc.cuh"

namespace lmoe {

// smem_desc_sw128 for an MN-major operand (64 consecutive M/N elements per
// 128-byte row, one row per k): SBO is the 1024-byte stride from one group of 8 k to
// the next, LBO the stride from one block of 64 M/N elements to the next.
__host__ __device__ constexpr uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
constexpr uint32_t kIdescBMnMajor = 1u << 16;  // B is MN-major

// L2 policy for copies of what will be read again.
__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// TMEM -> registers: 32 lanes x 32 bits, 16 consecutive columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// tc_mma_bf16_ts into some of D's lanes only: bit i of off[w] leaves lane
// 32 w + i as it is.
__device__ __forceinline__ void tc_mma_bf16_ts_lanes(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                     uint32_t accumulate, const uint32_t (&off)[4]) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
      : "memory");
}

}  // namespace lmoe
