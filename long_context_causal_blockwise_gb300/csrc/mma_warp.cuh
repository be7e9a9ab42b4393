// tcgen05 issue by a whole warp: every lane walks the same control flow and one
// elected lane's predicate guards the instruction itself.
//
// The tensor-core instructions take their descriptors and addresses from
// uniform registers. In a branch that one lane alone takes, values are per
// thread and have to be moved over for every instruction; walked by the whole
// warp, the address arithmetic is uniform from the start.
#pragma once

#include "common.cuh"

namespace lcb {

// 1 in one lane of a converged warp, 0 in the others.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}

// Bits [0, n) of a word.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// A value that all lanes hold, as one the compiler knows to be uniform.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// mbar_wait without a function call in the waiting path: a call keeps the
// values around it in the registers of the calling convention, and does not
// compile beside setmaxnreg.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                 const DevStatus& st, uint32_t where) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, kSleepHintNs)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > st.limit) {
      *abort_flag = 1;
      if (atomicOr(st.words, DEV_TIMEOUT) == 0) {
        st.words[1] = where | ((blockIdx.x & 0xffu)) | ((warp_id() & 0xffu) << 8);
        st.words[2] = blockIdx.x;
      }
      return false;
    }
  }
}

// The same by all lanes of a warp, with the same answer in each.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                               const DevStatus& st, uint32_t where) {
  return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, abort_flag, st, where));
}

__device__ __forceinline__ void tc_commit_if(uint64_t* bar, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem], as mma_ss, by the elected lane.
__device__ __forceinline__ void mma_ss_if(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], as mma_ts, by the elected lane.
__device__ __forceinline__ void mma_ts_if(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}

}  // namespace lcb
