// What the matrix products on tcgen05 share (linear.cu, expert_linear.cu): descriptors of operands of
// 16 bits, the ring of stages, single-thread roles run by whole warps.
#pragma once

#include <cudaTypedefs.h>

#include "moe_common.cuh"
#include "ops_common.cuh"

namespace moe {

// cuTensorMapEncodeTiled, or null where the driver has none (linear.cu).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

#if defined(__CUDACC__)

// Shared-memory matrix descriptor of an MN-major operand stored by TMA in boxes of 64
// elements (128 bytes, the swizzle span) x 64 k-rows: 8 KB from one box to the next,
// 1024 bytes from 8 k-rows to the next 8.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(8192 >> 4) << 16;  // leading-dimension offset: the next 64 elements
  d |= (uint64_t)(1024 >> 4) << 32;  // stride-dimension offset: the next 8 k
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Instruction descriptor: 16-bit A and B of one type, fp32 accumulator, M x N.
__device__ __forceinline__ uint32_t idesc_16bit(bool bf16, bool a_mn, bool b_mn, int M, int N) {
  const uint32_t t = bf16 ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The next stage of a ring. (A division by the ring's length, which only the launch knows,
// costs these single threads more than the rest of a step: with `n % stages` a step took
// 190 ns without any copy or product in it.)
__device__ __forceinline__ void next_stage(int& st, uint32_t& phase, int stages) {
  if (++st == stages) {
    st = 0;
    phase ^= 1;
  }
}

// One lane of a converged warp, the same one every time. The single-thread roles run as whole
// warps and ask this around what one thread issues: their addresses and descriptors then
// stay uniform values, which tcgen05 and TMA take as they are.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

constexpr long long kWaitNs = 4000000000LL;  // bound of every device-side wait

// Waits of a whole warp: every lane comes out with the same answer, so that no lane leaves
// a role that the others carry on with.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase, volatile int* abort, uint32_t* status,
                                          uint32_t detail) {
  return __all_sync(kAll, mbar_wait_bounded(bar, phase, abort, kWaitNs, status, detail));
}
__device__ __forceinline__ bool warp_pwait(uint64_t* bar, uint32_t phase, volatile int* abort, uint32_t* status,
                                           uint32_t detail) {
  return __all_sync(kAll, pwait(bar, phase, abort, kWaitNs, status, detail));
}

#endif  // __CUDACC__

}  // namespace moe
