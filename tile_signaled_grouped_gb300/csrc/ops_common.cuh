// Shared by the operators around the routed experts (router.cu, norm.cu, linear.cu):
// element types and the device check.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe_tsg.h"

namespace moe {

inline int type_bytes(int dtype) {
  return dtype == MOE_FP32 ? 4 : dtype == MOE_BF16 || dtype == MOE_FP16 ? 2 : 0;
}
inline bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// MOE_OK and the current device's SM count, MOE_ERR_CUDA without a device and
// MOE_ERR_UNSUPPORTED for any but compute capability 10.3. Two attribute reads on the
// first call for a device, a table after that (an entry is written whole, so callers
// on other threads see 0 or the count).
int ops_device(int* num_sms);

// The current device's status words of the operators ([0] code, [1] detail; sticky, read by
// moe_ops_status): where a device wait that ran out is recorded. Null if the runtime
// cannot tell.
uint32_t* ops_status();

constexpr size_t kSmemMax = 227 * 1024;  // shared memory of a CTA
// Lets `kernel` use all of it; once for each device (bit d of *ready).
cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>* ready);

#if defined(__CUDACC__)

// Launches a kernel that may start once every CTA of the kernel before it on the stream has
// allowed it (allow_dependent_launch) or left; it calls wait_prior_grid() before it reads or
// writes anything that kernel touches. After a kernel that allows nothing: an ordinary launch.
template <typename K, typename... A>
cudaError_t launch_behind(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Every earlier kernel of the stream is complete and its writes are visible.
__device__ __forceinline__ void wait_prior_grid() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr uint32_t kAll = 0xFFFFFFFFu;  // every lane of a warp
// The sum of the warp's values, in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// The two elements of a 32-bit word as fp32, and back (one conversion for both: single
// conversions of 16-bit types run at a quarter of its rate and need a merge each).
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A 16-byte vector of T as fp32, and back.
template <typename T>
struct Vec {
  static constexpr int kN = 16 / (int)sizeof(T);
};
template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[Vec<T>::kN]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(w[i]);
    } else {
      const float2 p = unpack2<T>(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[Vec<T>::kN]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4)
      w[i] = __float_as_uint(f[i]);
    else
      w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Element i of an array whose type is known at run time (the branch is uniform).
__device__ __forceinline__ float load_as_f32(const void* p, int dtype, long long i) {
  if (dtype == MOE_FP32) return __ldg(static_cast<const float*>(p) + i);
  const unsigned short u = __ldg(static_cast<const unsigned short*>(p) + i);
  return dtype == MOE_BF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}
__device__ __forceinline__ void store_from_f32(void* p, int dtype, long long i, float v) {
  if (dtype == MOE_FP32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == MOE_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

#endif  // __CUDACC__

}  // namespace moe
