// Shared by the operators around the routed experts (router.cu, norm.cu, linear.cu):
// element types and the device check.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

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

#if defined(__CUDACC__)

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
