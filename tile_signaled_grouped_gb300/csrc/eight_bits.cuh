// Checkpoints in 8 bits: blocks of 32 elements of a row share a scale 2^s, s in -127 .. 127 (stored as
// s + 127), the least for which the block's largest finite |x| is at most 448 2^s, the largest e4m3
// number; a code is x 2^-s rounded to e4m3, to nearest, ties to even. Scaling by a power of two is
// exact, so the rounding to the code is the only error: 2^-4 of x at most, or 2^-10 2^s. What is not
// finite becomes NaN (an infinity that came back as 448 2^s would hide an overflow).
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "ops_common.cuh"

namespace moe {

constexpr int kScaleBlock = 32;  // elements that share a scale
inline long long scale_blocks(long long c) { return (c + kScaleBlock - 1) / kScaleBlock; }

#if defined(__CUDACC__)

// The bits of |v|, 0 where v is not finite: their maximum over a block gives its scale.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}
// The stored scale of a block whose largest finite |x| has these bits: 448 is 1.75 2^8.
__device__ __forceinline__ uint32_t scale_of(uint32_t bits) {
  const int s = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(s, 0);
}
// 2^s and 2^-s of a stored scale; 2^-127 is a subnormal number.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s << 23);
}
__device__ __forceinline__ float scale_inverse(uint32_t s) {
  return __uint_as_float(s >= 254 ? 0x00400000u : (254u - s) << 23);
}

__device__ __forceinline__ float code_input(float v, float inverse) {
  return (__float_as_uint(v) & 0x7FFFFFFFu) == 0x7F800000u ? __uint_as_float(0x7FC00000u) : v * inverse;
}
__device__ __forceinline__ uint32_t encode2(float a, float b, float inverse) {
  return __nv_cvt_float2_to_fp8x2(make_float2(code_input(a, inverse), code_input(b, inverse)), __NV_SATFINITE,
                                  __NV_E4M3);
}
__device__ __forceinline__ uint8_t encode1(float a, float inverse) {
  return __nv_cvt_float_to_fp8(code_input(a, inverse), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// N consecutive codes of one block as they lie in memory (the address is a multiple of N), and times 2^s.
template <int N>
struct Codes {
  uint32_t w[(N + 3) / 4];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (N == 16) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else if constexpr (N == 8) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = u.x, w[1] = u.y;
    } else if constexpr (N == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      static_assert(N == 1, "16, 8, 4 or 1 codes");
      w[0] = __ldg(p);
    }
  }
  __device__ __forceinline__ void get(float scale, float (&f)[N]) const {
    if constexpr (N == 1) {
      f[0] = decode2(w[0]).x * scale;
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 d = decode2(w[i / 2] >> (16 * (i & 1)) & 0xFFFFu);
        f[2 * i] = d.x * scale;
        f[2 * i + 1] = d.y * scale;
      }
    }
  }
};
template <int N>
__device__ __forceinline__ void decode(const uint8_t* p, float scale, float (&f)[N]) {
  Codes<N> c;
  c.load(p);
  c.get(scale, f);
}

// N elements of a block, whose other elements the neighbouring lanes have (zeros outside the row),
// to codes and, by the block's first lane, the scale. Whole warps.
template <int N>
__device__ __forceinline__ void encode_block(const float (&f)[N], bool in, uint8_t* codes, uint8_t* scales,
                                             int lane) {
  constexpr int kLanes = kScaleBlock / N;
  uint32_t most = 0;
#pragma unroll
  for (int q = 0; q < N; ++q) most = max(most, finite_bits(f[q]));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) most = max(most, __shfl_xor_sync(kAll, most, o));
  if (!in) return;
  const uint32_t s = scale_of(most);
  const float inverse = scale_inverse(s);
  if constexpr (N == 1) {
    *codes = encode1(f[0], inverse);
  } else {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = encode2(f[4 * i], f[4 * i + 1], inverse) | encode2(f[4 * i + 2], f[4 * i + 3], inverse) << 16;
    if constexpr (N == 8)
      *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(codes) = w[0];
  }
  if (lane % kLanes == 0) *scales = (uint8_t)s;
}

// The same for eight elements of 16 bits as they lie in memory. The bits of |x| are in the order of
// |x|, so two elements at a time give the largest; only where that is not finite do the
// elements have to be looked at one by one. (131 instructions for eight elements of 16 bits by
// encode_block, 60 so.)
template <typename T>
__device__ __forceinline__ void encode_block16(const uint4& u, bool in, uint8_t* codes, uint8_t* scales, int lane) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu, kInf = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  uint32_t m = __vmaxu2(__vmaxu2(u.x & kAbs, u.y & kAbs), __vmaxu2(u.z & kAbs, u.w & kAbs));
  m = __vmaxu2(m, __shfl_xor_sync(kAll, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(kAll, m, 2));
  m = max(m & 0xFFFFu, m >> 16);
  if (__any_sync(kAll, m >= kInf)) {
    float f[8];
    unpack<T>(u, f);
    encode_block<8>(f, in, codes, scales, lane);
    return;
  }
  if (!in) return;
  const uint32_t s = scale_of(__float_as_uint(unpack2<T>(m).x));
  const float inverse = scale_inverse(s);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<T>(w[i]);
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(p.x * inverse, p.y * inverse), __NV_SATFINITE, __NV_E4M3);
  }
  *reinterpret_cast<uint2*>(codes) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  if ((lane & 3) == 0) *scales = (uint8_t)s;
}

#endif  // __CUDACC__

}  // namespace moe
