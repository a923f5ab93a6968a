// Checkpoints in 8 bits: blocks of 32 elements of a row share a scale 2^s, s in -127 .. 127 (stored as
// s + 127), the least for which the block's largest finite |x| is at most 448 2^s, the largest e4m3
// number; a code is x 2^-s rounded to e4m3, to nearest, ties to even. Scaling by a power of two is
// exact, so the rounding to the code is the only error: 2^-4 of x at most, or 2^-10 2^s. What is not
// finite becomes NaN (an infinity that came back as 448 2^s would hide an overflow). From 1.9375 2^e on, e the
// largest exponent of x's type, the nearest code stands for 2^(e + 1), an infinity in that type: there it
// is the one below, 1.875 2^e, which is within 2^-4 of x too.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "any_rows.cuh"
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
__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// N consecutive codes from code c of a row of `width`, as they lie in memory (zeros outside), and times
// 2^s. ANY: the row starts anywhere; else on N bytes, and whole vectors are inside or outside.
template <int N, bool ANY>
struct Codes {
  Words<N> v;
  __device__ __forceinline__ void load(const uint8_t* row, long long c, long long width) {
    if constexpr (ANY) {
      v = load_any<N>(row + c, bytes_left<uint8_t>(c, width));
    } else {
      v = Words<N>{};
      if (c < width) v = load_words<N>(row + c);
    }
  }
  __device__ __forceinline__ void get(float scale, float (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 d = decode2(v.w[i / 2] >> (16 * (i & 1)) & 0xFFFFu);
      f[2 * i] = d.x * scale;
      f[2 * i + 1] = d.y * scale;
    }
  }
};
// N elements from element e of a row of `width` and of codes that start anywhere; zeros outside it.
template <int N>
struct CodeWord {
  uint8_t code[N], scale[N];
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, long long e, long long width) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = e + i >= 0 && e + i < width;
      code[i] = in ? __ldg(codes + e + i) : 0;
      scale[i] = in ? __ldg(scales + (e + i) / kScaleBlock) : 0;
    }
  }
  __device__ __forceinline__ void get(long long, long long, float (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = decode2(code[i]).x * scale_value(scale[i]);
  }
};
// The codes of one element.
__device__ __forceinline__ float decode1(const uint8_t* p, float scale) { return decode2(__ldg(p)).x * scale; }

// The codes of N elements of T from element c of a row of `width`, and their block's scale, for elements
// whose largest finite |x| in the block (other lanes have the rest of it) has the bits `most`.
// PLAIN: all of the block are finite and below 1.9375 2^e. Whole warps where ANY.
template <typename T, bool ANY, bool PLAIN, int N>
__device__ __forceinline__ void store_codes(float (&f)[N], uint32_t most, uint8_t* codes, uint8_t* scales,
                                            long long c, long long width, int lane) {
  const uint32_t s = scale_of(most);
  const float inverse = scale_inverse(s);
  constexpr uint32_t kExponent = std::is_same<T, __half>::value ? 0x47000000u : 0x7F000000u;
  constexpr uint32_t kTop = kExponent | 0x780000u, kBelow = kExponent | 0x700000u;  // 1.9375 and 1.875
  if (!PLAIN && most >= kTop) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (finite_bits(f[i]) >= kTop) f[i] = copysignf(__uint_as_float(kBelow), f[i]);
  }
  Words<N> o;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float* g = f + 4 * i;
    if constexpr (PLAIN)
      o.w[i] = __nv_cvt_float2_to_fp8x2(make_float2(g[0] * inverse, g[1] * inverse), __NV_SATFINITE, __NV_E4M3) |
               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(g[2] * inverse, g[3] * inverse), __NV_SATFINITE,
                                                  __NV_E4M3) << 16;
    else
      o.w[i] = encode2(g[0], g[1], inverse) | encode2(g[2], g[3], inverse) << 16;
  }
  if constexpr (ANY)
    store_any<N, 1>(codes + c, c == 0, bytes_left<uint8_t>(c, width), o, lane, kOwn<true, true>);
  else if (c < width)
    store_words<N>(codes + c, o);
  if (c < width && c % kScaleBlock == 0 && (!ANY || lane < kOwn<true, true>)) scales[c / kScaleBlock] = (uint8_t)s;
}

// A lane's vector of a row to codes; the block's other elements are in the neighbouring lanes, c is a
// multiple of the vector. Whole warps. Of 16-bit types the bits of |x| are in the order of |x|, so two
// elements at a time give the largest; only where that is 1.9375 2^e or more do they have to be looked
// at one by one (131 instructions for eight elements one by one, 60 so).
template <typename T, bool ANY>
__device__ __forceinline__ void encode_vec(const RowVec<T, ANY>& x, uint8_t* codes, uint8_t* scales, long long c,
                                           long long width, int lane) {
  constexpr int N = Vec<T>::kN;
  float f[N];
  if constexpr (sizeof(T) == 2) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu, kTop = std::is_same<T, __half>::value ? 0x7BC0u : 0x7F78u;
    uint32_t m = __vmaxu2(__vmaxu2(x.v.w[0] & kAbs, x.v.w[1] & kAbs), __vmaxu2(x.v.w[2] & kAbs, x.v.w[3] & kAbs));
    m = __vmaxu2(m, __shfl_xor_sync(kAll, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(kAll, m, 2));
    m = max(m & 0xFFFFu, m >> 16);
    if (!__any_sync(kAll, m >= kTop)) {
      x.get(f);
      store_codes<T, ANY, true>(f, __float_as_uint(unpack2<T>(m).x), codes, scales, c, width, lane);
      return;
    }
  }
  x.get(f);
  uint32_t most = 0;
#pragma unroll
  for (int q = 0; q < N; ++q) most = max(most, finite_bits(f[q]));
#pragma unroll
  for (int o = 1; o < kScaleBlock / N; o <<= 1) most = max(most, __shfl_xor_sync(kAll, most, o));
  store_codes<T, ANY, false>(f, most, codes, scales, c, width, lane);
}

#endif  // __CUDACC__

}  // namespace moe
