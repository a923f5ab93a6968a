// Vectors of rows that start anywhere (on their element), for warps whose lanes hold neighbouring
// vectors of one row: 16, 8 or 4 bytes are read as the two aligned vectors that hold them, shifted
// together, and written as aligned vectors put together from neighbouring lanes. The last lanes of a
// warp are there for the lane before them: the next part of the row starts with them. Only the
// bytes at the ends of a row go one element at a time. (A lane for each element, with loads and
// stores of 2 bytes, took up to 3 times as long.)
#pragma once

#include "ops_common.cuh"

#if defined(__CUDACC__)

namespace moe {

template <int B>
struct Words {
  static_assert(B == 16 || B == 8 || B == 4, "a vector's bytes");
  uint32_t w[B / 4];
};
template <int B>
__device__ __forceinline__ Words<B> load_words(const void* p) {
  Words<B> v;
  if constexpr (B == 16) {
    const uint4 u = __ldg(static_cast<const uint4*>(p));
    v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
  } else if constexpr (B == 8) {
    const uint2 u = __ldg(static_cast<const uint2*>(p));
    v.w[0] = u.x, v.w[1] = u.y;
  } else {
    v.w[0] = __ldg(static_cast<const uint32_t*>(p));
  }
  return v;
}
template <int B>
__device__ __forceinline__ void store_words(void* p, const Words<B>& v) {
  if constexpr (B == 16)
    *static_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  else if constexpr (B == 8)
    *static_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
  else
    *static_cast<uint32_t*>(p) = v.w[0];
}
// B bytes from byte s (0 .. B - 1) of two vectors in a row.
template <int B>
__device__ __forceinline__ Words<B> shifted(const Words<B>& lo, const Words<B>& hi, uint32_t s) {
  constexpr int W = B / 4;
  uint32_t w[2 * W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    w[i] = lo.w[i];
    w[W + i] = hi.w[i];
  }
  if (B == 16 && (s & 8)) {
#pragma unroll
    for (int i = 0; i + 2 < 2 * W; ++i) w[i] = w[i + 2];
  }
  if (B >= 8 && (s & 4)) {
#pragma unroll
    for (int i = 0; i + 1 < 2 * W; ++i) w[i] = w[i + 1];
  }
  Words<B> v;
#pragma unroll
  for (int i = 0; i < W; ++i) v.w[i] = __funnelshift_r(w[i], w[i + 1], (s & 3) * 8);
  return v;
}

// Bytes from element c to the end of a row of `width`, at most 64 elements' (what is asked of them is less).
template <typename T>
__device__ __forceinline__ int bytes_left(long long c, long long width) {
  return (int)min(width - c, 64LL) * (int)sizeof(T);
}

// The B bytes at p, `left` bytes before its row's end; zeros past it. Reads whole aligned vectors with a
// byte of the row in them.
template <int B>
__device__ __forceinline__ Words<B> load_any(const void* p, int left) {
  const char* at = static_cast<const char*>(p);
  const int s = (int)(reinterpret_cast<uintptr_t>(at) & (B - 1));
  Words<B> lo{}, hi{};
  if (left > 0) lo = load_words<B>(at - s);
  if (s != 0 && left > B - s) hi = load_words<B>(at - s + B);
  Words<B> v = shifted<B>(lo, hi, s);
  if (left < B) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      const int n = left - 4 * i;  // bytes of this word
      v.w[i] &= n >= 4 ? 0xFFFFFFFFu : n > 0 ? (1u << (8 * n)) - 1 : 0u;
    }
  }
  return v;
}

// A lane's B bytes to p, those of the `left` before its row's end; `first`: p is the row's start. The
// lanes' vectors are neighbours, lane 0's first, and those from `own` on are stored by another warp.
// Whole warps, also lanes past the end. E: bytes of an element.
template <int B, int E>
__device__ __forceinline__ void store_any(void* p, bool first, int left, const Words<B>& v, int lane, int own) {
  char* at = static_cast<char*>(p);
  const int s = (int)(reinterpret_cast<uintptr_t>(at) & (B - 1));  // the same in every lane
  // The aligned vector that this lane's last s bytes begin, or its own.
  Words<B> o = v;
  if (s != 0) {
    Words<B> next;
#pragma unroll
    for (int i = 0; i < B / 4; ++i) next.w[i] = __shfl_down_sync(kAll, v.w[i], 1);
    o = shifted<B>(v, next, B - s);
  }
  const int need = s != 0 ? 2 * B - s : B;  // bytes of the row that make it whole
  if (lane >= own || left <= 0) return;
  if (left >= need) store_words<B>(at + need - B, o);
  if ((s != 0 && first) || left < need) {  // the ends of the row, by elements
#pragma unroll
    for (int i = 0; i < B / E; ++i) {
      const bool head = s != 0 && i * E < B - s;  // else of this lane's aligned vector
      if ((head ? first || left < B - s : left < need) && left >= (i + 1) * E) {
        const uint32_t w = v.w[i * E / 4] >> (8 * (i * E % 4));
        if (E == 4)
          *reinterpret_cast<uint32_t*>(at + i * E) = w;
        else if (E == 2)
          *reinterpret_cast<uint16_t*>(at + i * E) = (uint16_t)w;
        else
          *reinterpret_cast<uint8_t*>(at + i * E) = (uint8_t)w;
      }
    }
  }
}

// Lanes of a warp that store their vectors. CODES: blocks of 32 elements lie in whole groups of lanes.
template <bool ANY, bool CODES = false>
constexpr int kOwn = !ANY ? 32 : CODES ? 24 : 31;

// A lane's vector of a row of `width` elements, N of them from element c, as it lies in memory; zeros
// outside the row. ANY: the row starts anywhere; else on 16 bytes, and whole vectors are inside or
// outside.
template <typename T, bool ANY>
struct RowVec {
  static constexpr int N = Vec<T>::kN;
  Words<16> v;
  __device__ __forceinline__ void load(const T* row, long long c, long long width) {
    if constexpr (ANY) {
      v = load_any<16>(row + c, bytes_left<T>(c, width));
    } else {
      v = Words<16>{};
      if (c < width) v = load_words<16>(row + c);
    }
  }
  __device__ __forceinline__ uint4 raw() const { return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]); }
  __device__ __forceinline__ void get(float (&f)[N]) const { unpack<T>(raw(), f); }
};
// The same to a row, of the lanes before `own`. Whole warps where ANY.
template <bool ANY, typename T>
__device__ __forceinline__ void store_vec(T* row, long long c, long long width, const float (&f)[Vec<T>::kN], int lane,
                                          int own = kOwn<ANY>) {
  const uint4 u = pack<T>(f);
  if constexpr (ANY) {
    store_any<16, (int)sizeof(T)>(row + c, c == 0, bytes_left<T>(c, width), Words<16>{{u.x, u.y, u.z, u.w}}, lane, own);
  } else {
    if (c < width) *reinterpret_cast<uint4*>(row + c) = u;
  }
}

// Four bytes of a row a lane (two elements of 16 bits, one of 32), for kernels with many rows in and out,
// where the shifting of long vectors is most of the work (see the kernels that use them).
template <typename T>
struct RowWord {
  static constexpr int N = 4 / (int)sizeof(T);
  uint32_t a, b;  // the aligned words that hold the elements; put together once they are used, so that
                  // no load waits for another
  int odd;        // the elements begin in the middle of a
  // The elements from e of a row of `width`. Reads whole words with an element of the row in them.
  __device__ __forceinline__ void load(const T* row, long long e, long long width) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(row + e) & ~(uintptr_t)3);
    odd = N == 2 ? (int)(reinterpret_cast<uintptr_t>(row + e) >> 1 & 1) : 0;
    const bool second = N == 2 && e + 1 >= 0 && e + 1 < width;  // that element is in the row
    a = b = 0;
    if ((e >= 0 && e < width) || (odd == 0 && second)) a = __ldg(p);
    if (odd != 0 && second) b = __ldg(p + 1);
  }
  // Zeros outside the row.
  __device__ __forceinline__ void get(long long e, long long width, float (&f)[N]) const {
    if constexpr (N == 1) {
      f[0] = __uint_as_float(a);
    } else {
      const float2 p = unpack2<T>(__funnelshift_r(a, b, 16 * odd));
      f[0] = e >= 0 && e < width ? p.x : 0.f;
      f[1] = e + 1 >= 0 && e + 1 < width ? p.y : 0.f;
    }
  }
};
// The same for rows that mostly lie as the kernel's words do: one load for them, single elements else.
template <typename T>
struct LikeWord {
  static constexpr int N = 4 / (int)sizeof(T);
  uint32_t w;
  __device__ __forceinline__ void load(const T* row, long long e, long long width) {
    const T* p = row + e;
    if constexpr (N == 1) {
      w = e >= 0 && e < width ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
      if (e >= 0 && e + 1 < width && (reinterpret_cast<uintptr_t>(p) & 2) == 0) {
        w = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else {
        const uint32_t lo = e >= 0 && e < width ? __ldg(h) : 0u;
        w = lo | (e + 1 >= 0 && e + 1 < width ? (uint32_t)__ldg(h + 1) << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (N == 1) {
      f[0] = __uint_as_float(w);
    } else {
      const float2 p = unpack2<T>(w);
      f[0] = p.x;
      f[1] = p.y;
    }
  }
};
template <typename T>
__device__ __forceinline__ uint32_t pack_word(const float (&f)[4 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4)
    return __float_as_uint(f[0]);
  else
    return pack2<T>(f[0], f[1]);
}
// The elements from e, whose address lies on four bytes.
template <typename T>
__device__ __forceinline__ void store_word(T* row, long long e, long long width, uint32_t w) {
  T* p = row + e;
  if constexpr (sizeof(T) == 4) {
    if (e >= 0 && e < width) *reinterpret_cast<uint32_t*>(p) = w;
  } else {
    unsigned short* h = reinterpret_cast<unsigned short*>(p);
    if (e >= 0 && e + 1 < width) {
      *reinterpret_cast<uint32_t*>(p) = w;
    } else {
      if (e >= 0 && e < width) h[0] = (unsigned short)w;
      if (e + 1 >= 0 && e + 1 < width) h[1] = (unsigned short)(w >> 16);
    }
  }
}
// The elements from e of a whole warp's, anywhere: lanes are neighbours, lane 0's first.
template <typename T>
__device__ __forceinline__ void store_word_any(T* row, long long e, long long width, uint32_t w, int lane) {
  if (sizeof(T) == 4 || (reinterpret_cast<uintptr_t>(row + e) & 2) == 0) {  // the same in every lane
    store_word(row, e, width, w);
    return;
  }
  // The word before this lane's second element: the lane before has its first half.
  const uint32_t before = __shfl_up_sync(kAll, w, 1);
  unsigned short* h = reinterpret_cast<unsigned short*>(row + e);
  if (lane == 0) {
    if (e >= 0 && e < width) h[0] = (unsigned short)w;
  } else {
    store_word(row, e - 1, width, __byte_perm(before, w, 0x5432));
  }
  if (lane == 31 && e + 1 >= 0 && e + 1 < width) h[1] = (unsigned short)(w >> 16);
}

}  // namespace moe

#endif  // __CUDACC__
