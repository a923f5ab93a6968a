// Matrix product with bias, activation and residual in its epilogue, and its backward
// pass, on tcgen05.
//
//   forward   z = x W^T + b,  y = act(z) + r            x [M][K], W [N][K]
//   backward  dz = dy act'(z),  db = sum over rows of dz
//             dx = dz W  [M][K],   dW = dz^T x  [N][K]
//
// Every product is D[i][j] = sum_k A(i, k) B(j, k) with fp32 accumulators in TMEM; an
// operand lies in memory with k innermost (K-major) or with i or j innermost (MN-major):
//   forward  A = x (K),   B = W (K)        i = m, j = n, k = k
//   dx       A = dz (K),  B = W (MN)       i = m, j = k, k = n
//   dW       A = dz (MN), B = x (MN)       i = n, j = k, k = m
// TMA stages 64 k-elements of both operands with the 128-byte swizzle, and the tensor
// cores read either layout, so no operand is ever transposed in memory. The bounds of the
// tensor maps fill with zeros what lies past M, N and K.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "linear_tiles.h"
#include "moe_common.cuh"
#include "ops_common.cuh"

namespace moe {
namespace {

constexpr long long kWaitNs = 4000000000LL;  // bound of every device-side wait

// The sticky device status of these kernels: [0] code, [1] detail (moe_ops_status).
__device__ uint32_t g_status[4];

// ------------------------------------------------------------------- activations
__device__ __forceinline__ float fast_sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

constexpr float kGeluC0 = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluC1 = 0.044715f;

// The normal distribution: returns (1 + erf(z / sqrt(2))) / 2, and in *e exp(-z^2 / 2). The
// side of 0 that z is on has the tail q = erfc(|z| / sqrt(2)) / 2 = e t R(t), t = 1 / (1 + 0.44 |z| /
// sqrt(2)): without the exponential it falls only as 1 / |z|, and R is a polynomial fitted to it over
// |z| < 14, where e leaves fp32, with the largest relative error as small as degree 7 allows
// (1.9e-7; least squares reweighted by the errors, Lawson's method). So nothing cancels below 0,
// where 1 + erf keeps multiples of 6e-8 only (4 % of gelu at -5). Within (1.5 z^2 + 25) 2^-24 of
// itself: three roundings of the exponent, and 25 half steps for the rest. 4096 x 4096 x 1024
// with this gelu takes 42 us, 47 by erff, 67 by erfcf.
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  float t, x;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(fabsf(z), 0.44f * 0.7071067811865476f, 1.0f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(z * z * -0.7213475204444817f));  // log2(e) / 2
  float r = 0.035597959f;
  r = fmaf(r, t, -0.13891378f);
  r = fmaf(r, t, 0.14823441f);
  r = fmaf(r, t, -0.0099838804f);
  r = fmaf(r, t, 0.10784631f);
  r = fmaf(r, t, 0.10867608f);
  r = fmaf(r, t, 0.12443229f);
  r = fmaf(r, t, 0.12411071f);
  const float q = r * t * x;
  *e = x;
  return z < 0.f ? q : 1.0f - q;
}

// act(z). 0.5 (1 + tanh u) is the sigmoid of 2u. The fast exponential of v is within
// (2 + 1.2 |v|) 2^-23 of itself (1e-6 at 6, 1e-5 at 80) and the fast division within 2^-22, far
// below half a step of a 16-bit result; an fp32 result is off by that. Sigmoids below 2^-126 are 0.
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
  if (ACT == MOE_ACT_GELU) {
    float e;
    return z * normal_cdf(z, &e);
  }
  if (ACT == MOE_ACT_GELU_TANH) return z * fast_sigmoid(2.0f * kGeluC0 * (z + kGeluC1 * z * z * z));
  if (ACT == MOE_ACT_SILU) return z * fast_sigmoid(z);
  return z;
}
// act'(z). z is kept where it makes no infinities times zero: past 30 the derivatives are 1 to
// the last bit, and below -30 0 in fp32, but for silu's, z exp(z), which is below 1e-36 only
// from -88 on and 0 here. NaN stays (relu's derivative there is 0).
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  constexpr float kLow = ACT == MOE_ACT_SILU ? -100.f : -30.f;
  z = z > 30.f ? 30.f : z < kLow ? kLow : z;
  if (ACT == MOE_ACT_GELU) {
    float e;
    const float p = normal_cdf(z, &e);
    return fmaf(z * 0.3989422804014327f, e, p);  // 1 / sqrt(2 pi)
  }
  if (ACT == MOE_ACT_GELU_TANH) {
    const float q = fast_sigmoid(2.0f * kGeluC0 * (z + kGeluC1 * z * z * z));
    return q + z * q * (1.0f - q) * (2.0f * kGeluC0) * (1.0f + 3.0f * kGeluC1 * z * z);
  }
  if (ACT == MOE_ACT_SILU) {
    const float q = fast_sigmoid(z);
    return q * (1.0f + z * (1.0f - q));
  }
  return 1.f;
}

__device__ __forceinline__ void st_cluster_v4(uint32_t cl_addr, uint32_t x, uint32_t y, uint32_t z,
                                              uint32_t w) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cl_addr), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}
// The halves of a cluster barrier of every thread that orders no memory (a release costs 0.3 us here):
// after it every CTA of the cluster has started.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------- the epilogue
struct Epilogue {
  void* y;        // [I][ld_y] of ytype
  void* z;        // [I][ld_z] of dtype, before the activation, or null
  const void* r;  // [I][ld_r] of dtype or null
  const void* b;  // [J] of btype or null
  long long ld_y, ld_z, ld_r;
  int dtype, ytype, btype, act;
  int vy, vz, vr;  // bytes on which every row starts: 32, 16 or 0 (any)
  bool vb;         // b starts on 16 bytes
};

// Whether every row of the outputs and the residual starts on 16 bytes.
__host__ __device__ inline bool aligned_rows(const Epilogue& e) {
  return e.vy != 0 && (e.z == nullptr || e.vz != 0) && (e.r == nullptr || e.vr != 0);
}

// Eight elements of a row from column j: in one or two 16-byte accesses where `vec` and
// all eight are inside, else one by one.
__device__ __forceinline__ void load8(const void* p, int dtype, long long at, int n, bool vec, float (&f)[8]) {
  if (vec && n >= 8) {
    if (dtype == MOE_FP32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      const float4 u = __ldg(q), v = __ldg(q + 1);
      f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
      return;
    }
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(p) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (dtype == MOE_BF16) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = h.x;
        f[2 * i + 1] = h.y;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = i < n ? load_as_f32(p, dtype, at + i) : 0.f;
}
__device__ __forceinline__ void store8(void* p, int dtype, long long at, int n, bool vec, const float (&f)[8]) {
  if (vec && n >= 8) {
    if (dtype == MOE_FP32) {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
      q[0] = make_float4(f[0], f[1], f[2], f[3]);
      q[1] = make_float4(f[4], f[5], f[6], f[7]);
      return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (dtype == MOE_BF16) {
        w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      } else {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<unsigned short*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store_from_f32(p, dtype, at + i, f[i]);
}

template <int ACT>
__device__ __forceinline__ void act8(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = act_of<ACT>(v[i]);
}

// The bias of eight columns from j, n of them inside the matrix; zeros without one.
__device__ __forceinline__ void bias8(const Epilogue& e, int j, int n, float (&b)[8]) {
  if (e.b != nullptr) {
    load8(e.b, e.btype, j, n, e.vb, b);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) b[q] = 0.f;
  }
}

__device__ __forceinline__ void act8_any(float (&v)[8], int act) {
  switch (act) {  // the same for the whole grid
    case MOE_ACT_RELU: act8<MOE_ACT_RELU>(v); break;
    case MOE_ACT_GELU: act8<MOE_ACT_GELU>(v); break;
    case MOE_ACT_GELU_TANH: act8<MOE_ACT_GELU_TANH>(v); break;
    case MOE_ACT_SILU: act8<MOE_ACT_SILU>(v); break;
    default: break;
  }
}

// Elements at[0] .. at[7] of an array, those of `mask`, one by one: the type is asked once.
__device__ __forceinline__ void scatter8(void* p, int dtype, const long long (&at)[8], uint32_t mask,
                                         const float (&f)[8]) {
  if (dtype == MOE_FP32) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if ((mask >> q) & 1u) static_cast<float*>(p)[at[q]] = f[q];
  } else if (dtype == MOE_BF16) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if ((mask >> q) & 1u) static_cast<__nv_bfloat16*>(p)[at[q]] = __float2bfloat16_rn(f[q]);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if ((mask >> q) & 1u) static_cast<__half*>(p)[at[q]] = __float2half_rn(f[q]);
  }
}
// Eight sums at rows i[q] and columns j[q], those of `mask`, whose residuals are r.
__device__ __forceinline__ void finish_scattered(const Epilogue& e, const long long (&i)[8],
                                                 const long long (&j)[8], uint32_t mask, const float (&r)[8],
                                                 float (&v)[8]) {
  long long at[8];
  if (e.z != nullptr) {
#pragma unroll
    for (int q = 0; q < 8; ++q) at[q] = i[q] * e.ld_z + j[q];
    scatter8(e.z, e.dtype, at, mask, v);
  }
  act8_any(v, e.act);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    v[q] += r[q];
    at[q] = i[q] * e.ld_y + j[q];
  }
  scatter8(e.y, e.ytype, at, mask, v);
}

// Eight sums of row i from column j, n of them inside the matrix, to the outputs.
__device__ __forceinline__ void finish8(const Epilogue& e, long long i, int j, int n, const float (&b)[8],
                                        float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] += b[q];
  if (e.z != nullptr) store8(e.z, e.dtype, i * e.ld_z + j, n, e.vz != 0, v);
  act8_any(v, e.act);
  if (e.r != nullptr) {
    float t[8];
    load8(e.r, e.dtype, i * e.ld_r + j, n, e.vr != 0, t);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += t[q];
  }
  store8(e.y, e.ytype, i * e.ld_y + j, n, e.vy != 0, v);
}

// 32 sums of row i from column j, n of them inside the matrix, to the outputs: 32 bytes (a
// sector) a store where the rows allow it.
__device__ __forceinline__ void load32(const void* p, int dtype, long long at, float (&f)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float t[8];
    load8(p, dtype, at + 8 * c, 8, true, t);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[8 * c + q] = t[q];
  }
}
__device__ __forceinline__ void store32(void* p, int dtype, long long at, bool wide, const float (&f)[32]) {
  if (dtype != MOE_FP32 && wide) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (dtype == MOE_BF16) {
        w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      } else {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    unsigned short* q = static_cast<unsigned short*>(p) + at;
    st_global_v8(q, w);
    st_global_v8(q + 16, w + 8);
    return;
  }
  if (dtype == MOE_FP32 && wide) {
    float* q = static_cast<float*>(p) + at;
#pragma unroll
    for (int c = 0; c < 4; ++c) st_global_v8(q + 8 * c, reinterpret_cast<const uint32_t*>(f) + 8 * c);
    return;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float t[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) t[q] = f[8 * c + q];
    store8(p, dtype, at + 8 * c, 8, true, t);
  }
}
template <int ACT>
__device__ __forceinline__ void act32(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = act_of<ACT>(v[i]);
}
__device__ __forceinline__ void finish32(const Epilogue& e, long long i, int j, int n, float (&v)[32]) {
  if (n < 32 || !e.vb) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (8 * c < n) {
        float t[8], b[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) t[q] = v[8 * c + q];
        bias8(e, j + 8 * c, n - 8 * c, b);
        finish8(e, i, j + 8 * c, n - 8 * c, b, t);
      }
    }
    return;
  }
  if (e.b != nullptr) {
    float t[32];
    load32(e.b, e.btype, j, t);
#pragma unroll
    for (int q = 0; q < 32; ++q) v[q] += t[q];
  }
  if (e.z != nullptr) store32(e.z, e.dtype, i * e.ld_z + j, e.vz >= 32, v);
  switch (e.act) {  // the same for the whole grid
    case MOE_ACT_RELU: act32<MOE_ACT_RELU>(v); break;
    case MOE_ACT_GELU: act32<MOE_ACT_GELU>(v); break;
    case MOE_ACT_GELU_TANH: act32<MOE_ACT_GELU_TANH>(v); break;
    case MOE_ACT_SILU: act32<MOE_ACT_SILU>(v); break;
    default: break;
  }
  if (e.r != nullptr) {
    float t[32];
    load32(e.r, e.dtype, i * e.ld_r + j, t);
#pragma unroll
    for (int q = 0; q < 32; ++q) v[q] += t[q];
  }
  store32(e.y, e.ytype, i * e.ld_y + j, e.vy >= 32, v);
}

// act of a value whose kind is known at run time.
__device__ __forceinline__ float act_any(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return act_of<MOE_ACT_RELU>(z);
    case MOE_ACT_GELU: return act_of<MOE_ACT_GELU>(z);
    case MOE_ACT_GELU_TANH: return act_of<MOE_ACT_GELU_TANH>(z);
    case MOE_ACT_SILU: return act_of<MOE_ACT_SILU>(z);
    default: return z;
  }
}

// One sum of row i and column j to the outputs.
__device__ __forceinline__ void finish1(const Epilogue& e, long long i, long long j, float v) {
  if (e.b != nullptr) v += load_as_f32(e.b, e.btype, j);
  if (e.z != nullptr) store_from_f32(e.z, e.dtype, i * e.ld_z + j, v);
  v = act_any(v, e.act);
  if (e.r != nullptr) v += load_as_f32(e.r, e.dtype, i * e.ld_r + j);
  store_from_f32(e.y, e.ytype, i * e.ld_y + j, v);
}

// ------------------------------------------------------------------- tensor-core pieces
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

constexpr int kMaxStages = 8;
constexpr int kABytes = kTileI * kBlockK * 2;  // 16 KB
constexpr int kTileThreads = 256;

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

// Waits of a whole warp: every lane comes out with the same answer, so that no lane leaves
// a role that the others carry on with.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase, volatile int* abort, uint32_t detail) {
  return __all_sync(kAll, mbar_wait_bounded(bar, phase, abort, kWaitNs, g_status, detail));
}
__device__ __forceinline__ bool warp_pwait(uint64_t* bar, uint32_t phase, volatile int* abort, uint32_t detail) {
  return __all_sync(kAll, pwait(bar, phase, abort, kWaitNs, g_status, detail));
}

struct GemmArgs {
  CUtensorMap ta, tb;
  Epilogue e;
  int I, J, nk;       // nk: 64-element blocks of k
  int bn;             // columns of a tile: 16, 32, 64, 128 or 256 (64 or more if B is MN-major)
  int stages, blocks; // blocks: of k in a stage, one or two
  int splits, splits_log2;  // CTAs of a cluster that share a tile, each with a range of k
  int tiles_i, box_a; // box_a: rows of A's box (K-major)
  bool bf16;
};

struct TileSmem {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t done;
  uint32_t tmem;
  int abort;
};

__host__ __device__ constexpr size_t part_bytes(int bn) { return (size_t)kTileI * (bn + 4) * 4; }
// The sums of a split tile come from other CTAs, whose products may be done before this one's:
// they have memory of their own.
__host__ __device__ inline size_t tile_pipe_bytes(int bn, int blocks, int stages, int splits) {
  const size_t pipe = (size_t)stages * blocks * (kABytes + bn * 128);
  return splits > 1 ? pipe + part_bytes(bn) : pipe > part_bytes(bn) ? pipe : part_bytes(bn);
}

// This CTA's rows of a tile, `own` of them: rank, rank + S, ... The partial sums that all S CTAs
// of the cluster left in `part` ([S][128 / S][bn + 4]) are added in the order of the ranks and go
// through the epilogue. A thread keeps to eight columns, whose bias it has.
template <int S>
__device__ __forceinline__ void join_tile(const GemmArgs& a, const float* part, int rank, int own, int i0,
                                          int j, int c, const float (&bias)[8]) {
  constexpr int U = 2;
  const int chunks = a.bn / 8, pitch = a.bn + 4, each = kTileThreads / chunks, from = kTileI / S * pitch;
  const int n = a.J - j;
  if (n <= 0) return;
  for (int row0 = (int)threadIdx.x / chunks; row0 < own; row0 += U * each) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* at = part + min(row0 + u * each, own - 1) * pitch + c;
#pragma unroll
      for (int r = 0; r < S; ++r) {
        const float4 s = *reinterpret_cast<const float4*>(at + r * from);
        const float4 t = *reinterpret_cast<const float4*>(at + r * from + 4);
        const float w[8] = {s.x, s.y, s.z, s.w, t.x, t.y, t.z, t.w};
#pragma unroll
        for (int x = 0; x < 8; ++x) v[u][x] = r == 0 ? w[x] : v[u][x] + w[x];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row0 + u * each < own)
        finish8(a.e, i0 + rank + (long long)S * (row0 + u * each), j, n, bias, v[u]);
  }
}

// The same where rows do not start on 16 bytes: neighbouring threads take neighbouring
// columns, eight elements a thread at a time.
template <int S>
__device__ __forceinline__ void join_tile_any(const GemmArgs& a, const float* part, int rank, int own,
                                              int i0, int j0) {
  const int pitch = a.bn + 4, total = own * a.bn, shift = 31 - __clz(a.bn), from = kTileI / S * pitch;
  for (int it = (int)threadIdx.x; it < total; it += 8 * kTileThreads) {
    float v[8], r[8];
    long long i[8], j[8];
    uint32_t mask = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int x = min(it + u * kTileThreads, total - 1), c = x & (a.bn - 1), row = x >> shift;
      const float* at = part + row * pitch + c;
      mask |= (it + u * kTileThreads < total && j0 + c < a.J) ? 1u << u : 0u;
      i[u] = i0 + rank + (long long)S * row;
      j[u] = min(j0 + c, a.J - 1);
      r[u] = a.e.r != nullptr ? load_as_f32(a.e.r, a.e.dtype, i[u] * a.e.ld_r + j[u]) : 0.f;
      v[u] = a.e.b != nullptr ? load_as_f32(a.e.b, a.e.btype, j[u]) : 0.f;
      float sum = at[0];
#pragma unroll
      for (int q = 1; q < S; ++q) sum += at[q * from];
      v[u] += sum;
    }
    finish_scattered(a.e, i, j, mask, r, v);
  }
}
template <int S>
__device__ __forceinline__ void join(const GemmArgs& a, const float* part, int rank, int own, int i0, int j0,
                                     int c0, const float (&bias)[8]) {
  if (aligned_rows(a.e))
    join_tile<S>(a, part, rank, own, i0, j0 + c0, c0, bias);
  else
    join_tile_any<S>(a, part, rank, own, i0, j0);
}

// One tile of 128 x bn for each cluster of `splits` CTAs, each of which sums its range of
// k in its TMEM. The partial sums of a row then meet in the shared memory of one of them, which
// adds them in the order of the ranks and finishes the row. Warp 0
// loads, warp 1 issues the products, all eight warps empty TMEM. Bound by its start, the
// pipeline's first loads and the end: 333 x 517 x 1000 takes 8.1 us, 512 x 1024 x 1024 6.0 us, of
// which its products are 16 steps of 0.16 us. The CTA that finishes a row gets all its sums by
// stores, and no CTA waits for the others to have read: joining took 2.9 us where it takes 2.2
// (64 x 1024 x 1024 in four parts) as reads of the others' memory between two barriers.
template <bool AMN, bool BMN>
__global__ void __launch_bounds__(kTileThreads) linear_tile_kernel(const __grid_constant__ GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int b_bytes = a.bn * 128, block_bytes = kABytes + b_bytes, stage_bytes = a.blocks * block_bytes;
  TileSmem& sm = *reinterpret_cast<TileSmem*>(base + tile_pipe_bytes(a.bn, a.blocks, a.stages, a.splits));
  // Partial sums, [splits][128 / splits][bn + 4]; where the tile is not split, once the products are done.
  float* part = reinterpret_cast<float*>(base + (a.splits > 1 ? (size_t)a.stages * stage_bytes : 0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cols = a.bn < 32 ? 32 : a.bn;
  // (No 64-bit divisions and no loop of one thread here: they took 0.4 us of every launch.)
  const uint32_t rank = blockIdx.x & (uint32_t)(a.splits - 1), tile = blockIdx.x >> a.splits_log2;
  const uint32_t tj = tile / (uint32_t)a.tiles_i;
  const int i0 = (int)(tile - tj * (uint32_t)a.tiles_i) * kTileI, j0 = (int)tj * a.bn;
  const int k_lo = (int)(((long long)a.nk * rank) >> a.splits_log2);
  const int k_hi = (int)(((long long)a.nk * (rank + 1)) >> a.splits_log2);

  if (warp == 0) {
    if (lane < a.stages) {
      mbar_init(&sm.full[lane], 1);
      mbar_init(&sm.empty[lane], 1);
    }
    if (lane == 31) {
      mbar_init(&sm.done, 1);
      sm.abort = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(&sm.tmem, cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (a.splits > 1) cluster_arrive();  // waited for before this CTA writes to the others
  wait_prior_grid();  // behind a kernel that allows it, all of the above ran beside that one

  if (warp == 0) {
    const uint32_t bytes = (AMN ? kABytes : a.box_a * 128) + b_bytes;
    int issued = 0, st = 0;
    uint32_t phase = 1;
    for (int kb = k_lo; kb < k_hi; kb += a.blocks, ++issued) {
      if (!warp_wait(&sm.empty[st], phase, &sm.abort, 0x01000000u)) break;
      if (elect_one()) {
        uint8_t* as = base + (size_t)st * stage_bytes;
        const int n = min(a.blocks, k_hi - kb);
        mbar_arrive_expect_tx(&sm.full[st], n * bytes);
        for (int k = kb; k < kb + n; ++k, as += block_bytes) {
          uint8_t* bs = as + kABytes;
          if (AMN) {
            tma_load_2d(as, &a.ta, &sm.full[st], i0, k * kBlockK);
            tma_load_2d(as + 8192, &a.ta, &sm.full[st], i0 + 64, k * kBlockK);
          } else {
            tma_load_2d(as, &a.ta, &sm.full[st], k * kBlockK, i0);
          }
          if (BMN) {
            for (int c = 0; c < a.bn / 64; ++c)
              tma_load_2d(bs + c * 8192, &a.tb, &sm.full[st], j0 + c * 64, k * kBlockK);
          } else {
            tma_load_2d(bs, &a.tb, &sm.full[st], k * kBlockK, j0);
          }
        }
      }
      __syncwarp();
      next_stage(st, phase, a.stages);
    }
    if (*(volatile int*)&sm.abort) {  // the copies in flight land before the CTA leaves
      volatile int never = 0;
      for (int n = max(0, issued - a.stages); n < issued; ++n)
        mbar_wait_bounded(&sm.full[n % a.stages], (n / a.stages) & 1, &never, kWaitNs, g_status,
                          0x02000000u);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_16bit(a.bf16, AMN, BMN, kTileI, a.bn);
    const uint32_t s0 = (smem_u32(base) & 0x3FFFFu) >> 4;  // above lies the CTA's rank in its cluster
    const uint64_t da = (AMN ? sdesc_mn_sw128(0) : sdesc_k_sw128(0)) + s0;
    const uint64_t db = (BMN ? sdesc_mn_sw128(0) : sdesc_k_sw128(0)) + s0 + (kABytes >> 4);
    constexpr uint32_t step_a = (AMN ? 2048 : 32) >> 4, step_b = (BMN ? 2048 : 32) >> 4;
    int st = 0;
    uint32_t phase = 0, accumulate = 0, at = 0;  // at: the stage's offset in 16-byte units
    int kb = k_lo;
    for (; kb < k_hi; kb += a.blocks) {
      if (!warp_wait(&sm.full[st], phase, &sm.abort, 0x03000000u)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kBlockK / 16; ++k)
          tc_mma(tmem, da + at + k * step_a, db + at + k * step_b, idesc, k != 0 ? 1u : accumulate);
        if (a.blocks == 2 && kb + 1 < k_hi) {
          const uint32_t bt = at + (block_bytes >> 4);
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            tc_mma(tmem, da + bt + k * step_a, db + bt + k * step_b, idesc, 1u);
        }
        tc_commit(&sm.empty[st]);
      }
      __syncwarp();
      accumulate = 1;
      next_stage(st, phase, a.stages);
      at = st == 0 ? 0 : at + (stage_bytes >> 4);
    }
    if (kb < k_hi) {
      // A wait ran out, perhaps after warp 0 had issued all of its copies: those that may be in
      // flight, of this step and of the stages after it, land before the CTA leaves.
      volatile int never = 0;
      const unsigned long long t0 = globaltimer();
      for (int n = 0; n < a.stages && kb < k_hi; ++n, kb += a.blocks) {
        const long long left = kWaitNs - (long long)(globaltimer() - t0);
        mbar_wait_bounded(&sm.full[st], phase, &never, left > 0 ? left : 0, g_status, 0x05000000u);
        next_stage(st, phase, a.stages);
      }
    }
    // Also after a wait that ran out: no product outlives the CTA.
    __syncwarp();
    if (elect_one()) tc_commit(&sm.done);
  }
  __syncwarp();
  // The bias of the columns this thread will finish is on its way during the products.
  const int c0 = ((int)threadIdx.x % (a.bn / 8)) * 8;
  float bias[8];
  bias8(a.e, j0 + c0, a.J - j0 - c0, bias);
  volatile int never = 0;
  bool ok = mbar_wait_bounded(&sm.done, 0, &never, 2 * kWaitNs, g_status, 0x04000000u);
  ok = ok && *(volatile int*)&sm.abort == 0;
  __syncwarp();
  tc_fence_after();

  // Warp w reads lanes 32 (w & 3).. of TMEM, of column half w >> 2.
  const int rows = min(kTileI, a.I - i0);
  if (a.splits == 1 && aligned_rows(a.e)) {  // straight to the outputs
    const int q = warp & 3, row = q * 32 + lane;
    for (int c = (warp >> 2) * 32; c < a.bn; c += 64) {
      uint32_t v[32];
      tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c, v);
      tmem_ld_wait();
      float f[32];
#pragma unroll
      for (int x = 0; x < 32; ++x) f[x] = __uint_as_float(v[x]);
      const int n = min(a.bn - c, a.J - j0 - c);
      if (ok && row < rows && n > 0) finish32(a.e, i0 + row, j0 + c, n, f);
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, cols);
    return;
  }
  // TMEM to the memory of the CTA that finishes the row, whose wait is not one for its products.
  if (a.splits > 1)
    cluster_wait();
  else
    __syncthreads();  // every wait above is over: the pipeline's memory is free
  const int pitch = a.bn + 4;
  {
    const int row = (warp & 3) * 32 + lane, owner = row & (a.splits - 1);
    const int at = ((int)rank * (kTileI >> a.splits_log2) + (row >> a.splits_log2)) * pitch;
    const uint32_t to = (a.splits > 1 ? map_shared(part, (uint32_t)owner) : smem_u32(part)) + at * 4;
    for (int c = (warp >> 2) * 32; c < a.bn; c += 64) {
      uint32_t v[32];
      tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + c, v);
      tmem_ld_wait();
      if (row < rows) {
#pragma unroll
        for (int x = 0; x < 32; x += 4)
          if (c + x < a.bn) st_cluster_v4(to + (c + x) * 4, v[x], v[x + 1], v[x + 2], v[x + 3]);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (a.splits > 1) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, cols);
  if (!ok) return;
  const int own = (rows - (int)rank + a.splits - 1) >> a.splits_log2;
  switch (a.splits) {
    case 1: join_tile_any<1>(a, part, 0, own, i0, j0); break;
    case 2: join<2>(a, part, rank, own, i0, j0, c0, bias); break;
    case 4: join<4>(a, part, rank, own, i0, j0, c0, bias); break;
    default: join<8>(a, part, rank, own, i0, j0, c0, bias); break;
  }
}

// ------------------------------------------------------------------- CTA pairs
// Many tiles: a persistent kernel of clusters of two CTAs, each pair with one tcgen05.mma
// of 256 rows at a time (cta_group::2). A CTA stages its own 128 rows of A and half of B's
// columns, so a 256 x 256 x 64 step loads 64 KB for the pair; the accumulators of two
// tiles (2 x 256 columns of TMEM) alternate, so that eight epilogue warps empty one while
// the next is summed. The pairs take tiles in turn; eight row tiles share a group of
// columns, so the tiles in flight share their operands in L2. Bound by the tensor cores:
// 8192 x 8192 x 2048 with both outputs takes 161 to 172 us (1.6 to 1.7 PFLOP/s), 8192^3 646 us
// (1.7), both products of 4096^3 155 us (1.78).
constexpr int kPairMaxStages = 8;
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 32 * (2 + kPairEpiWarps);
constexpr int kPairGroup = 8;  // row tiles that walk the columns together

struct PairProduct {
  CUtensorMap ta, tb;
  Epilogue e;
  int I, J, nk;
  int tiles_i, tiles_j;
  bool a_mn, b_mn;
  bool any_rows;  // rows of the outputs or the residual that do not start on 16 bytes
};
constexpr int kPairCols = 256;   // columns of a tile
constexpr int kPairRounds = 24;  // tiles of a product that a pair takes at most by `live`

// One product, whose tiles the pairs take in turn (products = 1: tile p, p + pairs, ...), or
// the two of a backward pass in one launch. Then pair p takes, of product q in round k, the
// tile that its rank numbers among the live[q][k] pairs that take one; the ranks count from
// pair 0 in the first product and from the last pair in the second, so that the pairs with
// a tile less of the first get one more of the second.
struct PairArgs {
  PairProduct p[2];
  int products, stages;
  bool bf16;
  bool any_rows;  // of one of the products: a patch of shared memory for every epilogue warp
  uint16_t live[2][kPairRounds];
};

struct PairSmem {
  uint64_t full[kPairMaxStages], empty[kPairMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

constexpr int kPairStageBytes = kABytes + kPairCols * 64;  // a CTA's rows of A and half of B
constexpr int kPatchPitch = 33;
constexpr int kPatchBytes = kPairEpiWarps * 32 * kPatchPitch * 4;
size_t pair_smem_bytes(int stages, bool any_rows) {
  return 1024 + (size_t)stages * kPairStageBytes + (any_rows ? kPatchBytes : 0) + sizeof(PairSmem);
}

// The tiles of one pair in their order; every role of both CTAs walks the same.
struct PairWalk {
  const PairArgs& a;
  int pair, pairs;
  int q, ti, tj;  // the product and the tile, once next() has said there is one
  int k, base;

  __device__ __forceinline__ PairWalk(const PairArgs& args, int p, int n)
      : a(args), pair(p), pairs(n), q(0), ti(0), tj(0), k(0), base(0) {}

  __device__ __forceinline__ bool next() {
    int t;
    if (a.products == 1) {
      t = base + pair;
      base += pairs;
      if (t >= a.p[0].tiles_i * a.p[0].tiles_j) return false;
    } else {
      while (true) {
        const int rank = q == 0 ? pair : pairs - 1 - pair;
        const int live = k < kPairRounds ? a.live[q][k] : 0;
        if (rank < live) {
          t = base + rank;
          base += live;
          ++k;
          break;
        }
        if (q == 1) return false;
        q = 1;
        k = base = 0;
      }
    }
    // Groups of kPairGroup row tiles, inside a group column by column.
    const int cols = a.p[q].tiles_j, per = kPairGroup * cols, g = t / per, r = t - g * per;
    const int rows = min(kPairGroup, a.p[q].tiles_i - g * kPairGroup);
    tj = r / rows;
    ti = g * kPairGroup + r - tj * rows;
    return true;
  }
};

// n of eight values of one column, ld elements apart: the addresses are a running sum, and where all
// eight are inside no store has a condition (finish_scattered, with both for each element, took 4
// to 6 % longer for 1431 and 4096 rows of 7893).
template <typename T>
__device__ __forceinline__ void store_column(T* p, long long ld, int n, const float (&f)[8]) {
  if (n >= 8) {
#pragma unroll
    for (int q = 0; q < 8; ++q, p += ld) *p = from_f32<T>(f[q]);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q, p += ld)
      if (q < n) *p = from_f32<T>(f[q]);
  }
}
__device__ __forceinline__ void store_column(void* p, int dtype, long long at, long long ld, int n,
                                             const float (&f)[8]) {
  if (dtype == MOE_FP32)
    store_column(static_cast<float*>(p) + at, ld, n, f);
  else if (dtype == MOE_BF16)
    store_column(static_cast<__nv_bfloat16*>(p) + at, ld, n, f);
  else
    store_column(static_cast<__half*>(p) + at, ld, n, f);
}

// A warp's 32 x 32 sums (lane l has row l), `rows` x n of them inside the matrix, where rows do
// not start on 16 bytes: turned round in shared memory, so that the lanes are neighbouring
// columns of one row. (Without it, 34 us for a tile.)
__device__ __forceinline__ void finish_patch(const Epilogue& e, float* patch, long long i0, int rows, int j,
                                             int n, const float (&v)[32], int lane) {
  __syncwarp();  // the patch's last readers
#pragma unroll
  for (int x = 0; x < 32; ++x) patch[lane * kPatchPitch + x] = v[x];
  __syncwarp();
  if (lane >= n) return;
  const long long c = j + lane;
  const float bias = e.b != nullptr ? load_as_f32(e.b, e.btype, c) : 0.f;
  for (int r0 = 0; r0 < rows; r0 += 8) {
    const long long i = i0 + r0;
    const int m = rows - r0;
    float f[8], t[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int row = min(r, m - 1);
      t[r] = e.r != nullptr ? load_as_f32(e.r, e.dtype, (i + row) * e.ld_r + c) : 0.f;
      f[r] = patch[(r0 + row) * kPatchPitch + lane] + bias;
    }
    if (e.z != nullptr) store_column(e.z, e.dtype, i * e.ld_z + c, e.ld_z, m, f);
    act8_any(f, e.act);
#pragma unroll
    for (int r = 0; r < 8; ++r) f[r] += t[r];
    store_column(e.y, e.ytype, i * e.ld_y + c, e.ld_y, m, f);
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* after = base + (size_t)a.stages * kPairStageBytes;
  PairSmem& sm = *reinterpret_cast<PairSmem*>(after + (a.any_rows ? kPatchBytes : 0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool lead = crank == 0;
  PairWalk walk(a, blockIdx.x >> 1, gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&sm.full[i], 1);   // rank 0: its arrive.expect_tx (bytes of both CTAs)
      mbar_init(&sm.empty[i], 1);  // the leader's commit (multicast)
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.tfull[i], 1);                    // the leader's commit (multicast)
      mbar_init(&sm.tempty[i], 2 * kPairEpiWarps);   // rank 0: both CTAs' epilogue warps
    }
    mbar_init(&sm.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sm.abort = 0;
  }
  if (warp == 1) tmem_alloc_pair(&sm.tmem, 2 * kPairCols);
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync_all();  // both CTAs: barriers initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  wait_prior_grid();  // behind a kernel that allows it, all of the above ran beside that one

  if (warp == 0) {
    constexpr uint32_t bytes = 2 * kPairStageBytes;
    int n = 0, st = 0;
    uint32_t phase = 1;
    bool ok = true;
    while (ok && walk.next()) {
      const PairProduct& p = a.p[walk.q];
      const int i0 = walk.ti * 256 + (int)crank * 128;
      const int j0 = walk.tj * kPairCols + (int)crank * (kPairCols / 2);
      for (int kb = 0; kb < p.nk; ++kb, ++n) {
        if (!warp_pwait(&sm.empty[st], phase, &sm.abort, 0x11000000u)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* as = base + (size_t)st * kPairStageBytes;
          uint8_t* bs = as + kABytes;
          if (lead) mbar_arrive_expect_tx(&sm.full[st], bytes);
          const uint32_t fb = map_shared(&sm.full[st], 0);
          const int k0 = kb * kBlockK;
          if (p.a_mn) {
            tma_load_2d_pair(as, &p.ta, fb, i0, k0);
            tma_load_2d_pair(as + 8192, &p.ta, fb, i0 + 64, k0);
          } else {
            tma_load_2d_pair(as, &p.ta, fb, k0, i0);
          }
          if (p.b_mn) {
            for (int c = 0; c < kPairCols / 128; ++c)
              tma_load_2d_pair(bs + c * 8192, &p.tb, fb, j0 + c * 64, k0);
          } else {
            tma_load_2d_pair(bs, &p.tb, fb, k0, j0);
          }
        }
        __syncwarp();
        next_stage(st, phase, a.stages);
      }
    }
    // Every copy this CTA issued has landed once the products that read its stage are done.
    volatile int never = 0;
    const unsigned long long t0 = globaltimer();
    for (int i = max(0, n - a.stages); i < n; ++i) {
      const long long left = kWaitNs - (long long)(globaltimer() - t0);
      pwait(&sm.empty[i % a.stages], (i / a.stages) & 1, &never, left > 0 ? left : 0, g_status, 0x12000000u);
    }
  } else if (warp == 1 && lead) {
    const uint32_t s0 = (smem_u32(base) & 0x3FFFFu) >> 4;  // above lies the CTA's rank in its cluster
    int it = 0, st = 0;
    uint32_t phase = 0, at = 0;  // at: the stage's offset in 16-byte units
    bool ok = true;
    for (; ok && walk.next(); ++it) {
      const PairProduct& p = a.p[walk.q];
      const uint32_t idesc = idesc_16bit(a.bf16, p.a_mn, p.b_mn, 256, kPairCols);
      const uint64_t da = (p.a_mn ? sdesc_mn_sw128(0) : sdesc_k_sw128(0)) + s0;
      const uint64_t db = (p.b_mn ? sdesc_mn_sw128(0) : sdesc_k_sw128(0)) + s0 + (kABytes >> 4);
      const uint32_t step_a = (p.a_mn ? 2048 : 32) >> 4, step_b = (p.b_mn ? 2048 : 32) >> 4;
      const int acc = it & 1;
      if (!warp_pwait(&sm.tempty[acc], ((it >> 1) & 1) ^ 1, &sm.abort, 0x21000000u)) break;
      tc_fence_after();
      const uint32_t dt = tmem + (uint32_t)(acc * kPairCols);
      for (int kb = 0; kb < p.nk; ++kb) {
        if (!warp_pwait(&sm.full[st], phase, &sm.abort, 0x22000000u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            tc_mma_pair(dt, da + at + k * step_a, db + at + k * step_b, idesc, (kb | k) != 0 ? 1u : 0u);
          tc_commit_pair(&sm.empty[st], 0x3);
        }
        __syncwarp();
        next_stage(st, phase, a.stages);
        at = st == 0 ? 0 : at + (kPairStageBytes >> 4);
      }
      if (ok && elect_one()) tc_commit_pair(&sm.tfull[acc], 0x3);
      __syncwarp();
    }
    // Every product issued is done before either CTA frees TMEM or leaves.
    if (elect_one()) tc_commit_pair(&sm.drain, 0x1);
    __syncwarp();
    volatile int never = 0;
    pwait(&sm.drain, 0, &never, kWaitNs, g_status, 0x23000000u);
  } else if (warp >= 2) {
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quarter, half of the columns
    const uint32_t tempty[2] = {map_shared(&sm.tempty[0], 0), map_shared(&sm.tempty[1], 0)};
    int it = 0;
    for (; walk.next(); ++it) {
      const PairProduct& p = a.p[walk.q];
      const int acc = it & 1;
      if (!warp_pwait(&sm.tfull[acc], (it >> 1) & 1, &sm.abort, 0x31000000u)) break;
      tc_fence_after();
      const int row = walk.ti * 256 + (int)crank * 128 + q * 32 + lane;
      const uint32_t src = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kPairCols);
      const int c1 = (half + 1) * (kPairCols / 2);
#pragma unroll 1
      for (int c = half * (kPairCols / 2); c < c1; c += 32) {
        uint32_t v[32];
        __syncwarp();  // the stores of the columns before may have parted it; the load wants it whole
        tmem_ld32(src + c, v);
        tmem_ld_wait();
        if (c + 32 >= c1) {  // the accumulator is read: it may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty[acc]);
        }
        const int j = walk.tj * kPairCols + c;
        if (j >= p.J) continue;
        float f[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) f[x] = __uint_as_float(v[x]);
        if (p.any_rows)  // whole warps: row - lane is the first of its 32 rows
          finish_patch(p.e, reinterpret_cast<float*>(after) + (warp - 2) * 32 * kPatchPitch, row - lane,
                       min(32, p.I - (row - lane)), j, min(32, p.J - j), f, lane);
        else if (row < p.I)
          finish32(p.e, row, j, p.J - j, f);
      }
    }
  }
  // Both CTAs meet: the leader's products (which read both CTAs' shared memory and write
  // both CTAs' TMEM) are done, every copy has landed and every accumulator is read.
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * kPairCols);
}

// ------------------------------------------------------------------- few rows
// Up to 8 rows of x: the weights are read once, and their bytes are the bound, so they
// stream from global memory into registers, without the latency of a shared-memory
// pipeline, and the products are mma.sync (16 x 8 x 16; the tokens are its first eight rows,
// eight weight rows its columns). A sum over k may take the k in any order: lane (g, t)
// loads 16 bytes, elements 8 t .. 8 t + 7 of 32, of weight row g and of token row g, and
// gives the first four to one product and the rest to the next, where the products expect
// 2 t, 2 t + 1, 2 t + 8, 2 t + 9; both operands agree. `ks` warps share eight rows of the
// weights, each with a range of k; their sums are added in the warps' order. CTAs walk the
// rows of the weights, and the next batch of loads, of the next rows at the end of a row,
// is on its way while a batch is multiplied. One row by 2048 x 7168: 7.4 to 8.6 us (3.4 to
// 4 TB/s, of which 2 us are the launch and its first loads); by 8192 x 8192: 26 us, 5.2 TB/s.
// (16 rows of x in this form took 14 us for 2048 x 7168, where the tiles take 9.4.)
constexpr int kRowsMax = 8;  // rows of x
constexpr int kRowsWarps = 8;
constexpr int kRowsUnroll = 8;  // steps of 32 k whose loads are in flight together

struct RowsArgs {
  const void* x;
  const void* w;
  Epilogue e;
  long long ld_x, ld_w, blocks;  // blocks: of 8 (kRowsWarps / ks) weight rows
  int M, N, K, ks;
};

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load_tokens(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// The first n of eight elements, zeros for the others.
__device__ __forceinline__ uint4 load_tail(const unsigned short* p, int n) {
  unsigned short u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = i < n ? __ldg(p + i) : (unsigned short)0;
  return make_uint4(u[0] | (uint32_t)u[1] << 16, u[2] | (uint32_t)u[3] << 16, u[4] | (uint32_t)u[5] << 16,
                    u[6] | (uint32_t)u[7] << 16);
}
template <bool BF16>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool BF16>
__global__ void __launch_bounds__(32 * kRowsWarps, 2) linear_rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float part[2][kRowsWarps][8][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int per = kRowsWarps / a.ks;  // groups of eight weight rows in the CTA
  const int kw = warp % a.ks;
  // Rows past the end are stood in for by the last one (the first token): what they give is
  // not written, and no load needs a condition, which would keep a batch's loads apart.
  const unsigned short* x0 = static_cast<const unsigned short*>(a.x) + (g < a.M ? g * a.ld_x : 0) + t * 8;
  auto row_of = [&](long long block) {
    const long long n = min((block * per + warp / a.ks) * 8 + g, (long long)a.N - 1);
    return static_cast<const unsigned short*>(a.w) + n * a.ld_w + t * 8;
  };
  const int steps = (a.K + 31) / 32, full = a.K / 32;  // full: steps without a tail
  const int lo = (int)((long long)steps * kw / a.ks), hi = (int)((long long)steps * (kw + 1) / a.ks);
  const int end = min(hi, full);
  float d[4];
  auto product = [&](const uint4& w, const uint4& p) {
    mma_16x8x16<BF16>(d, p.x, 0u, p.y, 0u, w.x, w.y);
    mma_16x8x16<BF16>(d, p.z, 0u, p.w, 0u, w.z, w.w);
  };
  uint4 w[kRowsUnroll];
  const unsigned short* row = row_of(blockIdx.x);
  // A batch past the end loads its last step again and leaves the product out.
  if (lo < end) {
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) w[u] = load_stream(row + min(lo + u, end - 1) * 32);
  }
  int parity = 0;
  for (long long block = blockIdx.x; block < a.blocks; block += gridDim.x, parity ^= 1) {
    const unsigned short* after = block + gridDim.x < a.blocks ? row_of(block + gridDim.x) : row;
    d[0] = d[1] = d[2] = d[3] = 0.f;
    for (int s = lo; s < end; s += kRowsUnroll) {
      uint4 next[kRowsUnroll], p[kRowsUnroll];
#pragma unroll
      for (int u = 0; u < kRowsUnroll; ++u) p[u] = load_tokens(x0 + min(s + u, end - 1) * 32);
      const bool last = s + kRowsUnroll >= end;
      const unsigned short* from = last ? after : row;
      const int at = last ? lo : s + kRowsUnroll;
#pragma unroll
      for (int u = 0; u < kRowsUnroll; ++u) next[u] = load_stream(from + min(at + u, end - 1) * 32);
#pragma unroll
      for (int u = 0; u < kRowsUnroll; ++u)
        if (s + u < end) product(w[u], p[u]);
#pragma unroll
      for (int u = 0; u < kRowsUnroll; ++u) w[u] = next[u];
    }
    if (hi > full) {  // the tail of k
      const int k = full * 32;
      const bool vec = k + t * 8 + 8 <= a.K;
      product(vec ? load_stream(row + k) : load_tail(row + k, a.K - k - t * 8),
              vec ? load_tokens(x0 + k) : load_tail(x0 + k, a.K - k - t * 8));
    }
    row = after;
    part[parity][warp][g][2 * t] = d[0];
    part[parity][warp][g][2 * t + 1] = d[1];
    __syncthreads();
    // Output (token i, group q, column c): consecutive threads along the columns.
    const int wide = per * 8;
    for (int o = threadIdx.x; o < a.M * wide; o += blockDim.x) {
      const int i = o / wide, q = (o % wide) / 8, c = o % 8;
      const long long j = (block * per + q) * 8 + c;
      if (j >= a.N) continue;
      float v = 0.f;
      for (int r = 0; r < a.ks; ++r) v += part[parity][q * a.ks + r][i][c];
      finish1(a.e, i, j, v);
    }
  }
}

// ------------------------------------------------------------------- dz and db
struct ActGradArgs {
  const void* dy;
  const void* z;  // null without an activation
  void* dz;       // null: only the sums
  float* part;    // [gridDim.y][N] column sums, or null
  long long ld_dy, ld_z, ld_dz;
  int M, N, dtype, rows;  // rows of a CTA
};

// Eight elements of 16 bits as fp32.
__device__ __forceinline__ void unpack8(const uint4& u, int dtype, float (&f)[8]) {
  if (dtype == MOE_BF16)
    unpack<__nv_bfloat16>(u, f);
  else
    unpack<__half>(u, f);
}

// dz = dy act'(z) and its column sums, for the rows of a range; 256 columns a CTA. dz is
// rounded to the operands' type for the products; the sums take it unrounded. Bound by the
// bytes of dy, z and dz. VEC: rows on 16 bytes and N a multiple of 8; a thread takes eight
// columns of four rows at a time, warp w rows 4 w .. of every 32, and all eight loads leave
// before the first is used; the eight warps' sums are added in order: 10.9 us for 4096 x 1536
// (3.5 TB/s; cold, under a profiler). Otherwise a thread takes one column, so that neighbouring
// threads read neighbouring elements.
constexpr int kActRows = 4;
template <int ACT, bool VEC>
__global__ void __launch_bounds__(256) act_grad_kernel(const __grid_constant__ ActGradArgs a) {
  __shared__ float red[VEC ? 8 : 1][32][9];
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lo = blockIdx.y * a.rows, hi = min(a.M, lo + a.rows);
  const int c = blockIdx.x * 256 + threadIdx.x;  // the column whose sum this thread writes
  float sum = 0.f;
  if constexpr (VEC) {
    const int j = (blockIdx.x * 32 + lane) * 8;
    const unsigned short* dy = static_cast<const unsigned short*>(a.dy) + j;
    const unsigned short* z = static_cast<const unsigned short*>(a.z) + j;
    float s[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] = 0.f;
    if (j < a.N) {
      for (int i0 = lo + warp * kActRows; i0 < hi; i0 += 8 * kActRows) {
        uint4 du[kActRows], zu[kActRows];
#pragma unroll
        for (int r = 0; r < kActRows; ++r) {
          const long long i = min(i0 + r, hi - 1);
          du[r] = __ldg(reinterpret_cast<const uint4*>(dy + i * a.ld_dy));
          if (ACT != MOE_ACT_NONE) zu[r] = __ldg(reinterpret_cast<const uint4*>(z + i * a.ld_z));
        }
#pragma unroll
        for (int r = 0; r < kActRows; ++r) {
          if (i0 + r < hi) {
            float d[8];
            unpack8(du[r], a.dtype, d);
            if (ACT != MOE_ACT_NONE) {
              float v[8];
              unpack8(zu[r], a.dtype, v);
#pragma unroll
              for (int q = 0; q < 8; ++q) d[q] *= act_grad<ACT>(v[q]);
            }
            if (a.dz != nullptr) store8(a.dz, a.dtype, (long long)(i0 + r) * a.ld_dz + j, 8, true, d);
#pragma unroll
            for (int q = 0; q < 8; ++q) s[q] += d[q];
          }
        }
      }
    }
    if (a.part == nullptr) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) red[warp][lane][q] = s[q];
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += red[w][threadIdx.x >> 3][threadIdx.x & 7];
  } else {
    const int j = min(c, a.N - 1);
    for (int i0 = lo; i0 < hi; i0 += kActRows) {
      float d[kActRows], z[kActRows];
#pragma unroll
      for (int r = 0; r < kActRows; ++r) {
        const long long i = min(i0 + r, hi - 1);
        d[r] = load_as_f32(a.dy, a.dtype, i * a.ld_dy + j);
        z[r] = ACT != MOE_ACT_NONE ? load_as_f32(a.z, a.dtype, i * a.ld_z + j) : 0.f;
      }
#pragma unroll
      for (int r = 0; r < kActRows; ++r) {
        if (i0 + r < hi) {
          if (ACT != MOE_ACT_NONE) d[r] *= act_grad<ACT>(z[r]);
          if (a.dz != nullptr && c < a.N) store_from_f32(a.dz, a.dtype, (long long)(i0 + r) * a.ld_dz + c, d[r]);
          sum += d[r];
        }
      }
    }
    if (a.part == nullptr) return;
  }
  if (c < a.N) a.part[(size_t)blockIdx.y * a.N + c] = sum;
}

// db from the row ranges' sums: sixteen warps share the ranges, then their sums in order.
// Starts while the kernel before it ends, and the products behind it start beside it.
constexpr int kBiasWarps = 16;
__global__ void __launch_bounds__(32 * kBiasWarps)
    bias_grad_kernel(const float* part, int parts, int N, int btype, void* db) {
  __shared__ float red[kBiasWarps][32];
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < N) {
#pragma unroll 8
    for (int r = warp; r < parts; r += kBiasWarps) s += part[(size_t)r * N + c];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < N) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kBiasWarps; ++i) v += red[i][lane];
    store_from_f32(db, btype, c, v);
  }
}

// ------------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<void*> cached{nullptr};
  void* fn = cached.load(std::memory_order_relaxed);
  if (fn == nullptr) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    cached.store(fn, std::memory_order_relaxed);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

// Map of a row-major [rows][cols] matrix of 16-bit elements: boxes of box_rows x 64
// columns, 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* m, const void* p, bool bf16, long long rows, long long cols, long long ld,
              int box_rows) {
  const auto encode = encoder();
  if (encode == nullptr) return false;
  if (rows == 1) ld = (cols + 7) / 8 * 8;  // the stride of a single row is never used
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {(cuuint32_t)kBlockK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operand {
  const void* p;
  long long ld;
  bool mn;  // MN-major: [k][i or j] in memory
};

template <bool AMN, bool BMN>
cudaError_t launch_tile(const GemmArgs& a, int tiles, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(linear_tile_kernel<AMN, BMN>), &ready);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * a.splits));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes =
      1024 + tile_pipe_bytes(a.bn, a.blocks, a.stages, a.splits) + sizeof(TileSmem);
  cfg.stream = s;
  // May start beside the kernel before it, as launch_behind says: 64 x 1024 x 1024 4.8 us in a
  // graph and 5.3 without, 5.7 and 8.1 in calls one after another.
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)a.splits, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_tile_kernel<AMN, BMN>, a);
}

cudaError_t allow_pair_smem() {
  static std::atomic<uint64_t> ready{0};
  return allow_smem(reinterpret_cast<const void*>(linear_pair_kernel), &ready);
}

// Clusters of two resident at once on an idle GPU: all of a persistent launch has to be. The
// answer is 0 while the kernel may not take its shared memory; what was not told is not kept.
int pair_clusters(int num_sms) {
  static std::atomic<int> table[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return num_sms / 2;
  int n = table[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kSmemMax;
  if (allow_pair_smem() != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, linear_pair_kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return num_sms / 2;
  }
  n = std::min(n, num_sms / 2);
  table[dev].store(n, std::memory_order_relaxed);
  return n;
}

// A product D[i][j] = sum_k A(i, k) B(j, k) through the epilogue.
struct Product {
  Operand A, B;
  int I, J;
  long long K;
  Epilogue e;
  int nk() const { return (int)((K + kBlockK - 1) / kBlockK); }
  long long tiles256() const { return ((long long)I + 255) / 256 * (((long long)J + 255) / 256); }
};

bool pair_product(const Product& g, bool bf16, PairProduct* p) {
  p->e = g.e;
  p->I = g.I;
  p->J = g.J;
  p->nk = g.nk();
  p->tiles_i = (g.I + 255) / 256;
  p->tiles_j = (g.J + kPairCols - 1) / kPairCols;
  p->a_mn = g.A.mn;
  p->b_mn = g.B.mn;
  p->any_rows = !aligned_rows(g.e);
  return (g.A.mn ? make_map(&p->ta, g.A.p, bf16, g.K, g.I, g.A.ld, kBlockK)
                 : make_map(&p->ta, g.A.p, bf16, g.I, g.K, g.A.ld, kTileI)) &&
         (g.B.mn ? make_map(&p->tb, g.B.p, bf16, g.K, g.J, g.B.ld, kBlockK)
                 : make_map(&p->tb, g.B.p, bf16, g.J, g.K, g.B.ld, kPairCols / 2));
}

int launch_pairs(PairArgs& a, int pairs, cudaStream_t s) {
  a.any_rows = a.p[0].any_rows || (a.products == 2 && a.p[1].any_rows);
  a.stages = std::min<int>(kPairMaxStages, (int)((kSmemMax - pair_smem_bytes(0, a.any_rows)) / kPairStageBytes));
  if (allow_pair_smem() != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  const cudaError_t e = launch_behind(linear_pair_kernel, dim3(2 * pairs), dim3(kPairThreads),
                                      pair_smem_bytes(a.stages, a.any_rows), s, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int gemm_pair(const Product& g, bool bf16, int num_sms, cudaStream_t s) {
  PairArgs a;
  a.products = 1;
  a.bf16 = bf16;
  if (g.tiles256() > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  if (!pair_product(g, bf16, &a.p[0])) return MOE_ERR_CUDA;
  return launch_pairs(a, (int)std::min<long long>(pair_clusters(num_sms), g.tiles256()), s);
}

// How the pairs share the tiles of two products: the longer tiles (of `first`) in turn, then
// each of the others to the pairs with the least steps so far. Returns the steps of the pair
// with the most, or 0 where a pair would take more than kPairRounds tiles of one.
long long share_tiles(const Product& first, const Product& second, int pairs, uint16_t (*live)[kPairRounds]) {
  const long long n0 = first.tiles256(), n1 = second.tiles256();
  if (n0 > (long long)pairs * kPairRounds || n1 > (long long)pairs * kPairRounds) return 0;
  for (int k = 0; k < kPairRounds; ++k)
    live[0][k] = (uint16_t)std::max(0LL, std::min<long long>(pairs, n0 - (long long)k * pairs));
  // Pairs 0 .. more - 1 have `rounds` tiles of the first product, the others one less; a group's
  // pairs get their tiles of the second together, the last time perhaps only some of them.
  const long long rounds = (n0 + pairs - 1) / pairs;
  const int more = (int)(n0 - (rounds - 1) * pairs);
  const long long size[2] = {more, pairs - more};
  const long long load[2] = {rounds * first.nk(), (rounds - 1) * first.nk()};
  long long got[2] = {0, 0}, some[2] = {0, 0}, left = n1;
  while (left > 0) {
    const long long at0 = load[0] + got[0] * second.nk(), at1 = load[1] + got[1] * second.nk();
    const int g = size[1] == 0 || at0 < at1 ? 0 : 1;
    if (left >= size[g]) {
      ++got[g];
      left -= size[g];
    } else {
      some[g] = left;
      left = 0;
    }
  }
  long long most = 0;
  for (int g = 0; g < 2; ++g)
    if (size[g] > 0) most = std::max(most, load[g] + (got[g] + (some[g] > 0)) * second.nk());
  // live[1][k]: the pairs with more than k tiles. The ranks (from the last pair) hand them out
  // to the second group first, which has at least as many each.
  for (int k = 0; k < kPairRounds; ++k) {
    long long c = 0;
    for (int g = 0; g < 2; ++g) c += got[g] > k ? size[g] : got[g] == k ? some[g] : 0;
    live[1][k] = (uint16_t)c;
  }
  return got[0] > kPairRounds - 1 || got[1] > kPairRounds - 1 ? 0 : most;
}

// The product of a few token rows.
int gemm_rows(const moe_linear_args* p, const Epilogue& e, int num_sms, cudaStream_t s) {
  RowsArgs a;
  a.x = p->x;
  a.w = p->w;
  a.e = e;
  a.ld_x = p->ld_x;
  a.ld_w = p->ld_w;
  a.M = (int)p->M;
  a.N = (int)p->N;
  a.K = (int)p->K;
  // Fewer warps to a row of the weights, and so fewer sums to put together, while the rows
  // still make 1.4 CTAs for every SM, and where a warp would have less than a batch of k.
  const long long groups = (p->N + 7) / 8;
  a.ks = kRowsWarps;
  while (a.ks > 1 && (p->K < 32LL * kRowsUnroll * a.ks ||
                      10 * groups * (a.ks / 2) >= 14LL * num_sms * kRowsWarps))
    a.ks /= 2;
  const int per = kRowsWarps / a.ks;
  a.blocks = (p->N + 8 * per - 1) / (8 * per);
  const unsigned grid = (unsigned)std::min<long long>(a.blocks, 2 * num_sms);
  if (p->dtype == MOE_BF16)
    linear_rows_kernel<true><<<grid, 32 * kRowsWarps, 0, s>>>(a);
  else
    linear_rows_kernel<false><<<grid, 32 * kRowsWarps, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int gemm(const Product& g, bool bf16, int num_sms, cudaStream_t s) {
  const Operand &A = g.A, &B = g.B;
  const int I = g.I, J = g.J, nk = g.nk();
  const long long K = g.K;
  const TileChoice tc = choose_tiles(I, J, nk, B.mn, aligned_rows(g.e), num_sms);
  if (tc.bn < 0) return gemm_pair(g, bf16, num_sms, s);
  GemmArgs a{};
  a.e = g.e;
  a.I = I;
  a.J = J;
  a.nk = nk;
  a.bf16 = bf16;
  a.tiles_i = (I + kTileI - 1) / kTileI;
  a.bn = tc.bn;
  a.splits = tc.splits;
  const long long tiles = (long long)a.tiles_i * ((J + a.bn - 1) / a.bn);
  if (tiles * a.splits > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  while (1 << a.splits_log2 < a.splits) ++a.splits_log2;
  // Two blocks of k a stage share what a step of the single threads costs (0.27 us for a block of
  // 128 x 64 alone, 0.155 in pairs), where three such stages fit.
  a.blocks = a.bn <= (a.splits > 1 ? 64 : 128) ? 2 : 1;
  const size_t room = kSmemMax - 1024 - sizeof(TileSmem) - (a.splits > 1 ? part_bytes(a.bn) : 0);
  a.stages = (int)std::min<size_t>(kMaxStages, room / (a.blocks * (kABytes + a.bn * 128)));
  a.box_a = std::min(kTileI, (I + 7) / 8 * 8);
  const bool ok = (A.mn ? make_map(&a.ta, A.p, bf16, K, I, A.ld, kBlockK)
                        : make_map(&a.ta, A.p, bf16, I, K, A.ld, a.box_a)) &&
                  (B.mn ? make_map(&a.tb, B.p, bf16, K, J, B.ld, kBlockK)
                        : make_map(&a.tb, B.p, bf16, J, K, B.ld, a.bn));
  if (!ok) return MOE_ERR_CUDA;
  const cudaError_t rc = A.mn   ? launch_tile<true, true>(a, (int)tiles, s)
                         : B.mn ? launch_tile<false, true>(a, (int)tiles, s)
                                : launch_tile<false, false>(a, (int)tiles, s);
  if (rc != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// The two products of a backward pass: in one launch of the pair kernel where that is
// estimated to take less than one after the other.
int gemm_both(const Product& x, const Product& y, bool bf16, int num_sms, cudaStream_t s) {
  const Product& first = x.nk() >= y.nk() ? x : y;
  const Product& second = x.nk() >= y.nk() ? y : x;
  const int pairs = pair_clusters(num_sms);
  PairArgs a;
  const long long most =
      first.tiles256() + second.tiles256() >= pairs ? share_tiles(first, second, pairs, a.live) : 0;
  const double apart = choose_tiles(x.I, x.J, x.nk(), x.B.mn, aligned_rows(x.e), num_sms).us +
                       choose_tiles(y.I, y.J, y.nk(), y.B.mn, aligned_rows(y.e), num_sms).us;
  if (most > 0 && kPairStart + (double)most * kPairStep < apart) {
    a.products = 2;
    a.bf16 = bf16;
    if (!pair_product(first, bf16, &a.p[0]) || !pair_product(second, bf16, &a.p[1])) return MOE_ERR_CUDA;
    return launch_pairs(a, pairs, s);
  }
  const int rc = gemm(x, bf16, num_sms, s);
  return rc != MOE_OK ? rc : gemm(y, bf16, num_sms, s);
}

// Bytes on which every row of a matrix starts: 32, 16 or 0 (any).
int row_bytes(const void* p, long long ld, int dtype, long long rows) {
  for (const int b : {32, 16})
    if (aligned_to(p, b) && (rows == 1 || ld * type_bytes(dtype) % b == 0)) return b;
  return 0;
}

int check_linear(const moe_linear_args* p) {
  if (p == nullptr) return MOE_ERR_ARG;
  if (p->dtype != MOE_BF16 && p->dtype != MOE_FP16) return MOE_ERR_ARG;
  if (p->M < 0 || p->M > INT32_MAX / 2 || p->N < 1 || p->N > INT32_MAX / 2 || p->K < 1 ||
      p->K > INT32_MAX / 2)
    return MOE_ERR_ARG;
  if (p->act < MOE_ACT_NONE || p->act > MOE_ACT_SILU) return MOE_ERR_ARG;
  if (p->btype != p->dtype && p->btype != MOE_FP32) return MOE_ERR_ARG;
  return MOE_OK;
}
// A matrix that the tensor maps read: rows on 16 bytes.
bool check_operand(const void* q, long long ld, long long rows, long long cols) {
  return q != nullptr && aligned_to(q, 16) && (rows <= 1 || (ld >= cols && ld % 8 == 0 && ld <= INT32_MAX));
}
bool check_matrix(const void* q, long long ld, long long rows, long long cols, int dtype, bool need) {
  if (q == nullptr) return !need;
  return aligned_to(q, (size_t)type_bytes(dtype)) && (rows <= 1 || (ld >= cols && ld <= INT32_MAX));
}

// Backward workspace: dz (rows padded to 16 bytes), then the column sums' parts.
constexpr int kBiasParts = 256;  // row ranges of the column sums at most
size_t dz_bytes(long long M, long long N) { return ((size_t)M * ((N + 7) / 8 * 8) * 2 + 255) / 256 * 256; }

// A stream's device, current while this lives: the status words are one set for each device.
struct StreamDevice {
  int before = -1;
  bool ok = false;
  explicit StreamDevice(cudaStream_t s) {
    int dev = 0;
    if (cudaGetDevice(&before) != cudaSuccess) return;
    // The default streams have no device of their own.
    if (s == nullptr || s == cudaStreamLegacy || s == cudaStreamPerThread)
      dev = before;
    else if (cudaStreamGetDevice(s, &dev) != cudaSuccess)
      return;
    ok = dev == before || cudaSetDevice(dev) == cudaSuccess;
  }
  ~StreamDevice() {
    if (ok) cudaSetDevice(before);
  }
  StreamDevice(const StreamDevice&) = delete;
  StreamDevice& operator=(const StreamDevice&) = delete;
};

template <int ACT>
void launch_act_grad(const ActGradArgs& a, bool vec, dim3 grid, cudaStream_t s) {
  if (vec)
    act_grad_kernel<ACT, true><<<grid, 256, 0, s>>>(a);
  else
    act_grad_kernel<ACT, false><<<grid, 256, 0, s>>>(a);
}

}  // namespace

uint32_t* ops_status() {
  static std::atomic<void*> table[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return nullptr;
  void* p = table[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    table[dev].store(p, std::memory_order_relaxed);
  }
  return static_cast<uint32_t*>(p);
}

cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>* ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && ((ready->load(std::memory_order_relaxed) >> dev) & 1)) return cudaSuccess;
  // Dynamic shared memory on top of the kernel's own.
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)(kSmemMax - fa.sharedSizeBytes));
  if (e == cudaSuccess && dev < 64) ready->fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_linear(const moe_linear_args* p, moe_stream_t stream) {
  int rc = check_linear(p);
  if (rc != MOE_OK) return rc;
  if (p->ytype != p->dtype && p->ytype != MOE_FP32) return MOE_ERR_ARG;
  if (p->M == 0) return MOE_OK;
  if (!check_operand(p->x, p->ld_x, p->M, p->K) || !check_operand(p->w, p->ld_w, p->N, p->K) ||
      !check_matrix(p->y, p->ld_y, p->M, p->N, p->ytype, true) ||
      !check_matrix(p->z, p->ld_z, p->M, p->N, p->dtype, false) ||
      !check_matrix(p->r, p->ld_r, p->M, p->N, p->dtype, false) ||
      !aligned_to(p->b, (size_t)type_bytes(p->btype)))
    return MOE_ERR_ARG;
  int sms = 0;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  Epilogue e{};
  e.y = p->y;
  e.z = p->z;
  e.r = p->r;
  e.b = p->b;
  e.ld_y = p->ld_y;
  e.ld_z = p->ld_z;
  e.ld_r = p->ld_r;
  e.dtype = p->dtype;
  e.ytype = p->ytype;
  e.btype = p->btype;
  e.act = p->act;
  e.vy = row_bytes(p->y, p->ld_y, p->ytype, p->M);
  e.vz = row_bytes(p->z, p->ld_z, p->dtype, p->M);
  e.vr = row_bytes(p->r, p->ld_r, p->dtype, p->M);
  e.vb = aligned_to(p->b, 16);
  if (p->M <= kRowsMax) return gemm_rows(p, e, sms, reinterpret_cast<cudaStream_t>(stream));
  return gemm(Product{{p->x, p->ld_x, false}, {p->w, p->ld_w, false}, (int)p->M, (int)p->N, p->K, e},
              p->dtype == MOE_BF16, sms, reinterpret_cast<cudaStream_t>(stream));
}

size_t moe_linear_workspace(long long M, long long N) {
  if (M < 1 || N < 1) return 0;
  return dz_bytes(M, N) + (size_t)kBiasParts * N * sizeof(float);
}

int moe_linear_backward(const moe_linear_args* p, void* workspace, size_t workspace_bytes,
                        moe_stream_t stream) {
  int rc = check_linear(p);
  if (rc != MOE_OK) return rc;
  if (p->dwtype != p->dtype && p->dwtype != MOE_FP32) return MOE_ERR_ARG;
  if (!check_matrix(p->dw, p->ld_dw, p->N, p->K, p->dwtype, false) ||
      !aligned_to(p->db, (size_t)type_bytes(p->btype)))
    return MOE_ERR_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  if (p->M == 0) {  // no rows: the weights' gradients are zero
    if (p->dw == nullptr && p->db == nullptr) return MOE_OK;
    rc = ops_device(&sms);
    if (rc != MOE_OK) return rc;
    const size_t wt = (size_t)type_bytes(p->dwtype);
    const size_t pitch = (p->N > 1 ? (size_t)p->ld_dw : (size_t)p->K) * wt;
    if ((p->dw != nullptr && cudaMemset2DAsync(p->dw, pitch, 0, (size_t)p->K * wt, (size_t)p->N, s) !=
                                 cudaSuccess) ||
        (p->db != nullptr &&
         cudaMemsetAsync(p->db, 0, (size_t)p->N * type_bytes(p->btype), s) != cudaSuccess)) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    return MOE_OK;
  }
  const bool act = p->act != MOE_ACT_NONE;
  if (!check_matrix(p->dy, p->ld_dy, p->M, p->N, p->dtype, true) ||
      !check_matrix(p->z, p->ld_z, p->M, p->N, p->dtype, act) ||
      !check_matrix(p->dx, p->ld_dx, p->M, p->K, p->dtype, false) ||
      (p->dx != nullptr && !check_operand(p->w, p->ld_w, p->N, p->K)) ||
      (p->dw != nullptr && !check_operand(p->x, p->ld_x, p->M, p->K)) || workspace == nullptr ||
      !aligned_to(workspace, 256))
    return MOE_ERR_ARG;
  if (workspace_bytes < moe_linear_workspace(p->M, p->N)) return MOE_ERR_WORKSPACE;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  const int M = (int)p->M, N = (int)p->N;
  const bool bf16 = p->dtype == MOE_BF16;
  // dy itself where there is no activation and the tensor maps can read its rows.
  const bool copy = act || !check_operand(p->dy, p->ld_dy, M, N);
  const long long ld_dz = copy ? (p->N + 7) / 8 * 8 : p->ld_dy;
  const void* dz = copy ? workspace : p->dy;
  if (copy || p->db != nullptr) {
    ActGradArgs g{};
    g.dy = p->dy;
    g.z = p->z;
    g.dz = copy ? workspace : nullptr;
    g.part = p->db != nullptr ? reinterpret_cast<float*>(static_cast<char*>(workspace) + dz_bytes(M, N))
                              : nullptr;
    g.ld_dy = p->ld_dy;
    g.ld_z = p->ld_z;
    g.ld_dz = ld_dz;
    g.M = M;
    g.N = N;
    g.dtype = p->dtype;
    const bool vec = N % 8 == 0 && row_bytes(p->dy, p->ld_dy, p->dtype, M) != 0 &&
                     (!act || row_bytes(p->z, p->ld_z, p->dtype, M) != 0);
    const int bx = (N + 255) / 256;
    const int want = std::max(1, std::min(kBiasParts, 8 * sms / bx));  // ranges: eight CTAs an SM
    g.rows = ((M + want - 1) / want + 8 * kActRows - 1) / (8 * kActRows) * (8 * kActRows);
    const int by = (M + g.rows - 1) / g.rows;
    const dim3 grid((unsigned)bx, (unsigned)by);
    switch (p->act) {
      case MOE_ACT_RELU: launch_act_grad<MOE_ACT_RELU>(g, vec, grid, s); break;
      case MOE_ACT_GELU: launch_act_grad<MOE_ACT_GELU>(g, vec, grid, s); break;
      case MOE_ACT_GELU_TANH: launch_act_grad<MOE_ACT_GELU_TANH>(g, vec, grid, s); break;
      case MOE_ACT_SILU: launch_act_grad<MOE_ACT_SILU>(g, vec, grid, s); break;
      default: launch_act_grad<MOE_ACT_NONE>(g, vec, grid, s); break;
    }
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    if (p->db != nullptr && launch_behind(bias_grad_kernel, dim3((N + 31) / 32), dim3(32 * kBiasWarps), 0, s,
                                          (const float*)g.part, by, N, p->btype, p->db) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  Epilogue e{};
  e.dtype = p->dtype;
  e.btype = p->dtype;
  e.vb = true;
  Product to_x{{dz, ld_dz, false}, {p->w, p->ld_w, true}, M, (int)p->K, N, e};
  to_x.e.y = p->dx;
  to_x.e.ld_y = p->ld_dx;
  to_x.e.ytype = p->dtype;
  to_x.e.vy = row_bytes(p->dx, p->ld_dx, p->dtype, M);
  Product to_w{{dz, ld_dz, true}, {p->x, p->ld_x, true}, N, (int)p->K, M, e};
  to_w.e.y = p->dw;
  to_w.e.ld_y = p->ld_dw;
  to_w.e.ytype = p->dwtype;
  to_w.e.vy = row_bytes(p->dw, p->ld_dw, p->dwtype, N);
  if (p->dx != nullptr && p->dw != nullptr) return gemm_both(to_x, to_w, bf16, sms, s);
  if (p->dx != nullptr) return gemm(to_x, bf16, sms, s);
  if (p->dw != nullptr) return gemm(to_w, bf16, sms, s);
  return MOE_OK;
}

int moe_ops_status(moe_stream_t stream, int* code, int* detail) {
  uint32_t v[2] = {0, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const StreamDevice device(s);
  if (!device.ok || cudaMemcpyFromSymbolAsync(v, g_status, sizeof(v), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  if (code != nullptr) *code = (int)v[0];
  if (detail != nullptr) *detail = (int)v[1];
  return MOE_OK;
}

int moe_ops_status_clear(moe_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const StreamDevice device(s);
  void* p = device.ok ? ops_status() : nullptr;
  if (p == nullptr || cudaMemsetAsync(p, 0, sizeof(g_status), s) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
