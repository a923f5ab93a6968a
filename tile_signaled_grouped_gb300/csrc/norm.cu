// Layer norm of token rows with the residual stream's sum, and its backward pass.
//
// Forward, for each row of D elements:
//   z = x + r,  mean = sum z / D,  var = sum (z - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   y = (z - mean) rstd w + b
// z is kept in fp32 between the sum and the norm; y and the stored z are rounded once.
// A row is read once into the registers of one to 32 warps (EPT elements a thread), so the variance is the sum of squared distances from the mean: no difference
// of large sums. Bound by the bytes of the rows.
//
// Backward, with xhat = (z - mean) rstd and g = dy w:
//   dx = rstd (g - sum g / D - xhat sum(g xhat) / D) + dz
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
// A CTA walks rows; each thread owns the same columns of every row and sums their dw and
// db in registers; the CTAs' sums go to the workspace, and a second kernel adds them in
// a fixed order (no atomics: the same bits on every call).
//
// Rows longer than the registers hold are read three times (forward) or twice
// (backward) by a CTA of 1024 threads.
#include <algorithm>
#include <cmath>

#include "ops_common.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kNormParts = 304;   // CTAs of the backward kernel at most (two for each of 152 SMs)
constexpr int kLoopThreads = 1024;

struct NormArgs {
  const void* x;   // forward: x; backward: z
  const void* r;   // forward: residual or null; backward: dz or null
  const void* dy;  // backward
  const void* w;   // [D] or null (1)
  const void* b;   // [D] or null (0)
  void* y;         // forward: y; backward: dx
  void* z;         // forward: out z or null
  float* mean;     // [n]: out (or null) of the forward, in of the backward
  float* rstd;
  float* part;     // backward: [gridDim.x][2][D] sums of dw and db
  long long n, ld_x, ld_r, ld_dy, ld_y, ld_z;
  int D, wtype, wpr;  // wpr: warps of a row
  float eps;
  bool vx, vr, vdy, vy, vz;  // rows start on 16 bytes
  bool vw;                   // w and b start on 16 bytes
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

template <typename T>
struct Vec {
  static constexpr int kN = 16 / (int)sizeof(T);
};

// Elements [v N, v N + N) of a row of D as fp32; 0 past the row.
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int v, int D, bool vec, float (&f)[Vec<T>::kN]) {
  constexpr int N = Vec<T>::kN;
  const int c = v * N;
  if (vec && c + N <= D) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row) + v);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = c + i < D ? to_f32(row[c + i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store_vec(T* row, int v, int D, bool vec, const float (&f)[Vec<T>::kN]) {
  constexpr int N = Vec<T>::kN;
  const int c = v * N;
  if (vec && c + N <= D) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = from_f32<T>(f[i]);
    reinterpret_cast<uint4*>(row)[v] = u;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < D) row[c + i] = from_f32<T>(f[i]);
  }
}
// The same elements of w or b, of the rows' type or fp32; `none` where there is no array.
template <typename T>
__device__ __forceinline__ void load_param(const void* p, int wtype, int v, int D, bool vec, float none,
                                           float (&f)[Vec<T>::kN]) {
  constexpr int N = Vec<T>::kN;
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = none;
  } else if (sizeof(T) == 2 && wtype == MOE_FP32) {
    const float* q = static_cast<const float*>(p);
    const int c = v * N;
    if (vec && c + N <= D) {
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(q + c) + h);
        f[4 * h] = u.x;
        f[4 * h + 1] = u.y;
        f[4 * h + 2] = u.z;
        f[4 * h + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = c + i < D ? q[c + i] : 0.f;
    }
  } else {
    load_vec<T>(static_cast<const T*>(p), v, D, vec, f);
  }
}

// The sums of NV values over the wpr warps of a row, in every thread. red: NV x 32 floats
// of shared memory of this row's group; every thread of the CTA calls it. The warps' sums
// are added in the same order by every thread.
template <int NV>
__device__ __forceinline__ void row_sum(float (&s)[NV], float* red, int wpr, int w_in_row) {
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] = warp_sum(s[i]);
  if (wpr == 1) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) red[i * 32 + w_in_row] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] = warp_sum(lane < wpr ? red[i * 32 + lane] : 0.f);
}

// Warps of a CTA at most, by the elements a thread holds: what their registers allow.
constexpr int max_warps(int ept) { return ept == 8 ? 32 : 16; }

// wpr warps take a row, each thread EPT elements of it in 16-byte vectors.
template <typename T, int EPT>
__global__ void __launch_bounds__(32 * max_warps(EPT)) norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = Vec<T>::kN, PERV = EPT / N;
  __shared__ float red[2][32][32];  // [sum][row of the CTA][warp of the row]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / a.wpr, wr = warp % a.wpr, rows = (blockDim.x >> 5) / a.wpr;
  const long long row = (long long)blockIdx.x * rows + grp;
  const bool live = row < a.n;
  const long long rr = live ? row : 0;
  const T* x = static_cast<const T*>(a.x) + rr * a.ld_x;
  const T* r = a.r != nullptr ? static_cast<const T*>(a.r) + rr * a.ld_r : nullptr;
  const int t = wr * 32 + lane, step = a.wpr * 32;

  float f[PERV][N];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < PERV; ++i) {
    const int v = t + i * step;
    load_vec<T>(x, v, live ? a.D : 0, a.vx, f[i]);
    if (r != nullptr) {
      float g[N];
      load_vec<T>(r, v, live ? a.D : 0, a.vr, g);
#pragma unroll
      for (int e = 0; e < N; ++e) f[i][e] += g[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) s[0] += f[i][e];
  }
  row_sum<1>(s, red[0][grp], a.wpr, wr);
  const float mean = s[0] / (float)a.D;
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < PERV; ++i) {
    const int c = (t + i * step) * N;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = c + e < a.D ? f[i][e] - mean : 0.f;
      q[0] = fmaf(d, d, q[0]);
    }
  }
  row_sum<1>(q, red[1][grp], a.wpr, wr);
  if (!live) return;
  const float rstd = 1.0f / sqrtf(q[0] / (float)a.D + a.eps);
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
  T* z = a.z != nullptr ? static_cast<T*>(a.z) + row * a.ld_z : nullptr;
#pragma unroll
  for (int i = 0; i < PERV; ++i) {
    const int v = t + i * step;
    if (v * N >= a.D) break;
    if (z != nullptr) store_vec<T>(z, v, a.D, a.vz, f[i]);
    float w[N], b[N];
    load_param<T>(a.w, a.wtype, v, a.D, a.vw, 1.f, w);
    load_param<T>(a.b, a.wtype, v, a.D, a.vw, 0.f, b);
#pragma unroll
    for (int e = 0; e < N; ++e) f[i][e] = fmaf((f[i][e] - mean) * rstd, w[e], b[e]);
    store_vec<T>(y, v, a.D, a.vy, f[i]);
  }
}

// Rows of any length: one CTA a row, read three times.
template <typename T>
__global__ void __launch_bounds__(kLoopThreads) norm_long_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = Vec<T>::kN;
  __shared__ float red[2][32];
  const int wr = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* r = a.r != nullptr ? static_cast<const T*>(a.r) + row * a.ld_r : nullptr;
  auto load = [&](int v, float (&f)[N]) {
    load_vec<T>(x, v, a.D, a.vx, f);
    if (r != nullptr) {
      float g[N];
      load_vec<T>(r, v, a.D, a.vr, g);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] += g[e];
    }
  };
  float s[1] = {0.f}, q[1] = {0.f};
  const int nv = (a.D + N - 1) / N;
  for (int v = threadIdx.x; v < nv; v += blockDim.x) {
    float f[N];
    load(v, f);
#pragma unroll
    for (int e = 0; e < N; ++e) s[0] += f[e];
  }
  row_sum<1>(s, red[0], nw, wr);
  const float mean = s[0] / (float)a.D;
  for (int v = threadIdx.x; v < nv; v += blockDim.x) {
    float f[N];
    load(v, f);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = v * N + e < a.D ? f[e] - mean : 0.f;
      q[0] = fmaf(d, d, q[0]);
    }
  }
  row_sum<1>(q, red[1], nw, wr);
  const float rstd = 1.0f / sqrtf(q[0] / (float)a.D + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
  T* z = a.z != nullptr ? static_cast<T*>(a.z) + row * a.ld_z : nullptr;
  for (int v = threadIdx.x; v < nv; v += blockDim.x) {
    float f[N], w[N], b[N];
    load(v, f);
    if (z != nullptr) store_vec<T>(z, v, a.D, a.vz, f);
    load_param<T>(a.w, a.wtype, v, a.D, a.vw, 1.f, w);
    load_param<T>(a.b, a.wtype, v, a.D, a.vw, 0.f, b);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = fmaf((f[e] - mean) * rstd, w[e], b[e]);
    store_vec<T>(y, v, a.D, a.vy, f);
  }
}

// Backward. wpr warps take a row, the CTA's groups of warps take rows in turn.
template <typename T, int EPT>
__global__ void __launch_bounds__(32 * max_warps(EPT))
    norm_backward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = Vec<T>::kN, PERV = EPT / N;
  extern __shared__ float gather[];  // more than one row group: 2 x (EPT * wpr * 32)
  __shared__ float red[2][32][64];   // [row parity][row group][sum, warp]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / a.wpr, wr = warp % a.wpr, rows = (blockDim.x >> 5) / a.wpr;
  const int t = wr * 32 + lane, step = a.wpr * 32;
  const float inv_d = 1.0f / (float)a.D;

  float dw[PERV][N], db[PERV][N];
#pragma unroll
  for (int i = 0; i < PERV; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) dw[i][e] = db[i][e] = 0.f;

  int parity = 0;
  for (long long row0 = (long long)blockIdx.x * rows; row0 < a.n; row0 += (long long)gridDim.x * rows) {
    const long long row = row0 + grp;
    const bool live = row < a.n;
    const long long rr = live ? row : 0;
    const int D = live ? a.D : 0;
    const T* z = static_cast<const T*>(a.x) + rr * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + rr * a.ld_dy;
    const float mean = live ? __ldg(a.mean + row) : 0.f, rstd = live ? __ldg(a.rstd + row) : 0.f;
    float xh[PERV][N], g[PERV][N];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      load_vec<T>(z, v, D, a.vx, xh[i]);
      load_vec<T>(dy, v, D, a.vdy, g[i]);
    }
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      float w[N];
      load_param<T>(a.w, a.wtype, v, D, a.vw, 1.f, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        xh[i][e] = v * N + e < D ? (xh[i][e] - mean) * rstd : 0.f;
        dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
        db[i][e] += g[i][e];
        g[i][e] *= w[e];
        s[0] += g[i][e];
        s[1] = fmaf(g[i][e], xh[i][e], s[1]);
      }
    }
    row_sum<2>(s, red[parity][grp], a.wpr, wr);
    parity ^= 1;  // the next row's sums do not overwrite what a slow warp still reads
    if (!live) continue;
    const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
    const T* dz = a.r != nullptr ? static_cast<const T*>(a.r) + row * a.ld_r : nullptr;
    T* dx = static_cast<T*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      if (v * N >= D) break;
      float o[N];
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = 0.f;
      if (dz != nullptr) load_vec<T>(dz, v, D, a.vr, o);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = fmaf(rstd, g[i][e] - m1 - xh[i][e] * m2, o[e]);
      store_vec<T>(dx, v, D, a.vy, o);
    }
  }

  if (rows > 1) {
    // Add the row groups' sums in their order.
    const int width = PERV * step * N;
    for (int q = 0; q < rows; ++q) {
      __syncthreads();
      if (grp == q) {
#pragma unroll
        for (int i = 0; i < PERV; ++i)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            float* p = gather + ((size_t)i * N + e) * step + t;
            if (q > 0) {
              dw[i][e] += p[0];
              db[i][e] += p[width];
            }
            if (q + 1 < rows) {
              p[0] = dw[i][e];
              p[width] = db[i][e];
            }
          }
      }
    }
    if (grp != rows - 1) return;
  }
  float* pw = a.part + (size_t)blockIdx.x * 2 * a.D;
#pragma unroll
  for (int i = 0; i < PERV; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int c = (t + i * step) * N + e;
      if (c < a.D) {
        pw[c] = dw[i][e];
        pw[a.D + c] = db[i][e];
      }
    }
}

// Rows of any length: each thread adds its columns' products to the CTA's sums in the
// workspace (no other thread touches them).
template <typename T>
__global__ void __launch_bounds__(kLoopThreads) norm_backward_long_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = Vec<T>::kN;
  __shared__ float red[2][64];
  const int wr = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int nv = (a.D + N - 1) / N;
  const float inv_d = 1.0f / (float)a.D;
  float* pw = a.part + (size_t)blockIdx.x * 2 * a.D;
  float* pb = pw + a.D;
  for (int v = threadIdx.x; v < nv; v += blockDim.x)
    for (int e = 0; e < N; ++e)
      if (v * N + e < a.D) pw[v * N + e] = pb[v * N + e] = 0.f;
  int parity = 0;
  for (long long row = blockIdx.x; row < a.n; row += gridDim.x) {
    const T* z = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    auto load = [&](int v, float (&xh)[N], float (&d)[N], float (&w)[N]) {
      load_vec<T>(z, v, a.D, a.vx, xh);
      load_vec<T>(dy, v, a.D, a.vdy, d);
      load_param<T>(a.w, a.wtype, v, a.D, a.vw, 1.f, w);
#pragma unroll
      for (int e = 0; e < N; ++e) xh[e] = v * N + e < a.D ? (xh[e] - mean) * rstd : 0.f;
    };
    float s[2] = {0.f, 0.f};
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
      float xh[N], d[N], w[N];
      load(v, xh, d, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float g = d[e] * w[e];
        s[0] += g;
        s[1] = fmaf(g, xh[e], s[1]);
        if (v * N + e < a.D) {
          pw[v * N + e] = fmaf(d[e], xh[e], pw[v * N + e]);
          pb[v * N + e] += d[e];
        }
      }
    }
    row_sum<2>(s, red[parity], nw, wr);
    parity ^= 1;
    const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
    const T* dz = a.r != nullptr ? static_cast<const T*>(a.r) + row * a.ld_r : nullptr;
    T* dx = static_cast<T*>(a.y) + row * a.ld_y;
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
      float xh[N], d[N], w[N], o[N];
      load(v, xh, d, w);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = 0.f;
      if (dz != nullptr) load_vec<T>(dz, v, a.D, a.vr, o);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = fmaf(rstd, d[e] * w[e] - m1 - xh[e] * m2, o[e]);
      store_vec<T>(dx, v, a.D, a.vy, o);
    }
  }
}

// dw and db from the CTAs' sums: 32 columns a CTA, eight warps share the rows; then their
// eight sums in order.
__global__ void __launch_bounds__(256) norm_params_kernel(const float* part, int rows, int D, int wtype,
                                                         void* dw, void* db) {
  __shared__ float red[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f, q = 0.f;
  if (c < D)
    for (int r = warp; r < rows; r += 8) {
      const float* p = part + (size_t)r * 2 * D + c;
      s += p[0];
      q += p[D];
    }
  red[0][warp][lane] = s;
  red[1][warp][lane] = q;
  __syncthreads();
  if (warp < 2 && c < D) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += red[warp][i][lane];
    void* out = warp == 0 ? dw : db;
    if (out != nullptr) store_from_f32(out, wtype, c, v);
  }
}

int check_norm(const moe_norm_args* p) {
  if (p == nullptr || type_bytes(p->dtype) == 0) return MOE_ERR_ARG;
  if (p->wtype != p->dtype && p->wtype != MOE_FP32) return MOE_ERR_ARG;
  if (p->n < 0 || p->n > INT32_MAX || p->D < 1 || p->D > (1 << 24)) return MOE_ERR_ARG;
  if (!(p->eps >= 0.f) || !(p->eps < INFINITY)) return MOE_ERR_ARG;
  return MOE_OK;
}
// A matrix argument: present if `need`, element-aligned, with room for its rows.
bool check_rows(const void* q, long long ld, const moe_norm_args* p, bool need) {
  if (q == nullptr) return !need;
  return ld >= p->D && ld <= INT32_MAX && aligned_to(q, (size_t)type_bytes(p->dtype));
}
bool check_vec(const void* q, int dtype) { return aligned_to(q, (size_t)type_bytes(dtype)); }
// Whether every row of a matrix starts on 16 bytes.
bool rows16(const void* q, long long ld, const moe_norm_args* p) {
  return aligned_to(q, 16) && (p->n == 1 || ld * type_bytes(p->dtype) % 16 == 0);
}

// Warps of a row and of a CTA: a row lies in the registers of wpr warps, EPT elements a
// thread; short rows share a CTA of eight warps.
struct NormShape {
  int ept, wpr, warps;  // ept 0: the long-row kernel
};
NormShape norm_shape(const moe_norm_args* p, int num_sms, bool backward) {
  auto wpr = [&](int ept) { return (p->D + 32 * ept - 1) / (32 * ept); };
  // Few rows: as many threads a row as there are. Else few enough that a warp keeps
  // several loads in flight; the backward pass holds two sums for each element too.
  const bool few = p->n < 2 * num_sms;
  NormShape s{};
  s.ept = few || wpr(8) <= 4 ? 8 : backward || wpr(16) <= 8 ? 16 : 32;
  if (wpr(s.ept) > max_warps(s.ept)) s.ept = backward ? 16 : 32;
  s.wpr = wpr(s.ept);
  if (s.wpr > max_warps(s.ept)) return NormShape{0, 32, 32};
  s.warps = s.wpr * std::max(1, 8 / s.wpr);
  return s;
}

template <typename T>
void launch_forward(const NormArgs& a, const NormShape& sh, cudaStream_t s) {
  if (sh.ept == 0) {
    norm_long_kernel<T><<<(unsigned)a.n, kLoopThreads, 0, s>>>(a);
    return;
  }
  const int rows = sh.warps / sh.wpr, threads = 32 * sh.warps;
  const unsigned grid = (unsigned)((a.n + rows - 1) / rows);
  if (sh.ept == 8)
    norm_kernel<T, 8><<<grid, threads, 0, s>>>(a);
  else if (sh.ept == 16)
    norm_kernel<T, 16><<<grid, threads, 0, s>>>(a);
  else
    norm_kernel<T, 32><<<grid, threads, 0, s>>>(a);
}

template <typename T>
void launch_backward(const NormArgs& a, const NormShape& sh, int grid, cudaStream_t s) {
  if (sh.ept == 0) {
    norm_backward_long_kernel<T><<<grid, kLoopThreads, 0, s>>>(a);
    return;
  }
  const int rows = sh.warps / sh.wpr, threads = 32 * sh.warps;
  const size_t smem = rows > 1 ? (size_t)2 * sh.ept * sh.wpr * 32 * sizeof(float) : 0;
  if (sh.ept == 8)
    norm_backward_kernel<T, 8><<<grid, threads, smem, s>>>(a);
  else
    norm_backward_kernel<T, 16><<<grid, threads, smem, s>>>(a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_layer_norm(const moe_norm_args* p, moe_stream_t stream) {
  int rc = check_norm(p);
  if (rc != MOE_OK) return rc;
  if (p->n == 0) return MOE_OK;
  if (!check_rows(p->x, p->ld_x, p, true) || !check_rows(p->r, p->ld_r, p, false) ||
      !check_rows(p->y, p->ld_y, p, true) || !check_rows(p->z, p->ld_z, p, false) ||
      !check_vec(p->w, p->wtype) || !check_vec(p->b, p->wtype) || !aligned_to(p->mean, 4) ||
      !aligned_to(p->rstd, 4))
    return MOE_ERR_ARG;
  int sms = 0;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  NormArgs a{};
  a.x = p->x;
  a.r = p->r;
  a.w = p->w;
  a.b = p->b;
  a.y = p->y;
  a.z = p->z;
  a.mean = p->mean;
  a.rstd = p->rstd;
  a.n = p->n;
  a.ld_x = p->ld_x;
  a.ld_r = p->ld_r;
  a.ld_y = p->ld_y;
  a.ld_z = p->ld_z;
  a.D = p->D;
  a.wtype = p->wtype;
  a.eps = p->eps;
  a.vx = rows16(p->x, p->ld_x, p);
  a.vr = rows16(p->r, p->ld_r, p);
  a.vy = rows16(p->y, p->ld_y, p);
  a.vz = rows16(p->z, p->ld_z, p);
  a.vw = aligned_to(p->w, 16) && aligned_to(p->b, 16);
  const NormShape sh = norm_shape(p, sms, false);
  a.wpr = sh.wpr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->dtype == MOE_BF16)
    launch_forward<__nv_bfloat16>(a, sh, s);
  else if (p->dtype == MOE_FP16)
    launch_forward<__half>(a, sh, s);
  else
    launch_forward<float>(a, sh, s);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_layer_norm_workspace(long long n, int D) {
  if (n < 1 || D < 1) return 0;
  return (size_t)std::min<long long>(n, kNormParts) * 2 * (size_t)D * sizeof(float);
}

int moe_layer_norm_backward(const moe_norm_args* p, void* workspace, size_t workspace_bytes,
                            moe_stream_t stream) {
  int rc = check_norm(p);
  if (rc != MOE_OK) return rc;
  if (!check_vec(p->w, p->wtype) || !check_vec(p->dw, p->wtype) || !check_vec(p->db, p->wtype))
    return MOE_ERR_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  if (p->n == 0) {  // no rows: the sums are zero
    const size_t bytes = (size_t)p->D * type_bytes(p->wtype);
    if (p->dw == nullptr && p->db == nullptr) return MOE_OK;
    rc = ops_device(&sms);
    if (rc != MOE_OK) return rc;
    if ((p->dw != nullptr && cudaMemsetAsync(p->dw, 0, bytes, s) != cudaSuccess) ||
        (p->db != nullptr && cudaMemsetAsync(p->db, 0, bytes, s) != cudaSuccess))
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!check_rows(p->z, p->ld_z, p, true) || !check_rows(p->dy, p->ld_dy, p, true) ||
      !check_rows(p->dz, p->ld_dz, p, false) || !check_rows(p->dx, p->ld_dx, p, true) ||
      p->mean == nullptr || p->rstd == nullptr || !aligned_to(p->mean, 4) || !aligned_to(p->rstd, 4) ||
      workspace == nullptr || !aligned_to(workspace, 4))
    return MOE_ERR_ARG;
  if (workspace_bytes < moe_layer_norm_workspace(p->n, p->D)) return MOE_ERR_WORKSPACE;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  NormArgs a{};
  a.x = p->z;
  a.r = p->dz;
  a.dy = p->dy;
  a.w = p->w;
  a.y = p->dx;
  a.mean = p->mean;
  a.rstd = p->rstd;
  a.part = static_cast<float*>(workspace);
  a.n = p->n;
  a.ld_x = p->ld_z;
  a.ld_r = p->ld_dz;
  a.ld_dy = p->ld_dy;
  a.ld_y = p->ld_dx;
  a.D = p->D;
  a.wtype = p->wtype;
  a.vx = rows16(p->z, p->ld_z, p);
  a.vr = rows16(p->dz, p->ld_dz, p);
  a.vdy = rows16(p->dy, p->ld_dy, p);
  a.vy = rows16(p->dx, p->ld_dx, p);
  a.vw = aligned_to(p->w, 16);
  const NormShape sh = norm_shape(p, sms, true);
  a.wpr = sh.wpr;
  const int rows = sh.ept == 0 ? 1 : sh.warps / sh.wpr;
  const int grid = (int)std::min<long long>((p->n + rows - 1) / rows, std::min(kNormParts, 2 * sms));
  if (p->dtype == MOE_BF16)
    launch_backward<__nv_bfloat16>(a, sh, grid, s);
  else if (p->dtype == MOE_FP16)
    launch_backward<__half>(a, sh, grid, s);
  else
    launch_backward<float>(a, sh, grid, s);
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  if (p->dw != nullptr || p->db != nullptr)
    norm_params_kernel<<<(p->D + 31) / 32, 256, 0, s>>>(a.part, grid, p->D, p->wtype, p->dw, p->db);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
