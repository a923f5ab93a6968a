// Layer norm of token rows with the residual stream's sum, and its backward pass.
//
// Forward, for each row of D elements:
//   z = x + r,  mean = sum z / D,  var = sum (z - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   y = (z - mean) rstd w + b
// z is kept in fp32 between the sum and the norm; y and the stored z are rounded once.
// A row is read once into the registers of one to 32 warps (EPT elements a thread), so the
// variance is the sum of squared distances from the mean: no difference of large sums. Bound
// by the bytes of the rows.
//
// Backward, with xhat = (z - mean) rstd and g = dy w:
//   dx = rstd (g - sum g / D - xhat sum(g xhat) / D) + dz
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
// A CTA walks rows; each thread owns the same columns of every row and sums their dw and
// db in registers; the CTAs' sums go to the workspace, and a second kernel adds them in
// a fixed order (no atomics: the same bits on every call).
//
// Three forms: a row in registers (few rows), a ring of rows in shared memory (many), and rows
// longer than the registers hold, which a CTA of 1024 threads reads three times (forward) or
// twice (backward). One row of 7168 takes 3.9 us, 777 of 1531 in wider rows 5.2 us.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "moe_common.cuh"
#include "ops_common.cuh"

namespace moe {
namespace {

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
  int stages;        // ring kernels: rows of shared memory
  uint32_t* status;  // ring kernels: where a wait that ran out is recorded
};

// What a thread reads at once: N elements, a 16-byte vector of them (the rows start on 16
// bytes and D is a multiple of N) or one (neighbouring threads then take neighbouring
// elements: vectors taken apart would touch eight times the lines an access).
template <typename T, int N>
struct Word {
  using type = uint4;
};
template <typename T>
struct Word<T, 1> {
  using type = T;
};
__device__ __forceinline__ uint4 load_word(const uint4* p) { return __ldg(p); }
__device__ __forceinline__ float load_word(const float* p) { return __ldg(p); }
__device__ __forceinline__ __nv_bfloat16 load_word(const __nv_bfloat16* p) {
  return __ushort_as_bfloat16(__ldg(reinterpret_cast<const unsigned short*>(p)));
}
__device__ __forceinline__ __half load_word(const __half* p) {
  return __ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(p)));
}

// Words first, first + step, ... of a row of nv words, as fp32; zeros past it, and everywhere
// unless `live`. All loads leave before the first is used: none stands behind a condition
// (a word past the row is its last one, and is dropped afterwards).
template <typename T, int N, int PERV>
__device__ __forceinline__ void load_row(const T* row, int first, int step, int nv, bool live,
                                         float (&f)[PERV][N]) {
  using W = typename Word<T, N>::type;
  W u[PERV];
#pragma unroll
  for (int i = 0; i < PERV; ++i)
    u[i] = load_word(reinterpret_cast<const W*>(row) + min(first + i * step, nv - 1));
#pragma unroll
  for (int i = 0; i < PERV; ++i) {
    const bool in = live && first + i * step < nv;
    if constexpr (N == 1) {
      f[i][0] = to_f32(u[i]);
    } else {
      unpack<T>(u[i], f[i]);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) f[i][e] = in ? f[i][e] : 0.f;
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_word(T* row, int v, const float (&f)[N]) {
  if constexpr (N == 1)
    row[v] = from_f32<T>(f[0]);
  else
    reinterpret_cast<uint4*>(row)[v] = pack<T>(f);
}
// The same words of w or b, of the rows' type or fp32; `none` where there is no array. The
// type is asked once, and the loads come before a row's stores, which no later load may pass.
template <typename T, int N, int PERV>
__device__ __forceinline__ void load_params(const void* p, int wtype, int first, int step, int nv, float none,
                                            float (&f)[PERV][N]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < PERV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) f[i][e] = none;
  } else if (sizeof(T) == 2 && wtype == MOE_FP32) {
    const float* q = static_cast<const float*>(p);
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = min(first + i * step, nv - 1);
      if constexpr (N == 1) {
        f[i][0] = __ldg(q + v);
      } else {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
          const float4 u = __ldg(reinterpret_cast<const float4*>(q) + v * (N / 4) + h);
          f[i][4 * h] = u.x;
          f[i][4 * h + 1] = u.y;
          f[i][4 * h + 2] = u.z;
          f[i][4 * h + 3] = u.w;
        }
      }
    }
  } else {
    load_row<T, N, PERV>(static_cast<const T*>(p), first, step, nv, true, f);
  }
}

// The sums of NV values over the wpr warps of a row, in every thread. red: NV x 32 floats
// of shared memory of this row's group. The warps' sums are added in the same order by
// every thread. Every thread of the row's group calls it; they meet at barrier 1 + group.
// W: a power of two, at least wpr.
template <int NV, int W = 32>
__device__ __forceinline__ void row_sum(float (&s)[NV], float* red, int wpr, int w_in_row, int group) {
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] = warp_sum(s[i]);
  if (wpr == 1) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) red[i * 32 + w_in_row] = s[i];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * wpr) : "memory");
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] = (lane & (W - 1)) < wpr ? red[i * 32 + (lane & (W - 1))] : 0.f;
#pragma unroll
  for (int o = W / 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] += __shfl_xor_sync(kAll, s[i], o);
}

// Warps of a CTA at most, by the elements a thread holds: what their registers allow.
constexpr int max_warps(int ept) { return ept == 8 ? 32 : 16; }

// wpr warps take a row, each thread EPT elements of it.
template <typename T, int EPT, int N>
__global__ void __launch_bounds__(32 * max_warps(EPT)) norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int PERV = EPT / N;
  __shared__ float red[2][32][32];  // [sum][row of the CTA][warp of the row]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / a.wpr, wr = warp % a.wpr, rows = (blockDim.x >> 5) / a.wpr;
  const long long row = (long long)blockIdx.x * rows + grp;
  const bool live = row < a.n;
  const long long rr = live ? row : 0;
  const int t = wr * 32 + lane, step = a.wpr * 32, nv = a.D / N;

  float f[PERV][N];
  float s[1] = {0.f};
  load_row<T, N, PERV>(static_cast<const T*>(a.x) + rr * a.ld_x, t, step, nv, live, f);
  if (a.r != nullptr) {
    float g[PERV][N];
    load_row<T, N, PERV>(static_cast<const T*>(a.r) + rr * a.ld_r, t, step, nv, live, g);
#pragma unroll
    for (int i = 0; i < PERV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) f[i][e] += g[i][e];
  }
#pragma unroll
  for (int i = 0; i < PERV; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) s[0] += f[i][e];
  row_sum<1>(s, red[0][grp], a.wpr, wr, grp);
  const float mean = s[0] / (float)a.D;
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < PERV; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = t + i * step < nv ? f[i][e] - mean : 0.f;
      q[0] = fmaf(d, d, q[0]);
    }
  row_sum<1>(q, red[1][grp], a.wpr, wr, grp);
  if (!live) return;
  const float rstd = 1.0f / sqrtf(q[0] / (float)a.D + a.eps);
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
  T* z = a.z != nullptr ? static_cast<T*>(a.z) + row * a.ld_z : nullptr;
  constexpr int B = EPT > 16 ? 16 / N : PERV;  // words whose parameters are held at once
#pragma unroll
  for (int i0 = 0; i0 < PERV; i0 += B) {
    float w[B][N], b[B][N];
    load_params<T, N, B>(a.w, a.wtype, t + i0 * step, step, nv, 1.f, w);
    load_params<T, N, B>(a.b, a.wtype, t + i0 * step, step, nv, 0.f, b);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int v = t + (i0 + i) * step;
      if (v < nv) {
        if (z != nullptr) store_word<T, N>(z, v, f[i0 + i]);
#pragma unroll
        for (int e = 0; e < N; ++e) f[i0 + i][e] = fmaf((f[i0 + i][e] - mean) * rstd, w[i][e], b[i][e]);
        store_word<T, N>(y, v, f[i0 + i]);
      }
    }
  }
}

constexpr int kLoopWords = 4;  // words of a thread in flight in the long-row kernels

// Rows of any length: one CTA a row, read three times.
template <typename T, int N>
__global__ void __launch_bounds__(kLoopThreads) norm_long_kernel(const __grid_constant__ NormArgs a) {
  constexpr int P = kLoopWords;
  __shared__ float red[2][32];
  const int wr = threadIdx.x >> 5, nw = blockDim.x >> 5, step = blockDim.x, nv = a.D / N;
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* r = a.r != nullptr ? static_cast<const T*>(a.r) + row * a.ld_r : nullptr;
  auto load = [&](int v, float (&f)[P][N]) {
    load_row<T, N, P>(x, v, step, nv, true, f);
    if (r != nullptr) {
      float g[P][N];
      load_row<T, N, P>(r, v, step, nv, true, g);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) f[i][e] += g[i][e];
    }
  };
  float s[1] = {0.f}, q[1] = {0.f};
  for (int v = threadIdx.x; v < nv; v += P * step) {
    float f[P][N];
    load(v, f);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) s[0] += f[i][e];
  }
  row_sum<1>(s, red[0], nw, wr, 0);
  const float mean = s[0] / (float)a.D;
  for (int v = threadIdx.x; v < nv; v += P * step) {
    float f[P][N];
    load(v, f);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = v + i * step < nv ? f[i][e] - mean : 0.f;
        q[0] = fmaf(d, d, q[0]);
      }
  }
  row_sum<1>(q, red[1], nw, wr, 0);
  const float rstd = 1.0f / sqrtf(q[0] / (float)a.D + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ld_y;
  T* z = a.z != nullptr ? static_cast<T*>(a.z) + row * a.ld_z : nullptr;
  for (int v = threadIdx.x; v < nv; v += P * step) {
    float f[P][N], w[P][N], b[P][N];
    load(v, f);
    load_params<T, N, P>(a.w, a.wtype, v, step, nv, 1.f, w);
    load_params<T, N, P>(a.b, a.wtype, v, step, nv, 0.f, b);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (v + i * step >= nv) break;
      if (z != nullptr) store_word<T, N>(z, v + i * step, f[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) f[i][e] = fmaf((f[i][e] - mean) * rstd, w[i][e], b[i][e]);
      store_word<T, N>(y, v + i * step, f[i]);
    }
  }
}

// Backward. wpr warps take a row, the CTA's groups of warps take rows in turn.
template <typename T, int EPT, int N>
__global__ void __launch_bounds__(32 * max_warps(EPT))
    norm_backward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int PERV = EPT / N;
  allow_dependent_launch();
  extern __shared__ float gather[];  // more than one row group: 2 x (EPT * wpr * 32)
  __shared__ float red[2][32][64];   // [row parity][row group][sum, warp]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / a.wpr, wr = warp % a.wpr, rows = (blockDim.x >> 5) / a.wpr;
  const int t = wr * 32 + lane, step = a.wpr * 32, nv = a.D / N;
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
    const float mean = live ? __ldg(a.mean + row) : 0.f, rstd = live ? __ldg(a.rstd + row) : 0.f;
    float xh[PERV][N], g[PERV][N], o[PERV][N], w[PERV][N];
    float s[2] = {0.f, 0.f};
    load_row<T, N, PERV>(static_cast<const T*>(a.x) + rr * a.ld_x, t, step, nv, live, xh);
    load_row<T, N, PERV>(static_cast<const T*>(a.dy) + rr * a.ld_dy, t, step, nv, live, g);
    if (a.r != nullptr) {
      load_row<T, N, PERV>(static_cast<const T*>(a.r) + rr * a.ld_r, t, step, nv, live, o);
    } else {
#pragma unroll
      for (int i = 0; i < PERV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) o[i][e] = 0.f;
    }
    load_params<T, N, PERV>(a.w, a.wtype, t, step, nv, 1.f, w);
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        xh[i][e] = t + i * step < nv ? (xh[i][e] - mean) * rstd : 0.f;
        dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
        db[i][e] += g[i][e];
        g[i][e] *= w[i][e];
        s[0] += g[i][e];
        s[1] = fmaf(g[i][e], xh[i][e], s[1]);
      }
    }
    row_sum<2>(s, red[parity][grp], a.wpr, wr, grp);
    parity ^= 1;  // the next row's sums do not overwrite what a slow warp still reads
    if (!live) continue;
    const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
    T* dx = static_cast<T*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      if (v >= nv) break;
#pragma unroll
      for (int e = 0; e < N; ++e) o[i][e] = fmaf(rstd, g[i][e] - m1 - xh[i][e] * m2, o[i][e]);
      store_word<T, N>(dx, v, o[i]);
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
      const int v = t + i * step;
      if (v < nv) {
        pw[v * N + e] = dw[i][e];
        pw[a.D + v * N + e] = db[i][e];
      }
    }
}

// Rows of any length: each thread adds its columns' products to the CTA's sums in the
// workspace (no other thread touches them).
template <typename T, int N>
__global__ void __launch_bounds__(kLoopThreads)
    norm_backward_long_kernel(const __grid_constant__ NormArgs a) {
  constexpr int P = N > 1 ? 1 : kLoopWords;
  __shared__ float red[2][64];
  allow_dependent_launch();
  const int wr = threadIdx.x >> 5, nw = blockDim.x >> 5, step = blockDim.x, nv = a.D / N;
  const float inv_d = 1.0f / (float)a.D;
  float* pw = a.part + (size_t)blockIdx.x * 2 * a.D;
  float* pb = pw + a.D;
  for (int v = threadIdx.x; v < nv; v += step)
#pragma unroll
    for (int e = 0; e < N; ++e) pw[v * N + e] = pb[v * N + e] = 0.f;
  int parity = 0;
  for (long long row = blockIdx.x; row < a.n; row += gridDim.x) {
    const T* z = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    auto load = [&](int v, float (&xh)[P][N], float (&d)[P][N], float (&w)[P][N]) {
      load_row<T, N, P>(z, v, step, nv, true, xh);
      load_row<T, N, P>(dy, v, step, nv, true, d);
      load_params<T, N, P>(a.w, a.wtype, v, step, nv, 1.f, w);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) xh[i][e] = v + i * step < nv ? (xh[i][e] - mean) * rstd : 0.f;
    };
    float s[2] = {0.f, 0.f};
    for (int v = threadIdx.x; v < nv; v += P * step) {
      float xh[P][N], d[P][N], w[P][N], sw[P][N], sb[P][N];
      load(v, xh, d, w);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int c = min(v + i * step, nv - 1) * N + e;
          sw[i][e] = pw[c];
          sb[i][e] = pb[c];
        }
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float g = d[i][e] * w[i][e];
          s[0] += g;
          s[1] = fmaf(g, xh[i][e], s[1]);
          if (v + i * step < nv) {
            pw[(v + i * step) * N + e] = fmaf(d[i][e], xh[i][e], sw[i][e]);
            pb[(v + i * step) * N + e] = sb[i][e] + d[i][e];
          }
        }
    }
    row_sum<2>(s, red[parity], nw, wr, 0);
    parity ^= 1;
    const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
    const T* dz = a.r != nullptr ? static_cast<const T*>(a.r) + row * a.ld_r : nullptr;
    T* dx = static_cast<T*>(a.y) + row * a.ld_y;
    for (int v = threadIdx.x; v < nv; v += P * step) {
      float xh[P][N], d[P][N], w[P][N], o[P][N];
      load(v, xh, d, w);
      if (dz != nullptr) {
        load_row<T, N, P>(dz, v, step, nv, true, o);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int e = 0; e < N; ++e) o[i][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (v + i * step >= nv) break;
#pragma unroll
        for (int e = 0; e < N; ++e) o[i][e] = fmaf(rstd, d[i][e] * w[i][e] - m1 - xh[i][e] * m2, o[i][e]);
        store_word<T, N>(dx, v + i * step, o[i]);
      }
    }
  }
}

// ------------------------------------------------------------------- ring kernels
// Long matrices: persistent CTAs whose groups of warps keep the next rows coming in (bulk copies
// into a ring of shared memory), so that the loads never stop for the reductions of a row: the
// kernels above only load between a CTA's start and its first reduction (16384 x 4096 bf16 with
// a residual: 143 us against 94, 5.7 TB/s; backward of 8192 x 7168: 257 us against 85, 5.5 TB/s).
// wpr warps share a row; a CTA holds as many such groups as its warps allow, each with a ring of
// its own. Rows that start anywhere come as the 16-byte blocks that they touch, and vectors are
// shifted together from two neighbours (8192 x 4097 fp16 with a residual: 230 us by the element
// against 97, backward 239 against 139).
constexpr int kMaxRing = 4;  // 2, 3, 4 and 8 stages measured within 2 %
constexpr int kMaxGroups = 16;
// Elements a thread. What a row costs beside its elements (waits, reductions, addresses:
// some 200 instructions a thread) bounds these kernels before the memory does, so a thread
// takes as many as the registers hold: 32 forward (16 for rows that one warp holds so), 16
// backward with its two sums (8: 148 us against 89 for 8192 x 7168).
constexpr int kForwardEpt = 32, kBackwardEpt = 16;
constexpr long long kWaitNs = 4000000000LL;  // bound of every device-side wait

struct RingState {
  uint64_t full[kMaxRing];
  int abort;
  int stop;  // the first step whose row the leader did not see land in time; -1: none
};

// A group's ring: a stage holds a row of x (forward) or of z and dy (backward), and of r
// if there is one. What it can read from the launch's arguments it does not keep.
// AL: rows start on 16 bytes and D is a multiple of a vector. Otherwise a stage holds the
// 16-byte blocks that a row touches, and the row starts in it where it starts in the first.
template <typename T, bool BACK, bool AL>
struct Ring {
  const NormArgs& a;
  uint8_t* smem;
  RingState* st;
  int first, stride;  // the group's rows: first, first + stride, ...

  __device__ __forceinline__ uint32_t bytes() const { return (uint32_t)a.D * sizeof(T); }
  __device__ __forceinline__ uint32_t pitch() const { return AL ? bytes() : (bytes() + 15u) / 16u * 16u + 16u; }
  __device__ __forceinline__ int mats() const { return (BACK ? 2 : 1) + (a.r != nullptr ? 1 : 0); }
  // Matrix m's row in stage i.
  __device__ __forceinline__ const uint4* stage(int i, int m) const {
    return reinterpret_cast<const uint4*>(smem + (size_t)(i * mats() + m) * pitch());
  }
  // The blocks that a row of p touches, [*lo, *hi), without those that reach out of the matrix
  // (its first and last row alone have such).
  __device__ __forceinline__ void blocks(const T* p, long long ld, long long row, uintptr_t* lo,
                                         uintptr_t* hi) const {
    const uintptr_t begin = reinterpret_cast<uintptr_t>(p), at = begin + (uintptr_t)(row * ld) * sizeof(T);
    const uintptr_t end = begin + (uintptr_t)((a.n - 1) * ld + a.D) * sizeof(T);
    *lo = at & ~(uintptr_t)15;
    *hi = (at + bytes() + 15) & ~(uintptr_t)15;
    if (*lo < begin) *lo += 16;
    if (*hi > end) *hi -= 16;
  }
  // Row `row` of p to `to`: the blocks by a bulk copy; what lies outside them by hand.
  __device__ __forceinline__ void copy(uint8_t* to, const T* p, long long ld, long long row,
                                       uint64_t* bar) const {
    uintptr_t lo, hi;
    blocks(p, ld, row, &lo, &hi);
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) + (uintptr_t)(row * ld) * sizeof(T);
    uint8_t* place = to + (lo - (at & ~(uintptr_t)15));
    bulk_load(place, reinterpret_cast<const void*>(lo), (uint32_t)(hi - lo), bar);
  }
  __device__ __forceinline__ void edges(uint8_t* to, const T* p, long long ld, long long row) const {
    uintptr_t lo, hi;
    blocks(p, ld, row, &lo, &hi);
    const T* src = p + row * ld;
    T* dst = reinterpret_cast<T*>(to + (reinterpret_cast<uintptr_t>(src) & 15));
    for (int e = 0; e < a.D && reinterpret_cast<uintptr_t>(src + e) < lo; ++e) dst[e] = src[e];
    for (int e = a.D - 1; e >= 0 && reinterpret_cast<uintptr_t>(src + e) >= hi; --e) dst[e] = src[e];
  }
  __device__ __forceinline__ uint32_t size(const T* p, long long ld, long long row) const {
    uintptr_t lo, hi;
    blocks(p, ld, row, &lo, &hi);
    return (uint32_t)(hi - lo);
  }
  // The group's leader: stage i receives row `row`.
  __device__ __forceinline__ void load(int i, long long row) const {
    uint64_t* bar = &st->full[i];
    uint8_t* to = smem + (size_t)(i * mats()) * pitch();
    const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.dy);
    const T* r = static_cast<const T*>(a.r);
    uint8_t *to_dy = to + pitch(), *to_r = to + (BACK ? 2 : 1) * pitch();
    if constexpr (AL) {
      mbar_arrive_expect_tx(bar, bytes() * mats());
      bulk_load(to, x + row * a.ld_x, bytes(), bar);
      if (BACK) bulk_load(to_dy, dy + row * a.ld_dy, bytes(), bar);
      if (r != nullptr) bulk_load(to_r, r + row * a.ld_r, bytes(), bar);
    } else {
      if (row == 0 || row == a.n - 1) {
        edges(to, x, a.ld_x, row);
        if (BACK) edges(to_dy, dy, a.ld_dy, row);
        if (r != nullptr) edges(to_r, r, a.ld_r, row);
      }
      // Orders what was written by hand into the stage, now or before, with the copies.
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive_expect_tx(bar, size(x, a.ld_x, row) + (BACK ? size(dy, a.ld_dy, row) : 0u) +
                                     (r != nullptr ? size(r, a.ld_r, row) : 0u));
      copy(to, x, a.ld_x, row, bar);
      if (BACK) copy(to_dy, dy, a.ld_dy, row, bar);
      if (r != nullptr) copy(to_r, r, a.ld_r, row, bar);
    }
  }
  // The same once every thread has read the stage. After a wait of the leader's that ran out
  // nothing is loaded any more: that stage's copy may be in flight, and its barrier, still in
  // the old phase, must not be armed a second time.
  __device__ __forceinline__ void refill(int i, long long row) const {
    if (*(volatile int*)&st->stop < 0) load(i, row);
  }
};

// Every thread of the CTA, once `st` of its group is set; `leader`: the group's first thread.
template <typename T, bool BACK, bool AL>
__device__ __forceinline__ void ring_begin(const Ring<T, BACK, AL>& g, bool leader) {
  if (leader) {
    for (int i = 0; i < g.a.stages; ++i) mbar_init(&g.st->full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    g.st->abort = 0;
    g.st->stop = -1;
  }
  __syncthreads();
  if (leader)
    for (int i = 0; i < g.a.stages; ++i) {
      const long long row = g.first + (long long)i * g.stride;
      if (row < g.a.n) g.load(i, row);
    }
}
// The stage's phase is complete: the row of step `it` is there. After a wait that ran out the group carries on
// with what is there (the status says that its results are void), so that every thread
// meets the same barriers.
template <typename T, bool BACK, bool AL>
__device__ __forceinline__ void ring_wait(const Ring<T, BACK, AL>& g, int stage, int phase, bool leader,
                                          int it) {
  if (!mbar_wait_bounded(&g.st->full[stage], phase, &g.st->abort, kWaitNs, g.a.status, 0x51000000u) &&
      leader && g.st->stop < 0)
    g.st->stop = it;
}
// After an abort: the copies in flight land before the group leaves. It loaded all of its `rows`
// rows, or those up to the stages ahead of the step where it stopped.
template <typename T, bool BACK, bool AL>
__device__ __forceinline__ void ring_end(const Ring<T, BACK, AL>& g, bool leader, int rows) {
  if (leader && *(volatile int*)&g.st->abort) {
    volatile int never = 0;
    if (g.st->stop >= 0) rows = min(rows, g.st->stop + g.a.stages);
    for (int it = max(0, rows - g.a.stages); it < rows; ++it)
      mbar_wait_bounded(&g.st->full[it % g.a.stages], (it / g.a.stages) & 1, &never, kWaitNs, g.a.status,
                        0x52000000u);
  }
}

// Two fp32 values in a register pair: one instruction works on both (the same roundings as
// two). Backward of 8192 x 7168: 89 -> 86 us, of 2048 x 7168: 36 -> 32 us. The pairs need more
// registers: the forward kernel takes 128 a thread (with 64 they made it slower, 90 -> 98 us).
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  }
  __device__ __forceinline__ float2 get() const {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
  }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}
template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& u, F2 (&f)[Vec<T>::kN / 2]) {
  float g[Vec<T>::kN];
  unpack<T>(u, g);
#pragma unroll
  for (int i = 0; i < Vec<T>::kN / 2; ++i) f[i] = F2(g[2 * i], g[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const F2 (&f)[Vec<T>::kN / 2]) {
  float g[Vec<T>::kN];
#pragma unroll
  for (int i = 0; i < Vec<T>::kN / 2; ++i) {
    const float2 p = f[i].get();
    g[2 * i] = p.x;
    g[2 * i + 1] = p.y;
  }
  return pack<T>(g);
}
// Sixteen bytes from byte `at` (below 16) of two neighbouring words.
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, uint32_t at) {
  uint32_t w[5];
  switch (at >> 2) {  // the same for the whole warp
    case 0: w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x; break;
    case 1: w[0] = lo.y, w[1] = lo.z, w[2] = lo.w, w[3] = hi.x, w[4] = hi.y; break;
    case 2: w[0] = lo.z, w[1] = lo.w, w[2] = hi.x, w[3] = hi.y, w[4] = hi.z; break;
    default: w[0] = lo.w, w[1] = hi.x, w[2] = hi.y, w[3] = hi.z, w[4] = hi.w; break;
  }
  const uint32_t bits = (at & 3u) * 8u;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}
// Where a row of p starts in its first 16-byte block.
template <typename T>
__device__ __forceinline__ uint32_t block_offset(const T* p, long long ld, long long row) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(p + row * ld) & 15);
}
// Vector v of a row in the ring that starts `at` bytes into its first block.
template <bool AL>
__device__ __forceinline__ uint4 ring_vec(const uint4* row, int v, uint32_t at) {
  return AL ? row[v] : shifted(row[v], row[v + 1], at);
}
// Zeros past the row's D elements in its last vector.
template <typename T, bool AL>
__device__ __forceinline__ void trim(F2 (&f)[Vec<T>::kN / 2], int v, int D) {
  constexpr int N = Vec<T>::kN;
  if constexpr (!AL) {
    if (v * N + N <= D) return;
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float2 p = f[e].get();
      f[e] = F2(v * N + 2 * e < D ? p.x : 0.f, v * N + 2 * e + 1 < D ? p.y : 0.f);
    }
  }
}
// Vector v (v < nv) of each lane to a row of D elements; a warp's lanes hold neighbouring
// vectors. Where the row does not start on 16 bytes, the part of its neighbour's vector that
// belongs to a lane's 16-byte block comes to it by a shuffle, and only the ends of the warp's
// run of vectors and of the row are stored by the element. Every lane of the warp calls it.
template <typename T, bool AL>
__device__ __forceinline__ void store_vecs(T* row, int v, int nv, int D, const uint4& u) {
  constexpr int N = Vec<T>::kN;
  if constexpr (AL) {
    if (v < nv) reinterpret_cast<uint4*>(row)[v] = u;
  } else {
    const int lane = threadIdx.x & 31;
    const uint32_t at = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15);
    const int skip = (int)(at / sizeof(T));  // elements of a block that are the vector's before
    uint4 p;
    p.x = __shfl_up_sync(kAll, u.x, 1);
    p.y = __shfl_up_sync(kAll, u.y, 1);
    p.z = __shfl_up_sync(kAll, u.z, 1);
    p.w = __shfl_up_sync(kAll, u.w, 1);
    const uint4 b = at == 0 ? u : shifted(p, u, 16u - at);
    const bool joined = at == 0 || (lane > 0 && v > 0);  // b is the block from element v N - skip
    const int from = v * N - skip;
    if (v < nv && joined && from + N <= D) {
      *reinterpret_cast<uint4*>(row + from) = b;
    } else if (v < nv) {
      const uint4 src = make_uint4(joined ? b.x : u.x, joined ? b.y : u.y, joined ? b.z : u.z,
                                   joined ? b.w : u.w);
      const T* e = reinterpret_cast<const T*>(&src);
      const int first = joined ? from : v * N, count = min(joined ? N : N - skip, D - first);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < count) row[first + i] = e[i];
    }
    if (v < nv && skip > 0 && (lane == 31 || v + 1 == nv)) {  // no lane after this one takes its end
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i >= N - skip && v * N + i < D) row[v * N + i] = e[i];
    }
  }
}

// The parameters of a thread's columns, kept in registers as they lie in memory: WT is the
// rows' type or float.
template <typename T, typename WT>
struct Params {
  static constexpr int kWords = Vec<T>::kN * (int)sizeof(WT) / 16;  // 16-byte words of a vector
  uint4 u[kWords];
  // `none` without an array, and past its D elements.
  __device__ __forceinline__ void load(const void* p, int v, int D, float none) {
    constexpr int E = Vec<WT>::kN;
    const bool aligned = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int c = (v * kWords + i) * E;
      if (p != nullptr && aligned && c + E <= D) {
        u[i] = __ldg(static_cast<const uint4*>(p) + v * kWords + i);
      } else {
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
          f[e] = p != nullptr && c + e < D ? to_f32(static_cast<const WT*>(p)[c + e]) : none;
        u[i] = pack<WT>(f);
      }
    }
  }
  __device__ __forceinline__ void get(F2 (&f)[Vec<T>::kN / 2]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      // Unpacked anew for every row: left to itself the compiler keeps the unpacked values
      // over the loop, twice the registers, and spills.
      uint4 c = u[i];
      asm volatile("" : "+r"(c.x), "+r"(c.y), "+r"(c.z), "+r"(c.w));
      F2 q[Vec<WT>::kN / 2];
      unpack_pairs<WT>(c, q);
#pragma unroll
      for (int e = 0; e < Vec<WT>::kN / 2; ++e) f[i * (Vec<WT>::kN / 2) + e] = q[e];
    }
  }
};

// The parameters stand in shared memory as they lie in global memory (the registers are the
// row's). z leaves before the reductions, the row's distances from the mean replace it.
template <typename T, typename WT, int EPT, bool AL>
__global__ void __launch_bounds__(512, 1) norm_ring_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = Vec<T>::kN, PERV = EPT / N, WORDS = N * (int)sizeof(WT) / 16;
  extern __shared__ __align__(128) uint8_t ring_smem[];  // [2][D] parameters, then the rings
  __shared__ RingState rs[kMaxGroups];
  __shared__ float red[kMaxGroups][2][32];
  const int warp = threadIdx.x >> 5, grp = warp / a.wpr, wr = warp % a.wpr;
  const int groups = (blockDim.x >> 5) / a.wpr;
  const int t = wr * 32 + (threadIdx.x & 31), step = a.wpr * 32, nv = (a.D + N - 1) / N;
  const int words = nv * WORDS;  // 16-byte words of a parameter
  uint4* ws = reinterpret_cast<uint4*>(ring_smem);
  for (int i = threadIdx.x; i < nv; i += blockDim.x) {
    Params<T, WT> w, b;
    w.load(a.w, i, a.D, 1.f);
    b.load(a.b, i, a.D, 0.f);
#pragma unroll
    for (int h = 0; h < WORDS; ++h) {
      ws[i * WORDS + h] = w.u[h];
      ws[words + i * WORDS + h] = b.u[h];
    }
  }
  const int mats = a.r != nullptr ? 2 : 1;
  // At most 2^31 rows, and an index past n by less than a stride: 64 bits where it matters.
  const int first = (int)min((long long)blockIdx.x * groups + grp, a.n);
  Ring<T, false, AL> g{a, ring_smem + (size_t)words * 32, &rs[grp], first, (int)gridDim.x * groups};
  g.smem += (size_t)grp * a.stages * mats * g.pitch();
  ring_begin(g, t == 0);
  const float inv_d = 1.0f / (float)a.D;
  int it = 0, st = 0, phase = 0;
  for (long long row = g.first; row < a.n; row += g.stride, ++it) {
    T* y = static_cast<T*>(a.y) + row * a.ld_y;
    T* z = a.z != nullptr ? static_cast<T*>(a.z) + row * a.ld_z : nullptr;
    ring_wait(g, st, phase, t == 0, it);
    const uint4 *xs = g.stage(st, 0), *rs_row = g.stage(st, 1);
    const uint32_t at_x = AL ? 0u : block_offset(static_cast<const T*>(a.x), a.ld_x, row);
    const uint32_t at_r = AL || mats == 1 ? 0u : block_offset(static_cast<const T*>(a.r), a.ld_r, row);
    F2 f[PERV][N / 2];
    F2 s2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      if (v < nv) {
        unpack_pairs<T>(ring_vec<AL>(xs, v, at_x), f[i]);
        if (mats == 2) {
          F2 q[N / 2];
          unpack_pairs<T>(ring_vec<AL>(rs_row, v, at_r), q);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) f[i][e] = f[i][e] + q[e];
        }
        trim<T, AL>(f[i], v, a.D);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) s2 = s2 + f[i][e];
      }
    }
    float s[1] = {s2.get().x + s2.get().y};
    row_sum<1, 16>(s, red[grp][0], a.wpr, wr, grp);
    // Every thread has read the stage: it takes the row `stages` ahead. (row_sum's barrier orders
    // those reads before the copy; a group of one warp meets here.)
    __syncwarp();
    const long long next = row + (long long)a.stages * g.stride;
    if (t == 0 && next < a.n) g.refill(st, next);
    if (++st == a.stages) {
      st = 0;
      phase ^= 1;
    }
    const float mean = s[0] * inv_d;
    const F2 minus_mean(-mean, -mean);
    F2 q2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      if (z != nullptr) store_vecs<T, AL>(z, v, nv, a.D, pack_pairs<T>(f[i]));
      if (v < nv) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) f[i][e] = f[i][e] + minus_mean;
        trim<T, AL>(f[i], v, a.D);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) q2 = fma2(f[i][e], f[i][e], q2);
      }
    }
    float q[1] = {q2.get().x + q2.get().y};
    row_sum<1, 16>(q, red[grp][1], a.wpr, wr, grp);
    const float rstd = 1.0f / sqrtf(q[0] * inv_d + a.eps);
    if (t == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    const F2 rr(rstd, rstd);
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      if (AL && v >= nv) break;
#pragma unroll
      for (int h = 0; h < WORDS; ++h) {
        const int at = (AL ? v : min(v, nv - 1)) * WORDS + h;
        F2 wf[Vec<WT>::kN / 2], bf[Vec<WT>::kN / 2];
        unpack_pairs<WT>(ws[at], wf);
        unpack_pairs<WT>(ws[words + at], bf);
#pragma unroll
        for (int e = 0; e < Vec<WT>::kN / 2; ++e) {
          F2& x = f[i][h * (Vec<WT>::kN / 2) + e];
          x = fma2(x * rr, wf[e], bf[e]);
        }
      }
      store_vecs<T, AL>(y, v, nv, a.D, pack_pairs<T>(f[i]));
    }
  }
  ring_end(g, t == 0, it);
}

template <typename T, typename WT, int EPT, bool AL>
__global__ void __launch_bounds__(32 * max_warps(EPT))
    norm_backward_ring_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = Vec<T>::kN, PERV = EPT / N;
  allow_dependent_launch();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ RingState rs[kMaxGroups];
  __shared__ float red[kMaxGroups][2][64];
  const int warp = threadIdx.x >> 5, grp = warp / a.wpr, wr = warp % a.wpr;
  const int groups = (blockDim.x >> 5) / a.wpr;
  const int t = wr * 32 + (threadIdx.x & 31), step = a.wpr * 32, nv = (a.D + N - 1) / N;
  const float inv_d = 1.0f / (float)a.D;
  // At most 2^31 rows, and an index past n by less than a stride: 64 bits where it matters.
  const int first = (int)min((long long)blockIdx.x * groups + grp, a.n);
  Ring<T, true, AL> g{a, ring_smem, &rs[grp], first, (int)gridDim.x * groups};
  g.smem += (size_t)grp * a.stages * g.mats() * g.pitch();
  ring_begin(g, t == 0);

  Params<T, WT> w[PERV];
#pragma unroll
  for (int i = 0; i < PERV; ++i) {
    const int v = t + i * step;
    w[i].load(a.w, v, a.D, 1.f);
  }
  F2 dw[PERV][N / 2], db[PERV][N / 2];
#pragma unroll
  for (int i = 0; i < PERV; ++i)
#pragma unroll
    for (int e = 0; e < N / 2; ++e) dw[i][e] = db[i][e] = F2(0.f, 0.f);
  float mean_n = 0.f, rstd_n = 0.f;
  if (g.first < a.n) {
    mean_n = __ldg(a.mean + g.first);
    rstd_n = __ldg(a.rstd + g.first);
  }
  int it = 0, st = 0, phase = 0;
  for (long long row = g.first; row < a.n; row += g.stride, ++it) {
    const float mean = mean_n, rstd = rstd_n;
    if (row + g.stride < a.n) {  // the next row's, a row ahead
      mean_n = __ldg(a.mean + row + g.stride);
      rstd_n = __ldg(a.rstd + row + g.stride);
    }
    ring_wait(g, st, phase, t == 0, it);
    const uint4 *zs = g.stage(st, 0), *ds = g.stage(st, 1), *us = g.stage(st, 2);
    const uint32_t at_z = AL ? 0u : block_offset(static_cast<const T*>(a.x), a.ld_x, row);
    const uint32_t at_d = AL ? 0u : block_offset(static_cast<const T*>(a.dy), a.ld_dy, row);
    const uint32_t at_u =
        AL || a.r == nullptr ? 0u : block_offset(static_cast<const T*>(a.r), a.ld_r, row);
    const F2 minus_mean(-mean, -mean), rr(rstd, rstd);
    F2 xh[PERV][N / 2], d[PERV][N / 2];
    uint4 up[PERV];
    F2 s1(0.f, 0.f), s2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      if (v < nv) {
        F2 wf[N / 2];
        unpack_pairs<T>(ring_vec<AL>(zs, v, at_z), xh[i]);
        unpack_pairs<T>(ring_vec<AL>(ds, v, at_d), d[i]);
        if (a.r != nullptr) up[i] = ring_vec<AL>(us, v, at_u);
        w[i].get(wf);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) xh[i][e] = (xh[i][e] + minus_mean) * rr;
        trim<T, AL>(xh[i], v, a.D);
        trim<T, AL>(d[i], v, a.D);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          dw[i][e] = fma2(d[i][e], xh[i][e], dw[i][e]);
          db[i][e] = db[i][e] + d[i][e];
          d[i][e] = d[i][e] * wf[e];
          s1 = s1 + d[i][e];
          s2 = fma2(d[i][e], xh[i][e], s2);
        }
      }
    }
    float s[2] = {s1.get().x + s1.get().y, s2.get().x + s2.get().y};
    row_sum<2, 16>(s, red[grp][it & 1], a.wpr, wr, grp);
    __syncwarp();  // as in the forward kernel: the sums need nothing of `up`
    const long long next = row + (long long)a.stages * g.stride;
    if (t == 0 && next < a.n) g.refill(st, next);
    if (++st == a.stages) {
      st = 0;
      phase ^= 1;
    }
    const F2 m1(-s[0] * inv_d, -s[0] * inv_d), m2(-s[1] * inv_d, -s[1] * inv_d);
    T* dx = static_cast<T*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int i = 0; i < PERV; ++i) {
      const int v = t + i * step;
      if (AL && v >= nv) break;
      F2 o[N / 2];
      if (a.r != nullptr) {
        unpack_pairs<T>(up[i], o);
      } else {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) o[e] = F2(0.f, 0.f);
      }
#pragma unroll
      for (int e = 0; e < N / 2; ++e) o[e] = fma2(rr, fma2(xh[i][e], m2, d[i][e] + m1), o[e]);
      store_vecs<T, AL>(dx, v, nv, a.D, pack_pairs<T>(o));
    }
  }
  ring_end(g, t == 0, it);
  if (groups > 1) {
    F2* gather = reinterpret_cast<F2*>(ring_smem);  // 2 x (EPT x step floats), after the ring
    const int width = EPT * step / 2;
    for (int q = 0; q < groups; ++q) {  // the groups' sums in their order
      __syncthreads();
      if (grp == q) {
#pragma unroll
        for (int i = 0; i < PERV; ++i)
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            F2* p = gather + ((size_t)i * (N / 2) + e) * step + t;
            if (q > 0) {
              dw[i][e] = dw[i][e] + p[0];
              db[i][e] = db[i][e] + p[width];
            }
            if (q + 1 < groups) {
              p[0] = dw[i][e];
              p[width] = db[i][e];
            }
          }
      }
    }
    if (grp != groups - 1) return;
  }
  float* pw = a.part + (size_t)blockIdx.x * 2 * a.D;
#pragma unroll
  for (int i = 0; i < PERV; ++i) {
    const int v = t + i * step;
    if (v < nv)
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const int c = v * N + 2 * e;
        const float2 p = dw[i][e].get(), q = db[i][e].get();
        if (AL) {  // D is even: pairs on 8 bytes
          *reinterpret_cast<float2*>(pw + c) = p;
          *reinterpret_cast<float2*>(pw + a.D + c) = q;
        } else {
          if (c < a.D) pw[c] = p.x, pw[a.D + c] = q.x;
          if (c + 1 < a.D) pw[c + 1] = p.y, pw[a.D + c + 1] = q.y;
        }
      }
  }
}

// dw and db from the CTAs' sums: 32 columns a CTA, sixteen warps share the rows, then
// their sums in order. Launched to start while the kernel before it ends; it waits for
// that kernel's sums itself.
constexpr int kParamWarps = 16;
__global__ void __launch_bounds__(32 * kParamWarps)
    norm_params_kernel(const float* part, int rows, int D, int wtype, void* dw, void* db) {
  __shared__ float red[2][kParamWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  wait_prior_grid();
  float s = 0.f, q = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int r = warp; r < rows; r += kParamWarps) {
      const float* p = part + (size_t)r * 2 * D + c;
      s += p[0];
      q += p[D];
    }
  }
  red[0][warp][lane] = s;
  red[1][warp][lane] = q;
  __syncthreads();
  if (warp < 2 && c < D) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kParamWarps; ++i) v += red[warp][i][lane];
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
// Whether every row of a matrix (if there is one) starts on 16 bytes.
bool rows16(const void* q, long long ld, const moe_norm_args* p) {
  return q == nullptr || aligned_to(q, 16) && (p->n == 1 || ld * type_bytes(p->dtype) % 16 == 0);
}

// Warps of a row and of a CTA: a row lies in the registers of wpr warps, EPT elements a
// thread; short rows share a CTA of eight warps.
struct NormShape {
  int ept, wpr, warps;  // ept 0: the long-row kernel
};
NormShape norm_shape(const moe_norm_args* p, bool vec, int num_sms, bool backward) {
  auto wpr = [&](int ept) { return (p->D + 32 * ept - 1) / (32 * ept); };
  // Few rows: as many threads a row as there are. Else few enough that a warp keeps
  // several loads in flight; the backward pass holds two sums for each element too.
  const bool few = p->n < 2 * num_sms;
  NormShape s{};
  if (few)
    s.ept = 8;
  else if (backward)
    s.ept = p->D <= 256 || (!vec && wpr(8) <= max_warps(8)) ? 8 : 16;
  else if (!vec)
    s.ept = wpr(8) <= 16 ? 8 : wpr(16) <= 16 ? 16 : 32;
  else
    s.ept = p->D <= 256 ? 8 : p->D <= 512 || (p->D > 1024 && p->D <= 4096) ? 16 : 32;
  if (wpr(s.ept) > max_warps(s.ept)) s.ept = backward ? 16 : 32;
  s.wpr = wpr(s.ept);
  if (s.wpr > max_warps(s.ept)) return NormShape{0, 32, 32};
  s.warps = s.wpr * std::max(1, 8 / s.wpr);
  return s;
}

constexpr int kRingBytes = 200 * 1024;  // shared memory of an SM that the rings share

// Whether the ring kernel takes these rows, and its launch: 64 bytes a row or more, and enough
// rows that every group walks two or more. 16 warps an SM of 128 registers a thread: one CTA
// forward, one or two backward.
struct RingShape {
  bool aligned;
  int ept, wpr, groups, stages, ctas;  // ctas: on an SM; 0: not taken
  size_t smem;
};
RingShape ring_shape(const moe_norm_args* p, bool aligned, int mats, int num_sms, bool backward) {
  RingShape r{};
  const size_t bytes = (size_t)p->D * type_bytes(p->dtype);
  const size_t row = aligned ? bytes : (bytes + 15) / 16 * 16 + 16;  // in a stage
  r.aligned = aligned;
  r.ept = backward ? kBackwardEpt : p->D <= 512 ? 16 : kForwardEpt;
  r.wpr = (p->D + 32 * r.ept - 1) / (32 * r.ept);
  if (bytes < 64 || r.wpr > 16) return r;
  r.groups = std::max(1, (backward ? 8 : 16) / r.wpr);
  r.ctas = backward ? std::max(1, 16 / (r.wpr * r.groups)) : 1;
  const size_t params = backward ? 0 : 2 * ((size_t)p->D + 7) / 8 * 8 * type_bytes(p->wtype);
  const size_t stage = (size_t)r.groups * mats * row, room = kRingBytes / r.ctas;
  r.stages = room > params ? (int)std::min<size_t>(kMaxRing, (room - params) / stage) : 0;
  r.smem = params + r.stages * stage;
  // The groups' sums of the backward pass meet in the ring's memory.
  if (r.stages < 2 || p->n < 2LL * r.ctas * r.groups * num_sms ||
      (backward && r.groups > 1 && r.smem < (size_t)2 * r.ept * 32 * r.wpr * sizeof(float)))
    r.ctas = 0;
  return r;
}

template <typename K>
cudaError_t launch_ring(K kernel, std::atomic<uint64_t>* ready, const NormArgs& a, const RingShape& r,
                        int grid, cudaStream_t s) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), ready);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 32 * r.wpr * r.groups, r.smem, s>>>(a);
  return cudaGetLastError();
}
template <typename T, typename WT, bool AL>
cudaError_t launch_ring_as(bool backward, const NormArgs& a, const RingShape& r, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> ready_f{0}, ready_n{0}, ready_b{0};
  if (backward)
    return launch_ring(norm_backward_ring_kernel<T, WT, kBackwardEpt, AL>, &ready_b, a, r, grid, s);
  return r.ept == 16 ? launch_ring(norm_ring_kernel<T, WT, 16, AL>, &ready_n, a, r, grid, s)
                     : launch_ring(norm_ring_kernel<T, WT, kForwardEpt, AL>, &ready_f, a, r, grid, s);
}
template <typename T, typename WT>
cudaError_t launch_ring_of(bool backward, const NormArgs& a, const RingShape& r, int grid, cudaStream_t s) {
  return r.aligned ? launch_ring_as<T, WT, true>(backward, a, r, grid, s)
                   : launch_ring_as<T, WT, false>(backward, a, r, grid, s);
}
int run_ring(bool backward, int dtype, NormArgs& a, const RingShape& r, int grid, cudaStream_t s) {
  a.wpr = r.wpr;
  a.stages = r.stages;
  a.status = ops_status();
  if (a.status == nullptr) return MOE_ERR_CUDA;
  const bool wide = a.wtype == MOE_FP32;
  cudaError_t e;
  if (dtype == MOE_FP32)
    e = launch_ring_of<float, float>(backward, a, r, grid, s);
  else if (dtype == MOE_BF16)
    e = wide ? launch_ring_of<__nv_bfloat16, float>(backward, a, r, grid, s)
             : launch_ring_of<__nv_bfloat16, __nv_bfloat16>(backward, a, r, grid, s);
  else
    e = wide ? launch_ring_of<__half, float>(backward, a, r, grid, s)
             : launch_ring_of<__half, __half>(backward, a, r, grid, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T, int N>
void launch_forward(const NormArgs& a, const NormShape& sh, cudaStream_t s) {
  if (sh.ept == 0) {
    norm_long_kernel<T, N><<<(unsigned)a.n, kLoopThreads, 0, s>>>(a);
    return;
  }
  const int rows = sh.warps / sh.wpr, threads = 32 * sh.warps;
  const unsigned grid = (unsigned)((a.n + rows - 1) / rows);
  if (sh.ept == 8)
    norm_kernel<T, 8, N><<<grid, threads, 0, s>>>(a);
  else if (sh.ept == 16)
    norm_kernel<T, 16, N><<<grid, threads, 0, s>>>(a);
  else
    norm_kernel<T, 32, N><<<grid, threads, 0, s>>>(a);
}

template <typename T, int N>
void launch_backward(const NormArgs& a, const NormShape& sh, int grid, cudaStream_t s) {
  if (sh.ept == 0) {
    norm_backward_long_kernel<T, N><<<grid, kLoopThreads, 0, s>>>(a);
    return;
  }
  const int rows = sh.warps / sh.wpr, threads = 32 * sh.warps;
  const size_t smem = rows > 1 ? (size_t)2 * sh.ept * sh.wpr * 32 * sizeof(float) : 0;
  if (sh.ept == 8)
    norm_backward_kernel<T, 8, N><<<grid, threads, smem, s>>>(a);
  else
    norm_backward_kernel<T, 16, N><<<grid, threads, smem, s>>>(a);
}
template <typename T>
void launch_rows(bool backward, bool vec, const NormArgs& a, const NormShape& sh, int grid, cudaStream_t s) {
  constexpr int N = Vec<T>::kN;
  if (backward)
    vec ? launch_backward<T, N>(a, sh, grid, s) : launch_backward<T, 1>(a, sh, grid, s);
  else
    vec ? launch_forward<T, N>(a, sh, s) : launch_forward<T, 1>(a, sh, s);
}
int run_rows(bool backward, int dtype, bool vec, const NormArgs& a, const NormShape& sh, int grid,
             cudaStream_t s) {
  if (dtype == MOE_BF16)
    launch_rows<__nv_bfloat16>(backward, vec, a, sh, grid, s);
  else if (dtype == MOE_FP16)
    launch_rows<__half>(backward, vec, a, sh, grid, s);
  else
    launch_rows<float>(backward, vec, a, sh, grid, s);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
  const bool vec = (size_t)p->D * type_bytes(p->dtype) % 16 == 0 && rows16(p->x, p->ld_x, p) &&
                   rows16(p->r, p->ld_r, p) && rows16(p->y, p->ld_y, p) && rows16(p->z, p->ld_z, p) &&
                   aligned_to(p->w, 16) && aligned_to(p->b, 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int mats = p->r != nullptr ? 2 : 1;
  const RingShape ring = ring_shape(p, vec, mats, sms, false);
  if (ring.ctas > 0) return run_ring(false, p->dtype, a, ring, ring.ctas * sms, s);
  const NormShape sh = norm_shape(p, vec, sms, false);
  a.wpr = sh.wpr;
  return run_rows(false, p->dtype, vec, a, sh, 0, s);
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
      workspace == nullptr || !aligned_to(workspace, 16))
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
  const bool vec = (size_t)p->D * type_bytes(p->dtype) % 16 == 0 && rows16(p->z, p->ld_z, p) &&
                   rows16(p->dz, p->ld_dz, p) && rows16(p->dy, p->ld_dy, p) && rows16(p->dx, p->ld_dx, p) &&
                   aligned_to(p->w, 16);
  const int mats = p->dz != nullptr ? 3 : 2;
  const RingShape ring =
      ring_shape(p, vec, mats, sms, true);
  int grid;
  if (ring.ctas > 0) {
    grid = std::min(kNormParts, ring.ctas * sms);
    rc = run_ring(true, p->dtype, a, ring, grid, s);
    if (rc != MOE_OK) return rc;
  } else {
    const NormShape sh = norm_shape(p, vec, sms, true);
    a.wpr = sh.wpr;
    const int rows = sh.ept == 0 ? 1 : sh.warps / sh.wpr;
    grid = (int)std::min<long long>((p->n + rows - 1) / rows, std::min(kNormParts, 2 * sms));
    rc = run_rows(true, p->dtype, vec, a, sh, grid, s);
    if (rc != MOE_OK) return rc;
  }
  if (p->dw == nullptr && p->db == nullptr) return MOE_OK;
  const cudaError_t e = launch_behind(norm_params_kernel, dim3((p->D + 31) / 32), dim3(32 * kParamWarps), 0, s,
                                      (const float*)a.part, grid, p->D, p->wtype, p->dw, p->db);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
