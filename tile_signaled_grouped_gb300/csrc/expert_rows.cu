// Tokens as rows in the order of their experts, and back.
//
//   sort      slots (token t, choice j: t topk + j) by expert, earlier slots first:
//             offsets[e] .. offsets[e + 1] are expert e's rows, rows[slot] a slot's row, slots[row]
//             a row's slot
//   rows      r[rows[t, j]] = x[t]
//   combine   y[t] = sum_j w[t, j] r[rows[t, j]]           (w = 1: the gradient of x from that of r)
//   backward  dr[rows[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], r[rows[t, j]]>
//
// A slot whose expert is out of range has no row (-1), and the rows behind the last are zero. Every
// row that is read from `rows` is checked against the matrix: an index out of range is no row.
#include <algorithm>
#include <atomic>

#include "eight_bits.cuh"
#include "moe_common.cuh"
#include "ops_common.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------- the order
// A counting sort. The slots are cut into at most kSortChunks chunks of whole warps' ranges; a CTA
// counts its chunk's experts by warp, and after a scan over the experts, the chunks before and its
// warps, every warp walks its range in order and hands out rows: a slot's row is its warp's next one
// of its expert and the lanes before it with the same expert. Integer sums, so the order of
// the counting does not matter, and the result is the stable order always. One chunk (up to 2048
// slots) is one launch; otherwise a first launch leaves the chunks' counts.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortSlots = 4;      // slots of a lane at least, and read at a time
constexpr int kSortChunks = 148;   // a chunk is a CTA's work, and all of them are read by each
constexpr int kSortMaxExperts = 1024;

struct SortArgs {
  const int32_t* ids;
  int32_t *slots, *rows, *offsets;
  int32_t* counts;  // [chunks][E], with more than one chunk
  int n, E, per;    // per: slots of a lane
};

// Expert of a slot, E for none.
__device__ __forceinline__ int expert_at(const SortArgs& a, long long i, long long end) {
  if (i >= end) return a.E;
  const int e = __ldg(a.ids + i);
  return (unsigned)e < (unsigned)a.E ? e : a.E;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortArgs a) {
  __shared__ int count[kSortMaxExperts];
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) count[e] = 0;
  __syncthreads();
  allow_dependent_launch();
  wait_prior_grid();
  const long long lo = (long long)blockIdx.x * kSortThreads * a.per;
  const long long end = min((long long)a.n, lo + (long long)kSortThreads * a.per);
  for (long long i = lo + threadIdx.x; i < end; i += kSortThreads * kSortSlots) {
    int e[kSortSlots];
#pragma unroll
    for (int u = 0; u < kSortSlots; ++u) e[u] = expert_at(a, i + u * kSortThreads, end);
#pragma unroll
    for (int u = 0; u < kSortSlots; ++u)
      if (e[u] < a.E) atomicAdd(&count[e[u]], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.counts[(size_t)blockIdx.x * a.E + e] = count[e];
}

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int next[];  // [warps][E]: counts, then every warp's next row of each expert; [2][E]: sums
  __shared__ int scratch[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < (kSortWarps + 2) * a.E; i += kSortThreads) next[i] = 0;
  __syncthreads();
  allow_dependent_launch();
  wait_prior_grid();
  const long long lo = ((long long)blockIdx.x * kSortWarps + warp) * 32 * a.per;
  const long long end = min((long long)a.n, lo + 32LL * a.per);
  int* mine = next + warp * a.E;
  for (long long i = lo + lane; i < end; i += 32 * kSortSlots) {
    int e[kSortSlots];
#pragma unroll
    for (int u = 0; u < kSortSlots; ++u) e[u] = expert_at(a, i + u * 32, end);
#pragma unroll
    for (int u = 0; u < kSortSlots; ++u)
      if (e[u] < a.E) atomicAdd(&mine[e[u]], 1);
  }
  __syncthreads();
  // Every expert's rows of all chunks, and of the chunks before this one: the threads share the chunks'
  // counts, so that each has few to wait for.
  int* sum = next + kSortWarps * a.E;  // [2][E]
  if (gridDim.x > 1) {
    const int groups = max(1, kSortThreads / a.E);
    for (int i = threadIdx.x; i < groups * a.E; i += kSortThreads) {
      const int g = i / a.E, e = i - g * a.E;
      int all = 0, before = 0;
#pragma unroll 8
      for (int c = g; c < (int)gridDim.x; c += groups) {
        const int v = __ldcg(a.counts + (size_t)c * a.E + e);
        all += v;
        before += c < (int)blockIdx.x ? v : 0;
      }
      atomicAdd(&sum[e], all);
      atomicAdd(&sum[a.E + e], before);
    }
  } else {
    for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
      int all = 0;
      for (int w = 0; w < kSortWarps; ++w) all += next[w * a.E + e];
      sum[e] = all;
    }
  }
  __syncthreads();
  int all[2], before[2];  // of two neighbouring experts a thread
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = 2 * threadIdx.x + h;
    all[h] = e < a.E ? sum[e] : 0;
    before[h] = e < a.E ? sum[a.E + e] : 0;
  }
  int total;
  const int first = block_excl_scan(all[0] + all[1], scratch, &total);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = 2 * threadIdx.x + h;
    if (e >= a.E) continue;
    int at = first + (h == 1 ? all[0] : 0);
    if (blockIdx.x == 0) a.offsets[e] = at;
    at += before[h];
    for (int w = 0; w < kSortWarps; ++w) {
      const int v = next[w * a.E + e];
      next[w * a.E + e] = at;
      at += v;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = total;
  __syncthreads();
  for (long long i0 = lo; i0 < end; i0 += 32 * kSortSlots) {  // whole warps
    int e[kSortSlots];
#pragma unroll
    for (int u = 0; u < kSortSlots; ++u) e[u] = expert_at(a, i0 + u * 32 + lane, end);
#pragma unroll
    for (int u = 0; u < kSortSlots; ++u) {
      const long long i = i0 + u * 32 + lane;
      if (i - lane >= end) break;
      const uint32_t same = __match_any_sync(kAll, e[u]);
      int row = -1;
      if (e[u] < a.E) row = mine[e[u]] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (e[u] < a.E && lane == __ffs(same) - 1) mine[e[u]] += __popc(same);
      __syncwarp();
      if (i < end) a.rows[i] = row;
      if (row >= 0) a.slots[row] = (int)i;
    }
  }
  const long long all_threads = (long long)gridDim.x * kSortThreads;
  for (long long r = total + (long long)blockIdx.x * kSortThreads + threadIdx.x; r < a.n; r += all_threads)
    a.slots[r] = -1;
}

// ------------------------------------------------------------------- rows
struct RowsArgs {
  const void* x;         // rows: [T][ld_x]; backward: dy [T][ld_x]
  void* y;               // combine: out [T][ld_x]
  const void* r;         // combine, backward: [n][ld_r], or codes
  void* dr;              // rows, backward: out [n][ld_d]
  const uint8_t* scales; // backward: [n][ld_s] of the codes
  const float* w;        // [T][topk] or null
  float* dw;             // backward: out [T][topk]
  const int32_t* rows;   // [T][topk]
  const int32_t* total;  // offsets[E]
  long long T, n, D, ld_x, ld_r, ld_d, ld_s;  // D, ld_x and ld_d of the copy: in its units
  int topk;
};

// The row of a slot, or -1.
__device__ __forceinline__ int row_of(const RowsArgs& a, long long slot) {
  const int r = __ldg(a.rows + slot);
  return r >= 0 && r < a.n ? r : -1;
}

// Copies of token rows in units U of 16 bytes (or of one element, where rows do not start on 16
// bytes). A warp takes 128 units of a token: it reads them once and writes them to the token's
// topk rows. Bound by the bytes written: 8192 x 8 x 2048 bf16 48 us, floor 45. By elements 8192 x 8 x 2049 takes
// 55, and 8192 x 8 x 4096 from rows of 4101 as long as from rows of 4096, 91 us: what a token costs in
// instructions is shared by its rows.
constexpr int kRowWarps = 8, kCopyUnits = 4;
template <typename U>
__global__ void __launch_bounds__(32 * kRowWarps) expert_rows_kernel(const __grid_constant__ RowsArgs a) {
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * kRowWarps;
  const long long me = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const long long chunks = (a.D + 32 * kCopyUnits - 1) / (32 * kCopyUnits);
  const U* x = static_cast<const U*>(a.x);
  U* out = static_cast<U*>(a.dr);
  for (long long u = me; u < a.T * chunks; u += warps) {
    const long long t = u / chunks, c = (u - t * chunks) * 32 * kCopyUnits + lane;
    const int mine = lane < a.topk ? row_of(a, t * a.topk + lane) : -1;
    U v[kCopyUnits];
#pragma unroll
    for (int i = 0; i < kCopyUnits; ++i)
      if (c + 32 * i < a.D) v[i] = __ldg(x + t * a.ld_x + c + 32 * i);
    for (int j = 0; j < a.topk; ++j) {
      const int row = __shfl_sync(kAll, mine, j);
      if (row < 0) continue;
#pragma unroll
      for (int i = 0; i < kCopyUnits; ++i)
        if (c + 32 * i < a.D) out[row * a.ld_d + c + 32 * i] = v[i];
    }
  }
  const long long total = min(max((long long)__ldg(a.total), 0LL), a.n);
  for (long long row = total + me; row < a.n; row += warps)
    for (long long c = lane; c < a.D; c += 32) out[row * a.ld_d + c] = U{};
}

// The weighted sum of a token's rows, in the order of its slots, fp32. A warp takes 64 vectors of a
// token; four rows' loads leave before the first is added. A row that a slot has not is no term of
// the sum (not one times zero: what lies there may be NaN). Bound by the bytes of the rows.
// ANY: rows that do not start on 16 bytes.
constexpr int kSumSlots = 4, kSumUnits = 2;
template <typename T, bool ANY>
__global__ void __launch_bounds__(32 * kRowWarps) combine_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int N = Vec<T>::kN, kLanes = kOwn<ANY> * N, kSpan = kLanes * kSumUnits;
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * kRowWarps, chunks = (a.D + kSpan - 1) / kSpan;
  const T* r = static_cast<const T*>(a.r);
  for (long long u = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < a.T * chunks; u += warps) {
    const long long t = u / chunks, c = (u - t * chunks) * kSpan + lane * N;
    int mine = -1;
    float weight = 1.f;
    if (lane < a.topk) {
      mine = row_of(a, t * a.topk + lane);
      if (a.w != nullptr) weight = __ldg(a.w + t * a.topk + lane);
    }
    float sum[kSumUnits][N];
#pragma unroll
    for (int i = 0; i < kSumUnits; ++i)
#pragma unroll
      for (int q = 0; q < N; ++q) sum[i][q] = 0.f;
    for (int j0 = 0; j0 < a.topk; j0 += kSumSlots) {
      RowVec<T, ANY> v[kSumSlots][kSumUnits];
      int row[kSumSlots];
#pragma unroll
      for (int j = 0; j < kSumSlots; ++j) {
        row[j] = __shfl_sync(kAll, mine, min(j0 + j, 31));  // lanes from topk on have none
        if (row[j] < 0) continue;
#pragma unroll
        for (int i = 0; i < kSumUnits; ++i) v[j][i].load(r + row[j] * a.ld_r, c + kLanes * i, a.D);
      }
#pragma unroll
      for (int j = 0; j < kSumSlots; ++j) {
        const float w = __shfl_sync(kAll, weight, min(j0 + j, 31));
        if (row[j] < 0) continue;
#pragma unroll
        for (int i = 0; i < kSumUnits; ++i) {
          float f[N];
          v[j][i].get(f);
#pragma unroll
          for (int q = 0; q < N; ++q) sum[i][q] = fmaf(w, f[q], sum[i][q]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kSumUnits; ++i) {
      store_vec<ANY>(static_cast<T*>(a.y) + t * a.ld_x, c + kLanes * i, a.D, sum[i], lane);
    }
  }
}

// Elements of a row that was kept, a vector of T at a time, as they lie in memory.
template <typename T, bool EIGHT>
struct Kept {
  static constexpr int N = Vec<T>::kN;
  typename std::conditional<EIGHT, Codes<N, false>, RowVec<T, false>>::type u;
  uint8_t scale;
  __device__ __forceinline__ void load(const RowsArgs& a, long long row, int c, long long width) {
    if constexpr (EIGHT) {
      u.load(static_cast<const uint8_t*>(a.r) + row * a.ld_r, c, width);
      scale = c < width ? __ldg(a.scales + row * a.ld_s + c / kScaleBlock) : 0;
    } else {
      u.load(static_cast<const T*>(a.r) + row * a.ld_r, c, width);
    }
  }
  __device__ __forceinline__ void get(int, long long, float (&f)[N]) const {
    if constexpr (EIGHT)
      u.get(scale_value(scale), f);
    else
      u.get(f);
  }
};
// The same a word at a time, of rows that start anywhere.
template <typename T, bool EIGHT>
struct KeptWord {
  static constexpr int N = RowWord<T>::N;
  typename std::conditional<EIGHT, CodeWord<N>, RowWord<T>>::type u;
  __device__ __forceinline__ void load(const RowsArgs& a, long long row, int c, long long width) {
    if constexpr (EIGHT)
      u.load(static_cast<const uint8_t*>(a.r) + row * a.ld_r, a.scales + row * a.ld_s, c, width);
    else
      u.load(static_cast<const T*>(a.r) + row * a.ld_r, c, width);
  }
  __device__ __forceinline__ void get(int c, long long width, float (&f)[N]) const { u.get(c, width, f); }
};

// Gradients of the rows and weights. A CTA takes one token, its warps walk the row together: a
// vector of dy meets those of eight rows, which it is multiplied into (dw) and, times the weight,
// written to (dr). The warps' partial products are added in their order. EIGHT: the rows kept are codes.
// Bound by the bytes of the rows: all eight loads leave before the first is used, and 24 warps
// fit on an SM (as fp32 the eight vectors took 121 registers, and 328 us where this takes
// 126 for 4096 tokens of 8 x 7168 from codes). ANY: rows that start anywhere go by words (8192 tokens of
// 8 x 2049 take 208 us so, and 261 by vectors shifted together). DY_ANY: dy's alone start anywhere.
// SLOTS: rows at a time, and 8 / SLOTS vectors of each: of one, two or four rows a token as many loads are in
// flight as of eight (4096 x 1 x 7168 33 us by two rows, 51 by eight; 7273 x 1 x 6841 109 by four and 226;
// 8192 x 4 x 2048 from codes 40 by four, 48 by eight or two). At 80 registers, which 24 warps leave each, forms
// of 16-bit values by two rows spill 36 to 48 bytes, some others 4 to 32.
constexpr int kBackLoads = 8, kBackWarps = 24;
template <typename T, bool EIGHT, bool ANY, bool DY_ANY, int SLOTS>
__global__ void __launch_bounds__(32 * kBackWarps, 1) combine_backward_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int N = ANY ? RowWord<T>::N : Vec<T>::kN, kUnits = kBackLoads / SLOTS, kSpan = 32 * N * kUnits;
  __shared__ float part[kBackWarps][SLOTS];
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T* dr = static_cast<T*>(a.dr);
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const T* dy = static_cast<const T*>(a.x) + t * a.ld_x;
    for (int j0 = 0; j0 < a.topk; j0 += SLOTS) {
      int row[SLOTS];
      float w[SLOTS], dot[SLOTS];
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        const bool in = j0 + j < a.topk;
        row[j] = in ? row_of(a, t * a.topk + j0 + j) : -1;
        w[j] = in ? __ldg(a.w + t * a.topk + j0 + j) : 0.f;
        dot[j] = 0.f;
      }
      for (int c0 = warp * kSpan; c0 < a.D; c0 += warps * kSpan) {
        const int c = c0 + lane * N;
        if (!ANY && c >= a.D) break;
        typename std::conditional<ANY, KeptWord<T, EIGHT>, Kept<T, EIGHT>>::type v[SLOTS][kUnits];
        typename std::conditional<ANY, RowWord<T>, RowVec<T, DY_ANY>>::type x[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
          x[i].load(dy, c + 32 * N * i, ANY || DY_ANY || kUnits > 1 ? a.D : c + N);  // else c is inside
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          if (row[j] < 0) continue;
#pragma unroll
          for (int i = 0; i < kUnits; ++i) v[j][i].load(a, row[j], c + 32 * N * i, ANY || kUnits > 1 ? a.D : c + N);
        }
        float d[kUnits][N];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          if constexpr (ANY)
            x[i].get(c + 32 * N * i, a.D, d[i]);
          else
            x[i].get(d[i]);
        }
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          if (row[j] < 0) continue;
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            const int ci = c + 32 * N * i;
            float f[N];
            v[j][i].get(ci, a.D, f);
#pragma unroll
            for (int q = 0; q < N; ++q) dot[j] = fmaf(d[i][q], f[q], dot[j]);
#pragma unroll
            for (int q = 0; q < N; ++q) f[q] = w[j] * d[i][q];
            if constexpr (ANY)
              store_word_any(dr + row[j] * a.ld_d, ci, a.D, pack_word<T>(f), lane);
            else
              store_vec<false>(dr + row[j] * a.ld_d, ci, kUnits > 1 ? a.D : ci + N, f, lane);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        dot[j] = warp_sum(dot[j]);
        if (lane == 0) part[warp][j] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < SLOTS && j0 + (int)threadIdx.x < a.topk) {
        float s = 0.f;
        for (int v = 0; v < warps; ++v) s += part[v][threadIdx.x];
        a.dw[t * a.topk + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
  const long long total = min(max((long long)__ldg(a.total), 0LL), a.n);
  for (long long r = total + blockIdx.x; r < a.n; r += gridDim.x)
    for (long long c = threadIdx.x; c < a.D; c += blockDim.x) dr[r * a.ld_d + c] = from_f32<T>(0.f);
}

// ------------------------------------------------------------------- host side
constexpr long long kMaxRows = INT32_MAX / 2;

int check_rows(const moe_rows_args* p) {
  if (p == nullptr || p->T < 0 || p->topk < 1 || p->topk > 32 || p->T > kMaxRows / p->topk || p->E < 1 ||
      p->E > kSortMaxExperts || p->D < 1 || p->D > INT32_MAX / 2)
    return MOE_ERR_ARG;
  return type_bytes(p->dtype) == 0 ? MOE_ERR_ARG : MOE_OK;
}
bool check_order(const moe_rows_args* p) {
  return p->rows != nullptr && p->offsets != nullptr && aligned_to(p->rows, 4) && aligned_to(p->offsets, 4);
}
bool check_matrix(const void* q, long long ld, long long rows, long long cols, int bytes) {
  return q != nullptr && aligned_to(q, (size_t)bytes) && (rows <= 1 || (ld >= cols && ld <= INT32_MAX));
}
bool vector_rows(const void* q, long long ld, long long rows, int bytes, int vector) {
  return aligned_to(q, (size_t)vector) && (rows <= 1 || ld * bytes % vector == 0);
}
RowsArgs rows_args(const moe_rows_args* p) {
  RowsArgs a{};
  a.rows = p->rows;
  a.total = p->offsets + p->E;
  a.T = p->T;
  a.n = p->T * p->topk;
  a.D = p->D;
  a.ld_x = p->ld_x;
  a.ld_r = p->ld_r;
  a.ld_d = p->ld_dr;
  a.w = p->w;
  a.topk = p->topk;
  return a;
}
unsigned row_grid(long long units) {
  return (unsigned)std::min<long long>((units + kRowWarps - 1) / kRowWarps, 1 << 20);
}
int launched(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

template <typename U>
int launch_rows(const RowsArgs& a, cudaStream_t s) {
  const long long chunks = (a.D + 32 * kCopyUnits - 1) / (32 * kCopyUnits);
  return launched(launch_behind(expert_rows_kernel<U>, dim3(row_grid(a.T * chunks)), dim3(32 * kRowWarps), 0, s, a));
}

template <typename T>
int launch_combine(const RowsArgs& a, bool vec, cudaStream_t s) {
  const int span = (vec ? 32 : kOwn<true>) * Vec<T>::kN * kSumUnits;
  const dim3 grid(row_grid(a.T * ((a.D + span - 1) / span))), block(32 * kRowWarps);
  return launched(vec ? launch_behind(combine_kernel<T, false>, grid, block, 0, s, a)
                      : launch_behind(combine_kernel<T, true>, grid, block, 0, s, a));
}

template <typename T>
int launch_backward(const RowsArgs& a, bool vec, bool dy, int sms, cudaStream_t s) {
  // Warps of a token: four vectors of a lane each, eight warps at most; where the tokens then leave room on
  // the SMs, as many more as fill it.
  const long long width = a.D / (vec ? Vec<T>::kN : RowWord<T>::N);
  const long long few = std::min<long long>(8, std::max<long long>(1, width / 128));
  const long long fill = std::min<long long>({kBackWarps, (long long)kBackWarps * sms / a.T, (width + 31) / 32});
  const dim3 grid((unsigned)std::min<long long>(a.T, 1 << 20)), block(32 * (unsigned)std::max(few, fill));
  auto go = [&](auto* kernel) { return launched(launch_behind(kernel, grid, block, 0, s, a)); };
  auto slots = [&](auto n) {
    constexpr int N = decltype(n)::value, kAny = std::max(N, 4);
    if (a.scales != nullptr)
      return !vec ? go(combine_backward_kernel<T, true, true, false, kAny>)
             : dy ? go(combine_backward_kernel<T, true, false, false, N>)
                  : go(combine_backward_kernel<T, true, false, true, N>);
    return !vec ? go(combine_backward_kernel<T, false, true, false, kAny>)
           : dy ? go(combine_backward_kernel<T, false, false, false, N>)
                : go(combine_backward_kernel<T, false, false, true, N>);
  };
  return a.topk <= 2   ? slots(std::integral_constant<int, 2>{})
         : a.topk <= 4 ? slots(std::integral_constant<int, 4>{})
                       : slots(std::integral_constant<int, kBackLoads>{});
}

// Slots of a lane, so that there are at most kSortChunks chunks.
int sort_per(long long n) {
  const long long most = (long long)kSortThreads * kSortChunks;
  return (int)std::max<long long>(kSortSlots, (n + most - 1) / most);
}
long long sort_chunks(long long n) {
  const long long chunk = (long long)kSortThreads * sort_per(n);
  return std::max<long long>(1, (n + chunk - 1) / chunk);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_sort_experts_workspace(long long n, int E) {
  if (n < 1 || n > kMaxRows || E < 1 || E > kSortMaxExperts) return 0;
  const long long chunks = sort_chunks(n);
  return chunks > 1 ? (size_t)chunks * E * sizeof(int32_t) : 0;
}

int moe_sort_experts(const int32_t* ids, long long n, int E, int32_t* slots, int32_t* rows, int32_t* offsets,
                     void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (n < 0 || n > kMaxRows || E < 1 || E > kSortMaxExperts || offsets == nullptr || !aligned_to(offsets, 4) ||
      (n > 0 && (ids == nullptr || slots == nullptr || rows == nullptr)) || !aligned_to(ids, 4) ||
      !aligned_to(slots, 4) || !aligned_to(rows, 4))
    return MOE_ERR_ARG;
  const size_t need = moe_sort_experts_workspace(n, E);
  if (need > 0 && (workspace == nullptr || !aligned_to(workspace, 16))) return MOE_ERR_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  int sms = 0;
  const int rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  SortArgs a{ids, slots, rows, offsets, static_cast<int32_t*>(workspace), (int)n, E, sort_per(n)};
  const dim3 grid((unsigned)sort_chunks(n)), block(kSortThreads);
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(sort_kernel), &ready);
  if (e == cudaSuccess && grid.x > 1) e = launch_behind(sort_count_kernel, grid, block, 0, s, a);
  if (e == cudaSuccess)
    e = launch_behind(sort_kernel, grid, block, (size_t)(kSortWarps + 2) * E * sizeof(int), s, a);
  return launched(e);
}

int moe_expert_rows(const moe_rows_args* p, moe_stream_t stream) {
  int rc = check_rows(p);
  if (rc != MOE_OK) return rc;
  if (p->T == 0) return MOE_OK;
  const int b = type_bytes(p->dtype);
  if (!check_order(p) || !check_matrix(p->x, p->ld_x, p->T, p->D, b) ||
      !check_matrix(p->dr, p->ld_dr, p->T * p->topk, p->D, b))
    return MOE_ERR_ARG;
  int sms = 0;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  RowsArgs a = rows_args(p);
  a.x = p->x;
  a.dr = p->dr;
  if (p->D * b % 16 == 0 && vector_rows(p->x, p->ld_x, p->T, b, 16) && vector_rows(p->dr, p->ld_dr, a.n, b, 16)) {
    a.D = a.D * b / 16;
    a.ld_x = a.ld_x * b / 16;
    a.ld_d = a.ld_d * b / 16;
    return launch_rows<uint4>(a, s);
  }
  return b == 4 ? launch_rows<uint32_t>(a, s) : launch_rows<uint16_t>(a, s);
}

int moe_combine_experts(const moe_rows_args* p, moe_stream_t stream) {
  int rc = check_rows(p);
  if (rc != MOE_OK) return rc;
  if (p->T == 0) return MOE_OK;
  const int b = type_bytes(p->dtype);
  if (!check_order(p) || !check_matrix(p->y, p->ld_y, p->T, p->D, b) ||
      !check_matrix(p->r, p->ld_r, p->T * p->topk, p->D, b) || !aligned_to(p->w, 4))
    return MOE_ERR_ARG;
  int sms = 0;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  RowsArgs a = rows_args(p);
  a.y = p->y;
  a.ld_x = p->ld_y;
  a.r = p->r;
  const bool vec =
      p->D * b % 16 == 0 && vector_rows(p->y, p->ld_y, p->T, b, 16) && vector_rows(p->r, p->ld_r, a.n, b, 16);
  return p->dtype == MOE_FP32   ? launch_combine<float>(a, vec, s)
         : p->dtype == MOE_BF16 ? launch_combine<__nv_bfloat16>(a, vec, s)
                                : launch_combine<__half>(a, vec, s);
}

int moe_combine_experts_backward(const moe_rows_args* p, moe_stream_t stream) {
  int rc = check_rows(p);
  if (rc != MOE_OK) return rc;
  if (p->T == 0) return MOE_OK;
  const int b = type_bytes(p->dtype), kb = p->r_scales != nullptr ? 1 : b;
  const long long n = p->T * p->topk;
  if (!check_order(p) || !check_matrix(p->x, p->ld_x, p->T, p->D, b) || !check_matrix(p->r, p->ld_r, n, p->D, kb) ||
      !check_matrix(p->dr, p->ld_dr, n, p->D, b) || p->w == nullptr || !aligned_to(p->w, 4) || p->dw == nullptr ||
      !aligned_to(p->dw, 4) || (p->r_scales != nullptr && n > 1 && p->ld_scales < scale_blocks(p->D)))
    return MOE_ERR_ARG;
  int sms = 0;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  RowsArgs a = rows_args(p);
  a.x = p->x;
  a.r = p->r;
  a.dr = p->dr;
  a.scales = p->r_scales;
  a.ld_s = p->ld_scales;
  a.dw = p->dw;
  // A vector of codes has as many elements as one of 16 bytes of the type.
  const bool vec = p->D * b % 16 == 0 && vector_rows(p->dr, p->ld_dr, n, b, 16) &&
                   vector_rows(p->r, p->ld_r, n, kb, 16 / b * kb);
  const bool dy = vector_rows(p->x, p->ld_x, p->T, b, 16);
  return p->dtype == MOE_FP32   ? launch_backward<float>(a, vec, dy, sms, s)
         : p->dtype == MOE_BF16 ? launch_backward<__nv_bfloat16>(a, vec, dy, sms, s)
                                : launch_backward<__half>(a, vec, dy, sms, s);
}

}  // extern "C"
