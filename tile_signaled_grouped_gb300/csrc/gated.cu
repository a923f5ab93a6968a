// The gated activation of the experts, h = act(gate) up, and its backward pass, and checkpoints of
// activations in 8 bits (eight_bits.cuh has the format):
//
//   forward     h = act(gate) up, and the checkpoints of gate and up from the same reads
//   backward    dgate = dh up act'(gate), dup = dh act(gate), and h again, which the product
//               after it needs and nobody kept; gate and up as they were or from their checkpoints
//   checkpoint  codes and scales of a matrix;  restore: the matrix that they stand for
//
// Elementwise, so bound by the bytes; all arithmetic is fp32, each output is rounded once. A warp
// takes kUnits vectors of 16 bytes a lane, whose loads all leave before the first is used. A block
// of 32 elements lies in neighbouring lanes, whose largest |x| meet by shuffles. Rows that do not start on
// 16 bytes: any_rows.cuh.
#include <algorithm>

#include "activations.cuh"
#include "eight_bits.cuh"
#include "moe_common.cuh"
#include "ops_common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;

// Where a warp works: a row and its first column there.
struct Walk {
  long long chunks, units;  // units of a row; of all rows
  __device__ __forceinline__ Walk(long long n, long long c, int span) : chunks((c + span - 1) / span) {
    units = n * chunks;
  }
  __device__ __forceinline__ long long first() const {
    return (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  }
  __device__ __forceinline__ long long step() const { return (long long)gridDim.x * kWarps; }
};

// ------------------------------------------------------------------- checkpoint and restore
struct CheckArgs {
  void* x;
  uint8_t *codes, *scales;
  long long n, c, ld_x, ld_codes, ld_scales;
};
constexpr int kCheckUnits = 4;

template <typename T, bool ANY>
__global__ void __launch_bounds__(32 * kWarps) checkpoint_kernel(const __grid_constant__ CheckArgs a) {
  constexpr int N = Vec<T>::kN;
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  constexpr int kSpan = kOwn<ANY, true> * N;  // elements that a warp stores at a time
  const Walk k(a.n, a.c, kSpan * kCheckUnits);
  for (long long u = k.first(); u < k.units; u += k.step()) {
    const long long i = u / k.chunks, c0 = (u - i * k.chunks) * kSpan * kCheckUnits + lane * N;
    RowVec<T, ANY> v[kCheckUnits];
#pragma unroll
    for (int q = 0; q < kCheckUnits; ++q)
      v[q].load(static_cast<const T*>(a.x) + i * a.ld_x, c0 + kSpan * q, a.c);
#pragma unroll
    for (int q = 0; q < kCheckUnits; ++q) {
      encode_vec<T, ANY>(v[q], a.codes + i * a.ld_codes, a.scales + i * a.ld_scales, c0 + kSpan * q, a.c, lane);
    }
  }
}

// N codes a lane: 16, in two or four stores, where they start on 16 bytes.
template <typename T, int N, bool ANY>
__global__ void __launch_bounds__(32 * kWarps) restore_kernel(const __grid_constant__ CheckArgs a) {
  constexpr int kUnits = N == 16 ? 2 : 4, kStore = Vec<T>::kN;
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  constexpr int kSpan = kOwn<ANY> * N;
  const Walk k(a.n, a.c, kSpan * kUnits);
  for (long long u = k.first(); u < k.units; u += k.step()) {
    const long long i = u / k.chunks, c0 = (u - i * k.chunks) * kSpan * kUnits + lane * N;
    T* x = static_cast<T*>(a.x) + i * a.ld_x;
    Codes<N, ANY> v[kUnits];
    uint8_t s[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      const long long c = c0 + kSpan * q;
      v[q].load(a.codes + i * a.ld_codes, c, a.c);
      s[q] = c < a.c ? __ldg(a.scales + i * a.ld_scales + c / kScaleBlock) : 0;
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      float f[N];
      v[q].get(scale_value(s[q]), f);
#pragma unroll
      for (int p = 0; p < N; p += kStore) {
        float o[kStore];
#pragma unroll
        for (int e = 0; e < kStore; ++e) o[e] = f[p + e];
        store_vec<ANY>(x, c0 + kSpan * q + p, a.c, o, lane);
      }
    }
  }
}

// ------------------------------------------------------------------- the gated activation
struct GatedArgs {
  const void *gate, *up, *dh;
  void *h, *dgate, *dup;
  uint8_t *gate_codes, *up_codes, *gate_scales, *up_scales;
  long long n, c, ld_gate, ld_up, ld_h, ld_dh, ld_dgate, ld_dup;
  long long ld_codes, ld_scales;
};
constexpr int kGatedUnits = 2;

template <typename T, int ACT, bool ANY, bool KEEP>
__global__ void __launch_bounds__(32 * kWarps) gated_kernel(const __grid_constant__ GatedArgs a) {
  constexpr int N = Vec<T>::kN;
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  constexpr int kLanes = kOwn<ANY, KEEP>, kSpan = kLanes * N;
  const Walk k(a.n, a.c, kSpan * kGatedUnits);
  for (long long u = k.first(); u < k.units; u += k.step()) {
    const long long i = u / k.chunks, c0 = (u - i * k.chunks) * kSpan * kGatedUnits + lane * N;
    RowVec<T, ANY> g[kGatedUnits], v[kGatedUnits];
#pragma unroll
    for (int q = 0; q < kGatedUnits; ++q) {
      g[q].load(static_cast<const T*>(a.gate) + i * a.ld_gate, c0 + kSpan * q, a.c);
      v[q].load(static_cast<const T*>(a.up) + i * a.ld_up, c0 + kSpan * q, a.c);
    }
#pragma unroll
    for (int q = 0; q < kGatedUnits; ++q) {
      const long long c = c0 + kSpan * q;
      if (KEEP) {
        encode_vec<T, ANY>(g[q], a.gate_codes + i * a.ld_codes, a.gate_scales + i * a.ld_scales, c, a.c, lane);
        encode_vec<T, ANY>(v[q], a.up_codes + i * a.ld_codes, a.up_scales + i * a.ld_scales, c, a.c, lane);
      }
      float x[N], h[N];
      g[q].get(x);
      v[q].get(h);
#pragma unroll
      for (int e = 0; e < N; ++e) h[e] *= act_of<ACT>(x[e]);
      store_vec<ANY>(static_cast<T*>(a.h) + i * a.ld_h, c, a.c, h, lane, kLanes);
    }
  }
}

template <typename T, int ACT, bool ANY, bool KEPT>
__global__ void __launch_bounds__(32 * kWarps) gated_backward_kernel(const __grid_constant__ GatedArgs a) {
  constexpr int N = Vec<T>::kN;
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  constexpr int kSpan = kOwn<ANY> * N;
  const Walk k(a.n, a.c, kSpan * kGatedUnits);
  for (long long u = k.first(); u < k.units; u += k.step()) {
    const long long i = u / k.chunks, c0 = (u - i * k.chunks) * kSpan * kGatedUnits + lane * N;
    typename std::conditional<KEPT, Codes<N, ANY>, RowVec<T, ANY>>::type g[kGatedUnits], v[kGatedUnits];
    uint8_t gs[kGatedUnits], vs[kGatedUnits];
    RowVec<T, ANY> d[kGatedUnits];
#pragma unroll
    for (int q = 0; q < kGatedUnits; ++q) {
      const long long c = c0 + kSpan * q;
      if constexpr (KEPT) {
        g[q].load(static_cast<const uint8_t*>(a.gate) + i * a.ld_codes, c, a.c);
        v[q].load(static_cast<const uint8_t*>(a.up) + i * a.ld_codes, c, a.c);
        const long long scale = i * a.ld_scales + c / kScaleBlock;
        gs[q] = c < a.c ? __ldg(a.gate_scales + scale) : 0;
        vs[q] = c < a.c ? __ldg(a.up_scales + scale) : 0;
      } else {
        g[q].load(static_cast<const T*>(a.gate) + i * a.ld_gate, c, a.c);
        v[q].load(static_cast<const T*>(a.up) + i * a.ld_up, c, a.c);
      }
      d[q].load(static_cast<const T*>(a.dh) + i * a.ld_dh, c, a.c);
    }
#pragma unroll
    for (int q = 0; q < kGatedUnits; ++q) {
      const long long c = c0 + kSpan * q;
      float x[N], y[N], dh[N], o[N];
      if constexpr (KEPT) {
        g[q].get(scale_value(gs[q]), x);
        v[q].get(scale_value(vs[q]), y);
      } else {
        g[q].get(x);
        v[q].get(y);
      }
      d[q].get(dh);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float slope;
        x[e] = act_both<ACT>(x[e], &slope);
        o[e] = dh[e] * y[e] * slope;
      }
      store_vec<ANY>(static_cast<T*>(a.dgate) + i * a.ld_dgate, c, a.c, o, lane);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = dh[e] * x[e];
      store_vec<ANY>(static_cast<T*>(a.dup) + i * a.ld_dup, c, a.c, o, lane);
      if (a.h != nullptr) {
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = x[e] * y[e];
        store_vec<ANY>(static_cast<T*>(a.h) + i * a.ld_h, c, a.c, o, lane);
      }
    }
  }
}

// The same for whole values in rows that start anywhere: a word of 4 bytes a lane, by the place of dgate, as
// which the other outputs mostly lie; the inputs are read by their own places. (By vectors shifted together,
// with 600 instructions a vector, 65536 rows of 2049 took 602 us; this takes 343. From codes it is the other
// way round: 491 by vectors, 725 by words.)
constexpr int kWordUnits = 4;
template <typename T, int ACT>
__global__ void __launch_bounds__(32 * kWarps) gated_backward_words_kernel(const __grid_constant__ GatedArgs a) {
  constexpr int N = LikeWord<T>::N;
  allow_dependent_launch();
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const Walk k(a.n, a.c + N - 1, 32 * N * kWordUnits);
  for (long long u = k.first(); u < k.units; u += k.step()) {
    const long long i = u / k.chunks;
    T* dgate = static_cast<T*>(a.dgate) + i * a.ld_dgate;
    const int lead = N == 2 && (reinterpret_cast<uintptr_t>(dgate) & 2) != 0 ? 1 : 0;
    const long long e0 = ((u - i * k.chunks) * 32 * kWordUnits + lane) * N - lead;
    LikeWord<T> g[kWordUnits], v[kWordUnits], d[kWordUnits];
#pragma unroll
    for (int q = 0; q < kWordUnits; ++q) {
      const long long e = e0 + 32 * N * q;
      g[q].load(static_cast<const T*>(a.gate) + i * a.ld_gate, e, a.c);
      v[q].load(static_cast<const T*>(a.up) + i * a.ld_up, e, a.c);
      d[q].load(static_cast<const T*>(a.dh) + i * a.ld_dh, e, a.c);
    }
#pragma unroll
    for (int q = 0; q < kWordUnits; ++q) {
      const long long e = e0 + 32 * N * q;
      float x[N], y[N], dh[N], o[N];
      g[q].get(x);
      v[q].get(y);
      d[q].get(dh);
#pragma unroll
      for (int p = 0; p < N; ++p) {
        float slope;
        x[p] = act_both<ACT>(x[p], &slope);
        o[p] = dh[p] * y[p] * slope;
      }
      store_word(dgate, e, a.c, pack_word<T>(o));
#pragma unroll
      for (int p = 0; p < N; ++p) o[p] = dh[p] * x[p];
      store_word_any(static_cast<T*>(a.dup) + i * a.ld_dup, e, a.c, pack_word<T>(o), lane);
      if (a.h != nullptr) {
#pragma unroll
        for (int p = 0; p < N; ++p) o[p] = x[p] * y[p];
        store_word_any(static_cast<T*>(a.h) + i * a.ld_h, e, a.c, pack_word<T>(o), lane);
      }
    }
  }
}

// ------------------------------------------------------------------- host side
constexpr long long kMaxSize = INT32_MAX / 2;

bool check_matrix(const void* q, long long ld, long long rows, long long cols, int bytes) {
  return q != nullptr && aligned_to(q, (size_t)bytes) && (rows <= 1 || (ld >= cols && ld <= INT32_MAX));
}
bool vector_rows(const void* q, long long ld, long long rows, int bytes, int vector) {
  return aligned_to(q, (size_t)vector) && (rows <= 1 || ld * bytes % vector == 0);
}
unsigned grid_of(long long n, long long c, int span) {
  const long long units = n * ((c + span - 1) / span);
  return (unsigned)std::min<long long>((units + kWarps - 1) / kWarps, 1 << 20);
}
int launched(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

template <typename T>
int launch_checkpoint(const CheckArgs& a, bool vec, bool restore, cudaStream_t s) {
  constexpr int N = Vec<T>::kN;
  const dim3 block(32 * kWarps);
  if (restore && vec && a.c % 16 == 0 && vector_rows(a.codes, a.ld_codes, a.n, 1, 16))
    return launched(
        launch_behind(restore_kernel<T, 16, false>, dim3(grid_of(a.n, a.c, 32 * 16 * 2)), block, 0, s, a));
  const int lanes = vec ? 32 : restore ? kOwn<true> : kOwn<true, true>;
  const dim3 grid(grid_of(a.n, a.c, lanes * kCheckUnits * N));
  if (restore)
    return launched(vec ? launch_behind(restore_kernel<T, N, false>, grid, block, 0, s, a)
                        : launch_behind(restore_kernel<T, N, true>, grid, block, 0, s, a));
  return launched(vec ? launch_behind(checkpoint_kernel<T, false>, grid, block, 0, s, a)
                      : launch_behind(checkpoint_kernel<T, true>, grid, block, 0, s, a));
}

int checkpoint(const moe_checkpoint_args* p, bool restore, moe_stream_t stream) {
  if (p == nullptr || p->n < 0 || p->n > kMaxSize || p->c < 1 || p->c > kMaxSize) return MOE_ERR_ARG;
  const int b = type_bytes(p->dtype);
  if (b == 0) return MOE_ERR_ARG;
  if (p->n == 0) return MOE_OK;
  if (!check_matrix(p->x, p->ld_x, p->n, p->c, b) || !check_matrix(p->codes, p->ld_codes, p->n, p->c, 1) ||
      !check_matrix(p->scales, p->ld_scales, p->n, scale_blocks(p->c), 1))
    return MOE_ERR_ARG;
  int sms = 0;
  const int rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  CheckArgs a{p->x,      static_cast<uint8_t*>(p->codes), p->scales, p->n, p->c, p->ld_x, p->ld_codes,
              p->ld_scales};
  // Whole blocks in one run of memory: one long row.
  if (a.n > 1 && a.c % kScaleBlock == 0 && a.ld_x == a.c && a.ld_codes == a.c &&
      a.ld_scales == a.c / kScaleBlock) {
    a.c *= a.n;
    a.n = 1;
  }
  const bool vec = a.c * b % 16 == 0 && vector_rows(a.x, a.ld_x, a.n, b, 16) &&
                   vector_rows(a.codes, a.ld_codes, a.n, 1, 16 / b);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return p->dtype == MOE_FP32   ? launch_checkpoint<float>(a, vec, restore, s)
         : p->dtype == MOE_BF16 ? launch_checkpoint<__nv_bfloat16>(a, vec, restore, s)
                                : launch_checkpoint<__half>(a, vec, restore, s);
}

template <typename T, int ACT>
int launch_gated(const GatedArgs& a, bool vec, bool kept, bool backward, cudaStream_t s) {
  const bool words = backward && !kept && !vec;
  const int lanes = vec || words ? 32 : kept && !backward ? kOwn<true, true> : kOwn<true>;
  const dim3 grid(grid_of(a.n, a.c, lanes * (words ? kWordUnits * LikeWord<T>::N : kGatedUnits * Vec<T>::kN)));
  const dim3 block(32 * kWarps);
  auto go = [&](auto* v, auto* e) {
    return launched(vec ? launch_behind(v, grid, block, 0, s, a) : launch_behind(e, grid, block, 0, s, a));
  };
  if (backward)
    return kept ? go(gated_backward_kernel<T, ACT, false, true>, gated_backward_kernel<T, ACT, true, true>)
                : go(gated_backward_kernel<T, ACT, false, false>, gated_backward_words_kernel<T, ACT>);
  return kept ? go(gated_kernel<T, ACT, false, true>, gated_kernel<T, ACT, true, true>)
              : go(gated_kernel<T, ACT, false, false>, gated_kernel<T, ACT, true, false>);
}
template <typename T>
int launch_gated(int act, const GatedArgs& a, bool vec, bool kept, bool backward, cudaStream_t s) {
  switch (act) {
    case MOE_ACT_RELU: return launch_gated<T, MOE_ACT_RELU>(a, vec, kept, backward, s);
    case MOE_ACT_GELU: return launch_gated<T, MOE_ACT_GELU>(a, vec, kept, backward, s);
    case MOE_ACT_GELU_TANH: return launch_gated<T, MOE_ACT_GELU_TANH>(a, vec, kept, backward, s);
    case MOE_ACT_SILU: return launch_gated<T, MOE_ACT_SILU>(a, vec, kept, backward, s);
    default: return launch_gated<T, MOE_ACT_NONE>(a, vec, kept, backward, s);
  }
}

int gated(const moe_gated_args* p, bool backward, moe_stream_t stream) {
  if (p == nullptr || p->n < 0 || p->n > kMaxSize || p->c < 1 || p->c > kMaxSize) return MOE_ERR_ARG;
  if ((p->dtype != MOE_BF16 && p->dtype != MOE_FP16) || p->act < MOE_ACT_NONE || p->act > MOE_ACT_SILU)
    return MOE_ERR_ARG;
  if (p->n == 0) return MOE_OK;
  const bool kept = p->gate_scales != nullptr;
  if (kept != (p->up_scales != nullptr)) return MOE_ERR_ARG;
  const int in = backward && kept ? 1 : 2;
  const long long ld_gate = in == 1 ? p->c : p->ld_gate, ld_up = in == 1 ? p->c : p->ld_up;
  if (!check_matrix(p->gate, ld_gate, p->n, p->c, in) || !check_matrix(p->up, ld_up, p->n, p->c, in))
    return MOE_ERR_ARG;
  if (backward) {
    if (!check_matrix(p->dh, p->ld_dh, p->n, p->c, 2) || !check_matrix(p->dgate, p->ld_dgate, p->n, p->c, 2) ||
        !check_matrix(p->dup, p->ld_dup, p->n, p->c, 2) ||
        (p->h != nullptr && !check_matrix(p->h, p->ld_h, p->n, p->c, 2)))
      return MOE_ERR_ARG;
  } else if (!check_matrix(p->h, p->ld_h, p->n, p->c, 2) ||
             (kept != (p->gate_codes != nullptr)) || (kept != (p->up_codes != nullptr))) {
    return MOE_ERR_ARG;
  }
  int sms = 0;
  const int rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  GatedArgs a{};
  a.gate = p->gate;
  a.up = p->up;
  a.dh = p->dh;
  a.h = p->h;
  a.dgate = p->dgate;
  a.dup = p->dup;
  a.gate_codes = static_cast<uint8_t*>(p->gate_codes);
  a.up_codes = static_cast<uint8_t*>(p->up_codes);
  a.gate_scales = p->gate_scales;
  a.up_scales = p->up_scales;
  a.n = p->n;
  a.c = p->c;
  a.ld_gate = ld_gate;
  a.ld_up = ld_up;
  a.ld_h = p->ld_h;
  a.ld_dh = p->ld_dh;
  a.ld_dgate = p->ld_dgate;
  a.ld_dup = p->ld_dup;
  a.ld_codes = a.c;
  a.ld_scales = scale_blocks(a.c);
  auto whole = [&](const void* q, long long ld) { return q == nullptr || ld == a.c; };
  // Whole blocks in one run of memory: one long row.
  if (a.n > 1 && a.c % kScaleBlock == 0 && a.ld_gate == a.c && a.ld_up == a.c && whole(a.h, a.ld_h) &&
      (!backward || (a.ld_dh == a.c && a.ld_dgate == a.c && a.ld_dup == a.c))) {
    a.c *= a.n;
    a.n = 1;
  }
  auto rows = [&](const void* q, long long ld) { return q == nullptr || vector_rows(q, ld, a.n, 2, 16); };
  bool vec = a.c % 8 == 0 && rows(a.h, a.ld_h);
  if (backward)
    vec = vec && rows(a.dh, a.ld_dh) && rows(a.dgate, a.ld_dgate) && rows(a.dup, a.ld_dup);
  if (in == 1)
    vec = vec && aligned_to(a.gate, 8) && aligned_to(a.up, 8);
  else
    vec = vec && rows(a.gate, a.ld_gate) && rows(a.up, a.ld_up);
  if (kept && !backward) vec = vec && aligned_to(a.gate_codes, 8) && aligned_to(a.up_codes, 8);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return p->dtype == MOE_BF16 ? launch_gated<__nv_bfloat16>(p->act, a, vec, kept, backward, s)
                              : launch_gated<__half>(p->act, a, vec, kept, backward, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_checkpoint(const moe_checkpoint_args* p, moe_stream_t stream) { return checkpoint(p, false, stream); }
int moe_restore(const moe_checkpoint_args* p, moe_stream_t stream) { return checkpoint(p, true, stream); }
int moe_gated(const moe_gated_args* p, moe_stream_t stream) { return gated(p, false, stream); }
int moe_gated_backward(const moe_gated_args* p, moe_stream_t stream) { return gated(p, true, stream); }

}  // extern "C"
