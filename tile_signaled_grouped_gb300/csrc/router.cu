// Routing to experts from their scores, with a balance bias, groups and renormalised
// weights, and its backward pass.
//
// Forward, for each token with scores l_e:
//   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e) / sum_i exp(l_i)
//   c_e = s_e + b_e                                   (selection only)
//   the groups of E / G consecutive experts with the largest sums of their group_top
//   largest c_e stay; the k largest c_e of those are chosen (equal: lower id or group)
//   w_j = s_j                 or  s_j / (sum of the chosen s)      times `scale`
//
// A warp takes a token, its experts in the lanes' registers. At many tokens neither memory nor
// the issue slots (68 % full) are the bound, but both the instructions and the rounds that follow
// one another: 16384 x 256 with a bias and 4 of 8 groups, k = 8, takes 16 us (1.1 TB/s of scores)
// for 670 warp instructions a token: 75 to load, 75 for the scores, 55 to sort a lane's eight,
// 125 for the groups, 20 a round, 50 to find the ids, 40 to judge how close the order is, 75
// for the weights. 1.7 of the 16 us pass while the last tokens decided in 64 bits end. At few
// tokens it is bound by its chain of warp reductions: 3.2 us for one.
//
// Which experts are chosen is decided as in 64 bits. The scores are computed in 32 bits
// with a known error bound; where two neighbours in the order of the winners (or the
// last group kept and the first one dropped) lie within it, those that may belong on
// either side are scored again in 64 bits and ordered by that. Without a bias the order of
// the c_e is that of the l_e, which needs no rounding, so only sums of group scores can be
// close then.
#include <algorithm>
#include <atomic>

#include "moe_common.cuh"
#include "ops_common.cuh"
#include "route_topk.cuh"

namespace moe {

int ops_device(int* num_sms) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> table[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  int sms = dev < kMaxDevices ? table[dev].load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;
    if (dev < kMaxDevices) table[dev].store(sms, std::memory_order_relaxed);
  }
  *num_sms = sms;
  return MOE_OK;
}

namespace {

constexpr int kRouterWarps = 8;

struct RouterArgs {
  const void* logits;
  const float* bias;    // [E] or null
  int32_t* ids;         // [n][k]
  float* w;             // [n][k]
  const float* dw;      // backward: [n][k]
  void* dl;             // backward: [n][ld_dl]
  long long n, ld, ld_dl;
  int dtype, E, k, G, TG, GT, score, renorm;
  bool vec;  // rows (and the bias) can be read and written by vectors of four
  int lpg, lpg_log2;  // lanes of a group: the largest power of two that leaves each one its own
  float scale;
};

// The largest and the smallest value of the warp without its NaN; NaN if there is no other.
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float redux_min(float v) {
  float r;
  asm("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// The largest value of the warp; NaN counts as -inf.
__device__ __forceinline__ float warp_max(float v) { return redux_max(v == v ? v : -INFINITY); }
// Within 5 steps of fp32 (expf 2, the fast division 2, two roundings); an exponential that
// the fast division takes for infinity (beyond 2^126) belongs to a score below 1e-37.
__device__ __forceinline__ float sigmoid(float l) { return __fdividef(1.0f, 1.0f + expf(-l)); }
// For the order alone: within 4 * 2^-23 of s, not relative to it. exp(-l) = 2^(-l log2 e) is off
// by (1.5 + |l|) 2^-23 of itself (the product's rounding, 2^-22.5 for ex2), which s (1 - s)
// turns into less than 0.5 * 2^-23; the sum's rounding and the reciprocal add 2 s 2^-23.
__device__ __forceinline__ float sigmoid_near(float l) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}

// The two largest of (a, b, ...) so far.
template <typename F>
__device__ __forceinline__ void top2(F v, F& t1, F& t2) {
  t2 = v > t1 ? t1 : (v > t2 ? v : t2);
  t1 = v > t1 ? v : t1;
}

// What the order is decided by in 64 bits: the token's scores, and the sum of its
// exponentials for a softmax (the whole warp computes it).
struct Exact {
  const RouterArgs& a;
  const void* row;
  double mx, sum;
  __device__ Exact(const RouterArgs& args, const void* r, int lane) : a(args), row(r), mx(-INFINITY), sum(0) {
    if (a.score != MOE_SCORE_SOFTMAX) return;
    for (int e = lane; e < a.E; e += 32) {
      const double l = load_as_f32(row, a.dtype, e);
      mx = l > mx ? l : mx;
    }
    for (int o = 16; o; o >>= 1) {
      const double v = __shfl_xor_sync(kAll, mx, o);
      mx = v > mx ? v : mx;
    }
    if (mx == -INFINITY) return;
    for (int e = lane; e < a.E; e += 32) sum += exp((double)load_as_f32(row, a.dtype, e) - mx);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  }
  // c of expert e (NaN: -inf).
  __device__ double at(int e) const {
    const double l = load_as_f32(row, a.dtype, e);
    double c = a.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-l)) : sum == 0.0 ? 0.0 : exp(l - mx) / sum;
    if (a.bias != nullptr) c += (double)__ldg(a.bias + e);
    return c == c ? c : -INFINITY;
  }
};

// This group's score in 64 bits, in every lane.
__device__ double exact_group(const Exact& x, int g, int lane) {
  const int per = x.a.E / x.a.G;
  double t1 = -INFINITY, t2 = -INFINITY;
  for (int i = lane; i < per; i += 32) top2(x.at(g * per + i), t1, t2);
  for (int o = 16; o; o >>= 1) {
    const double u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
    top2(u1, t1, t2);
    top2(u2, t1, t2);
  }
  return x.a.GT > 1 && per > 1 ? t1 + t2 : t1;
}

// Group g's score stands in lane g (g < G); `may` and `sure` are the groups that may be and
// that are certainly kept. The rest of the TG places goes by the 64-bit scores.
__device__ __noinline__ uint32_t settle_groups(const RouterArgs& a, const void* row, uint32_t may,
                                               uint32_t sure, int lane) {
  const Exact x(a, row, lane);
  double mine = -INFINITY;
  for (uint32_t m = may; m; m &= m - 1) {
    const double v = exact_group(x, __ffs(m) - 1, lane);
    if (lane == __ffs(m) - 1) mine = v;
  }
  int rank = 0;
  for (uint32_t m = may; m; m &= m - 1) {
    const int h = __ffs(m) - 1;
    const double o = __shfl_sync(kAll, mine, h);
    rank += (o > mine) | ((o == mine) & (h < lane));
  }
  return sure | (__ballot_sync(kAll, rank < a.TG - __popc(sure)) & may);
}

// rank_groups where the last group kept and the first one dropped are too close to call.
__device__ __noinline__ uint32_t settle_ranks(const RouterArgs& a, const void* row, float sum, float last,
                                              float first, float tol, int lane) {
  const float s = __shfl_sync(kAll, sum, min(lane * a.lpg, 31));  // lane g: group g's
  const uint32_t in = a.G < 32 ? (1u << a.G) - 1u : kAll;
  const uint32_t sure = __ballot_sync(kAll, s > last + tol) & in;
  const uint32_t out = __ballot_sync(kAll, s < first - tol) & in;
  const uint32_t kept = settle_groups(a, row, in & ~(sure | out), sure, lane);
  const int g = lane >> a.lpg_log2;
  return __ballot_sync(kAll, g < a.G && ((kept >> (g & 31)) & 1u));
}

// Which groups stay: bits g LPG .. g LPG + LPG - 1 of the result are group g's, and so are those
// lanes, each of which brings the two largest values t1 and t2 that it saw. A group's lanes share
// its comparisons with the others. eps: what a value may be off by beside the rounding of a sum
// with a bias; negative where none is.
template <int LPG, bool WHOLE>
__device__ __forceinline__ uint32_t rank_groups_of(const RouterArgs& a, const void* row, float t1, float t2,
                                                   bool sums, float eps, float smax, int lane) {
#pragma unroll
  for (int o = LPG / 2; o; o >>= 1) {
    const float u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
    t2 = fmaxf(fminf(t1, u1), fmaxf(t2, u2));
    t1 = fmaxf(t1, u1);
  }
  const float sum = sums ? t1 + t2 : t1;
  const int G = WHOLE ? 32 / LPG : a.G, g = lane / LPG, q = lane % LPG;
  int rank = 0;
#pragma unroll
  for (int h0 = 0; h0 < 32 / LPG; h0 += LPG) {
    if (!WHOLE && h0 >= G) break;
    const int h = h0 + q;
    const float o = __shfl_sync(kAll, sum, h * LPG);  // h past the last group does not count
    rank += (h < G) & ((o > sum) | ((o == sum) & (h < g)));
  }
#pragma unroll
  for (int o = LPG / 2; o; o >>= 1) rank += __shfl_xor_sync(kAll, rank, o);
  const bool in = g < G, stays = in && rank < a.TG;
  const uint32_t kept = __ballot_sync(kAll, stays);
  if (eps >= 0.f) {
    // What two sums may differ by and still be in the other order. The largest finite term
    // counts, not the sum: a sum of two can cancel.
    float m = smax;
    if (a.bias != nullptr) {
      m = fabsf(t1) < INFINITY ? fmaxf(m, fabsf(t1)) : m;
      m = redux_max(fabsf(t2) < INFINITY ? fmaxf(m, fabsf(t2)) : m);
    }
    const float tol = 4.f * eps + 0x1p-21f * m;
    const float last = redux_min(stays ? sum : NAN), first = redux_max(in && !stays ? sum : NAN);
    // Not for -inf - -inf, where the ids have decided, nor where every group stays.
    if (last - first <= tol) return settle_ranks(a, row, sum, last, first, tol, lane);
  }
  return kept;
}
template <bool WHOLE>
__device__ __forceinline__ uint32_t rank_groups(const RouterArgs& a, const void* row, float t1, float t2,
                                                bool sums, float eps, float smax, int lane) {
  switch (a.lpg_log2) {  // unrolled, less than half the instructions of loops over a.lpg
    case 0: return rank_groups_of<1, WHOLE>(a, row, t1, t2, sums, eps, smax, lane);
    case 1: return rank_groups_of<2, WHOLE>(a, row, t1, t2, sums, eps, smax, lane);
    case 2: return rank_groups_of<4, WHOLE>(a, row, t1, t2, sums, eps, smax, lane);
    case 3: return rank_groups_of<8, WHOLE>(a, row, t1, t2, sums, eps, smax, lane);
    default: return rank_groups_of<16, WHOLE>(a, row, t1, t2, sums, eps, smax, lane);
  }
}

// Slot `lane`'s id where the m candidates in lanes 0.. (id in lane) hold every expert that
// may be among the k: ordered by their 64-bit values, equal ones by id.
__device__ __noinline__ int settle_slots(const RouterArgs& a, const void* row, int id, int m, int lane) {
  const Exact x(a, row, lane);
  const double mine = lane < m ? x.at(id) : -INFINITY;
  int rank = 0;
  for (int h = 0; h < m; ++h) {
    const double o = __shfl_sync(kAll, mine, h);
    const int oe = __shfl_sync(kAll, id, h);
    rank += (o > mine) | ((o == mine) & (oe < id));
  }
  int got = 0;
  for (int h = 0; h < m; ++h) {  // lane h's candidate goes to slot rank
    const int r = __shfl_sync(kAll, rank, h), oe = __shfl_sync(kAll, id, h);
    if (r == lane) got = oe;
  }
  return got;
}

// The k experts of the groups `kept` by their 64-bit values, where more than 32 of them may
// be among the k; returns the id of slot `lane`. buf: E doubles of shared memory.
__device__ __noinline__ int settle_all(const RouterArgs& a, const void* row, uint32_t kept, double* buf,
                                       int lane) {
  const int per = a.E / a.G;
  const Exact x(a, row, lane);
  __syncwarp();
  for (int e = lane; e < a.E; e += 32) buf[e] = x.at(e);
  __syncwarp();
  uint32_t taken = 0;  // bit i: this lane's expert lane + 32 i
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int be = 0x7FFFFFFF;
    for (int i = 0, e = lane; e < a.E; ++i, e += 32) {
      const bool ok = !((taken >> i) & 1u) && (a.G == 1 || ((kept >> (e / per * a.lpg)) & 1u));
      if (ok && (be == 0x7FFFFFFF || buf[e] > bv)) {
        bv = buf[e];
        be = e;
      }
    }
    for (int o = 16; o; o >>= 1) {
      const double ov = __shfl_xor_sync(kAll, bv, o);
      const int oe = __shfl_xor_sync(kAll, be, o);
      const bool take = oe != 0x7FFFFFFF && (be == 0x7FFFFFFF || ov > bv || (ov == bv && oe < be));
      bv = take ? ov : bv;
      be = take ? oe : be;
    }
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
    if (lane == j) mine = be;
  }
  __syncwarp();
  return mine;
}

// The normalised weight of slot `lane` (0 in lanes >= k) before `scale`: t is its score,
// mx and inv the token's maximum and 1 / sum (softmax that is not renormalised).
__device__ __forceinline__ float slot_weight(const RouterArgs& a, float t, bool in, float mx, float inv) {
  if (!a.renorm) {
    if (!in) return 0.f;
    if (a.score == MOE_SCORE_SIGMOID) return sigmoid(t);
    return mx == -INFINITY ? 0.f : expf(t - mx) * inv;
  }
  if (a.score == MOE_SCORE_SIGMOID) {
    const float s = in ? sigmoid(t) : 0.f;
    const float S = warp_sum(s);
    if (!(S < 1e-20f)) return s / S;
    // Scores that leave the range of 32 bits: the ratio from their logarithms, which
    // here are the l themselves (log s = l - log(1 + exp(l)), exp(l) < 1e-20).
  }
  const float m = warp_max(in ? t : -INFINITY);
  const float e = in && m != -INFINITY ? expf(t - m) : 0.f;
  const float S = warp_sum(e);
  return S == 0.f ? 0.f : e / S;
}

// A lane's values, the largest first: sorting networks of 1, 5 and 19 comparators (Batcher).
template <int PER>
__device__ __forceinline__ void sort_values(float (&v)[PER]) {
  auto order = [&](int i, int j) {
    const float x = v[i], y = v[j];
    v[i] = fmaxf(x, y);
    v[j] = fminf(x, y);
  };
  if constexpr (PER == 2) {
    order(0, 1);
  } else if constexpr (PER == 4) {
    order(0, 1), order(2, 3), order(0, 2), order(1, 3), order(1, 2);
  } else if constexpr (PER == 8) {
    order(0, 1), order(2, 3), order(4, 5), order(6, 7);
    order(0, 2), order(1, 3), order(4, 6), order(5, 7);
    order(1, 2), order(5, 6);
    order(0, 4), order(1, 5), order(2, 6), order(3, 7);
    order(2, 4), order(3, 5);
    order(1, 2), order(3, 4), order(5, 6);
  }
}

// Four or eight scores of a lane, as one or two vector loads.
template <int PER>
__device__ __forceinline__ void load_scores(const void* row, int dtype, int e0, float (&l)[PER]) {
  if (dtype == MOE_FP32) {
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + e0 + i));
      l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < PER; i += 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(row) + e0 + i));
    const float2 p = dtype == MOE_BF16 ? unpack2<__nv_bfloat16>(v.x) : unpack2<__half>(v.x);
    const float2 q = dtype == MOE_BF16 ? unpack2<__nv_bfloat16>(v.y) : unpack2<__half>(v.y);
    l[i] = p.x, l[i + 1] = p.y, l[i + 2] = q.x, l[i + 3] = q.y;
  }
}

// A lane's values to shared memory and back: vectors of up to four beside the other lanes' (no
// bank conflicts, which one run of eight for each lane would have).
template <int PER>
__device__ __forceinline__ void put_values(float* vals, int lane, const float (&v)[PER]) {
  if constexpr (PER >= 4) {
#pragma unroll
    for (int i = 0; i < PER; i += 4)
      reinterpret_cast<float4*>(vals)[i * 8 + lane] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) vals[i * 32 + lane] = v[i];
  }
}
template <int PER>
__device__ __forceinline__ void get_values(const float* vals, int lane, float (&v)[PER]) {
  if constexpr (PER >= 4) {
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const float4 u = reinterpret_cast<const float4*>(vals)[i * 8 + lane];
      v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = vals[i * 32 + lane];
  }
}
constexpr int kSlotBytes = 33 * 8 + 8;
template <int PER>
constexpr int kWarpBytes = kSlotBytes + 32 * (2 * PER + (PER <= 8 ? 2 : 0)) * (int)sizeof(float);

// Lane l holds experts PER l .. PER l + PER - 1. Up to PER = 8 it sorts their values once, its
// best in a register and the rest in shared memory, from where a round's winner takes its next;
// which expert a value was is found after the rounds, from the values' places (a sort of pairs
// and lists shifted in registers took 23 us where this takes 16). Above, each round looks
// through the lane's candidates again. WHOLE: E = 32 PER and a power of two of groups, so that a
// group is a run of whole lanes: its two largest values are among the heads of those lanes'
// lists, and a group that goes takes its lanes along. Otherwise the values that groups are
// judged by pass through shared memory. Six CTAs an SM: 3 % faster than the four of 64 registers.
template <int PER, bool WHOLE>
__global__ void __launch_bounds__(32 * kRouterWarps, PER <= 8 ? 6 : 1)
    router_kernel(const __grid_constant__ RouterArgs a) {
  static_assert(!WHOLE || PER <= 8, "sorted lists");
  extern __shared__ double2 smem_d[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tok = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
  if (tok >= a.n) return;
  // A warp's shared memory: 33 slots, the values (PER <= 8, or of groups) and the lanes' lists
  // of them (PER <= 8), which the 64-bit values may replace.
  char* mem = reinterpret_cast<char*>(smem_d) + (size_t)warp * kWarpBytes<PER>;
  float2* slot = reinterpret_cast<float2*>(mem);
  double* buf = reinterpret_cast<double*>(mem + kSlotBytes);
  float* vals = reinterpret_cast<float*>(buf);
  float* list = vals + 32 * PER;
  const int tb = a.dtype == MOE_FP32 ? 4 : 2, e0 = lane * PER;
  const void* row = static_cast<const char*>(a.logits) + (size_t)tok * a.ld * tb;

  float c[PER];  // the scores, then what experts are ordered by (NaN: -inf)
  if (WHOLE && PER >= 4 && a.vec) {
    if constexpr (PER >= 4) load_scores<PER>(row, a.dtype, e0, c);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      c[i] = WHOLE || e0 + i < a.E ? load_as_f32(row, a.dtype, e0 + i) : -INFINITY;
  }
  const bool sums = a.G > 1 && a.GT > 1 && a.E > a.G;  // groups are judged by sums of scores
  const bool by_score = a.bias != nullptr || sums;     // else by the l themselves
  float mx = 0.f, inv = 1.f;
  const bool soft = a.score == MOE_SCORE_SOFTMAX && (by_score || !a.renorm);
  float s[PER];
  if (soft) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, c[i]);
    mx = warp_max(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = mx == -INFINITY ? 0.f : expf(c[i] - mx);
      sum += s[i];
    }
    sum = warp_sum(sum);
    if (mx != -INFINITY) inv = 1.0f / sum;
  }
  auto score_of = [&](float l) {
    return a.score == MOE_SCORE_SIGMOID ? sigmoid_near(l) : mx == -INFINITY ? 0.f : expf(l - mx) * inv;
  };
  if (a.bias != nullptr) {
    float b[PER];
    if (WHOLE && PER >= 4 && a.vec) {
      if constexpr (PER >= 4) load_scores<PER>(a.bias, MOE_FP32, e0, b);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) b[i] = WHOLE || e0 + i < a.E ? __ldg(a.bias + e0 + i) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = (soft ? s[i] * inv : sigmoid_near(c[i])) + b[i];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) c[i] = fmaxf(c[i], -INFINITY);  // of NaN and a number the number
  // How far a score in 32 bits may be off: 5 steps of fp32 for the sigmoid; for the softmax
  // 3 for the exponential and its argument, PER + 5 additions in the sum, 2 for the rest.
  // At most `eps` for scores up to smax; c adds its own rounding.
  const float smax = a.score == MOE_SCORE_SIGMOID ? 1.0f : inv;
  const float eps = (a.score == MOE_SCORE_SIGMOID ? 6.f : PER + 12.f) * 0x1p-23f * smax;
  const float group_eps = by_score ? eps : -1.f;  // judged by the l themselves, nothing is rounded

  uint32_t kept = kAll;
  uint32_t open = 0;  // bit i: this lane's candidate i may be chosen
  if constexpr (!WHOLE) {
    if (a.G > 1) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i < a.E) {
          const float v = a.bias == nullptr && sums ? score_of(c[i]) : c[i];
          vals[e0 + i] = v == v ? v : -INFINITY;
        }
      __syncwarp();
      const int per = a.E / a.G, g = lane >> a.lpg_log2;
      float t1 = -INFINITY, t2 = -INFINITY;
      if (g < a.G)
        for (int i = lane & (a.lpg - 1); i < per; i += a.lpg) top2(vals[g * per + i], t1, t2);
      kept = rank_groups<WHOLE>(a, row, t1, t2, sums, group_eps, smax, lane);
      int q = e0 / per, r = e0 % per;  // of expert e0 + i: its group, its place there
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        open |= (e0 + i < a.E && ((kept >> ((q << a.lpg_log2) & 31)) & 1u)) ? 1u << i : 0u;
        const bool next = ++r == per;
        r = next ? 0 : r;
        q += next;
      }
      __syncwarp();  // what is chosen from takes their place
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) open |= e0 + i < a.E ? 1u << i : 0u;
    }
  }

  // Rounds: the warp's best candidate each. Round j's winner writes slot j. NaN: no candidate.
  float head = NAN;  // PER <= 8: this lane's best, then the rest in their order from list[at]
  int at = lane * (PER + 1);
  if constexpr (PER <= 8) {
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = (open >> i) & 1u ? c[i] : NAN;
    }
    put_values<PER>(vals, lane, c);
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = fmaxf(c[i], -INFINITY);  // after every candidate
    }
    sort_values<PER>(c);
    const int n = WHOLE ? PER : __popc(open);
#pragma unroll
    for (int i = 1; i < PER; ++i) list[at + i - 1] = i < n ? c[i] : NAN;
    list[at + PER - 1] = NAN;
    head = n > 0 ? c[0] : NAN;
    if (WHOLE && a.G > 1) {
      float t1 = c[0], t2 = PER > 1 ? c[PER > 1 ? 1 : 0] : -INFINITY;
      if (a.bias == nullptr && sums) {
        t1 = score_of(t1);
        t2 = PER > 1 ? score_of(t2) : t2;
        t1 = t1 == t1 ? t1 : -INFINITY;
        t2 = t2 == t2 ? t2 : -INFINITY;
      }
      kept = rank_groups<WHOLE>(a, row, t1, t2, sums, group_eps, smax, lane);
      head = (kept >> lane) & 1u ? head : NAN;
    }
  }
  int rounds = 0;
  float past = NAN;  // the last round's
  auto round = [&] {
    float v = head;
    int bi = -1;
    if constexpr (PER > 8) {
      v = NAN;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const bool better = ((open >> i) & 1u) & ((c[i] > v) | (bi < 0));
        v = better ? c[i] : v;
        bi = better ? i : bi;
      }
    }
    past = redux_max(v);
    // Equal ones: the lowest id is the lowest lane's, whose candidates are in that order too.
    const bool win = lane == __ffs(__ballot_sync(kAll, v == past)) - 1;
    if (win) {
      slot[rounds] = make_float2(v, __int_as_float(PER > 8 ? e0 + bi : at));
      if constexpr (PER > 8)
        open &= ~(1u << bi);
      else
        head = list[at++];
    }
    ++rounds;
  };
  const int need = a.bias != nullptr ? a.k + 1 : a.k;  // with a bias, the next in line too
  // The id of slot `lane` in the lanes that have one (the last round may have found none).
  auto slot_id = [&] {
    __syncwarp();
    int id = 0;
    if (lane < rounds - (past == past ? 0 : 1)) {
      const float2 w = slot[lane];
      id = __float_as_int(w.y);
      if constexpr (PER <= 8) {
        // The value's place among its lane's candidates: of the equal ones that whose rank, the
        // larger ones and those before it, was the winner's place in the list.
        const int from = id / (PER + 1);
        float v[PER];
        get_values<PER>(vals, from, v);
        uint32_t same = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) same |= v[i] == w.x ? 1u << i : 0u;
        if (same & (same - 1)) {
          int skip = id % (PER + 1);
#pragma unroll
          for (int i = 0; i < PER; ++i) skip -= v[i] > w.x;
          for (; skip > 0; --skip) same &= same - 1;
        }
        id = from * PER + __ffs(same) - 1;
      }
    }
    return id;
  };
  while (rounds < need) round();
  int my_id = slot_id();
  if (a.bias != nullptr) {
    // Neighbours of the order within their error, unless score and bias are equal (then
    // the ids decide, as they did).
    auto differ = [&] {
      const int ni = __shfl_down_sync(kAll, my_id, 1);
      return lane < 31 && (load_as_f32(row, a.dtype, my_id) != load_as_f32(row, a.dtype, ni) ||
                           __ldg(a.bias + my_id) != __ldg(a.bias + ni));
    };
    bool close = false;
    if (lane < a.k) {
      const float x = slot[lane].x, y = lane + 1 < a.k ? slot[lane + 1].x : past;
      close = x - y <= 2.f * eps + 0x1p-22f * (fabsf(x) + fabsf(y));
    }
    const uint32_t pairs = __ballot_sync(kAll, close);
    if (pairs != 0) {
      const bool unlike = differ();
      bool open_order = close && (unlike || lane == 31);
      const uint32_t last = 1u << (a.k - 1);
      if (__any_sync(kAll, open_order) || (pairs & last)) {
        // Every candidate that may be among the k: those within the error of the k-th. Behind an
        // equal one in line there may be one that differs.
        const float border = slot[a.k - 1].x;
        const float low = border - (2.f * eps + 0x1p-21f * fabsf(border));
        while (past >= low && rounds <= 32) round();
        my_id = slot_id();
        const int m = min(rounds - 1, 32);  // `rounds` counts the one below `low`, or that found none
        open_order |= differ() & (lane >= a.k - 1) & (lane + 1 < m);
        if (past >= low)
          my_id = settle_all(a, row, kept, buf, lane);
        else if (__any_sync(kAll, open_order))
          my_id = settle_slots(a, row, my_id, m, lane);
      }
    }
  }

  const bool in = lane < a.k;
  const float t = in ? load_as_f32(row, a.dtype, my_id) : 0.f;
  const float w = slot_weight(a, t, in, mx, inv);
  if (in) {
    a.ids[tok * a.k + lane] = my_id;
    a.w[tok * a.k + lane] = a.scale * w;
  }
}

// Backward. With g_j = scale * dw_j and r_j the weight before `scale`:
//   sigmoid:              dl_j = g_j s_j (1 - s_j)
//   sigmoid, renormalised dl_j = r_j (g_j - sum_i g_i r_i) (1 - s_j)
//   softmax, renormalised dl_j = r_j (g_j - sum_i g_i r_i)
//   softmax               dl_e = p_e ((g_j where e is chosen, else 0) - sum_i g_i p_i)
// zero for the other experts except in the last, the only one that reads every score.
// A warp takes a token, lane l experts PER l .. PER l + PER - 1: the chosen experts' values
// reach their lanes through shared memory, and the row leaves in vectors. Bound by the
// row's bytes and, at these lengths, by the instructions a row costs.
template <int PER>
__global__ void __launch_bounds__(32 * kRouterWarps)
    router_backward_kernel(const __grid_constant__ RouterArgs a) {
  extern __shared__ double2 smem_d[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * PER;
  const long long tok = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
  if (tok >= a.n) return;
  float* g = reinterpret_cast<float*>(smem_d) + (size_t)warp * 32 * PER;  // [32 PER], to E and beyond
  const int tb = a.dtype == MOE_FP32 ? 4 : 2;
  const void* row = static_cast<const char*>(a.logits) + (size_t)tok * a.ld * tb;
  void* out = static_cast<char*>(a.dl) + (size_t)tok * a.ld_dl * tb;
  const bool whole = a.E == 32 * PER && a.vec;  // vectors of four; `vec` covers both matrices

  const int id = lane < a.k ? __ldg(a.ids + tok * a.k + lane) : -1;
  const bool in = id >= 0 && id < a.E;  // others have no gradient
  const float t = in ? load_as_f32(row, a.dtype, id) : 0.f;
  const float gj = in ? a.scale * __ldg(a.dw + tok * a.k + lane) : 0.f;
  const bool all = a.score == MOE_SCORE_SOFTMAX && !a.renorm;
  float p[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) g[lane + 32 * i] = 0.f;
  float mx = 0.f, inv = 1.f;
  if (all) {
    if (PER >= 4 && whole) {
      if constexpr (PER >= 4) load_scores<PER>(row, a.dtype, e0, p);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) p[i] = e0 + i < a.E ? load_as_f32(row, a.dtype, e0 + i) : -INFINITY;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, p[i]);
    mx = warp_max(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      p[i] = mx == -INFINITY ? 0.f : expf(p[i] - mx);
      sum += p[i];
    }
    sum = warp_sum(sum);
    inv = mx == -INFINITY ? 0.f : 1.0f / sum;
  }
  const float r = slot_weight(a, t, in, mx, inv);
  const float dot = a.renorm || all ? warp_sum(in ? gj * r : 0.f) : 0.f;
  float d = r * (a.renorm ? gj - dot : gj);
  if (a.score == MOE_SCORE_SIGMOID) d *= sigmoid(-t);  // 1 - s
  __syncwarp();
  if (in) g[id] = all ? gj : d;
  __syncwarp();
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = g[e0 + i];
    if (all) v[i] = p[i] * inv * (v[i] - dot);
  }
  if (PER >= 4 && whole) {
    if constexpr (PER >= 4) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        if (a.dtype == MOE_FP32) {
          *reinterpret_cast<float4*>(static_cast<float*>(out) + e0 + i) =
              make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
          const uint2 u = a.dtype == MOE_BF16
                              ? make_uint2(pack2<__nv_bfloat16>(v[i], v[i + 1]),
                                           pack2<__nv_bfloat16>(v[i + 2], v[i + 3]))
                              : make_uint2(pack2<__half>(v[i], v[i + 1]), pack2<__half>(v[i + 2], v[i + 3]));
          *reinterpret_cast<uint2*>(static_cast<unsigned short*>(out) + e0 + i) = u;
        }
      }
    }
  } else {
    // Rows of any length: neighbouring lanes write neighbouring experts.
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) g[e0 + i] = v[i];
    __syncwarp();
    for (int e = lane; e < a.E; e += 32) store_from_f32(out, a.dtype, e, g[e]);
  }
}

int check_router(const moe_router_cfg* c, int dtype, long long n, long long ld) {
  if (c == nullptr || type_bytes(dtype) == 0) return MOE_ERR_ARG;
  if (c->E < 1 || c->E > 1024 || c->topk < 1 || c->topk > std::min(c->E, 32)) return MOE_ERR_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_ARG;
  if (c->groups < 1 || c->groups > 32 || c->E % c->groups) return MOE_ERR_ARG;
  if (c->topk_groups < 1 || c->topk_groups > c->groups) return MOE_ERR_ARG;
  if (c->group_top != 1 && c->group_top != 2) return MOE_ERR_ARG;
  if (c->topk > c->topk_groups * (c->E / c->groups)) return MOE_ERR_ARG;
  if (c->renorm != 0 && c->renorm != 1) return MOE_ERR_ARG;
  if (!(c->scale - c->scale == 0.f)) return MOE_ERR_ARG;  // finite
  if (n < 0 || n > INT32_MAX || ld < c->E || ld > INT32_MAX) return MOE_ERR_ARG;
  return MOE_OK;
}

RouterArgs router_args(const moe_router_cfg* c, int dtype, long long n, long long ld) {
  RouterArgs a{};
  a.n = n;
  a.ld = ld;
  a.dtype = dtype;
  a.E = c->E;
  a.k = c->topk;
  a.G = c->groups;
  a.TG = c->topk_groups;
  a.GT = c->group_top;
  while ((2 << a.lpg_log2) * a.G <= 32) ++a.lpg_log2;
  a.lpg = 1 << a.lpg_log2;
  a.score = c->score;
  a.renorm = c->renorm;
  a.scale = c->scale;
  return a;
}

// Tokens (warps) of a CTA: eight, four above 512 experts (8 E bytes of shared memory each).
int router_warps(int E) { return E <= 512 ? kRouterWarps : kRouterWarps / 2; }

template <int PER>
void launch_router(const RouterArgs& a, cudaStream_t s) {
  const int warps = router_warps(a.E);
  const unsigned grid = (unsigned)((a.n + warps - 1) / warps);
  const size_t smem = (size_t)warps * kWarpBytes<PER>;
  if constexpr (PER <= 8) {
    if (a.E == 32 * PER && (a.G & (a.G - 1)) == 0) {
      router_kernel<PER, true><<<grid, 32 * warps, smem, s>>>(a);
      return;
    }
  }
  router_kernel<PER, false><<<grid, 32 * warps, smem, s>>>(a);
}

template <int PER>
void launch_router_backward(const RouterArgs& a, cudaStream_t s) {
  const int warps = router_warps(a.E);
  router_backward_kernel<PER><<<(unsigned)((a.n + warps - 1) / warps), 32 * warps,
                                (size_t)warps * 32 * PER * sizeof(float), s>>>(a);
}

}  // namespace

int router_forward(const moe_router_cfg* cfg, const void* logits, int dtype, long long n, long long ld,
                   const float* bias, int32_t* ids, float* w, cudaStream_t s) {
  int rc = check_router(cfg, dtype, n, ld);
  if (rc != MOE_OK) return rc;
  if (n == 0) return MOE_OK;
  if (logits == nullptr || ids == nullptr || w == nullptr) return MOE_ERR_ARG;
  if (!aligned_to(logits, (size_t)type_bytes(dtype)) || !aligned_to(bias, 4) || !aligned_to(ids, 4) ||
      !aligned_to(w, 4))
    return MOE_ERR_ARG;
  int sms = 0;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  RouterArgs a = router_args(cfg, dtype, n, ld);
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.w = w;
  a.vec = aligned_to(logits, 16) && ld % 8 == 0 && aligned_to(bias, 16);
  if (a.E <= 32) launch_router<1>(a, s);
  else if (a.E <= 64) launch_router<2>(a, s);
  else if (a.E <= 128) launch_router<4>(a, s);
  else if (a.E <= 256) launch_router<8>(a, s);
  else if (a.E <= 512) launch_router<16>(a, s);
  else launch_router<32>(a, s);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_router_backward(const moe_router_cfg* cfg, const float* d_w, const void* logits,
                                   const int32_t* ids, int dtype, long long n, long long ld,
                                   void* d_logits, long long ld_d, moe_stream_t stream) {
  int rc = check_router(cfg, dtype, n, ld);
  if (rc != MOE_OK) return rc;
  if (ld_d < cfg->E || ld_d > INT32_MAX) return MOE_ERR_ARG;
  if (n == 0) return MOE_OK;
  if (d_w == nullptr || logits == nullptr || ids == nullptr || d_logits == nullptr) return MOE_ERR_ARG;
  const size_t tb = (size_t)type_bytes(dtype);
  if (!aligned_to(d_w, 4) || !aligned_to(ids, 4) || !aligned_to(logits, tb) || !aligned_to(d_logits, tb))
    return MOE_ERR_ARG;
  int sms = 0;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  RouterArgs a = router_args(cfg, dtype, n, ld);
  a.dw = d_w;
  a.logits = logits;
  a.ids = const_cast<int32_t*>(ids);
  a.dl = d_logits;
  a.ld_dl = ld_d;
  a.vec = aligned_to(logits, 16) && ld % 8 == 0 && aligned_to(d_logits, 16) && ld_d % 8 == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.E <= 32) launch_router_backward<1>(a, s);
  else if (a.E <= 64) launch_router_backward<2>(a, s);
  else if (a.E <= 128) launch_router_backward<4>(a, s);
  else if (a.E <= 256) launch_router_backward<8>(a, s);
  else if (a.E <= 512) launch_router_backward<16>(a, s);
  else launch_router_backward<32>(a, s);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
