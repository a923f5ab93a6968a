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
// A warp takes a token; lane l holds experts l, l + 32, ... in registers. Bound by
// instructions at many tokens (the scores are 4 E bytes and the selection some hundred
// warp instructions), by its chain of warp reductions at few.
//
// Which experts are chosen is decided as in 64 bits. The scores are computed in 32 bits
// with a known error bound; where two neighbours in the order of the winners (or the
// last group kept and the first one dropped) lie within it, the token is decided again
// with 64-bit scores. Without a bias the order of the c_e is that of the l_e, which
// needs no rounding, so only sums of group scores can be close then.
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

constexpr uint32_t kAll = 0xFFFFFFFFu;
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
  float scale;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// The largest value of the warp; NaN counts as -inf.
__device__ __forceinline__ float warp_max(float v) {
  return key_float(__reduce_max_sync(kAll, float_key(v == v ? v : -INFINITY)));
}
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// The two largest of (a, b, ...) so far.
template <typename F>
__device__ __forceinline__ void top2(F v, F& t1, F& t2) {
  t2 = v > t1 ? t1 : (v > t2 ? v : t2);
  t1 = v > t1 ? v : t1;
}

// Bit g of the result: group g stays. val: the E values a group is judged by, in shared
// memory. Lanes share the groups evenly (a power of two of lanes for each). *last and
// *first receive the smallest score kept and the largest dropped (-inf if none is).
template <typename F>
__device__ __forceinline__ uint32_t keep_groups(const RouterArgs& a, const F* val, int lane, F* last,
                                                F* first) {
  int lpg = 1;
  while (lpg * 2 * a.G <= 32) lpg *= 2;
  const int per = a.E / a.G, g = lane / lpg, sub = lane % lpg;
  const F low = -INFINITY;
  F t1 = low, t2 = low;
  if (g < a.G)
    for (int i = sub; i < per; i += lpg) top2(val[g * per + i], t1, t2);
  for (int o = lpg / 2; o; o >>= 1) {
    const F u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
    top2(u1, t1, t2);
    top2(u2, t1, t2);
  }
  F sum = a.GT > 1 && per > 1 ? t1 + t2 : t1;
  sum = __shfl_sync(kAll, sum, min(lane * lpg, 31));  // lane g: group g
  int rank = 0;
  for (int h = 0; h < a.G; ++h) {
    const F o = __shfl_sync(kAll, sum, h);
    rank += (o > sum) | ((o == sum) & (h < lane));
  }
  const uint32_t in = __ballot_sync(kAll, lane < a.G);
  const uint32_t kept = __ballot_sync(kAll, rank < a.TG) & in;
  const uint32_t at_last = __ballot_sync(kAll, rank == a.TG - 1) & in;
  const uint32_t at_first = __ballot_sync(kAll, rank == a.TG) & in;
  const F vl = __shfl_sync(kAll, sum, at_last ? __ffs(at_last) - 1 : 0);
  const F vf = __shfl_sync(kAll, sum, at_first ? __ffs(at_first) - 1 : 0);
  *last = vl;
  *first = at_first ? vf : low;
  return kept;
}

// The token decided with 64-bit scores; returns the id of slot `lane` (lane < k). buf:
// E doubles of shared memory. Rare, so short rather than fast.
__device__ __noinline__ int route_exact(const RouterArgs& a, const void* row, double* buf, int lane) {
  __syncwarp();
  double mx = -INFINITY, sum = 0;
  if (a.score == MOE_SCORE_SOFTMAX) {
    for (int e = lane; e < a.E; e += 32) {
      const double l = load_as_f32(row, a.dtype, e);
      mx = l > mx ? l : mx;
    }
    for (int o = 16; o; o >>= 1) {
      const double v = __shfl_xor_sync(kAll, mx, o);
      mx = v > mx ? v : mx;
    }
    for (int e = lane; e < a.E; e += 32) {
      const double v = mx == -INFINITY ? 0.0 : exp((double)load_as_f32(row, a.dtype, e) - mx);
      sum += v;
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  }
  for (int e = lane; e < a.E; e += 32) {
    const double l = load_as_f32(row, a.dtype, e);
    double c = a.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-l))
               : sum == 0.0                 ? 0.0
                                            : exp(l - mx) / sum;
    if (a.bias != nullptr) c += (double)__ldg(a.bias + e);
    buf[e] = c == c ? c : -INFINITY;
  }
  __syncwarp();
  uint32_t kept = kAll;
  if (a.G > 1) {
    double x, y;
    kept = keep_groups<double>(a, buf, lane, &x, &y);
    __syncwarp();
  }
  if (a.bias == nullptr) {  // the order of the c is that of the scores
    for (int e = lane; e < a.E; e += 32) {
      const float l = load_as_f32(row, a.dtype, e);
      buf[e] = l == l ? l : -INFINITY;
    }
    __syncwarp();
  }
  const int per = a.E / a.G;
  uint32_t taken = 0;  // bit i: this lane's expert lane + 32 i
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int be = 0x7FFFFFFF;
    for (int i = 0, e = lane; e < a.E; ++i, e += 32) {
      const bool ok = !((taken >> i) & 1u) && (a.G == 1 || ((kept >> (e / per)) & 1u));
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

// PER: experts a lane holds. Registers for the sorted list of a lane up to PER = 8; above,
// each round looks through the lane's candidates again.
template <int PER>
__global__ void __launch_bounds__(32 * kRouterWarps) router_kernel(const __grid_constant__ RouterArgs a) {
  extern __shared__ double smem_d[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tok = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
  if (tok >= a.n) return;
  double* buf = smem_d + (size_t)warp * a.E;
  const int tb = a.dtype == MOE_FP32 ? 4 : 2;
  const void* row = static_cast<const char*>(a.logits) + (size_t)tok * a.ld * tb;

  float l[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < a.E ? load_as_f32(row, a.dtype, e) : -INFINITY;
  }
  const bool sums = a.G > 1 && a.GT > 1 && a.E > a.G;  // groups are judged by sums of scores
  const bool by_score = a.bias != nullptr || sums;     // else by the l themselves
  float mx = 0.f, inv = 1.f;
  if (a.score == MOE_SCORE_SOFTMAX && (by_score || !a.renorm)) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, l[i]);
    mx = warp_max(m);
    float sum = 0.f;
    if (mx != -INFINITY) {
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += expf(l[i] - mx);
      sum = warp_sum(sum);
      inv = 1.0f / sum;
    }
  }
  float c[PER];  // what experts are ordered by (NaN: -inf)
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    float v = l[i];
    if (by_score && e < a.E) {
      const float s = a.score == MOE_SCORE_SIGMOID ? sigmoid(l[i])
                      : mx == -INFINITY            ? 0.f
                                                   : expf(l[i] - mx) * inv;
      const float g = a.bias != nullptr ? s + __ldg(a.bias + e) : s;
      if (a.bias != nullptr) v = g;
      if (a.G > 1) reinterpret_cast<float*>(buf)[e] = g == g ? g : -INFINITY;
    } else if (a.G > 1 && e < a.E) {
      reinterpret_cast<float*>(buf)[e] = v == v ? v : -INFINITY;
    }
    c[i] = v == v ? v : -INFINITY;
  }
  // How far a score in 32 bits may be off: expf 2 ulp, the sum of the softmax PER + 5
  // additions, a few roundings more; at most `eps` for s <= smax. c adds its own rounding.
  const float smax = a.score == MOE_SCORE_SIGMOID ? 1.0f : inv;
  const float eps = (PER + 16) * 0x1p-23f * smax;

  uint32_t kept = kAll;
  bool close = false;
  if (a.G > 1) {
    __syncwarp();
    float last, first;
    kept = keep_groups<float>(a, reinterpret_cast<const float*>(buf), lane, &last, &first);
    if (by_score) {
      float cm = 0.f;  // the largest finite |c|: a sum of two can cancel
      if (a.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const float v = fabsf(c[i]);
          cm = v < INFINITY ? fmaxf(cm, v) : cm;
        }
        cm = warp_max(cm);
      }
      close = last - first <= 4.f * eps + 0x1p-21f * fmaxf(cm, smax);  // -inf - -inf: not close
    }
    __syncwarp();
  }
  const int per = a.E / a.G;
  uint32_t my_key = 0, my_id = 0;  // round `lane`'s winner; round k's (the next in line) too
  const int rounds = a.bias != nullptr ? a.k + 1 : a.k;
  uint32_t past_key = 0;  // k = 32: the next in line has no lane of its own
  if (PER <= 8) {
    int e[PER];
    int left = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      e[i] = lane + 32 * i;
      const bool ok = e[i] < a.E && (a.G == 1 || ((kept >> (e[i] / per)) & 1u));
      c[i] = ok ? c[i] : -INFINITY;
      e[i] = ok ? e[i] : 0x7FFFFFFF;  // after every candidate, the ones at -inf too
      left += ok;
    }
    route_sort<PER>(c, e);
    for (int j = 0; j < rounds; ++j) {
      const uint32_t key = left > 0 ? float_key(c[0]) : 0u;  // 0: no candidate (keys are larger)
      const uint32_t kmax = __reduce_max_sync(kAll, key);
      const uint32_t emin = __reduce_min_sync(kAll, key == kmax ? (uint32_t)e[0] : kAll);
      const bool win = left > 0 && (uint32_t)e[0] == emin;
#pragma unroll
      for (int i = 0; i + 1 < PER; ++i) {
        c[i] = win ? c[i + 1] : c[i];
        e[i] = win ? e[i + 1] : e[i];
      }
      left -= win;
      my_key = lane == j ? kmax : my_key;
      my_id = lane == j ? emin : my_id;
      past_key = kmax;
    }
  } else {
    uint32_t open = 0;  // bit i: this lane's candidate i may still be chosen
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      open |= (e < a.E && (a.G == 1 || ((kept >> (e / per)) & 1u))) ? 1u << i : 0u;
    }
    for (int j = 0; j < rounds; ++j) {
      float bv = -INFINITY;
      int bi = -1;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const bool better = ((open >> i) & 1u) & ((c[i] > bv) | (bi < 0));
        bv = better ? c[i] : bv;
        bi = better ? i : bi;
      }
      const uint32_t be = bi >= 0 ? (uint32_t)(lane + 32 * bi) : kAll;
      const uint32_t key = bi >= 0 ? float_key(bv) : 0u;
      const uint32_t kmax = __reduce_max_sync(kAll, key);
      const uint32_t emin = __reduce_min_sync(kAll, key == kmax ? be : kAll);
      open &= (bi >= 0 && be == emin) ? ~(1u << bi) : kAll;
      my_key = lane == j ? kmax : my_key;
      my_id = lane == j ? emin : my_id;
      past_key = kmax;
    }
  }
  if (a.bias != nullptr) {
    // Neighbours of the order within their error, unless score and bias are equal (then
    // the ids decide, as they did).
    uint32_t nk = __shfl_down_sync(kAll, my_key, 1);
    const uint32_t ni = __shfl_down_sync(kAll, my_id, 1);
    if (lane == 31) nk = past_key;  // only asked for k = 32
    bool amb = false;
    if (lane < a.k && nk != 0u) {
      const float x = key_float(my_key), y = key_float(nk);
      amb = x - y <= 2.f * eps + 0x1p-22f * (fabsf(x) + fabsf(y));
      if (amb && lane < 31 && (int)my_id < a.E && (int)ni < a.E)
        amb = load_as_f32(row, a.dtype, my_id) != load_as_f32(row, a.dtype, ni) ||
              __ldg(a.bias + my_id) != __ldg(a.bias + ni);
    }
    close |= __any_sync(kAll, amb);
  }
  if (close) my_id = (uint32_t)route_exact(a, row, buf, lane);

  const bool in = lane < a.k;
  const float t = in ? load_as_f32(row, a.dtype, my_id) : 0.f;
  const float w = slot_weight(a, t, in, mx, inv);
  if (in) {
    a.ids[tok * a.k + lane] = (int32_t)my_id;
    a.w[tok * a.k + lane] = a.scale * w;
  }
}

// Backward. With g_j = scale * dw_j and r_j the weight before `scale`:
//   sigmoid:              dl_j = g_j s_j (1 - s_j)
//   sigmoid, renormalised dl_j = r_j (g_j - sum_i g_i r_i) (1 - s_j)
//   softmax, renormalised dl_j = r_j (g_j - sum_i g_i r_i)
//   softmax               dl_e = p_e ((g_j where e is chosen, else 0) - sum_i g_i p_i)
// zero for the other experts except in the last, the only one that reads every score.
// A warp takes a token and writes its whole row: the row is put together in shared
// memory, so that the stores are coalesced. Bound by the row's bytes.
__global__ void __launch_bounds__(32 * kRouterWarps)
    router_backward_kernel(const __grid_constant__ RouterArgs a) {
  extern __shared__ double smem_d[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tok = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
  if (tok >= a.n) return;
  float* g = reinterpret_cast<float*>(smem_d) + (size_t)warp * a.E;
  const int tb = a.dtype == MOE_FP32 ? 4 : 2;
  const void* row = static_cast<const char*>(a.logits) + (size_t)tok * a.ld * tb;
  void* out = static_cast<char*>(a.dl) + (size_t)tok * a.ld_dl * tb;

  for (int e = lane; e < a.E; e += 32) g[e] = 0.f;
  const int id = lane < a.k ? __ldg(a.ids + tok * a.k + lane) : -1;
  const bool in = id >= 0 && id < a.E;  // others have no gradient
  const float t = in ? load_as_f32(row, a.dtype, id) : 0.f;
  const float gj = in ? a.scale * __ldg(a.dw + tok * a.k + lane) : 0.f;
  const bool all = a.score == MOE_SCORE_SOFTMAX && !a.renorm;
  float mx = 0.f, inv = 1.f;
  if (all) {
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, load_as_f32(row, a.dtype, e));
    mx = warp_max(m);
    float sum = 0.f;
    if (mx != -INFINITY)
      for (int e = lane; e < a.E; e += 32) sum += expf(load_as_f32(row, a.dtype, e) - mx);
    sum = warp_sum(sum);
    inv = 1.0f / sum;
  }
  const float r = slot_weight(a, t, in, mx, inv);
  const float dot = a.renorm || all ? warp_sum(in ? gj * r : 0.f) : 0.f;
  float d = r * (a.renorm ? gj - dot : gj);
  if (a.score == MOE_SCORE_SIGMOID) d *= sigmoid(-t);  // 1 - s
  __syncwarp();
  if (in) g[id] = all ? gj : d;
  __syncwarp();
  for (int e = lane; e < a.E; e += 32) {
    float v = g[e];
    if (all) v = mx == -INFINITY ? 0.f : expf(load_as_f32(row, a.dtype, e) - mx) * inv * (v - dot);
    store_from_f32(out, a.dtype, e, v);
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
  router_kernel<PER><<<(unsigned)((a.n + warps - 1) / warps), 32 * warps,
                       (size_t)warps * a.E * sizeof(double), s>>>(a);
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
  const int warps = router_warps(a.E);
  router_backward_kernel<<<(unsigned)((n + warps - 1) / warps), 32 * warps,
                           (size_t)warps * a.E * sizeof(float), reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
