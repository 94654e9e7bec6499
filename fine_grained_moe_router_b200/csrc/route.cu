// Routing with a choice-only balance bias and expert groups, and its gradient.
//
// Per token, from fp32 logits l [E]:
//   s_e = softmax(l)_e  or  sigmoid(l)_e
//   c_e = s_e + B_e, -inf where l_e = -inf         (decides, carries no weight)
//   group value = sum of the group's group_top largest c; the topk_groups
//   best groups stay, and the K largest c of their experts are chosen, in the
//   order (c descending, index ascending)
//   w_k = scale * s_k  or  scale * s_k / sum_j s_j.
// "Kimi K3 专家路由不均衡诊断" §四 balances the load by a bias on the score
// (here it stays out of the weights); "MoE architecture in production" §2.3
// is the gating network.
//
// The choice is exact: it equals the choice on 64-bit scores. One warp takes
// one token. It selects on fp32 scores first and looks at the gaps that decided
// (between neighbours of the chosen order, the first expert left out, and the
// last group kept against the best one dropped). A gap within the error bound
// of the fp32 scores sends the whole token through the same selection on
// 64-bit scores.
#include "common.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "select.cuh"

namespace moe {

namespace {

constexpr int kRouteWarps = 8;
constexpr unsigned kFull = 0xffffffffu;

// Relative error bounds of one fp32 score, with a factor of two to spare:
// sigmoid is expf (2 ulp), an add and a division; softmax adds the rounding
// of l - max, which the exponential multiplies by up to |l - max| < 104.
constexpr float kSigmoidRel = 1.f / (1 << 20);
constexpr float kSoftmaxRel = 1.f / (1 << 16);

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float sigmoid32(float l) {
  // exp of the negative magnitude: no overflow on either side
  const float z = expf(-fabsf(l));
  return (l >= 0.f ? 1.f : z) / (1.f + z);
}

// Groups kept, as a bit mask over groups (lane g works on group g). `value`:
// group g's value in lane g. *near: the last kept and the first dropped value
// are within rel * (their magnitudes + 4 b_max) of each other.
template <typename V>
__device__ __forceinline__ unsigned keep_groups(V value, int groups, int kept, V rel, V b_max,
                                                bool* near) {
  const int lane = threadIdx.x & 31;
  int rank = 0;
  for (int g = 0; g < groups; ++g) {
    const V v = __shfl_sync(kFull, value, g);
    rank += (v > value || (v == value && g < lane)) ? 1 : 0;
  }
  const unsigned mask = __ballot_sync(kFull, lane < groups && rank < kept);
  const unsigned last = __ballot_sync(kFull, lane < groups && rank == kept - 1);
  const unsigned next = __ballot_sync(kFull, lane < groups && rank == kept);
  if (near && next && last) {
    const V a = __shfl_sync(kFull, value, __ffs(last) - 1);
    const V b = __shfl_sync(kFull, value, __ffs(next) - 1);
    *near |= b > (V)-INFINITY && a - b <= rel * (fabs(a) + fabs(b) + 4 * b_max);
  }
  return mask;
}

// Sum of the `top` (1 or 2) largest of c[0..n).
template <typename V>
__device__ __forceinline__ V group_value(const V* c, int n, int top) {
  V a = (V)-INFINITY, b = (V)-INFINITY;
  for (int i = 0; i < n; ++i) {
    const V v = c[i];
    if (v > a) {
      b = a;
      a = v;
    } else if (v > b) {
      b = v;
    }
  }
  return top == 2 ? a + b : a;
}

// The selection on 64-bit scores, from the token's logits in shared memory.
// c: E doubles of scratch of this warp. Returns the expert of slot `lane`.
__device__ __noinline__ int select64(const moe_route_desc& d, const float* l, const float* bias,
                                     double* c) {
  const int lane = threadIdx.x & 31, E = d.E;
  double m = 0.0, den = 1.0;
  if (d.score == MOE_SCORE_SOFTMAX) {
    float mx = -INFINITY;
    for (int e = lane; e < E; e += 32) mx = fmaxf(mx, l[e]);
    m = (double)warp_max(mx);
    double sum = 0.0;
    for (int e = lane; e < E; e += 32)
      if (l[e] > -INFINITY) sum += exp((double)l[e] - m);
    den = warp_sum(sum);
  }
  for (int e = lane; e < E; e += 32) {
    const double v = (double)l[e];
    double x = -INFINITY;
    if (l[e] > -INFINITY) {
      const double s = d.score == MOE_SCORE_SOFTMAX ? exp(v - m) / den : 1.0 / (1.0 + exp(-v));
      x = s + (bias ? (double)bias[e] : 0.0);
    }
    c[e] = x == x ? x : -INFINITY;
  }
  __syncwarp();
  if (d.topk_groups < d.groups) {
    const int size = E / d.groups;
    const double value =
        lane < d.groups ? group_value(c + lane * size, size, d.group_top) : -INFINITY;
    const unsigned mask = keep_groups<double>(value, d.groups, d.topk_groups, 0, 0, nullptr);
    for (int e = lane; e < E; e += 32)
      if (!((mask >> (e / size)) & 1u)) c[e] = NAN;   // NaN: never the largest below
    __syncwarp();
  }
  int mine = 0;
  for (int k = 0; k < d.K; ++k) {
    double bv = -INFINITY;
    int be = INT_MAX;
    for (int e = lane; e < E; e += 32)
      if (c[e] > bv || (c[e] == bv && be == INT_MAX)) {
        bv = c[e];
        be = e;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double ov = __shfl_xor_sync(kFull, bv, o);
      const int oe = __shfl_xor_sync(kFull, be, o);
      if (oe != INT_MAX && (be == INT_MAX || ov > bv || (ov == bv && oe < be))) {
        bv = ov;
        be = oe;
      }
    }
    if (lane == k) mine = be;
    if ((be & 31) == lane) c[be] = NAN;
    __syncwarp();
  }
  return mine;
}

// NJ: experts per lane (expert e = lane + 32 j).
template <int NJ>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const moe_route_desc d, const float* __restrict__ logits, int n_parts,
                 size_t part_stride, const float* __restrict__ bias, int32_t* __restrict__ idx,
                 float* __restrict__ w, float* __restrict__ logits_out) {
  extern __shared__ __align__(16) uint8_t route_smem[];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= d.T) return;
  const int E = d.E, K = d.K;
  double* c64 = reinterpret_cast<double*>(route_smem) + (size_t)warp * E;
  float* l_row = reinterpret_cast<float*>(route_smem + (size_t)kRouteWarps * E * sizeof(double)) +
                 (size_t)warp * E;
  const float* src = logits + (size_t)t * E;

  float l[NJ], c[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < E ? src[e] : -INFINITY;
  }
  for (int p = 1; p < n_parts; ++p)   // partial sums of a split gate product, in split order
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + 32 * j;
      if (e < E) l[j] = __fadd_rn(l[j], src[p * part_stride + e]);
    }
  float b_max = 0.f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 32 * j;
    c[j] = 0.f;
    if (e < E) {
      l_row[e] = l[j];
      if (logits_out) logits_out[(size_t)t * E + e] = l[j];
      if (bias) {
        c[j] = bias[e];
        if (isfinite(c[j])) b_max = fmaxf(b_max, fabsf(c[j]));
      }
    }
  }
  const bool soft = d.score == MOE_SCORE_SOFTMAX;
  float m = 0.f, den = 1.f;
  if (soft) {
    float mx = l[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) mx = fmaxf(mx, l[j]);
    m = warp_max(mx);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) sum += l[j] > -INFINITY ? expf(l[j] - m) : 0.f;
    den = warp_sum(sum);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const float s = soft ? expf(l[j] - m) / den : sigmoid32(l[j]);
    c[j] = l[j] > -INFINITY ? s + c[j] : -INFINITY;
    if (!(c[j] == c[j])) c[j] = -INFINITY;
  }
  if (bias) b_max = warp_max(b_max);
  const float rel = soft ? kSoftmaxRel : kSigmoidRel;
  bool near = false;
  uint32_t key[NJ];
  unsigned mask = kFull;
  const int size = E / d.groups;
  if (d.topk_groups < d.groups) {
    float* c32 = reinterpret_cast<float*>(c64);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (lane + 32 * j < E) c32[lane + 32 * j] = c[j];
    __syncwarp();
    const float value =
        lane < d.groups ? group_value(c32 + lane * size, size, d.group_top) : -INFINITY;
    mask = keep_groups<float>(value, d.groups, d.topk_groups, rel, b_max, &near);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 32 * j;
    key[j] = (e < E && ((mask >> (e / size)) & 1u)) ? score_key(c[j]) : 0u;
  }
  // K rounds of a warp arg-max, and one more for the best expert left out
  int mine = 0;
  float prev = INFINITY;
  for (int k = 0; k <= K; ++k) {
    uint32_t bk = 0u;
    int be = INT_MAX;
    float bs = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (key[j] > bk) {
        bk = key[j];
        be = lane + 32 * j;
        bs = c[j];
      }
    const uint32_t top = __reduce_max_sync(kFull, bk);
    if (top == 0u) break;
    const int e = __reduce_min_sync(kFull, bk == top ? be : INT_MAX);
    const float v = __shfl_sync(kFull, bs, e & 31);
    near |= v > -INFINITY && prev - v <= rel * (fabsf(prev) + fabsf(v) + 2.f * b_max);
    prev = v;
    if (lane == k) mine = e;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (e == lane + 32 * j) key[j] = 0u;
  }
  __syncwarp();
  if (near) mine = select64(d, l_row, bias, c64);   // the same in every lane

  // weights of slot `lane`
  float s = 0.f;
  const float lk = lane < K ? l_row[mine] : -INFINITY;
  if (d.renorm) {
    // the largest chosen exponential is divided out of numerator and
    // denominator, so scores too small for fp32 keep their ratios
    float top = warp_max(lk);
    if (!soft) top = fminf(top, 0.f);
    if (lk > -INFINITY) {
      if (soft)
        s = expf(lk - top);
      else
        s = lk >= 0.f ? 1.f / (1.f + expf(-lk)) : expf(lk - top) / (1.f + expf(lk));
    }
    float sum = 0.f;
    for (int j = 0; j < K; ++j) sum += __shfl_sync(kFull, s, j);
    s = sum > 0.f ? s / sum : 0.f;
  } else if (lk > -INFINITY) {
    s = soft ? expf(lk - m) / den : sigmoid32(lk);
  }
  if (lane < K) {
    idx[(size_t)t * K + lane] = mine;
    w[(size_t)t * K + lane] = s * d.scale;
  }
}

// Gradient of the weights with respect to the logits, the choice held fixed:
//   renormalised:  dl_k = scale r_k p_k (g_k - sum_j g_j p_j), p_k = s_k / sum,
//                  r_k = 1 (softmax) or 1 - s_k (sigmoid); other entries 0
//   sigmoid:       dl_k = scale g_k s_k (1 - s_k);           other entries 0
//   softmax:       dl_e = s_e (q_e - sum_j q_j s_j), q = scale g at the chosen
// 1 - s is computed as the sigmoid of -l. An index outside [0, E) takes no
// part; an expert named twice receives both contributions, in slot order.
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const moe_route_desc d, const float* __restrict__ logits,
                          const int32_t* __restrict__ idx, const float* __restrict__ d_w,
                          float* __restrict__ d_logits) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= d.T) return;
  const int E = d.E, K = d.K;
  const float* row = logits + (size_t)t * E;
  const bool soft = d.score == MOE_SCORE_SOFTMAX;
  int e = -1;
  float g = 0.f, lk = -INFINITY;
  if (lane < K) {
    e = idx[(size_t)t * K + lane];
    if ((unsigned)e < (unsigned)E) {
      g = d_w[(size_t)t * K + lane] * d.scale;
      lk = row[e];
    } else {
      e = -1;
    }
  }
  const bool live = lk > -INFINITY;
  float v = 0.f;   // contribution of slot `lane` to its expert
  float m = 0.f, den = 1.f, dot = 0.f;
  const bool whole = soft && !d.renorm;
  if (d.renorm) {
    float top = warp_max(lk), p = 0.f;
    if (!soft) top = fminf(top, 0.f);
    if (live) {
      if (soft)
        p = expf(lk - top);
      else
        p = lk >= 0.f ? 1.f / (1.f + expf(-lk)) : expf(lk - top) / (1.f + expf(lk));
    }
    const float sum = warp_sum(p);
    p = sum > 0.f ? p / sum : 0.f;
    const float mean = warp_sum(g * p);
    v = p * (g - mean) * (soft ? 1.f : sigmoid32(-lk));
    if (!live) v = 0.f;
  } else if (!soft) {
    v = live ? g * sigmoid32(lk) * sigmoid32(-lk) : 0.f;
  } else {
    float mx = -INFINITY;
    for (int i = lane; i < E; i += 32) mx = fmaxf(mx, row[i]);
    m = warp_max(mx);
    float sum = 0.f;
    for (int i = lane; i < E; i += 32) sum += row[i] > -INFINITY ? expf(row[i] - m) : 0.f;
    den = warp_sum(sum);
    dot = warp_sum(live ? g * (expf(lk - m) / den) : 0.f);
    v = g;
  }
  for (int i = lane; i < (E + 31) / 32 * 32; i += 32) {
    float q = 0.f;
    for (int k = 0; k < K; ++k) {
      const int ek = __shfl_sync(kFull, e, k);
      const float vk = __shfl_sync(kFull, v, k);
      if (ek == i) q += vk;
    }
    if (i < E) {
      if (whole) {
        const float x = row[i];
        q = x > -INFINITY ? expf(x - m) / den * (q - dot) : 0.f;
      }
      d_logits[(size_t)t * E + i] = q;
    }
  }
}

}  // namespace

cudaError_t launch_route(const moe_route_desc& d, const float* logits, int n_parts,
                         size_t part_stride, const float* bias, int32_t* idx, float* w,
                         float* logits_out, cudaStream_t st) {
  if (d.T == 0) return cudaSuccess;
  const dim3 grid((d.T + kRouteWarps - 1) / kRouteWarps);
  const size_t smem = (size_t)kRouteWarps * d.E * (sizeof(double) + sizeof(float));
#define MOE_ROUTE_CASE(NJ)                                                                     \
  if (d.E <= 32 * NJ)                                                                          \
    return launch_pdl(route_kernel<NJ>, grid, dim3(kRouteWarps * 32), smem, st, d, logits,     \
                      n_parts, part_stride, bias, idx, w, logits_out);
  MOE_ROUTE_CASE(1) MOE_ROUTE_CASE(2) MOE_ROUTE_CASE(4) MOE_ROUTE_CASE(8) MOE_ROUTE_CASE(16)
#undef MOE_ROUTE_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_backward(const moe_route_desc& d, const float* logits,
                                  const int32_t* idx, const float* d_w, float* d_logits,
                                  cudaStream_t st) {
  if (d.T == 0) return cudaSuccess;
  return launch_pdl(route_backward_kernel, dim3((d.T + kRouteWarps - 1) / kRouteWarps),
                    dim3(kRouteWarps * 32), 0, st, d, logits, idx, d_w, d_logits);
}

}  // namespace moe
