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
// one token. It selects on 32-bit keys first, and then looks at the gaps that
// decided: between neighbours of the chosen order, to the first expert left
// out, and between the last group kept and the best one dropped. Where a gap is
// within the error bound of the keys, 64-bit scores decide: of the K + 1 best
// alone if these are clear of the others, or of the whole token (select64).
//
// Bound by instructions, not by its 4 T E bytes, so a token should cost few:
//   - a group owns whole lanes (2^log_l of them), a lane NJ consecutive experts
//     of it: a group's value is a few shuffles;
//   - a key is c + max|B| (never negative, so its bits order like integers) with
//     the lane's slot in the lowest bits: one maximum finds value and place;
//   - a lane keeps its two best keys at hand and looks through its NJ again only
//     when it has won twice.
// Measured on B200, 256 experts in 8 groups, K = 8: 21 us for 16384 tokens (838
// instructions a token; 98 us with experts strided over the lanes and an index
// carried with every score), 3.4 us for one token, 4.0 for 64, where one token in
// a hundred or so takes the 64-bit way. Softmax scores: 23, and 25 with a quarter of
// the experts masked.
#include "common.cuh"
#include "kernels_block.cuh"
#include "launch.cuh"

namespace moe {

namespace {

constexpr int kRouteWarps = 8;
constexpr unsigned kFull = 0xffffffffu;

// Bounds on the error of a pair of scores, relative to their sum. Sigmoid: the
// exponent's rounding (|l| 2^-24, for |l| <= 16), ex2.approx (2^-22), rcp.approx
// (2^-23) and three roundings, below 2^-19. Softmax: the rounding of l - max,
// which the exponential multiplies by up to |l - max| < 104, and the sum's,
// below 2^-17. The key's cut (its slot bits) comes on top, and kFloor for sigmoids
// of l < -16, where |l| 2^-24 s stays below 2^-41.
constexpr float kSigmoidRel = 0x1p-18f;
constexpr float kSoftmaxRel = 0x1p-16f;
constexpr float kFloor = 0x1p-39f;

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float sigmoid32(float l) {
  // exp of the negative magnitude: no overflow on either side, and a divisor
  // in [1, 2], where the fast division is good to 2 ulp
  const float z = expf(-fabsf(l));
  return __fdividef(l >= 0.f ? 1.f : z, 1.f + z);
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The sigmoid that selects (bounds above). Past +-87 all logits look alike here,
// which kFloor covers: 64 bits tell them apart.
__device__ __forceinline__ float sigmoid_select(float l) {
  l = fminf(fmaxf(l, -87.f), 87.f);
  return rcp_approx(1.f + exp2_approx(l * -1.44269504088896340736f));
}

// Score of a chosen logit up to a factor common to the chosen ones, `top` being
// the largest of them: the largest exponential is divided out, so that scores
// too small for fp32 keep their ratios.
__device__ __forceinline__ float chosen_score(float l, float top, bool soft) {
  if (soft) return expf(l - top);
  if (top >= -60.f) return sigmoid32(l);
  return expf(l - top) / (1.f + expf(l));
}

// Where a token's experts are: lane g * 2^log_l + i of group g holds the NJ
// experts from g * size + i * NJ on, those of them inside the group.
struct RouteLayout {
  int size, groups, log_l;
};

// The two largest of two pairs (first >= second).
template <typename V>
__device__ __forceinline__ void merge2(V& a1, V& a2, V b1, V b2) {
  a2 = max(min(a1, b1), max(a2, b2));
  a1 = max(a1, b1);
}
template <typename V>
__device__ __forceinline__ void merge_group(V& a1, V& a2, int log_l) {
  for (int o = 1; o < (1 << log_l); o <<= 1) {
    const V b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
    merge2(a1, a2, b1, b2);
  }
}

// Logit of expert e of a token: the partial sums of a split gate product are
// added in split order.
__device__ __forceinline__ float logit_at(const float* row, int e, int n_parts,
                                          size_t part_stride) {
  float l = row[e];
  for (int p = 1; p < n_parts; ++p) l = __fadd_rn(l, row[p * part_stride + e]);
  return l;
}

// The selection on 64-bit scores. Returns the expert of slot `lane`.
template <int NJ>
__device__ __noinline__ int select64(const moe_route_desc& d, const RouteLayout& q,
                                     const float* row, int n_parts, size_t part_stride,
                                     const float* bias) {
  const int lane = threadIdx.x & 31;
  const int first = (lane & ((1 << q.log_l) - 1)) * NJ;   // inside the group
  const int e0 = (lane >> q.log_l) * q.size + first;
  const int n = (lane >> q.log_l) < q.groups ? min(NJ, q.size - first) : 0;
  double c[NJ];
  float mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const float l = j < n ? logit_at(row, e0 + j, n_parts, part_stride) : -INFINITY;
    c[j] = (double)l;
    mx = fmaxf(mx, l);
  }
  // no branches around the exponentials: those of a lane overlap
  double m = 0.0, scale = 1.0;
  const bool soft = d.score == MOE_SCORE_SOFTMAX;
  if (soft) m = (double)warp_max(mx);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool live = c[j] > -INFINITY;
    const double z = exp(soft ? c[j] - m : -c[j]);
    c[j] = !live ? -INFINITY : soft ? z : 1.0 / (1.0 + z);
  }
  if (soft) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) sum += c[j] > -INFINITY ? c[j] : 0.0;
    scale = warp_sum(sum);
  }
  double a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    double x = soft ? c[j] / scale : c[j];
    if (bias && j < n) x += (double)bias[e0 + j];
    c[j] = x == x ? x : -INFINITY;
    merge2(a1, a2, c[j], (double)-INFINITY);
  }
  unsigned left = n >= 32 ? kFull : (1u << max(n, 0)) - 1u;   // slots not taken yet
  if (q.groups > 1) {
    merge_group(a1, a2, q.log_l);
    const double value = d.group_top == 2 ? a1 + a2 : a1;
    const int group = lane >> q.log_l;
    int rank = 0;
    for (int g = 0; g < q.groups; ++g) {
      const double v = __shfl_sync(kFull, value, g << q.log_l);
      rank += (v > value || (v == value && g < group)) ? 1 : 0;
    }
    if (rank >= d.topk_groups) left = 0u;
  }
  // order-preserving 64-bit keys (0: not there); -0.0 ties with 0.0
  unsigned long long key[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const unsigned long long u = __double_as_longlong(c[j] + 0.0);
    key[j] = !((left >> j) & 1u) ? 0ull : (u >> 63) ? ~u : (u | (1ull << 63));
  }
  // K rounds of a warp maximum, high words first; the lowest lane of equals
  // holds the lowest index
  int mine = 0;
  for (int k = 0; k < d.K; ++k) {
    unsigned long long best = 0ull;
    int be = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (key[j] > best) {
        best = key[j];
        be = j;
      }
    const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
    const uint32_t top_hi = __reduce_max_sync(kFull, hi);
    const uint32_t top_lo = __reduce_max_sync(kFull, hi == top_hi ? lo : 0u);
    const int who = __ffs(__ballot_sync(kFull, hi == top_hi && lo == top_lo)) - 1;
    const int e = __shfl_sync(kFull, e0 + be, who);
    if (lane == k) mine = e;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (lane == who && j == be) key[j] = 0ull;
  }
  return mine;
}

// kVec: the lane's experts are NJ / 4 aligned 16-byte vectors.
template <int NJ, bool kVec>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const moe_route_desc d, const RouteLayout q, const float* __restrict__ logits,
                 int n_parts, size_t part_stride, const float* __restrict__ bias,
                 int32_t* __restrict__ idx, float* __restrict__ w,
                 float* __restrict__ logits_out) {
  __shared__ uint2 route_best[kRouteWarps][kMaxK + 2];
  pdl_wait();
  pdl_trigger();
  constexpr int kSlotBits = NJ <= 1 ? 0 : NJ <= 2 ? 1 : NJ <= 4 ? 2 : NJ <= 8 ? 3 : NJ <= 16 ? 4 : 5;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= d.T) return;
  const int E = d.E, K = d.K;
  const float* src = logits + (size_t)t * E;
  const int first = (lane & ((1 << q.log_l) - 1)) * NJ;
  const int e0 = (lane >> q.log_l) * q.size + first;
  const int n = (lane >> q.log_l) < q.groups ? min(NJ, q.size - first) : 0;

  float l[NJ], c[NJ];
  if (kVec) {   // n is NJ or at most 0
#pragma unroll
    for (int j = 0; j < NJ; j += 4) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), b = {};
      if (n > 0) {
        v = *reinterpret_cast<const float4*>(src + e0 + j);
        for (int p = 1; p < n_parts; ++p) {
          const float4 u = *reinterpret_cast<const float4*>(src + p * part_stride + e0 + j);
          v.x = __fadd_rn(v.x, u.x);
          v.y = __fadd_rn(v.y, u.y);
          v.z = __fadd_rn(v.z, u.z);
          v.w = __fadd_rn(v.w, u.w);
        }
        if (logits_out) *reinterpret_cast<float4*>(logits_out + (size_t)t * E + e0 + j) = v;
        if (bias) b = *reinterpret_cast<const float4*>(bias + e0 + j);
      }
      l[j] = v.x; l[j + 1] = v.y; l[j + 2] = v.z; l[j + 3] = v.w;
      c[j] = b.x; c[j + 1] = b.y; c[j + 2] = b.z; c[j + 3] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      l[j] = -INFINITY;
      c[j] = 0.f;
      if (j < n) {
        l[j] = logit_at(src, e0 + j, n_parts, part_stride);
        if (logits_out) logits_out[(size_t)t * E + e0 + j] = l[j];
        if (bias) c[j] = bias[e0 + j];
      }
    }
  }
  const bool soft = d.score == MOE_SCORE_SOFTMAX;
  float b_max = 0.f;
  if (bias) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (fabsf(c[j]) < INFINITY) b_max = fmaxf(b_max, fabsf(c[j]));
    b_max = warp_max(b_max);
  }
  float m = 0.f, den = 1.f;
  if (soft) {
    float mx = l[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) mx = fmaxf(mx, l[j]);
    m = warp_max(mx);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      l[j] = l[j] > -INFINITY ? expf(l[j] - m) : -INFINITY;
      sum += l[j] > -INFINITY ? l[j] : 0.f;
    }
    den = warp_sum(sum);
  }
  const float inv_den = 1.f / den;
  // keys: 0 for no expert, or one of choice -inf. A score that underflows (a finite
  // mask) has the smallest other key: its group is worth its best expert's score, and
  // what that key blurs is far below kFloor, so that 64 bits decide it.
  constexpr uint32_t kSlots = (1u << kSlotBits) - 1u;
  uint32_t key[NJ], k1 = 0u, k2 = 0u;   // k1 >= k2: the lane's best keys left
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const float s = soft ? l[j] * inv_den : sigmoid_select(l[j]);
    const float v = l[j] > -INFINITY ? s + (c[j] + b_max) : -INFINITY;
    const uint32_t bits = max(__float_as_uint(v), kSlots + 1u);
    key[j] = v >= 0.f ? (bits & ~kSlots) | (kSlots - (uint32_t)j) : 0u;
    merge2(k1, k2, key[j], 0u);
  }
  // error bound of the difference of two keys' values, for a sum of magnitudes
  const float rel = (soft ? kSoftmaxRel : kSigmoidRel) + 0x1p-22f * (float)(1u << kSlotBits);
  bool whole = false;   // the whole token on 64-bit scores
  if (q.groups > 1) {
    uint32_t g1 = k1, g2 = k2;
    merge_group(g1, g2, q.log_l);
    const int group = lane >> q.log_l;
    // the group's value, with the group in the lowest five bits
    const float sum = __uint_as_float(g1) + (d.group_top == 2 ? __uint_as_float(g2) : 0.f);
    uint32_t value = 31u - (uint32_t)group;
    if (d.group_top == 2 ? g2 != 0u : g1 != 0u) value |= __float_as_uint(sum) & ~31u;
    // the lanes of a group share the comparisons with the other groups
    int rank = 0;
    const int lanes = 1 << q.log_l, turn = lane & (lanes - 1);
    for (int g = 0; g < q.groups; g += lanes) {
      const int h = min(g + turn, q.groups - 1);
      const uint32_t v = __shfl_sync(kFull, value, h << q.log_l);
      rank += g + turn < q.groups && v > value ? 1 : 0;
    }
    for (int o = 1; o < lanes; o <<= 1) rank += __shfl_xor_sync(kFull, rank, o);
    const bool real = group < q.groups;
    const unsigned last = __ballot_sync(kFull, real && rank == d.topk_groups - 1);
    const unsigned next = __ballot_sync(kFull, real && rank == d.topk_groups);
    const float a = __uint_as_float(__shfl_sync(kFull, value, __ffs(last) - 1) & ~31u);
    const float b = __uint_as_float(__shfl_sync(kFull, value, __ffs(next) - 1) & ~31u);
    // `not above`, here and below: values past fp32's range (a bias near its end) have
    // no difference that compares, and are close
    whole = a == 0.f || !(a - b > fmaf(rel + 0x1p-17f, a + b + 4.f * b_max, kFloor));
    if (rank >= d.topk_groups) k1 = k2 = 0u;
  }
  // rounds of a warp maximum: the K best, the first left out and the one after.
  // Lanes with equal keys win together; the count of wins shows it afterwards.
  uint2* best = route_best[threadIdx.x >> 5];
  if (lane < kMaxK + 2) best[lane] = make_uint2(0u, 0u);
  __syncwarp();
  int wins = 0;
  for (int k = 0; k < K + 2; ++k) {
    const uint32_t top = __reduce_max_sync(kFull, k1);
    if (k1 == top && top != 0u) {
      best[k] = make_uint2(top, (uint32_t)lane);
      ++wins;
      k1 = k2;
      k2 = 0u;
      if (k1 == 0u) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) merge2(k1, k2, key[j] < top ? key[j] : 0u, 0u);
      }
    }
  }
  __syncwarp();
  const uint2 candidate = lane < K + 2 ? best[lane] : make_uint2(0u, 0u);
  const uint32_t got = candidate.x;   // key and lane of candidate `lane`
  const int from = (int)candidate.y;
  wins = __reduce_add_sync(kFull, wins);
  int mine = (from >> q.log_l) * q.size + (from & ((1 << q.log_l) - 1)) * NJ +
             (int)(kSlots - (got & kSlots));
  float lk = got ? logit_at(src, mine, n_parts, part_stride) : -INFINITY;
  {
    const float a = __uint_as_float(got & ~kSlots);
    const uint32_t below = __shfl_down_sync(kFull, got, 1);
    const float b = __uint_as_float(below & ~kSlots);
    const bool close = below != 0u && !(a - b > fmaf(rel, a + b + 2.f * b_max, kFloor));
    // bit k: candidates k and k + 1 are too close to tell
    const unsigned close_to = __ballot_sync(kFull, lane <= K && close);
    const unsigned found = __ballot_sync(kFull, got != 0u);
    const bool decides = (close_to & ((1u << K) - 1u)) != 0u;
    // the K + 1 best, or the K best, are clear of all others
    const bool clear = !((close_to >> (K - 1)) & (close_to >> K) & 1u);
    // a softmax without a bias orders like its logits where different logits have
    // different 64-bit scores: from 2^-20 on they are 2^-43 apart, far more than
    // the exponential and the division round, and down to m - 600 neither underflows
    const bool by_logits = fabsf(lk) >= 0x1p-20f && lk >= m - 600.f;
    whole |= ((found >> (K - 1)) & 1u) == 0u || wins != __popc(found);
    whole |= decides && (!clear || (soft && (bias || (lane <= K && got && !by_logits))));
    whole = __any_sync(kFull, whole);
    if (whole) {
      mine = select64<NJ>(d, q, src, n_parts, part_stride, bias);
      lk = lane < K ? logit_at(src, mine, n_parts, part_stride) : -INFINITY;
    } else if (decides) {
      const int n_c = min(K + 1 - (int)((close_to >> K) & 1u), __popc(found));
      double v = (double)lk;
      if (!soft && lane < n_c)
        v = 1.0 / (1.0 + exp(-v)) + (bias ? (double)bias[mine] : 0.0);
      int rank = 0;
      for (int j = 0; j < n_c; ++j) {
        const double o = __shfl_sync(kFull, v, j);
        const int e = __shfl_sync(kFull, mine, j);
        rank += (o > v || (o == v && e < mine)) ? 1 : 0;
      }
      if (lane >= n_c) rank = lane;
      int to = lane;
      for (int j = 0; j < n_c; ++j)
        if (__shfl_sync(kFull, rank, j) == lane) to = j;
      mine = __shfl_sync(kFull, mine, to);
      lk = __shfl_sync(kFull, lk, to);
    }
  }
  if (lane >= K) lk = -INFINITY;

  // weights of slot `lane`
  float s = 0.f;
  if (d.renorm) {
    const float top = warp_max(lk);   // by the whole warp
    s = lk > -INFINITY ? chosen_score(lk, top, soft) : 0.f;
    const float sum = warp_sum(s);
    s = sum > 0.f ? __fdividef(s, sum) : 0.f;
  } else if (lk > -INFINITY) {
    s = soft ? expf(lk - m) * inv_den : sigmoid32(lk);
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
//
// Bound by its 4 T E bytes of output (and of logits, for a whole softmax row):
// 16383 x 128, softmax, 5.2 us (2.7 at the copy rate), 16384 x 256, sigmoid, 5.9.
// A warp writes a row as if no expert were chosen, in vectors of V floats, and
// then the K chosen entries over it.
template <int V>
struct FloatVec;
template <>
struct FloatVec<1> {
  using T = float;
};
template <>
struct FloatVec<4> {
  using T = float4;
};

// kRow: vectors of a row per lane, rounded up to 1, 2 or 4 (16 of single floats).
template <int V, int kRow>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const moe_route_desc d, const float* __restrict__ logits,
                          const int32_t* __restrict__ idx, const float* __restrict__ d_w,
                          float* __restrict__ d_logits) {
  using Vec = typename FloatVec<V>::T;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= d.T) return;
  const int E = d.E, K = d.K, nvec = E / V;
  const float* row = logits + (size_t)t * E;
  float* out = d_logits + (size_t)t * E;
  const bool soft = d.score == MOE_SCORE_SOFTMAX;
  const bool whole = soft && !d.renorm;
  float x[kRow][V];
  if (whole)
#pragma unroll
    for (int i = 0; i < kRow; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) x[i][j] = -INFINITY;
      if (lane + 32 * i < nvec)
        *reinterpret_cast<Vec*>(x[i]) = reinterpret_cast<const Vec*>(row)[lane + 32 * i];
    }
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
  float base = 0.f, p = 0.f;
  if (whole) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kRow; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) mx = fmaxf(mx, x[i][j]);
    const float m = warp_max(mx);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kRow; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[i][j] = x[i][j] > -INFINITY ? expf(x[i][j] - m) : 0.f;
        sum += x[i][j];
      }
    const float inv = 1.f / warp_sum(sum);
    p = live ? expf(lk - m) * inv : 0.f;
    const float dot = warp_sum(g * p);
    v = g * p;                        // the chosen expert's own part,
    base = -dot;                      // on top of p * base in every entry
#pragma unroll
    for (int i = 0; i < kRow; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) x[i][j] = x[i][j] > 0.f ? x[i][j] * inv * base : 0.f;
  } else if (d.renorm) {
    const float top = warp_max(lk);
    float share = live ? chosen_score(lk, top, soft) : 0.f;
    const float sum = warp_sum(share);
    share = sum > 0.f ? share / sum : 0.f;
    const float mean = warp_sum(g * share);
    if (live) v = share * (g - mean) * (soft ? 1.f : sigmoid32(-lk));
  } else if (live) {
    v = g * sigmoid32(lk) * sigmoid32(-lk);
  }
#pragma unroll
  for (int i = 0; i < kRow; ++i)
    if (lane + 32 * i < nvec) {
      if (!whole)
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][j] = 0.f;
      reinterpret_cast<Vec*>(out)[lane + 32 * i] = *reinterpret_cast<const Vec*>(x[i]);
    }
  // slots of one expert: the lowest adds them up
  const unsigned same = __match_any_sync(kFull, e);
  if (__any_sync(kFull, e >= 0 && (same & (same - 1)) != 0)) {
    float total = 0.f;
    for (int k = 0; k < K; ++k) {
      const float vk = __shfl_sync(kFull, v, k);
      if ((same >> k) & 1u) total += vk;
    }
    v = total;
  }
  __syncwarp();   // the row's stores of other lanes come first
  if (e >= 0 && lane == __ffs(same) - 1) out[e] = live ? fmaf(p, base, v) : 0.f;
}

}  // namespace

cudaError_t launch_route(const moe_route_desc& d, const float* logits, int n_parts,
                         size_t part_stride, const float* bias, int32_t* idx, float* w,
                         float* logits_out, cudaStream_t st) {
  if (d.T == 0) return cudaSuccess;
  // groups that are all kept do not decide anything
  RouteLayout q;
  q.groups = d.topk_groups < d.groups ? d.groups : 1;
  q.size = d.E / q.groups;
  q.log_l = 5;
  while ((q.groups << q.log_l) > 32) --q.log_l;
  const int nj = (q.size + (1 << q.log_l) - 1) >> q.log_l;
  const dim3 grid((d.T + kRouteWarps - 1) / kRouteWarps);
#define MOE_ROUTE_CASE(NJ)                                                                     \
  if (nj <= NJ) {                                                                              \
    /* vectors: every lane full or empty, and every address a multiple of 16 bytes */          \
    if (NJ % 4 == 0 && q.size % NJ == 0 && part_stride % 4 == 0)                               \
      return launch_pdl(route_kernel<NJ, NJ % 4 == 0>, grid, dim3(kRouteWarps * 32), 0, st, d, \
                        q, logits, n_parts, part_stride, bias, idx, w, logits_out);            \
    return launch_pdl(route_kernel<NJ, false>, grid, dim3(kRouteWarps * 32), 0, st, d, q,      \
                      logits, n_parts, part_stride, bias, idx, w, logits_out);                 \
  }
  MOE_ROUTE_CASE(1) MOE_ROUTE_CASE(2) MOE_ROUTE_CASE(3) MOE_ROUTE_CASE(4) MOE_ROUTE_CASE(6)
  MOE_ROUTE_CASE(8) MOE_ROUTE_CASE(12) MOE_ROUTE_CASE(16) MOE_ROUTE_CASE(32)
#undef MOE_ROUTE_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_backward(const moe_route_desc& d, const float* logits,
                                  const int32_t* idx, const float* d_w, float* d_logits,
                                  cudaStream_t st) {
  if (d.T == 0) return cudaSuccess;
  const dim3 grid((d.T + kRouteWarps - 1) / kRouteWarps);
  auto k = d.E % 4      ? route_backward_kernel<1, kMaxE / 32>
           : d.E <= 128 ? route_backward_kernel<4, 1>
           : d.E <= 256 ? route_backward_kernel<4, 2>
                        : route_backward_kernel<4, 4>;
  return launch_pdl(k, grid, dim3(kRouteWarps * 32), 0, st, d, logits, idx, d_w, d_logits);
}

}  // namespace moe
