// The linear layer for a few tokens (a decode step): y = act(x W^T + b) + r on
// CUDA cores. "MoE architecture in production" §3.1 (Linear).
//
// Bound by reading W once. Tensor-core tiles would spend their time on rows that
// are not there and on starting up. Here a warp reads 16-byte pieces of kRows
// rows of W straight into registers and multiplies them with the same pieces of
// x (fp32 sums, in a fixed order, two elements to an instruction); the warps of a
// block split the reduction, so that a thousand rows keep every SM's memory pipes
// full. Measured on B200, bf16, 4096 x 4096, weights in L2: 5.1 us for one token, 6.5
// for two, 9.5 for four and 14.9 for eight; on the tensor cores 12.8 for any of them.
// 14336 rows of 4096 from memory: 22.5 us for one token, 5.2 TB/s.
#include "common.cuh"
#include "kernels_block.cuh"
#include "launch.cuh"
#include "linear_epilogue.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

constexpr int kRows = 4;       // rows of W per warp
// Pieces of a row on their way at a time, and blocks per SM that the registers are
// cut for, by the tokens: left to the compiler (four pieces, two to four blocks), two
// tokens took 7.1 us instead of 6.7 and eight (1024 x 1024) 4.0 instead of 3.0; more
// blocks spill.
constexpr int pieces(int kT) { return kT == 1 || kT == 4 ? 2 : 1; }
constexpr int blocks_per_sm(int kT) { return kT <= 2 ? 4 : 2; }
constexpr int kFewWarps = 8;

// Sums over the lanes of N values (a power of two up to 32) at a time: each exchange
// halves the values a lane carries on, so that lane l ends with value l / (32 / N).
template <int N, int kOff = 16>
__device__ __forceinline__ float sums_over_lanes(const float (&v)[N], int lane) {
  if constexpr (kOff == 0) {
    return v[0];
  } else if constexpr (N == 1) {
    const float w[1] = {v[0] + __shfl_xor_sync(0xffffffffu, v[0], kOff)};
    return sums_over_lanes<1, kOff / 2>(w, lane);
  } else {
    const bool hi = lane & kOff;
    float w[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float give = hi ? v[j] : v[j + N / 2], keep = hi ? v[j + N / 2] : v[j];
      w[j] = keep + __shfl_xor_sync(0xffffffffu, give, kOff);
    }
    return sums_over_lanes<N / 2, kOff / 2>(w, lane);
  }
}

// kT: tokens, rounded up to 1, 2, 4 or 8. warps_k: warps that split a row's
// reduction (1, 2, 4 or 8); the block's other warps take other rows.
template <typename T, int kT, int kAct>
__global__ void __launch_bounds__(kFewWarps * 32, blocks_per_sm(kT))
    linear_few_kernel(const moe_linear_desc d, int warps_k, const T* __restrict__ x,
                      const T* __restrict__ w, const LinearEpilogue epi) {
  using V = RowVec<T>;
  __shared__ float part[kFewWarps][kRows * kT];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nvec = d.in / V::N;
  const int slice = warp % warps_k;
  const int row0 = (blockIdx.x * (kFewWarps / warps_k) + warp / warps_k) * kRows;
  constexpr int P = V::N / 2, kSums = kRows * kT;
  Pair acc[kSums];
#pragma unroll
  for (int i = 0; i < kSums; ++i) acc[i] = pair_of(0.f);
  const uint4* wv = reinterpret_cast<const uint4*>(w);
  const uint4* xv = reinterpret_cast<const uint4*>(x);
  constexpr int kUnroll = pieces(kT);
#pragma unroll kUnroll
  for (int c = slice * 32 + lane; c < nvec; c += 32 * warps_k) {
    uint4 wr[kRows], xr[kT];
#pragma unroll
    for (int r = 0; r < kRows; ++r)   // rows past the last one repeat it: not stored
      wr[r] = __ldg(wv + (size_t)min(row0 + r, d.out - 1) * nvec + c);
#pragma unroll
    for (int t = 0; t < kT; ++t)
      xr[t] = t < d.T ? __ldg(xv + (size_t)t * nvec + c) : make_uint4(0, 0, 0, 0);
    Pair f[kRows][P];
#pragma unroll
    for (int r = 0; r < kRows; ++r) unpack_pairs<T>(wr[r], f[r]);
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      Pair g[P];
      unpack_pairs<T>(xr[t], g);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < P; ++i) acc[t * kRows + r] = fma2(f[r][i], g[i], acc[t * kRows + r]);
    }
  }
  float sum[kSums];
#pragma unroll
  for (int i = 0; i < kSums; ++i) sum[i] = sum_of(acc[i]);
  const float mine = sums_over_lanes(sum, lane);
  if (lane % (32 / kSums) == 0) part[warp][lane / (32 / kSums)] = mine;
  __syncthreads();
  // one output per thread: neighbours hold neighbouring columns of a token
  const int group = threadIdx.x / (kRows * kT), i = threadIdx.x % (kRows * kT);
  if (group >= kFewWarps / warps_k) return;
  const int t = i / kRows;
  const int col = (blockIdx.x * (kFewWarps / warps_k) + group) * kRows + i % kRows;
  if (t >= d.T || col >= d.out) return;
  float z = 0.f;
  for (int s = 0; s < warps_k; ++s) z += part[group * warps_k + s][i];
  const size_t o = (size_t)t * d.out + col;
  if (epi.bias) z += to_f32(static_cast<const T*>(epi.bias)[col]);
  if (epi.pre) static_cast<T*>(epi.pre)[o] = from_f32<T>(z);
  z = linear_act2<T, kAct>(make_float2(z, 0.f)).x;
  if (epi.residual) z += to_f32(static_cast<const T*>(epi.residual)[o]);
  static_cast<T*>(epi.out)[o] = from_f32<T>(z);
}

template <typename T, int kT>
cudaError_t few(const moe_linear_desc& d, const void* x, const void* w, const LinearEpilogue& epi,
                cudaStream_t st) {
  const int nvec = d.in / RowVec<T>::N;
  // eight pieces per lane and row at least, fewer where there would
  // not be 16 warps per SM
  int warps_k = 1;
  const int row_groups = (d.out + kRows - 1) / kRows;
  while (warps_k < kFewWarps && nvec >= 64 * warps_k &&
         (nvec >= 512 * warps_k || row_groups * warps_k < 16 * kPlanSms))
    warps_k *= 2;
  const int per_block = kRows * (kFewWarps / warps_k);
  auto k = d.act == MOE_ACT_GELU   ? linear_few_kernel<T, kT, MOE_ACT_GELU>
           : d.act == MOE_ACT_SILU ? linear_few_kernel<T, kT, MOE_ACT_SILU>
                                   : linear_few_kernel<T, kT, MOE_ACT_NONE>;
  return launch_pdl(k, dim3((d.out + per_block - 1) / per_block), dim3(kFewWarps * 32), 0, st, d,
                    warps_k, static_cast<const T*>(x), static_cast<const T*>(w), epi);
}

template <typename T>
cudaError_t few_tokens(const moe_linear_desc& d, const void* x, const void* w,
                       const LinearEpilogue& epi, cudaStream_t st) {
  if (d.T <= 1) return few<T, 1>(d, x, w, epi, st);
  if (d.T <= 2) return few<T, 2>(d, x, w, epi, st);
  return d.T <= 4 ? few<T, 4>(d, x, w, epi, st) : few<T, 8>(d, x, w, epi, st);
}

}  // namespace

bool linear_few_tokens(const moe_linear_desc& d) {
  if (d.dtype == MOE_F32) return d.T <= 8;   // no tensor-core form
  if (d.T <= 2) return true;
  // The arithmetic grows with the tokens, the tensor cores' time hardly does. us here
  // and there: four tokens, 4096 x 8192 15.9 and 14.6 (19.9 and 19.5 with weights from
  // memory), 4096 x 14336 34.6 and 27.4; eight, 2048 x 2048 6.5 and 9.3, 4096 to 2048 9.3
  // and 10.6, 4096 x 4096 14.9 and 12.8. Wide outputs fill the tensor cores' units
  // without a split of the reduction: eight tokens, 1024 to 8192, 9.6 and 7.8.
  const long long weights = (long long)d.in * d.out;
  if (d.T <= 4) return weights <= (1LL << 25);
  return d.T <= 8 && weights <= (d.out <= 4096 ? 1LL << 23 : 1LL << 21);
}

cudaError_t launch_linear_few(const moe_linear_desc& d, const void* x, const void* w,
                              const LinearEpilogue& epi, cudaStream_t st) {
  return d.dtype == MOE_BF16 ? few_tokens<__nv_bfloat16>(d, x, w, epi, st)
                             : few_tokens<float>(d, x, w, epi, st);
}

}  // namespace moe
