// The linear layer for a few tokens (a decode step): y = act(x W^T + b) + r on
// CUDA cores. "MoE architecture in production" §3.1 (Linear).
//
// Bound by reading W once. Tensor-core tiles would spend their time on rows that
// are not there and on starting up. Here a warp reads 16-byte pieces of kRows
// rows of W straight into registers and multiplies them with the same pieces of
// x (fp32 sums, in a fixed order); the warps of a block split the reduction, so
// that a thousand rows keep every SM's memory pipes full. The arithmetic grows
// with the tokens: bf16, 4096 x 4096, took 9.7 us for one token, 10.8 for two and
// 17.1 for four, on the tensor cores 15 for any of them, so that bf16 comes here
// with up to two tokens. fp32 has no tensor-core form and comes with up to eight.
#include "common.cuh"
#include "kernels_block.cuh"
#include "launch.cuh"
#include "linear_epilogue.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

constexpr int kRows = 4;       // rows of W per warp
constexpr int kFewWarps = 8;

// kT: tokens, rounded up to 1, 2, 4 or 8. warps_k: warps that split a row's
// reduction (1, 2, 4 or 8); the block's other warps take other rows.
template <typename T, int kT, int kAct>
__global__ void __launch_bounds__(kFewWarps * 32)
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
  float acc[kRows][kT];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int t = 0; t < kT; ++t) acc[r][t] = 0.f;
  const uint4* wv = reinterpret_cast<const uint4*>(w);
  const uint4* xv = reinterpret_cast<const uint4*>(x);
#pragma unroll 4
  for (int c = slice * 32 + lane; c < nvec; c += 32 * warps_k) {
    uint4 wr[kRows], xr[kT];
#pragma unroll
    for (int r = 0; r < kRows; ++r)   // rows past the last one repeat it: not stored
      wr[r] = __ldg(wv + (size_t)min(row0 + r, d.out - 1) * nvec + c);
#pragma unroll
    for (int t = 0; t < kT; ++t)
      xr[t] = t < d.T ? __ldg(xv + (size_t)t * nvec + c) : make_uint4(0, 0, 0, 0);
    float f[kRows][V::N];
#pragma unroll
    for (int r = 0; r < kRows; ++r) V::unpack(wr[r], f[r]);
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float g[V::N];
      V::unpack(xr[t], g);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < V::N; ++i) acc[r][t] = fmaf(f[r][i], g[i], acc[r][t]);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float v = acc[r][t];
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) part[warp][t * kRows + r] = v;
    }
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
  // eight pieces per lane and row (their loads overlap), fewer where there would
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
  if (d.dtype == MOE_F32) return d.T <= 8;
  const long long weights = (long long)d.in * d.out;
  return d.T <= (weights <= (1LL << 21) ? 8 : weights <= (1LL << 25) ? 4 : 2);
}

cudaError_t launch_linear_few(const moe_linear_desc& d, const void* x, const void* w,
                              const LinearEpilogue& epi, cudaStream_t st) {
  return d.dtype == MOE_BF16 ? few_tokens<__nv_bfloat16>(d, x, w, epi, st)
                             : few_tokens<float>(d, x, w, epi, st);
}

}  // namespace moe
