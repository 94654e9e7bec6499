// The linear layer's CUDA-core parts: the fp32 products, and the activation's
// gradient with the bias gradient's column sums.
#include "common.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "linear_epilogue.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

// fp32 layers: true FFMA products (no tensor-core type keeps 24 bits). 64 x 64
// tiles of C, 16 reduction elements per step, 4 x 4 outputs per thread. The
// sums of kRun elements are added up apart: rounding errors then grow with
// sqrt(kRun) + sqrt(K / kRun) and not with sqrt(K).
constexpr int kSB = 64, kSK = 16, kRun = 128;

// Element (row, k) of an operand stored [rows, K], or [K, rows] when kMn.
template <bool kMn>
__device__ __forceinline__ void load_tile(float (*dst)[kSB + 4], const float* p, int r0, int k0,
                                          int rows, int K) {
#pragma unroll
  for (int i = threadIdx.x; i < kSB * kSK; i += 256) {
    // neighbouring threads walk the dimension that is contiguous in memory
    const int r = kMn ? i % kSB : i / kSK, k = kMn ? i / kSB : i % kSK;
    const bool in = r0 + r < rows && k0 + k < K;
    dst[k][r] = !in ? 0.f
                    : kMn ? p[(size_t)(k0 + k) * rows + r0 + r] : p[(size_t)(r0 + r) * K + k0 + k];
  }
}

template <bool kAMn, bool kBMn, int kAct>
__global__ void __launch_bounds__(256)
    linear_simt_kernel(int M, int N, int K, const float* __restrict__ A,
                       const float* __restrict__ B, const LinearEpilogue epi) {
  __shared__ __align__(16) float sa[kSK][kSB + 4], sb[kSK][kSB + 4];
  pdl_wait();
  pdl_trigger();
  const int m0 = blockIdx.y * kSB, n0 = blockIdx.x * kSB;
  const int tr = threadIdx.x / 16 * 4, tc = threadIdx.x % 16 * 4;
  float total[4][4] = {}, c[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += kSK) {
    if (k0 % kRun == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          total[i][j] += c[i][j];
          c[i][j] = 0.f;
        }
    load_tile<kAMn>(sa, A, m0, k0, M, K);
    load_tile<kBMn>(sb, B, n0, k0, N, K);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSK; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(&sa[k][tr]);
      const float4 b = *reinterpret_cast<const float4*>(&sb[k][tc]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = fmaf(av[i], bv[j], c[i][j]);
    }
    __syncthreads();
  }
  const int col = n0 + tc;
  if (col >= N) return;   // N is a multiple of 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] += total[i][j];
    if (m0 + tr + i < M)
      linear_finish<float, kAct>(epi, (size_t)(m0 + tr + i) * N + col, col, c[i]);
  }
}

// One block: kGradRows rows by 32 vectors of columns; thread = one vector of
// columns, every eighth row.
template <typename T, int kAct>
__global__ void __launch_bounds__(256)
    linear_act_grad_kernel(int rows, int cols, const T* __restrict__ dy,
                           const T* __restrict__ pre, T* __restrict__ dz,
                           float* __restrict__ parts) {
  using V = RowVec<T>;
  __shared__ float buf[8][32 * V::N];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int nvec = cols / V::N, i = blockIdx.x * 32 + lane;
  const int r1 = min(rows, (int)(blockIdx.y + 1) * kGradRows);
  float s[V::N];
#pragma unroll
  for (int k = 0; k < V::N; ++k) s[k] = 0.f;
  if (i < nvec)
    for (int r = blockIdx.y * kGradRows + slice; r < r1; r += 8) {
      const size_t o = (size_t)r * nvec + i;
      float g[V::N], z[V::N];
      V::unpack(reinterpret_cast<const uint4*>(dy)[o], g);
      if (kAct != MOE_ACT_NONE) {
        V::unpack(reinterpret_cast<const uint4*>(pre)[o], z);
#pragma unroll
        for (int k = 0; k < V::N; ++k) g[k] *= linear_act_grad<T, kAct>(z[k]);
        reinterpret_cast<uint4*>(dz)[o] = V::pack(g);
      }
#pragma unroll
      for (int k = 0; k < V::N; ++k) s[k] += g[k];
    }
  if (!parts) return;
#pragma unroll
  for (int k = 0; k < V::N; ++k) buf[slice][lane * V::N + k] = s[k];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * V::N; c += 256) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += buf[q][c];
    const int col = blockIdx.x * 32 * V::N + c;
    if (col < cols) parts[(size_t)blockIdx.y * cols + col] = t;
  }
}

template <typename T>
cudaError_t act_grad(const moe_linear_desc& d, const void* dy, const void* pre, void* dz,
                     float* parts, cudaStream_t st) {
  const int nvec = d.out / RowVec<T>::N;
  const dim3 grid((nvec + 31) / 32, (d.T + kGradRows - 1) / kGradRows);
  auto k = d.act == MOE_ACT_GELU   ? linear_act_grad_kernel<T, MOE_ACT_GELU>
           : d.act == MOE_ACT_SILU ? linear_act_grad_kernel<T, MOE_ACT_SILU>
                                   : linear_act_grad_kernel<T, MOE_ACT_NONE>;
  return launch_pdl(k, grid, dim3(256), 0, st, d.T, d.out, (const T*)dy, (const T*)pre, (T*)dz,
                    parts);
}

template <bool kAMn, bool kBMn>
cudaError_t simt(int M, int N, int K, const float* A, const float* B, const LinearEpilogue& epi,
                 cudaStream_t st) {
  const dim3 grid((N + kSB - 1) / kSB, (M + kSB - 1) / kSB);
  auto k = epi.act == MOE_ACT_GELU   ? linear_simt_kernel<kAMn, kBMn, MOE_ACT_GELU>
           : epi.act == MOE_ACT_SILU ? linear_simt_kernel<kAMn, kBMn, MOE_ACT_SILU>
                                     : linear_simt_kernel<kAMn, kBMn, MOE_ACT_NONE>;
  return launch_pdl(k, grid, dim3(256), 0, st, M, N, K, A, B, epi);
}

}  // namespace

cudaError_t launch_linear_act_grad(const moe_linear_desc& d, const void* dy, const void* pre,
                                   void* dz, float* parts, cudaStream_t st) {
  return d.dtype == MOE_BF16 ? act_grad<__nv_bfloat16>(d, dy, pre, dz, parts, st)
                             : act_grad<float>(d, dy, pre, dz, parts, st);
}

cudaError_t launch_linear_simt(int M, int N, int K, const float* A, bool a_mn, const float* B,
                               bool b_mn, const LinearEpilogue& epi, cudaStream_t st) {
  if (a_mn) return simt<true, true>(M, N, K, A, B, epi, st);
  return b_mn ? simt<false, true>(M, N, K, A, B, epi, st)
              : simt<false, false>(M, N, K, A, B, epi, st);
}

}  // namespace moe
