// The linear layer's CUDA-core parts: the fp32 products, and the activation's
// gradient with the bias gradient's column sums.
#include "common.cuh"
#include "kernels_block.cuh"
#include "launch.cuh"
#include "linear_epilogue.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

// fp32 layers: true FFMA products (no tensor-core type keeps 24 bits). A block
// takes a tile of kB x kB of C. Its groups of 128 threads take the reduction's
// steps of kSK elements in turn (a chain of steps is a chain of trips to memory),
// and their sums are added in order at the end. The next step's elements travel
// from memory to registers while the products of this one are formed, then to
// the other half of shared memory. A group adds up the sums of kRun steps apart:
// rounding errors then grow with sqrt(kRun kSK) + sqrt(K / (kRun kSK)) and not
// with sqrt(K). Measured (fp32, 512 x 1024 x 1024): 133 us with one group and
// without the steps' overlap, 43 with it, 35 with two groups.
constexpr int kSK = 16, kRun = 8, kSimtThreads = 128;

// A step's elements of an operand stored [rows, K], or [K, rows] when kMn, as
// 16-byte vectors along the stored rows (K and rows then are multiples of 4).
template <int kB, bool kMn>
struct StepLoad {
  static constexpr int kVecs = kB * kSK / 4 / kSimtThreads;
  float4 v[kVecs];

  __device__ __forceinline__ static void at(int i, int& r, int& k) {
    if (kMn) {
      r = i % (kB / 4) * 4;
      k = i / (kB / 4);
    } else {
      r = i / (kSK / 4);
      k = i % (kSK / 4) * 4;
    }
  }
  __device__ __forceinline__ void load(const float* p, int r0, int k0, int rows, int K) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      int r, k;
      at((threadIdx.x & (kSimtThreads - 1)) + j * kSimtThreads, r, k);
      v[j] = r0 + r < rows && k0 + k < K
                 ? *reinterpret_cast<const float4*>(kMn ? p + (size_t)(k0 + k) * rows + r0 + r
                                                        : p + (size_t)(r0 + r) * K + k0 + k)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void store(float (*dst)[kB + 4]) const {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      int r, k;
      at((threadIdx.x & (kSimtThreads - 1)) + j * kSimtThreads, r, k);
      if (kMn) {
        *reinterpret_cast<float4*>(&dst[k][r]) = v[j];
      } else {
        dst[k][r] = v[j].x;
        dst[k + 1][r] = v[j].y;
        dst[k + 2][r] = v[j].z;
        dst[k + 3][r] = v[j].w;
      }
    }
  }
};

// kB = 64: 8 x 4 outputs per thread; kB = 32: 2 x 4.
template <int kB, int kGroups, bool kAMn, bool kBMn, int kAct>
__global__ void __launch_bounds__(kSimtThreads * kGroups)
    linear_simt_kernel(int M, int N, int K, const float* __restrict__ A,
                       const float* __restrict__ B, const LinearEpilogue epi) {
  constexpr int kTN = 4, kTM = kB * kB / kSimtThreads / kTN;
  __shared__ __align__(16) float tiles[kGroups][2][2][kSK][kB + 4];
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x / kSimtThreads, thread = threadIdx.x & (kSimtThreads - 1);
  const int m0 = blockIdx.y * kB, n0 = blockIdx.x * kB;
  const int tr = thread / (kB / kTN) * kTM, tc = thread % (kB / kTN) * kTN;
  float total[kTM][kTN] = {}, c[kTM][kTN] = {};
  StepLoad<kB, kAMn> a;
  StepLoad<kB, kBMn> b;
  a.load(A, m0, group * kSK, M, K);
  b.load(B, n0, group * kSK, N, K);
  int half = 0, step = 0;
  for (int k0 = group * kSK; k0 < K; k0 += kGroups * kSK, half ^= 1, ++step) {
    float(*sa)[kB + 4] = tiles[group][half][0];
    float(*sb)[kB + 4] = tiles[group][half][1];
    a.store(sa);
    b.store(sb);
    // one barrier of the group per step: the other half was last read before the
    // barrier of the step before
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kSimtThreads) : "memory");
    a.load(A, m0, k0 + kGroups * kSK, M, K);
    b.load(B, n0, k0 + kGroups * kSK, N, K);
    if (step % kRun == 0)
#pragma unroll
      for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int j = 0; j < kTN; ++j) {
          total[i][j] += c[i][j];
          c[i][j] = 0.f;
        }
#pragma unroll
    for (int k = 0; k < kSK; ++k) {
      float av[kTM];
#pragma unroll
      for (int i = 0; i < kTM; i += 2)
        *reinterpret_cast<float2*>(av + i) = *reinterpret_cast<const float2*>(&sa[k][tr + i]);
      const float4 b4 = *reinterpret_cast<const float4*>(&sb[k][tc]);
      const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int j = 0; j < kTN; ++j) c[i][j] = fmaf(av[i], bv[j], c[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int j = 0; j < kTN; ++j) c[i][j] += total[i][j];
  // the groups' sums through shared memory, [output][thread], added by group 0
  static_assert(sizeof(tiles) >= (size_t)(kGroups - 1) * kB * kB * sizeof(float),
                "the tiles' memory holds the other groups' sums");
  float* sums = &tiles[0][0][0][0][0];
  __syncthreads();
  if (group > 0)
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j)
        sums[((group - 1) * kTM * kTN + i * kTN + j) * kSimtThreads + thread] = c[i][j];
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int g = 0; g < kGroups - 1; ++g)
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j)
        c[i][j] += sums[(g * kTM * kTN + i * kTN + j) * kSimtThreads + thread];
  const int col = n0 + tc;
  if (col >= N) return;   // N is a multiple of 4
#pragma unroll
  for (int i = 0; i < kTM; ++i)
    if (m0 + tr + i < M)
      linear_finish<float, kAct>(epi, (size_t)(m0 + tr + i) * N + col, col, c[i]);
}

// One block: kGradRows rows by 32 vectors of columns; thread = one vector of
// columns, every eighth row, kAtOnce of them at a time: with an activation two, so
// that four blocks of 64 registers a thread share an SM. (4096 x 14336, gelu: 74 us
// with four rows, 65 with two, 54 the floor. Blocks of up to 256 vectors, a
// thread per column, were slower at every size measured.)

template <typename T, int kAct>
__global__ void __launch_bounds__(256, 4)
    linear_act_grad_kernel(int rows, int cols, const T* __restrict__ dy,
                           const T* __restrict__ pre, T* __restrict__ dz,
                           float* __restrict__ parts) {
  using V = RowVec<T>;
  constexpr int kWidth = 32, kSlices = 256 / kWidth, kAtOnce = kAct == MOE_ACT_NONE ? 4 : 2;
  __shared__ float buf[kSlices][kWidth * V::N];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (kWidth - 1), slice = threadIdx.x / kWidth;
  const int nvec = cols / V::N, i = blockIdx.x * kWidth + lane;
  const int r1 = min(rows, (int)(blockIdx.y + 1) * kGradRows);
  float s[V::N];
#pragma unroll
  for (int k = 0; k < V::N; ++k) s[k] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int r0 = blockIdx.y * kGradRows + slice; i < nvec && r0 < r1; r0 += kSlices * kAtOnce) {
    uint4 gv[kAtOnce], zv[kAtOnce];   // rows on their way together
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int r = r0 + kSlices * j;
      const size_t o = (size_t)r * nvec + i;
      gv[j] = r < r1 ? __ldcs(reinterpret_cast<const uint4*>(dy) + o) : zero;
      if (kAct != MOE_ACT_NONE)
        zv[j] = r < r1 ? __ldcs(reinterpret_cast<const uint4*>(pre) + o) : zero;
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int r = r0 + kSlices * j;
      float g[V::N], z[V::N];
      V::unpack(gv[j], g);
      if (kAct != MOE_ACT_NONE) {
        V::unpack(zv[j], z);
#pragma unroll
        for (int k = 0; k < V::N; k += 2) {
          const float2 f = linear_act_grad2<T, kAct>(make_float2(z[k], z[k + 1]));
          g[k] *= f.x;
          g[k + 1] *= f.y;
        }
        if (r < r1) reinterpret_cast<uint4*>(dz)[(size_t)r * nvec + i] = V::pack(g);
      }
#pragma unroll
      for (int k = 0; k < V::N; ++k) s[k] += g[k];
    }
  }
  if (!parts) return;
#pragma unroll
  for (int k = 0; k < V::N; ++k) buf[slice][lane * V::N + k] = s[k];
  __syncthreads();
  for (int c = threadIdx.x; c < kWidth * V::N; c += 256) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < kSlices; ++q) t += buf[q][c];
    const int col = blockIdx.x * kWidth * V::N + c;
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

template <int kB, int kGroups, bool kAMn, bool kBMn>
cudaError_t simt(int M, int N, int K, const float* A, const float* B, const LinearEpilogue& epi,
                 cudaStream_t st) {
  const dim3 grid((N + kB - 1) / kB, (M + kB - 1) / kB);
  auto k = epi.act == MOE_ACT_GELU   ? linear_simt_kernel<kB, kGroups, kAMn, kBMn, MOE_ACT_GELU>
           : epi.act == MOE_ACT_SILU ? linear_simt_kernel<kB, kGroups, kAMn, kBMn, MOE_ACT_SILU>
                                     : linear_simt_kernel<kB, kGroups, kAMn, kBMn, MOE_ACT_NONE>;
  return launch_pdl(k, grid, dim3(kSimtThreads * kGroups), 0, st, M, N, K, A, B, epi);
}

// Large tiles do more products per element read; small ones spread a small
// result over the SMs.
template <bool kAMn, bool kBMn>
cudaError_t simt_tiles(int M, int N, int K, const float* A, const float* B,
                       const LinearEpilogue& epi, cudaStream_t st) {
  const long long large = (long long)((M + 63) / 64) * ((N + 63) / 64);
  return large >= kPlanSms / 2 ? simt<64, 2, kAMn, kBMn>(M, N, K, A, B, epi, st)
                               : simt<32, 4, kAMn, kBMn>(M, N, K, A, B, epi, st);
}

}  // namespace

cudaError_t launch_linear_act_grad(const moe_linear_desc& d, const void* dy, const void* pre,
                                   void* dz, float* parts, cudaStream_t st) {
  return d.dtype == MOE_BF16 ? act_grad<__nv_bfloat16>(d, dy, pre, dz, parts, st)
                             : act_grad<float>(d, dy, pre, dz, parts, st);
}

cudaError_t launch_linear_simt(int M, int N, int K, const float* A, bool a_mn, const float* B,
                               bool b_mn, const LinearEpilogue& epi, cudaStream_t st) {
  if (a_mn) return simt_tiles<true, true>(M, N, K, A, B, epi, st);
  return b_mn ? simt_tiles<false, true>(M, N, K, A, B, epi, st)
              : simt_tiles<false, false>(M, N, K, A, B, epi, st);
}

}  // namespace moe
