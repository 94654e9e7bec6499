// Gradient of the combine y[t] = sum_k w[t,k] y_rows[inv[t,k]]:
//   d_y_rows[inv[t,k]] = w[t,k] dy[t]      (rounded to the layer dtype: the
//                        operand type of the experts' backward products)
//   d_w[t,k] = <dy[t], y_rows[inv[t,k]]>   (fp32)
// "Kimi K3 fine-grained MoE under high concurrency", section "物理通信拓扑"
// (combine phase). A shared expert's output has the gradient dy itself.
//
// Bound by memory: the K fp32 expert rows of a token are read once and the K
// gradient rows written once. One block per token: each thread keeps its piece
// of dy in registers and walks the K copies, whose loads do not depend on one
// another; the K inner products are reduced together at the end.
#include "common.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const T* __restrict__ dy, const float* __restrict__ y_rows,
                            const float* __restrict__ w, const int32_t* __restrict__ inv,
                            T* __restrict__ d_rows, float* __restrict__ d_w, int T_, int H,
                            int K) {
  using V = RowVec<T>;
  __shared__ float buf[kThreads / 32][kMaxK];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x;
  const unsigned rows = (unsigned)T_ * (unsigned)K;
  float dot[kMaxK];
#pragma unroll
  for (int k = 0; k < kMaxK; ++k) dot[k] = 0.f;
  for (int i = threadIdx.x; i < H / V::N; i += kThreads) {
    float g[V::N];
    V::unpack(reinterpret_cast<const uint4*>(dy)[(size_t)t * (H / V::N) + i], g);
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
      if (k >= K) break;
      const int r = inv[(size_t)t * K + k];
      if ((unsigned)r >= rows) continue;   // a copy that the dispatch did not place
      const float wk = w[(size_t)t * K + k];
      const float4* src = reinterpret_cast<const float4*>(y_rows + (size_t)r * H + i * V::N);
      float o[V::N];
#pragma unroll
      for (int q = 0; q < V::N / 4; ++q) {
        const float4 f = __ldcs(src + q);
        dot[k] = fmaf(g[4 * q], f.x, dot[k]);
        dot[k] = fmaf(g[4 * q + 1], f.y, dot[k]);
        dot[k] = fmaf(g[4 * q + 2], f.z, dot[k]);
        dot[k] = fmaf(g[4 * q + 3], f.w, dot[k]);
      }
#pragma unroll
      for (int q = 0; q < V::N; ++q) o[q] = wk * g[q];
      reinterpret_cast<uint4*>(d_rows)[(size_t)r * (H / V::N) + i] = V::pack(o);
    }
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < kMaxK; ++k) {
    if (k >= K) break;
#pragma unroll
    for (int o = 16; o; o >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
    if (lane == 0) buf[warp][k] = dot[k];
  }
  __syncthreads();
  if (threadIdx.x < K) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += buf[i][threadIdx.x];
    d_w[(size_t)t * K + threadIdx.x] = s;
  }
}

}  // namespace

cudaError_t launch_combine_backward(const moe_layer_desc& d, const void* dy, const float* y_rows,
                                    const float* w, const int32_t* inv, void* d_rows, float* d_w,
                                    cudaStream_t st) {
  if (d.T == 0) return cudaSuccess;
  if (d.dtype == MOE_BF16)
    return launch_pdl(combine_backward_kernel<__nv_bfloat16>, dim3(d.T), dim3(kThreads), 0, st,
                      (const __nv_bfloat16*)dy, y_rows, w, inv, (__nv_bfloat16*)d_rows, d_w, d.T,
                      d.H, d.K);
  return launch_pdl(combine_backward_kernel<float>, dim3(d.T), dim3(kThreads), 0, st,
                    (const float*)dy, y_rows, w, inv, (float*)d_rows, d_w, d.T, d.H, d.K);
}

}  // namespace moe
