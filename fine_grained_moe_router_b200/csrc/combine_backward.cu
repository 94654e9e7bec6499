// Gradient of the combine y[t] = sum_k w[t,k] y_rows[inv[t,k]]:
//   d_y_rows[inv[t,k]] = w[t,k] dy[t]      (rounded to the layer dtype: the
//                        operand type of the experts' backward products)
//   d_w[t,k] = <dy[t], y_rows[inv[t,k]]>   (fp32)
// "Kimi K3 fine-grained MoE under high concurrency", section "物理通信拓扑"
// (combine phase). A shared expert's output has the gradient dy itself.
//
// Bound by memory: the K fp32 expert rows of a token are read once and the K
// gradient rows written once. A group of threads takes a token: each thread keeps
// its piece of dy in registers and walks the K copies, whose loads do not depend
// on one another; the K inner products are reduced together at the end. A group
// is as wide as a row needs (one warp to 256 threads), and a batch too small to
// fill the SMs gives each copy a group of its own.
#include "common.cuh"
#include "kernels_block.cuh"
#include "launch.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// `width` threads per group (a power of two, 32 to 256); a group takes the copies
// [k0, k0 + n_k) of token t, n_k = K or 1 (then blockIdx.y is the copy). kCopies:
// n_k rounded up to 1, 2, 4, 8 or 16; kAtOnce: copies whose rows a thread has on
// their way together. (4096 tokens x 8 x 4096, bf16: 147 us one by one, 144 by
// fours, 134 by eights, 0.96 of the measured copy rate; but 16384 x 1 x 4096:
// 110 us one by one, 214 by eights.)
template <typename T, int kCopies, int kAtOnce>
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const T* __restrict__ dy, const float* __restrict__ y_rows,
                            const float* __restrict__ w, const int32_t* __restrict__ inv,
                            T* __restrict__ d_rows, float* __restrict__ d_w, int T_, int H,
                            int K, int n_k, int width) {
  using V = RowVec<T>;
  __shared__ float buf[kThreads / 32][kCopies];
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x / width, thread = threadIdx.x & (width - 1);
  const int t = blockIdx.x * (kThreads / width) + group, k0 = n_k == K ? 0 : blockIdx.y;
  const unsigned rows = (unsigned)T_ * (unsigned)K;
  const size_t copy0 = (size_t)t * K + k0;
  const int nvec = H / V::N;
  float dot[kCopies];
#pragma unroll
  for (int k = 0; k < kCopies; ++k) dot[k] = 0.f;
  if (t < T_)
    for (int i = thread; i < nvec; i += width) {
      float g[V::N];
      V::unpack(reinterpret_cast<const uint4*>(dy)[(size_t)t * nvec + i], g);
#pragma unroll
      for (int kb = 0; kb < kCopies; kb += kAtOnce) {
        if (kb >= n_k) break;
        // the rows of kAtOnce copies are on their way together; a copy that the
        // dispatch did not place (r out of range) is left out
        int r[kAtOnce];
        float4 f[kAtOnce][V::N / 4];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          r[j] = kb + j < n_k ? inv[copy0 + kb + j] : -1;
          const bool live = (unsigned)r[j] < rows;
          const float4* src =
              reinterpret_cast<const float4*>(y_rows + (live ? (size_t)r[j] : 0) * H + i * V::N);
#pragma unroll
          for (int q = 0; q < V::N / 4; ++q)
            f[j][q] = live ? __ldcs(src + q) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          if ((unsigned)r[j] >= rows) continue;
          const float wk = w[copy0 + kb + j];
          float o[V::N];
#pragma unroll
          for (int q = 0; q < V::N / 4; ++q) {
            float& s = dot[kb + j];
            s = fmaf(g[4 * q], f[j][q].x, s);
            s = fmaf(g[4 * q + 1], f[j][q].y, s);
            s = fmaf(g[4 * q + 2], f[j][q].z, s);
            s = fmaf(g[4 * q + 3], f[j][q].w, s);
          }
#pragma unroll
          for (int q = 0; q < V::N; ++q) o[q] = wk * g[q];
          reinterpret_cast<uint4*>(d_rows)[(size_t)r[j] * nvec + i] = V::pack(o);
        }
      }
    }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    if (k >= n_k) break;
#pragma unroll
    for (int o = 16; o; o >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
    if (lane == 0) buf[warp][k] = dot[k];
  }
  __syncthreads();
  if (thread < n_k && t < T_) {
    float s = 0.f;
    for (int i = 0; i < width / 32; ++i) s += buf[group * (width / 32) + i][thread];
    d_w[copy0 + thread] = s;
  }
}

template <typename T>
cudaError_t combine_backward(const moe_layer_desc& d, const void* dy, const float* y_rows,
                             const float* w, const int32_t* inv, void* d_rows, float* d_w,
                             cudaStream_t st) {
  int width = 32;
  while (width < kThreads && width < d.H / RowVec<T>::N) width *= 2;
  const int per_block = kThreads / width, blocks = (d.T + per_block - 1) / per_block;
  const bool split = d.K > 1 && blocks < 2 * kPlanSms;
  const int n_k = split ? 1 : d.K;
  auto kernel = n_k == 1   ? combine_backward_kernel<T, 1, 1>
                : n_k == 2 ? combine_backward_kernel<T, 2, 2>
                : n_k <= 4 ? combine_backward_kernel<T, 4, 4>
                : n_k <= 8 ? combine_backward_kernel<T, 8, 8>
                           : combine_backward_kernel<T, 16, 8>;
  return launch_pdl(kernel, dim3(blocks, split ? d.K : 1), dim3(kThreads), 0, st,
                    static_cast<const T*>(dy), y_rows, w, inv, static_cast<T*>(d_rows), d_w,
                    d.T, d.H, d.K, n_k, width);
}

}  // namespace

cudaError_t launch_combine_backward(const moe_layer_desc& d, const void* dy, const float* y_rows,
                                    const float* w, const int32_t* inv, void* d_rows, float* d_w,
                                    cudaStream_t st) {
  if (d.T == 0) return cudaSuccess;
  return d.dtype == MOE_BF16
             ? combine_backward<__nv_bfloat16>(d, dy, y_rows, w, inv, d_rows, d_w, st)
             : combine_backward<float>(d, dy, y_rows, w, inv, d_rows, d_w, st);
}

}  // namespace moe
