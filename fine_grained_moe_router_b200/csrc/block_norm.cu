// The norms around a block in one pass over the row, and their gradients.
//
//   u  = y                        or  rms(y) * w_post      (norm after the block)
//   h' = h + alpha * gate * u     (gate: 1, per channel, per token or per element)
//   x  = rms(h') * w_pre          (norm before the next block)
//   rms(v) = v / sqrt(mean(v^2) + eps)
// Each part is optional. The layer itself adds no residual ("Kimi K3
// fine-grained MoE under high concurrency" adds it at the combine); this is the
// step that does.
//
// Bound by memory: every element of h, y, h' and x moves once. A block takes
// whole rows, one after the other, and holds a row in registers between its
// reductions. Rows ahead are on their way into shared memory meanwhile
// (cp.async, each thread its own 16-byte pieces, so no barrier guards them).
// What is the same for every row stays in registers: alpha, the post-norm's
// weight and the channel gate as one factor. All sums are fp32; h' feeds the
// second norm before it is rounded to be stored. Measured on B200, bf16, 16384 x
// 4096: 85 us, 6.3 TB/s (137 us with rows loaded when they are due); one row 2.6.
#include "common.cuh"
#include "kernels_block.cuh"
#include "launch.cuh"
#include "row_ring.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

struct NormFwd {
  const void *h, *y, *w_post, *gate, *w_pre;
  void *h_out, *x;
};

template <typename T, int VPT, int kStages, int kMaxThreads, int kBlocks>
__global__ void __launch_bounds__(kMaxThreads, kBlocks)
    block_norm_kernel(const NormFwd a, const moe_norm_desc d) {
  using V = RowVec<T>;
  extern __shared__ uint4 norm_ring[];
  __shared__ SumBuffers sums;
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int nvec = d.H / V::N;
  const bool full = d.gate == MOE_GATE_FULL;
  const RowRing<3, kStages, VPT> ring{{a.h, a.y, full ? a.gate : nullptr}, nvec,
                                      norm_ring + threadIdx.x};
#pragma unroll
  for (int s = 0; s < kStages; ++s) ring.fetch(blockIdx.x + s * gridDim.x, d.T, s);
  float wg[VPT][V::N], wn[VPT][V::N];
  block_factor<T, VPT>(wg, a.w_post, a.gate, d, nvec);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = v * blockDim.x + threadIdx.x;
    V::unpack(a.w_pre && i < nvec ? vec_at(a.w_pre, i) : make_uint4(0, 0, 0, 0), wn[v]);
  }
  const float inv_h = 1.f / (float)d.H;
  int stage = 0;
  for (int t = blockIdx.x; t < d.T; t += gridDim.x) {
    const size_t row = (size_t)t * nvec;
    ring.wait();
    float f[VPT][V::N], u[VPT][V::N];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      V::unpack(*ring.at(stage, 0, v), f[v]);
      if (a.y) {
        V::unpack(*ring.at(stage, 1, v), u[v]);
        if (a.w_post)
#pragma unroll
          for (int k = 0; k < V::N; ++k) ss = fmaf(u[v][k], u[v][k], ss);
#pragma unroll
        for (int k = 0; k < V::N; ++k) u[v][k] *= wg[v][k];
        if (full) {
          float q[V::N];
          V::unpack(*ring.at(stage, 2, v), q);
#pragma unroll
          for (int k = 0; k < V::N; ++k) u[v][k] *= q[k];
        }
      }
    }
    ring.fetch(t + kStages * gridDim.x, d.T, stage);
    if (++stage == kStages) stage = 0;
    if (a.y) {
      float scale = 1.f;
      if (a.w_post) {
        scale = rsqrtf(block_sum(ss, sums, turn) * inv_h + d.eps);
      }
      if (d.gate == MOE_GATE_TOKEN) scale *= to_f32(reinterpret_cast<const T*>(a.gate)[t]);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int k = 0; k < V::N; ++k) f[v][k] = fmaf(scale, u[v][k], f[v][k]);
    }
    if (a.h_out)
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int i = v * blockDim.x + threadIdx.x;
        if (i < nvec) put_vec(a.h_out, row + i, V::pack(f[v]));
      }
    if (!a.w_pre) continue;
    ss = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int k = 0; k < V::N; ++k) ss = fmaf(f[v][k], f[v][k], ss);
    const float r = rsqrtf(block_sum(ss, sums, turn) * inv_h + d.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
#pragma unroll
      for (int k = 0; k < V::N; ++k) f[v][k] *= r * wn[v][k];
      if (i < nvec) put_vec(a.x, row + i, V::pack(f[v]));
    }
  }
}

template <typename T>
cudaError_t norm_forward(const moe_norm_desc& d, const NormFwd& a, int sms, cudaStream_t st) {
  const RowShape r = row_shape(d.H / RowVec<T>::N, 512, 1024);
  const int grid = std::min(d.T, sms * r.blocks_per_sm);
  static std::atomic<bool> one[64], two[64];
  return r.vpt == 1 ? launch_rows(block_norm_kernel<T, 1, 2, 512, 2>, one, grid, r,
                                  ring_bytes(r, 3, 2), st, a, d)
                    : launch_rows(block_norm_kernel<T, 2, 2, 1024, 1>, two, grid, r,
                                  ring_bytes(r, 3, 2), st, a, d);
}

}  // namespace

cudaError_t launch_block_norm(const moe_norm_desc& d, const void* h, const void* y,
                              const void* w_post, const void* gate, const void* w_pre,
                              void* h_out, void* x, int sms, cudaStream_t st) {
  const NormFwd a{h, y, w_post, gate, w_pre, h_out, x};
  return d.dtype == MOE_BF16 ? norm_forward<__nv_bfloat16>(d, a, sms, st)
                             : norm_forward<float>(d, a, sms, st);
}

}  // namespace moe
