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
// second norm before it is rounded to be stored. Each form is a kernel of its own,
// and two elements go through one instruction (a kernel that looked at the form as
// it ran took 48 us for the second norm alone, now 42; 85 for all of it). Measured
// on B200, bf16, 16384 x 4096: 84 us, 6.4 TB/s (137 us with rows loaded when they
// are due); one row 2.2.
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

// kPre: norm before the next block. kBlock: 0 no block output, 1 as it is, 2 with a
// norm after the block. kGate: 0 none or per channel, 1 per token, 2 per element.
template <typename T, int VPT, int kStages, int kThreads, bool kPre, int kBlock, int kGate>
__global__ void __launch_bounds__(kThreads)
    block_norm_kernel(const NormFwd a, const moe_norm_desc d) {
  using V = RowVec<T>;
  constexpr int P = V::N / 2, kIn = 1 + (kBlock > 0) + (kGate == 2);
  extern __shared__ uint4 norm_ring[];
  __shared__ SumBuffers sums;
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int nvec = d.H / V::N;
  RowRing<kIn, kStages, VPT> ring;
  ring.nvec = nvec;
  ring.mine = norm_ring + threadIdx.x;
  ring.in[0] = a.h;
  if constexpr (kBlock > 0) ring.in[1] = a.y;
  if constexpr (kGate == 2) ring.in[2] = a.gate;
#pragma unroll
  for (int s = 0; s < kStages; ++s) ring.fetch(blockIdx.x + s * gridDim.x, d.T, s);
  Pair wg[VPT][P], wn[VPT][P];
  if constexpr (kBlock > 0) block_factor<T, VPT>(wg, a.w_post, a.gate, d, nvec);
  if constexpr (kPre)
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      unpack_pairs<T>(i < nvec ? vec_at(a.w_pre, i) : make_uint4(0, 0, 0, 0), wn[v]);
    }
  const float inv_h = 1.f / (float)d.H;
  int stage = 0;
  for (int t = blockIdx.x; t < d.T; t += gridDim.x) {
    const size_t row = (size_t)t * nvec;
    ring.wait();
    Pair f[VPT][P], u[VPT][P];
    Pair ss = pair_of(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      unpack_pairs<T>(*ring.at(stage, 0, v), f[v]);
      if constexpr (kBlock > 0) {
        unpack_pairs<T>(*ring.at(stage, 1, v), u[v]);
        if (kBlock == 2)
#pragma unroll
          for (int k = 0; k < P; ++k) ss = fma2(u[v][k], u[v][k], ss);
#pragma unroll
        for (int k = 0; k < P; ++k) u[v][k] = mul2(u[v][k], wg[v][k]);
      }
      if constexpr (kGate == 2) {
        Pair q[P];
        unpack_pairs<T>(*ring.at(stage, 2, v), q);
#pragma unroll
        for (int k = 0; k < P; ++k) u[v][k] = mul2(u[v][k], q[k]);
      }
    }
    if constexpr (kBlock > 0) {
      float scale = 1.f;
      if (kBlock == 2) scale = rsqrtf(block_sum(sum_of(ss), sums, turn) * inv_h + d.eps);
      if (kGate == 1) scale *= to_f32(reinterpret_cast<const T*>(a.gate)[t]);
      const Pair by = pair_of(scale);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int i = v * blockDim.x + threadIdx.x;
#pragma unroll
        for (int k = 0; k < P; ++k) f[v][k] = fma2(by, u[v][k], f[v][k]);
        if (a.h_out && i < nvec) put_vec(a.h_out, row + i, pack_pairs<T>(f[v]));
      }
    }
    // not before h' is stored: reads ahead of those writes take 96 us instead of 84
    ring.fetch(t + kStages * gridDim.x, d.T, stage);
    if (++stage == kStages) stage = 0;
    if constexpr (kPre) {
      ss = pair_of(0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int k = 0; k < P; ++k) ss = fma2(f[v][k], f[v][k], ss);
      const Pair r = pair_of(rsqrtf(block_sum(sum_of(ss), sums, turn) * inv_h + d.eps));
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int i = v * blockDim.x + threadIdx.x;
#pragma unroll
        for (int k = 0; k < P; ++k) f[v][k] = mul2(f[v][k], mul2(r, wn[v][k]));
        if (i < nvec) put_vec(a.x, row + i, pack_pairs<T>(f[v]));
      }
    }
  }
}

// One vector per thread up to 512 of them, two beyond. 1536 threads of an SM instead
// of 1024 take 96 us instead of 84, 512 take 103.
constexpr int kOneUpTo = 512;
constexpr int kThreadsPerSm = 1024;

template <typename T, bool kPre, int kBlock, int kGate>
cudaError_t launch_form(const moe_norm_desc& d, const NormFwd& a, int sms, cudaStream_t st) {
  const RowShape r = row_shape(d.H / RowVec<T>::N, kOneUpTo, kThreadsPerSm);
  const int grid = std::min(d.T, sms * r.blocks_per_sm);
  // a third stage helps where h is the only input (42 us instead of 45) and costs
  // with the block's output beside it (95 instead of 84)
  constexpr int kStages = kBlock ? 2 : 3;
  const size_t smem = ring_bytes(r, 1 + (kBlock > 0) + (kGate == 2), kStages);
  static std::atomic<bool> set[2][64];
  return r.vpt == 1 ? launch_rows(block_norm_kernel<T, 1, kStages, 512, kPre, kBlock, kGate>, set[0],
                                  grid, r, smem, st, a, d)
                    : launch_rows(block_norm_kernel<T, 2, kStages, 1024, kPre, kBlock, kGate>, set[1],
                                  grid, r, smem, st, a, d);
}

template <typename T, bool kPre, int kBlock>
cudaError_t launch_gate(const moe_norm_desc& d, const NormFwd& a, int sms, cudaStream_t st) {
  if (d.gate == MOE_GATE_TOKEN) return launch_form<T, kPre, kBlock, 1>(d, a, sms, st);
  if (d.gate == MOE_GATE_FULL) return launch_form<T, kPre, kBlock, 2>(d, a, sms, st);
  return launch_form<T, kPre, kBlock, 0>(d, a, sms, st);
}

template <typename T>
cudaError_t norm_forward(const moe_norm_desc& d, const NormFwd& a, int sms, cudaStream_t st) {
  if (!a.y) return launch_form<T, true, 0, 0>(d, a, sms, st);
  if (a.w_post)
    return a.w_pre ? launch_gate<T, true, 2>(d, a, sms, st)
                   : launch_gate<T, false, 2>(d, a, sms, st);
  return a.w_pre ? launch_gate<T, true, 1>(d, a, sms, st) : launch_gate<T, false, 1>(d, a, sms, st);
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
