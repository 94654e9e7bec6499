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
// second norm before it is rounded to be stored.
#include <atomic>

#include "common.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

struct NormFwd {
  const void *h, *y, *w_post, *gate, *w_pre;
  void *h_out, *x;
};
struct NormBwd {
  const void *d_h_out, *d_x, *h_out, *y, *w_post, *gate, *w_pre;
  void *d_h, *d_y, *d_gate;
  float* parts;   // [grid, n_parts, H] column sums of each block
  int at_post, at_gate, at_pre, n_parts;   // -1: not wanted
};

// Sums of N values over the block, in a fixed order. Two buffers taken in turn
// let one barrier do per reduction: a buffer is written again only after every
// thread has passed the barrier of the reduction in between.
struct SumBuffers {
  float v[2][3 * 32];
};
template <int N>
__device__ __forceinline__ void block_sums(float (&s)[N], SumBuffers& bufs, int& turn) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  const int n_warps = blockDim.x >> 5;
  if (n_warps == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* buf = bufs.v[turn ^= 1];
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[32 * i + warp] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = lane < n_warps ? buf[32 * i + lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
}

__device__ __forceinline__ uint4 vec_at(const void* p, size_t i) {
  return reinterpret_cast<const uint4*>(p)[i];
}
__device__ __forceinline__ void put_vec(void* p, size_t i, const uint4& v) {
  reinterpret_cast<uint4*>(p)[i] = v;
}

// A ring of kStages rows of up to kIn inputs in shared memory. A thread copies
// and reads its own vectors only (vector v * blockDim.x + threadIdx.x of a row).
template <int kIn, int kStages, int VPT>
struct RowRing {
  const void* in[kIn];
  int nvec;
  uint4* mine;

  __device__ __forceinline__ uint4* at(int stage, int i, int v) const {
    return mine + (size_t)((stage * kIn + i) * VPT + v) * blockDim.x;
  }
  // Starts the copies of row t (past the last row: none) as one group.
  __device__ __forceinline__ void fetch(int t, int T, int stage) const {
    if (t < T) {
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        if (!in[i]) continue;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int c = v * blockDim.x + threadIdx.x;
          const bool on = c < nvec;   // past the row's end: zeros
          const uint4* src = reinterpret_cast<const uint4*>(in[i]) + (size_t)t * nvec + (on ? c : 0);
          const uint32_t dst = (uint32_t)__cvta_generic_to_shared(at(stage, i, v));
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                       "r"(on ? 16 : 0)
                       : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  }
};

// alpha * w_post * (channel gate) of the thread's columns.
template <typename T, int VPT>
__device__ __forceinline__ void block_factor(float (&f)[VPT][RowVec<T>::N], const void* w_post,
                                             const void* gate, const moe_norm_desc& d, int nvec) {
  using V = RowVec<T>;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = v * blockDim.x + threadIdx.x;
    const bool in = i < nvec;
#pragma unroll
    for (int k = 0; k < V::N; ++k) f[v][k] = d.alpha;
    float u[V::N];
    if (in && w_post) {
      V::unpack(vec_at(w_post, i), u);
#pragma unroll
      for (int k = 0; k < V::N; ++k) f[v][k] *= u[k];
    }
    if (in && d.gate == MOE_GATE_CHANNEL) {
      V::unpack(vec_at(gate, i), u);
#pragma unroll
      for (int k = 0; k < V::N; ++k) f[v][k] *= u[k];
    }
  }
}

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
    float ss[1] = {0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      V::unpack(*ring.at(stage, 0, v), f[v]);
      if (a.y) {
        V::unpack(*ring.at(stage, 1, v), u[v]);
        if (a.w_post)
#pragma unroll
          for (int k = 0; k < V::N; ++k) ss[0] = fmaf(u[v][k], u[v][k], ss[0]);
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
        block_sums(ss, sums, turn);
        scale = rsqrtf(ss[0] * inv_h + d.eps);
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
    ss[0] = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int k = 0; k < V::N; ++k) ss[0] = fmaf(f[v][k], f[v][k], ss[0]);
    block_sums(ss, sums, turn);
    const float r = rsqrtf(ss[0] * inv_h + d.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
#pragma unroll
      for (int k = 0; k < V::N; ++k) f[v][k] *= r * wn[v][k];
      if (i < nvec) put_vec(a.x, row + i, V::pack(f[v]));
    }
  }
}

// With r = 1/rms, n = v r and d = dL/d(n w):
//   dL/dv = r d w - v r^3 mean(d w v),   dL/dw = sum over tokens of d n.
// The row's first reduction takes both sums of squares and the pre-norm's inner
// product, the second the post-norm's, so the norms' statistics are not kept
// from the forward pass. With g = dL/dh' and n = y r, the column sums of g n
// (times a token or full gate) give both the post-norm's and the channel gate's
// gradient: what they differ by is the same for every row.
template <typename T, int VPT, int kStages, int kMaxThreads, int kBlocks>
__global__ void __launch_bounds__(kMaxThreads, kBlocks)
    block_norm_backward_kernel(const NormBwd a, const moe_norm_desc d) {
  using V = RowVec<T>;
  extern __shared__ uint4 norm_ring[];
  __shared__ SumBuffers sums;
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int nvec = d.H / V::N;
  const bool full = d.gate == MOE_GATE_FULL, pre = a.w_pre != nullptr;
  const RowRing<5, kStages, VPT> ring{{a.d_h_out, pre ? a.d_x : nullptr, pre ? a.h_out : nullptr,
                                       a.y, full ? a.gate : nullptr},
                                      nvec, norm_ring + threadIdx.x};
#pragma unroll
  for (int s = 0; s < kStages; ++s) ring.fetch(blockIdx.x + s * gridDim.x, d.T, s);
  float wg[VPT][V::N], wn[VPT][V::N], s_n[VPT][V::N], s_pre[VPT][V::N];
  block_factor<T, VPT>(wg, a.w_post, a.gate, d, nvec);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = v * blockDim.x + threadIdx.x;
    V::unpack(pre && i < nvec ? vec_at(a.w_pre, i) : make_uint4(0, 0, 0, 0), wn[v]);
#pragma unroll
    for (int k = 0; k < V::N; ++k) s_n[v][k] = s_pre[v][k] = 0.f;
  }
  const float inv_h = 1.f / (float)d.H;
  int stage = 0;
  for (int t = blockIdx.x; t < d.T; t += gridDim.x) {
    const size_t row = (size_t)t * nvec;
    ring.wait();
    uint4 xv[VPT], hv[VPT], yv[VPT];
    float g[VPT][V::N];
    float s[3] = {0.f, 0.f, 0.f};   // sums of h'^2, h' d_x w, y^2
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      V::unpack(a.d_h_out ? *ring.at(stage, 0, v) : make_uint4(0, 0, 0, 0), g[v]);
      float p[V::N], q[V::N];
      if (pre) {
        xv[v] = *ring.at(stage, 1, v);
        hv[v] = *ring.at(stage, 2, v);
        V::unpack(xv[v], q);
        V::unpack(hv[v], p);
#pragma unroll
        for (int k = 0; k < V::N; ++k) {
          s[0] = fmaf(p[k], p[k], s[0]);
          s[1] = fmaf(p[k] * q[k], wn[v][k], s[1]);
        }
      }
      if (a.y) {
        yv[v] = *ring.at(stage, 3, v);
        V::unpack(yv[v], p);
#pragma unroll
        for (int k = 0; k < V::N; ++k) s[2] = fmaf(p[k], p[k], s[2]);
      }
    }
    uint4 qv[VPT];
    if (full)
#pragma unroll
      for (int v = 0; v < VPT; ++v) qv[v] = *ring.at(stage, 4, v);
    ring.fetch(t + kStages * gridDim.x, d.T, stage);
    if (++stage == kStages) stage = 0;
    if (pre || a.w_post) block_sums(s, sums, turn);
    const float r_post = a.w_post ? rsqrtf(s[2] * inv_h + d.eps) : 1.f;
    if (pre) {
      const float r = rsqrtf(s[0] * inv_h + d.eps);
      const float c = s[1] * inv_h * r * r * r;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float p[V::N], q[V::N];
        V::unpack(xv[v], q);
        V::unpack(hv[v], p);
#pragma unroll
        for (int k = 0; k < V::N; ++k) {
          s_pre[v][k] = fmaf(p[k] * q[k], r, s_pre[v][k]);
          g[v][k] = fmaf(-c, p[k], fmaf(q[k] * wn[v][k], r, g[v][k]));
        }
      }
    }
    if (a.d_h)
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int i = v * blockDim.x + threadIdx.x;
        if (i < nvec) put_vec(a.d_h, row + i, V::pack(g[v]));
      }
    if (!a.y) continue;
    const float gate_t =
        d.gate == MOE_GATE_TOKEN ? to_f32(reinterpret_cast<const T*>(a.gate)[t]) : 1.f;
    float dot[1] = {0.f};   // sum of g wg y (times a full gate)
    const float rn = r_post * gate_t;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float y[V::N];
      V::unpack(yv[v], y);
      if (full) {
        float q[V::N], dg[V::N];
        V::unpack(qv[v], q);
#pragma unroll
        for (int k = 0; k < V::N; ++k) {
          dg[k] = g[v][k] * wg[v][k] * (y[k] * r_post);
          g[v][k] *= q[k];
        }
        const int i = v * blockDim.x + threadIdx.x;
        if (a.d_gate && i < nvec) put_vec(a.d_gate, row + i, V::pack(dg));
      }
#pragma unroll
      for (int k = 0; k < V::N; ++k) {
        const float gy = g[v][k] * y[k];
        s_n[v][k] = fmaf(gy, rn, s_n[v][k]);
        dot[0] = fmaf(gy, wg[v][k], dot[0]);
      }
    }
    const bool token = d.gate == MOE_GATE_TOKEN && a.d_gate;
    if (a.w_post || token) block_sums(dot, sums, turn);
    if (token && threadIdx.x == 0) reinterpret_cast<float*>(a.d_gate)[t] = dot[0] * r_post;
    if (!a.d_y) continue;
    const float c = a.w_post ? dot[0] * gate_t * inv_h * r_post * r_post * r_post : 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      float y[V::N];
      V::unpack(yv[v], y);
#pragma unroll
      for (int k = 0; k < V::N; ++k) y[k] = fmaf(-c, y[k], g[v][k] * wg[v][k] * rn);
      if (i < nvec) put_vec(a.d_y, row + i, V::pack(y));
    }
  }
  // this block's column sums
  auto put = [&](int at, const float (&s)[VPT][V::N], float alpha, const void* by) {
    if (at < 0) return;
    float* out = a.parts + ((size_t)blockIdx.x * a.n_parts + at) * d.H;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      if (i >= nvec) continue;
      float f[V::N];
#pragma unroll
      for (int k = 0; k < V::N; ++k) f[k] = 1.f;
      if (by) V::unpack(vec_at(by, i), f);
#pragma unroll
      for (int k = 0; k < V::N; k += 4)
        *reinterpret_cast<float4*>(out + (size_t)i * V::N + k) =
            make_float4(s[v][k] * f[k] * alpha, s[v][k + 1] * f[k + 1] * alpha,
                        s[v][k + 2] * f[k + 2] * alpha, s[v][k + 3] * f[k + 3] * alpha);
    }
  };
  put(a.at_post, s_n, d.alpha, d.gate == MOE_GATE_CHANNEL ? a.gate : nullptr);
  put(a.at_gate, s_n, d.alpha, a.w_post);
  put(a.at_pre, s_pre, 1.f, nullptr);
}

// out[at][c] = sum over the n_blocks partial rows, in a fixed order: 32
// strided partial sums, added in order.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ parts,
                                                           int n_blocks, int n_parts, int H,
                                                           const ColumnSums o) {
  __shared__ float buf[32][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < H)
    for (int b = slice; b < n_blocks; b += 32)
      s += parts[((size_t)b * n_parts + blockIdx.y) * H + c];
  buf[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += buf[i][lane];
    o.out[blockIdx.y][c] = s;
  }
}

// Launch shape of a row width: one vector per thread up to 512 (forward) or 1024
// (backward) of them, two beyond; as many resident blocks as fill an SM.
struct RowShape {
  int threads, vpt, per_sm;
};
RowShape row_shape(int nvec, int one_up_to) {
  RowShape r;
  r.vpt = nvec <= one_up_to ? 1 : 2;
  r.threads = ((nvec + r.vpt - 1) / r.vpt + 31) / 32 * 32;
  r.per_sm = std::max(1, std::min(32, 1024 / r.threads));
  return r;
}
size_t ring_bytes(const RowShape& r, int inputs, int stages) {
  return (size_t)r.threads * r.vpt * inputs * stages * sizeof(uint4);
}

template <typename Kernel, typename Args>
cudaError_t launch_rows(Kernel kernel, std::atomic<bool>* set, int grid, const RowShape& r,
                        size_t smem, cudaStream_t st, const Args& a, const moe_norm_desc& d) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3(grid), dim3(r.threads), smem, st, a, d);
}

constexpr int kOneFwd = 512, kOneBwd = 1024;

template <typename T>
cudaError_t norm_forward(const moe_norm_desc& d, const NormFwd& a, int sms, cudaStream_t st) {
  const RowShape r = row_shape(d.H / RowVec<T>::N, kOneFwd);
  const int grid = std::min(d.T, sms * r.per_sm);
  static std::atomic<bool> one[64], two[64];
  return r.vpt == 1 ? launch_rows(block_norm_kernel<T, 1, 2, 512, 2>, one, grid, r,
                                  ring_bytes(r, 3, 2), st, a, d)
                    : launch_rows(block_norm_kernel<T, 2, 2, 1024, 1>, two, grid, r,
                                  ring_bytes(r, 3, 2), st, a, d);
}

template <typename T>
cudaError_t norm_backward(const moe_norm_desc& d, const NormBwd& a, int grid, cudaStream_t st) {
  const RowShape r = row_shape(d.H / RowVec<T>::N, kOneBwd);
  static std::atomic<bool> one[64], two[64];
  return r.vpt == 1 ? launch_rows(block_norm_backward_kernel<T, 1, 2, 1024, 1>, one, grid, r,
                                  ring_bytes(r, 5, 2), st, a, d)
                    : launch_rows(block_norm_backward_kernel<T, 2, 1, 1024, 1>, two, grid, r,
                                  ring_bytes(r, 5, 1), st, a, d);
}

}  // namespace

// Blocks of the backward pass: each leaves one row of column sums.
int block_norm_backward_grid(const moe_norm_desc& d, int sms) {
  const int nvec = d.H / (d.dtype == MOE_BF16 ? 8 : 4);
  return std::min(d.T, sms * row_shape(nvec, kOneBwd).per_sm);
}

cudaError_t launch_column_sums(const float* parts, int n_blocks, int n_out, int H,
                               const ColumnSums& o, cudaStream_t st) {
  return launch_pdl(column_sums_kernel, dim3((H + 31) / 32, n_out), dim3(1024), 0, st, parts,
                    n_blocks, n_out, H, o);
}

cudaError_t launch_block_norm(const moe_norm_desc& d, const void* h, const void* y,
                              const void* w_post, const void* gate, const void* w_pre,
                              void* h_out, void* x, int sms, cudaStream_t st) {
  const NormFwd a{h, y, w_post, gate, w_pre, h_out, x};
  return d.dtype == MOE_BF16 ? norm_forward<__nv_bfloat16>(d, a, sms, st)
                             : norm_forward<float>(d, a, sms, st);
}

cudaError_t launch_block_norm_backward(const moe_norm_desc& d, const void* d_h_out,
                                       const void* d_x, const void* h_out, const void* y,
                                       const void* w_post, const void* gate, const void* w_pre,
                                       void* d_h, void* d_y, float* d_w_post, void* d_gate,
                                       float* d_w_pre, float* parts, int sms, cudaStream_t st) {
  NormBwd a{d_h_out, d_x, h_out, y, w_post, gate, w_pre, d_h, d_y, d_gate, parts, -1, -1, -1, 0};
  ColumnSums o{};
  if (d_w_post) {
    o.out[a.n_parts] = d_w_post;
    a.at_post = a.n_parts++;
  }
  if (d_gate && d.gate == MOE_GATE_CHANNEL) {
    o.out[a.n_parts] = static_cast<float*>(d_gate);
    a.at_gate = a.n_parts++;
  }
  if (d_w_pre) {
    o.out[a.n_parts] = d_w_pre;
    a.at_pre = a.n_parts++;
  }
  const int grid = block_norm_backward_grid(d, sms);
  if (d.T > 0) {
    const cudaError_t e = d.dtype == MOE_BF16 ? norm_backward<__nv_bfloat16>(d, a, grid, st)
                                              : norm_backward<float>(d, a, grid, st);
    if (e != cudaSuccess) return e;
  }
  if (!a.n_parts) return cudaSuccess;
  return launch_column_sums(parts, grid, a.n_parts, d.H, o, st);
}

}  // namespace moe
