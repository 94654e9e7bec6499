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
// whole rows, holds the row in registers between its reductions, and keeps the
// weights (the same for every row) in registers over the rows it takes. All
// sums are fp32; h' feeds the second norm before it is rounded to be stored.
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

// Sum of (a, b) over the block, in a fixed order. Two buffers taken in turn let
// one barrier do per reduction: a buffer is written again only after every
// thread has passed the barrier of the reduction in between.
struct SumBuffers {
  float v[2][64];
};
__device__ __forceinline__ float2 block_sum2(float a, float b, SumBuffers& bufs, int& turn) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int n_warps = blockDim.x >> 5;
  if (n_warps == 1) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* buf = bufs.v[turn ^= 1];
  if (lane == 0) {
    buf[2 * warp] = a;
    buf[2 * warp + 1] = b;
  }
  __syncthreads();
  a = lane < n_warps ? buf[2 * lane] : 0.f;
  b = lane < n_warps ? buf[2 * lane + 1] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  return make_float2(a, b);
}

__device__ __forceinline__ uint4 vec_at(const void* p, size_t i) {
  return reinterpret_cast<const uint4*>(p)[i];
}

template <typename T, int VPT, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads)
    block_norm_kernel(const NormFwd a, const moe_norm_desc d) {
  using V = RowVec<T>;
  __shared__ SumBuffers sums;
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int nvec = d.H / V::N;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 wp[VPT], wn[VPT], gc[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = v * blockDim.x + threadIdx.x;
    const bool in = i < nvec;
    wp[v] = in && a.w_post ? vec_at(a.w_post, i) : zero;
    wn[v] = in && a.w_pre ? vec_at(a.w_pre, i) : zero;
    gc[v] = in && d.gate == MOE_GATE_CHANNEL ? vec_at(a.gate, i) : zero;
  }
  const float inv_h = 1.f / (float)d.H;
  for (int t = blockIdx.x; t < d.T; t += gridDim.x) {
    const size_t row = (size_t)t * nvec;
    uint4 hv[VPT], yv[VPT];
    float f[VPT][V::N];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      hv[v] = i < nvec ? vec_at(a.h, row + i) : zero;
      yv[v] = i < nvec && a.y ? vec_at(a.y, row + i) : zero;
    }
    float r_post = 1.f;
    if (a.w_post) {
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        V::unpack(yv[v], f[v]);
#pragma unroll
        for (int k = 0; k < V::N; ++k) ss = fmaf(f[v][k], f[v][k], ss);
      }
      r_post = rsqrtf(block_sum2(ss, 0.f, sums, turn).x * inv_h + d.eps);
    }
    float scale = d.alpha;
    if (d.gate == MOE_GATE_TOKEN) scale *= to_f32(reinterpret_cast<const T*>(a.gate)[t]);
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      V::unpack(hv[v], f[v]);
      if (a.y) {
        float u[V::N], g[V::N];
        V::unpack(yv[v], u);
        if (a.w_post) {
          V::unpack(wp[v], g);
#pragma unroll
          for (int k = 0; k < V::N; ++k) u[k] *= r_post * g[k];
        }
        if (d.gate == MOE_GATE_CHANNEL || d.gate == MOE_GATE_FULL) {
          V::unpack(d.gate == MOE_GATE_CHANNEL ? gc[v] : i < nvec ? vec_at(a.gate, row + i) : zero,
                    g);
#pragma unroll
          for (int k = 0; k < V::N; ++k) u[k] *= g[k];
        }
#pragma unroll
        for (int k = 0; k < V::N; ++k) f[v][k] = fmaf(scale, u[k], f[v][k]);
      }
      if (a.h_out && i < nvec) reinterpret_cast<uint4*>(a.h_out)[row + i] = V::pack(f[v]);
#pragma unroll
      for (int k = 0; k < V::N; ++k) ss = fmaf(f[v][k], f[v][k], ss);
    }
    if (!a.w_pre) continue;
    const float r_pre = rsqrtf(block_sum2(ss, 0.f, sums, turn).x * inv_h + d.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      float g[V::N];
      V::unpack(wn[v], g);
#pragma unroll
      for (int k = 0; k < V::N; ++k) f[v][k] *= r_pre * g[k];
      if (i < nvec) reinterpret_cast<uint4*>(a.x)[row + i] = V::pack(f[v]);
    }
  }
}

// With r = 1/rms and n = v r, d = dL/d(n w): dL/dv = r (d w - n mean(d w n)),
// dL/dw = sum over tokens of d n. The row's first reduction takes both sums of
// squares and the pre-norm's inner product, the second the post-norm's and the
// token gate's, so the norms' statistics are not kept from the forward pass.
template <typename T, int VPT, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads)
    block_norm_backward_kernel(const NormBwd a, const moe_norm_desc d) {
  using V = RowVec<T>;
  __shared__ SumBuffers sums;
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int nvec = d.H / V::N;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const bool channel = d.gate == MOE_GATE_CHANNEL, full = d.gate == MOE_GATE_FULL;
  uint4 wp[VPT], wn[VPT], gc[VPT];
  float s_post[VPT][V::N], s_gate[VPT][V::N], s_pre[VPT][V::N];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = v * blockDim.x + threadIdx.x;
    const bool in = i < nvec;
    wp[v] = in && a.w_post ? vec_at(a.w_post, i) : zero;
    wn[v] = in && a.w_pre ? vec_at(a.w_pre, i) : zero;
    gc[v] = in && channel ? vec_at(a.gate, i) : zero;
#pragma unroll
    for (int k = 0; k < V::N; ++k) s_post[v][k] = s_gate[v][k] = s_pre[v][k] = 0.f;
  }
  const float inv_h = 1.f / (float)d.H;
  for (int t = blockIdx.x; t < d.T; t += gridDim.x) {
    const size_t row = (size_t)t * nvec;
    uint4 gv[VPT], xv[VPT], hv[VPT], yv[VPT], qv[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      const bool in = i < nvec;
      gv[v] = in && a.d_h_out ? vec_at(a.d_h_out, row + i) : zero;
      xv[v] = in && a.w_pre ? vec_at(a.d_x, row + i) : zero;
      hv[v] = in && a.w_pre ? vec_at(a.h_out, row + i) : zero;
      yv[v] = in && a.y ? vec_at(a.y, row + i) : zero;
      qv[v] = in && full ? vec_at(a.gate, row + i) : gc[v];
    }
    float hh = 0.f, hd = 0.f, yy = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float p[V::N], q[V::N], w[V::N];
      if (a.w_pre) {
        V::unpack(hv[v], p);
        V::unpack(xv[v], q);
        V::unpack(wn[v], w);
#pragma unroll
        for (int k = 0; k < V::N; ++k) {
          hh = fmaf(p[k], p[k], hh);
          hd = fmaf(p[k], q[k] * w[k], hd);
        }
      }
      if (a.w_post) {
        V::unpack(yv[v], p);
#pragma unroll
        for (int k = 0; k < V::N; ++k) yy = fmaf(p[k], p[k], yy);
      }
    }
    float r_pre = 0.f, c_pre = 0.f, r_post = 1.f;
    if (a.w_pre) {
      const float2 s = block_sum2(hh, hd, sums, turn);
      r_pre = rsqrtf(s.x * inv_h + d.eps);
      c_pre = s.y * r_pre * r_pre * inv_h;   // mean(d w n) * r = c_pre; n = h r
    }
    if (a.w_post) r_post = rsqrtf(block_sum2(yy, 0.f, sums, turn).x * inv_h + d.eps);
    const float gate_t =
        d.gate == MOE_GATE_TOKEN ? to_f32(reinterpret_cast<const T*>(a.gate)[t]) : 1.f;
    // g = dL/dh'
    float g[VPT][V::N];
    float dot = 0.f, du = 0.f;   // sum d(n) n, and sum of the token gate's products
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      V::unpack(gv[v], g[v]);
      if (a.w_pre) {
        float p[V::N], q[V::N], w[V::N];
        V::unpack(hv[v], p);
        V::unpack(xv[v], q);
        V::unpack(wn[v], w);
#pragma unroll
        for (int k = 0; k < V::N; ++k) {
          s_pre[v][k] = fmaf(q[k], p[k] * r_pre, s_pre[v][k]);
          g[v][k] = fmaf(r_pre, fmaf(q[k], w[k], -p[k] * c_pre), g[v][k]);
        }
      }
      if (a.d_h && i < nvec) reinterpret_cast<uint4*>(a.d_h)[row + i] = V::pack(g[v]);
      if (a.y) {
        float n[V::N], w[V::N], q[V::N], dg[V::N];
        V::unpack(yv[v], n);
        V::unpack(wp[v], w);
        V::unpack(qv[v], q);
#pragma unroll
        for (int k = 0; k < V::N; ++k) {
          g[v][k] *= d.alpha;   // from here on: dL/d(gate * u)
          n[k] *= r_post;
          const float wk = a.w_post ? w[k] : 1.f;
          const float gate = channel || full ? q[k] : gate_t;
          dg[k] = g[v][k] * n[k] * wk;              // dL/dgate of this element
          s_gate[v][k] += dg[k];
          s_post[v][k] = fmaf(g[v][k] * gate, n[k], s_post[v][k]);
          du += dg[k];
          g[v][k] *= gate * wk;                      // dL/dn
          dot = fmaf(g[v][k], n[k], dot);
        }
        if (full && a.d_gate && i < nvec)
          reinterpret_cast<uint4*>(a.d_gate)[row + i] = V::pack(dg);
      }
    }
    if (!a.y) continue;
    const float2 s = block_sum2(dot, du, sums, turn);
    if (d.gate == MOE_GATE_TOKEN && a.d_gate && threadIdx.x == 0)
      reinterpret_cast<float*>(a.d_gate)[t] = s.y;
    const float c_post = a.w_post ? s.x * inv_h : 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      float n[V::N];
      V::unpack(yv[v], n);
#pragma unroll
      for (int k = 0; k < V::N; ++k) n[k] = r_post * fmaf(-n[k] * r_post, c_post, g[v][k]);
      if (a.d_y && i < nvec) reinterpret_cast<uint4*>(a.d_y)[row + i] = V::pack(n);
    }
  }
  // this block's column sums
  auto put = [&](int at, const float (&s)[VPT][V::N]) {
    if (at < 0) return;
    float* out = a.parts + ((size_t)blockIdx.x * a.n_parts + at) * d.H;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      if (i >= nvec) continue;
#pragma unroll
      for (int k = 0; k < V::N; k += 4)
        *reinterpret_cast<float4*>(out + (size_t)i * V::N + k) =
            make_float4(s[v][k], s[v][k + 1], s[v][k + 2], s[v][k + 3]);
    }
  };
  put(a.at_post, s_post);
  put(a.at_gate, s_gate);
  put(a.at_pre, s_pre);
}

// out[at][c] = sum over the n_blocks partial rows, in a fixed order: eight
// strided partial sums, added in order.
__global__ void __launch_bounds__(256) column_sums_kernel(const float* __restrict__ parts,
                                                          int n_blocks, int n_parts, int H,
                                                          const ColumnSums o) {
  __shared__ float buf[8][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < H)
    for (int b = slice; b < n_blocks; b += 8)
      s += parts[((size_t)b * n_parts + blockIdx.y) * H + c];
  buf[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += buf[i][lane];
    o.out[blockIdx.y][c] = s;
  }
}

int row_threads(int nvec, int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; }

template <typename T>
cudaError_t norm_forward(const moe_norm_desc& d, const NormFwd& a, int sms, cudaStream_t st) {
  const int nvec = d.H / RowVec<T>::N;
  const int vpt = nvec <= 256 ? 1 : 2;
  const int threads = row_threads(nvec, vpt);
  const int grid = std::min(d.T, sms * std::max(1, std::min(32, 1536 / threads)));
  return launch_pdl(vpt == 1 ? block_norm_kernel<T, 1, 256> : block_norm_kernel<T, 2, 1024>, dim3(grid),
                    dim3(threads), 0, st, a, d);
}

template <typename T>
cudaError_t norm_backward(const moe_norm_desc& d, const NormBwd& a, int grid, cudaStream_t st) {
  const int nvec = d.H / RowVec<T>::N;
  const int vpt = nvec <= 512 ? 1 : 2;
  return launch_pdl(
      vpt == 1 ? block_norm_backward_kernel<T, 1, 512> : block_norm_backward_kernel<T, 2, 1024>, dim3(grid),
      dim3(row_threads(nvec, vpt)), 0, st, a, d);
}

}  // namespace

// Blocks of the backward pass: each leaves one row of column sums.
int block_norm_backward_grid(const moe_norm_desc& d, int sms) {
  const int nvec = d.H / (d.dtype == MOE_BF16 ? 8 : 4);
  const int threads = row_threads(nvec, nvec <= 512 ? 1 : 2);
  return std::min(d.T, sms * std::max(1, std::min(16, 1024 / threads)));
}

cudaError_t launch_column_sums(const float* parts, int n_blocks, int n_out, int H,
                               const ColumnSums& o, cudaStream_t st) {
  return launch_pdl(column_sums_kernel, dim3((H + 31) / 32, n_out), dim3(256), 0, st, parts,
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
