// Gradients of the norms around a block (block_norm.cu):
// with r = 1/rms, n = v r and d = dL/d(n w),
//   dL/dv = r d w - v r^3 mean(d w v),   dL/dw = sum over tokens of d n.
// The row's first reduction takes both sums of squares and the pre-norm's inner
// product, the second the post-norm's, so the norms' statistics are not kept
// from the forward pass. With g = dL/dh' and n = y r, the column sums of g n
// (times a token or full gate) give both the post-norm's and the channel gate's
// gradient: what they differ by is the same for every row.
//
// Bound by memory at wide rows: 16384 x 4096, bf16, 135 us, 6.0 TB/s; 8192 x 8192
// with a full gate 169 us, 6.4 TB/s. Before: 310 us in one kernel for all forms
// (677 instructions per vector and warp, now 372, and spills), 190 with the row
// held in registers across the reductions (half as many threads an SM), 171 with
// one vector per thread. Of the copy rate 0.85 at 8192 elements (channel gate), 0.77 at
// 7168 and 0.68 at 5120, where a block of fewer threads has an SM to itself, and 0.40
// past 8192 bf16 elements: 64 registers a thread, and spills in the forms with a norm
// before the next block.
#include "common.cuh"
#include "kernels_block.cuh"
#include "launch.cuh"
#include "row_ring.cuh"
#include "row_vec.cuh"

namespace moe {

namespace {

struct NormBwd {
  const void *d_h_out, *d_x, *h_out, *y, *w_post, *gate, *w_pre;
  void *d_h, *d_y, *d_gate;
  float* parts;   // [grid, n_parts, H] column sums of each block
  int at_post, at_gate, at_pre, n_parts;   // -1: not wanted
};

// kPre: norm before the next block. kBlock: 0 no block output, 1 as it is, 2 with a
// norm after the block. kGate: 0 none or per channel, 1 per token, 2 per element.
template <typename T, int VPT, int kStages, int kThreads, bool kPre, int kBlock, int kGate>
__global__ void __launch_bounds__(kThreads)
    block_norm_backward_kernel(const NormBwd a, const moe_norm_desc d) {
  using V = RowVec<T>;
  constexpr int P = V::N / 2;
  constexpr int kIn = 1 + 2 * kPre + (kBlock > 0) + (kGate == 2);
  constexpr int kAtX = 1, kAtH = 2, kAtY = 1 + 2 * kPre, kAtGate = kAtY + 1;
  extern __shared__ uint4 norm_ring[];
  __shared__ SumBuffers sums;
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int nvec = d.H / V::N;
  RowRing<kIn, kStages, VPT> ring;
  ring.nvec = nvec;
  ring.mine = norm_ring + threadIdx.x;
  ring.in[0] = a.d_h_out;
  if constexpr (kPre) {
    ring.in[kAtX] = a.d_x;
    ring.in[kAtH] = a.h_out;
  }
  if constexpr (kBlock > 0) ring.in[kAtY] = a.y;
  if constexpr (kGate == 2) ring.in[kAtGate] = a.gate;
#pragma unroll
  for (int s = 0; s < kStages; ++s) ring.fetch(blockIdx.x + s * gridDim.x, d.T, s);
  Pair wg[VPT][P], wn[VPT][P], s_n[VPT][P], s_pre[VPT][P];
  if constexpr (kBlock > 0) block_factor<T, VPT>(wg, a.w_post, a.gate, d, nvec);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = v * blockDim.x + threadIdx.x;
    if (kPre) unpack_pairs<T>(i < nvec ? vec_at(a.w_pre, i) : make_uint4(0, 0, 0, 0), wn[v]);
#pragma unroll
    for (int k = 0; k < P; ++k) s_n[v][k] = s_pre[v][k] = pair_of(0.f);
  }
  const float inv_h = 1.f / (float)d.H;
  int stage = 0;
  for (int t = blockIdx.x; t < d.T; t += gridDim.x) {
    const size_t row = (size_t)t * nvec;
    ring.wait();
    // the row stays in shared memory and is read again after each reduction:
    // held in registers, it would leave room for half as many threads
    Pair g[VPT][P];
    const Pair zero = pair_of(0.f);
    Pair hh2 = zero, hd2 = zero, yy2 = zero;   // sums of h'^2, h' d_x w, y^2
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      unpack_pairs<T>(a.d_h_out ? *ring.at(stage, 0, v) : make_uint4(0, 0, 0, 0), g[v]);
      Pair p[P], q[P];
      if constexpr (kPre) {
        unpack_pairs<T>(*ring.at(stage, kAtX, v), q);
        unpack_pairs<T>(*ring.at(stage, kAtH, v), p);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          hh2 = fma2(p[k], p[k], hh2);
          hd2 = fma2(mul2(p[k], q[k]), wn[v][k], hd2);
        }
      }
      if constexpr (kBlock == 2) {
        unpack_pairs<T>(*ring.at(stage, kAtY, v), p);
#pragma unroll
        for (int k = 0; k < P; ++k) yy2 = fma2(p[k], p[k], yy2);
      }
    }
    float hh = sum_of(hh2), hd = sum_of(hd2), yy = sum_of(yy2);
    if (kPre)
      block_sum3(hh, hd, yy, sums, turn);
    else if (kBlock == 2)
      yy = block_sum(yy, sums, turn);
    const float r_post = kBlock == 2 ? rsqrtf(yy * inv_h + d.eps) : 1.f;
    if constexpr (kPre) {
      const float r1 = rsqrtf(hh * inv_h + d.eps);
      const Pair r = pair_of(r1), minus_c = pair_of(-hd * inv_h * r1 * r1 * r1);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        Pair p[P], q[P];
        unpack_pairs<T>(*ring.at(stage, kAtX, v), q);
        unpack_pairs<T>(*ring.at(stage, kAtH, v), p);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          s_pre[v][k] = fma2(mul2(p[k], q[k]), r, s_pre[v][k]);
          g[v][k] = fma2(minus_c, p[k], fma2(mul2(q[k], wn[v][k]), r, g[v][k]));
        }
      }
    }
    if (a.d_h)
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int i = v * blockDim.x + threadIdx.x;
        if (i < nvec) put_vec(a.d_h, row + i, pack_pairs<T>(g[v]));
      }
    if constexpr (kBlock > 0) {
      const float gate_t = kGate == 1 ? to_f32(reinterpret_cast<const T*>(a.gate)[t]) : 1.f;
      Pair dot2 = zero;   // sum of g wg y (times a full gate)
      const Pair rn = pair_of(r_post * gate_t);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        Pair y[P];
        unpack_pairs<T>(*ring.at(stage, kAtY, v), y);
        if constexpr (kGate == 2) {
          Pair q[P], dg[P];
          unpack_pairs<T>(*ring.at(stage, kAtGate, v), q);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            dg[k] = mul2(mul2(g[v][k], wg[v][k]), mul2(y[k], pair_of(r_post)));
            g[v][k] = mul2(g[v][k], q[k]);
          }
          const int i = v * blockDim.x + threadIdx.x;
          if (a.d_gate && i < nvec) put_vec(a.d_gate, row + i, pack_pairs<T>(dg));
        }
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const Pair gy = mul2(g[v][k], y[k]);
          s_n[v][k] = fma2(gy, rn, s_n[v][k]);
          dot2 = fma2(gy, wg[v][k], dot2);
        }
      }
      float dot = sum_of(dot2);
      if (kBlock == 2 || kGate == 1) dot = block_sum(dot, sums, turn);
      if (kGate == 1 && a.d_gate && threadIdx.x == 0)
        reinterpret_cast<float*>(a.d_gate)[t] = dot * r_post;
      const Pair minus_c =
          pair_of(kBlock == 2 ? -dot * gate_t * inv_h * r_post * r_post * r_post : 0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int i = v * blockDim.x + threadIdx.x;
        Pair y[P];
        unpack_pairs<T>(*ring.at(stage, kAtY, v), y);
#pragma unroll
        for (int k = 0; k < P; ++k)
          y[k] = fma2(minus_c, y[k], mul2(mul2(g[v][k], wg[v][k]), rn));
        if (a.d_y && i < nvec) put_vec(a.d_y, row + i, pack_pairs<T>(y));
      }
    }
    ring.fetch(t + kStages * gridDim.x, d.T, stage);
    if (++stage == kStages) stage = 0;
  }
  // this block's column sums
  auto put = [&](int at, const Pair (&s)[VPT][P], float alpha, const void* by) {
    if (at < 0) return;
    float* out = a.parts + ((size_t)blockIdx.x * a.n_parts + at) * d.H;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = v * blockDim.x + threadIdx.x;
      if (i >= nvec) continue;
      Pair f[P];
#pragma unroll
      for (int k = 0; k < P; ++k) f[k] = pair_of(1.f);
      if (by) unpack_pairs<T>(vec_at(by, i), f);
#pragma unroll
      for (int k = 0; k < P; k += 2) {
        const float2 lo = floats_of(mul2(mul2(s[v][k], f[k]), pair_of(alpha)));
        const float2 hi = floats_of(mul2(mul2(s[v][k + 1], f[k + 1]), pair_of(alpha)));
        *reinterpret_cast<float4*>(out + (size_t)i * V::N + 2 * k) =
            make_float4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  };
  put(a.at_post, s_n, d.alpha, d.gate == MOE_GATE_CHANNEL ? a.gate : nullptr);
  put(a.at_gate, s_n, d.alpha, a.w_post);
  put(a.at_pre, s_pre, 1.f, nullptr);
}

// out[at][c] = sum over the n_blocks partial rows, in a fixed order: a thread
// takes four columns and every 128th row, then the 128 sums of a column are
// added up. n_blocks rows are a few MB, most of them in L2: enough threads
// have to ask for them at once.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ parts,
                                                           int n_blocks, int n_parts, int H,
                                                           const ColumnSums o) {
  __shared__ float buf[32][129];   // [column][slice], padded against bank conflicts
  pdl_wait();
  pdl_trigger();
  const int four = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + four * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H)   // H is a multiple of 4
#pragma unroll 4
    for (int b = slice; b < n_blocks; b += 128) {
      const float4 v = *reinterpret_cast<const float4*>(
          parts + ((size_t)b * n_parts + blockIdx.y) * H + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  buf[4 * four][slice] = s.x;
  buf[4 * four + 1][slice] = s.y;
  buf[4 * four + 2][slice] = s.z;
  buf[4 * four + 3][slice] = s.w;
  // a warp per column: four of the 128 sums in each lane, then the lanes
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;   // warp = column
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) v += buf[warp][lane + 32 * i];
  v = sum_lanes(v, 16);
  if (lane == 0 && blockIdx.x * 32 + warp < H) o.out[blockIdx.y][blockIdx.x * 32 + warp] = v;
}

// Vectors per thread: the work of a row that does not go with its width (sums
// over the block, addresses, waiting) is shared by twice the elements at two.
constexpr int kOneUpTo = 128;
constexpr int kThreadsPerSm = 512;

template <typename T, bool kPre, int kBlock, int kGate>
cudaError_t launch_form(const moe_norm_desc& d, const NormBwd& a, int grid, cudaStream_t st) {
  const RowShape r = row_shape(d.H / RowVec<T>::N, kOneUpTo, kThreadsPerSm);
  constexpr int kIn = 1 + 2 * kPre + (kBlock > 0) + (kGate == 2);
  static std::atomic<bool> set[3][64];
  if (r.vpt == 1)
    return launch_rows(block_norm_backward_kernel<T, 1, 2, 128, kPre, kBlock, kGate>, set[0],
                       grid, r, ring_bytes(r, kIn, 2), st, a, d);
  if (r.threads <= 512)
    return launch_rows(block_norm_backward_kernel<T, 2, 2, 512, kPre, kBlock, kGate>, set[1],
                       grid, r, ring_bytes(r, kIn, 2), st, a, d);
  // the widest rows: one row ahead has to do
  return launch_rows(block_norm_backward_kernel<T, 2, 1, 1024, kPre, kBlock, kGate>, set[2], grid,
                     r, ring_bytes(r, kIn, 1), st, a, d);
}

template <typename T, bool kPre, int kBlock>
cudaError_t launch_gate(const moe_norm_desc& d, const NormBwd& a, int grid, cudaStream_t st) {
  if (d.gate == MOE_GATE_TOKEN) return launch_form<T, kPre, kBlock, 1>(d, a, grid, st);
  if (d.gate == MOE_GATE_FULL) return launch_form<T, kPre, kBlock, 2>(d, a, grid, st);
  return launch_form<T, kPre, kBlock, 0>(d, a, grid, st);
}

template <typename T>
cudaError_t norm_backward(const moe_norm_desc& d, const NormBwd& a, int grid, cudaStream_t st) {
  if (!a.y)
    return a.w_pre ? launch_form<T, true, 0, 0>(d, a, grid, st)
                   : launch_form<T, false, 0, 0>(d, a, grid, st);
  if (a.w_post)
    return a.w_pre ? launch_gate<T, true, 2>(d, a, grid, st)
                   : launch_gate<T, false, 2>(d, a, grid, st);
  return a.w_pre ? launch_gate<T, true, 1>(d, a, grid, st) : launch_gate<T, false, 1>(d, a, grid, st);
}

}  // namespace

// Blocks of the backward pass. Each leaves a row of column sums, so that a block
// should take more than one row; but a row after the other is a chain of trips to
// memory (777 x 1004 fp32: 12.8 us with eight rows per block at least, 9.8 with
// two).
int block_norm_backward_grid(const moe_norm_desc& d, int sms) {
  const int nvec = d.H / (d.dtype == MOE_BF16 ? 8 : 4);
  const RowShape r = row_shape(nvec, kOneUpTo, kThreadsPerSm);
  return std::min(d.T, std::max(sms, std::min(sms * r.blocks_per_sm, d.T / 2)));
}

cudaError_t launch_column_sums(const float* parts, int n_blocks, int n_out, int H,
                               const ColumnSums& o, cudaStream_t st) {
  return launch_pdl(column_sums_kernel, dim3((H + 31) / 32, n_out), dim3(1024), 0, st, parts,
                    n_blocks, n_out, H, o);
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
