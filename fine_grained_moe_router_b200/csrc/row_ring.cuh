// Whole rows, one after the other, by a block: what the norms' forward and
// backward kernels share.
#pragma once

#include <atomic>

#include "common.cuh"
#include "launch.cuh"
#include "row_vec.cuh"

namespace moe {
namespace {

// Sums over the block, in a fixed order, in every thread. Two buffers taken in
// turn let one barrier do per reduction: a buffer is written again only after
// every thread has passed the barrier of the reduction in between.
struct SumBuffers {
  float v[2][3 * 32];
};

__device__ __forceinline__ float sum_lanes(float v, int from) {
#pragma unroll
  for (int o = from; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum of the warps' entries j, j + 8, ... of a buffer.
__device__ __forceinline__ float sum_entries(const float* buf, int j, int n_warps) {
  float v = j < n_warps ? buf[j] : 0.f;
  for (j += 8; j < n_warps; j += 8) v += buf[j];
  return v;
}

__device__ __forceinline__ float block_sum(float a, SumBuffers& bufs, int& turn) {
  a = sum_lanes(a, 16);
  const int n_warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (n_warps == 1) return a;
  float* buf = bufs.v[turn ^= 1];
  if (lane == 0) buf[threadIdx.x >> 5] = a;
  __syncthreads();
  return sum_lanes(lane < n_warps ? buf[lane] : 0.f, 16);
}

// Three sums at once: each exchange halves the values a lane carries on, so
// that lanes 0-7 end with a, 8-15 with b and 16-23 with c.
__device__ __forceinline__ void block_sum3(float& a, float& b, float& c, SumBuffers& bufs,
                                           int& turn) {
  const int lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
  const bool hi = lane & 16, second = lane & 8;
  float x = (hi ? c : a) + __shfl_xor_sync(0xffffffffu, hi ? a : c, 16);
  float y = (hi ? 0.f : b) + __shfl_xor_sync(0xffffffffu, hi ? b : 0.f, 16);
  x = (second ? y : x) + __shfl_xor_sync(0xffffffffu, second ? x : y, 8);
  x = sum_lanes(x, 4);
  if (n_warps > 1) {
    float* buf = bufs.v[turn ^= 1];
    const int which = lane >> 3;
    if ((lane & 7) == 0 && which < 3) buf[32 * which + (threadIdx.x >> 5)] = x;
    __syncthreads();
    x = sum_lanes(which < 3 ? sum_entries(buf + 32 * which, lane & 7, n_warps) : 0.f, 4);
  }
  a = __shfl_sync(0xffffffffu, x, 0);
  b = __shfl_sync(0xffffffffu, x, 8);
  c = __shfl_sync(0xffffffffu, x, 16);
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
__device__ __forceinline__ void block_factor(Pair (&f)[VPT][RowVec<T>::N / 2], const void* w_post,
                                             const void* gate, const moe_norm_desc& d, int nvec) {
  constexpr int P = RowVec<T>::N / 2;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = v * blockDim.x + threadIdx.x;
    const bool in = i < nvec;
#pragma unroll
    for (int k = 0; k < P; ++k) f[v][k] = pair_of(d.alpha);
    Pair u[P];
    if (in && w_post) {
      unpack_pairs<T>(vec_at(w_post, i), u);
#pragma unroll
      for (int k = 0; k < P; ++k) f[v][k] = mul2(f[v][k], u[k]);
    }
    if (in && d.gate == MOE_GATE_CHANNEL) {
      unpack_pairs<T>(vec_at(gate, i), u);
#pragma unroll
      for (int k = 0; k < P; ++k) f[v][k] = mul2(f[v][k], u[k]);
    }
  }
}

// Launch shape of a row width: `vpt` vectors per thread from more than `one_up_to`
// of them on, and as many resident blocks as `per_sm` threads of an SM hold.
struct RowShape {
  int threads, vpt, blocks_per_sm;
};
inline RowShape row_shape(int nvec, int one_up_to, int per_sm) {
  RowShape r;
  r.vpt = nvec <= one_up_to ? 1 : 2;
  r.threads = ((nvec + r.vpt - 1) / r.vpt + 31) / 32 * 32;
  r.blocks_per_sm = std::max(1, std::min(32, per_sm / r.threads));
  return r;
}
inline size_t ring_bytes(const RowShape& r, int inputs, int stages) {
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

}  // namespace
}  // namespace moe
