// Epilogue arithmetic of the linear layer, shared by its tensor-core and
// CUDA-core kernels: y = act(z) + r, z = sum + bias.
#pragma once

#include "common.cuh"
#include "row_vec.cuh"

namespace moe {

// Where an output tile goes. All rows have stride `ld` elements.
struct LinearEpilogue {
  void* out;              // [M, ld]
  const void* bias;       // [ld] or null
  const void* residual;   // [M, ld] or null; may be `out`
  void* pre;              // [M, ld] or null: z
  int act;                // moe_act
};

template <int kAct>
__device__ __forceinline__ float linear_act(float z) {
  if (kAct == MOE_ACT_GELU) return gelu_erf(z);
  // SiLU: exp of a large -z overflows to infinity and the quotient goes to -0
  if (kAct == MOE_ACT_SILU) return z / (1.f + expf(-z));
  return z;
}

// dz = dy * act'(z)
template <int kAct>
__device__ __forceinline__ float linear_act_grad(float z) {
  if (kAct == MOE_ACT_GELU)   // Phi(z) + z phi(z)
    return 0.5f * (1.f + erff(z * 0.70710678118654752440f)) +
           z * (0.39894228040143267794f * expf(-0.5f * z * z));
  if (kAct == MOE_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-z));
    return s * fmaf(z, 1.f - s, 1.f);
  }
  return 1.f;
}

// Finishes N consecutive columns (one 16-byte vector of the element type) of
// one row: v holds the sums, o the element offset of the first column.
template <typename T, int kAct>
__device__ __forceinline__ void linear_finish(const LinearEpilogue& e, size_t o, int col,
                                              float* v) {
  using V = RowVec<T>;
  float u[V::N];
  if (e.bias) {
    V::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(e.bias) + col), u);
#pragma unroll
    for (int i = 0; i < V::N; ++i) v[i] += u[i];
  }
  if (e.pre) *reinterpret_cast<uint4*>(static_cast<T*>(e.pre) + o) = V::pack(v);
#pragma unroll
  for (int i = 0; i < V::N; ++i) v[i] = linear_act<kAct>(v[i]);
  if (e.residual) {
    V::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(e.residual) + o), u);
#pragma unroll
    for (int i = 0; i < V::N; ++i) v[i] += u[i];
  }
  *reinterpret_cast<uint4*>(static_cast<T*>(e.out) + o) = V::pack(v);
}

}  // namespace moe
