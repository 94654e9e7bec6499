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

// Upper tail of the normal distribution, Phi(-|z|) = erfc(x) / 2 with
// x = |z| / sqrt 2: erfc(x) = t H(t) exp(-x^2), t = 1 / (1 + x / 2). H is a
// degree-8 minimax fit (relative error 4.3e-8) of erfcx(x) / t over x in
// [0, 10], made for this file. In fp32 the error is below 1.5e-7 absolute and
// 7e-7 relative for |z| < 4: what a bf16 result hides. `e` is exp(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float z, float e) {
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(fabsf(z), 0.35355339059327376f, 1.f)));
  float h = -0.05906904116272926f;
  h = fmaf(h, t, 0.28457534313201904f);
  h = fmaf(h, t, -0.48720064759254456f);
  h = fmaf(h, t, 0.2780679762363434f);
  h = fmaf(h, t, -0.026626206934452057f);
  h = fmaf(h, t, 0.2026870846748352f);
  h = fmaf(h, t, 0.24310371279716492f);
  h = fmaf(h, t, 0.282375305891037f);
  h = fmaf(h, t, 0.28208643198013306f);
  return 0.5f * (h * t) * e;
}
__device__ __forceinline__ float exp_minus_half_square(float z) {   // exp(-z^2 / 2)
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * z * -0.72134752044448170368f));
  return e;
}

// The activation, to the accuracy of the layer's element type T.
template <typename T, int kAct>
__device__ __forceinline__ float linear_act(float z) {
  if (kAct == MOE_ACT_GELU) {
    if (sizeof(T) == 4) return gelu_erf(z);
    const float q = normal_tail(z, exp_minus_half_square(z));
    return z * (z >= 0.f ? 1.f - q : q);
  }
  // SiLU: exp of a large -z overflows to infinity and the quotient goes to -0
  if (kAct == MOE_ACT_SILU)
    return sizeof(T) == 4 ? z / (1.f + expf(-z)) : __fdividef(z, 1.f + __expf(-z));
  return z;
}

// dz = dy * act'(z)
template <typename T, int kAct>
__device__ __forceinline__ float linear_act_grad(float z) {
  if (kAct == MOE_ACT_GELU) {   // Phi(z) + z phi(z)
    constexpr float kInvSqrt2Pi = 0.39894228040143267794f;
    if (sizeof(T) == 4)
      return 0.5f * (1.f + erff(z * 0.70710678118654752440f)) +
             z * (kInvSqrt2Pi * expf(-0.5f * z * z));
    const float e = exp_minus_half_square(z), q = normal_tail(z, e);
    return fmaf(z, kInvSqrt2Pi * e, z >= 0.f ? 1.f - q : q);
  }
  if (kAct == MOE_ACT_SILU) {
    const float s = sizeof(T) == 4 ? 1.f / (1.f + expf(-z)) : __fdividef(1.f, 1.f + __expf(-z));
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
  for (int i = 0; i < V::N; ++i) v[i] = linear_act<T, kAct>(v[i]);
  if (e.residual) {
    V::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(e.residual) + o), u);
#pragma unroll
    for (int i = 0; i < V::N; ++i) v[i] += u[i];
  }
  *reinterpret_cast<uint4*>(static_cast<T*>(e.out) + o) = V::pack(v);
}

}  // namespace moe
