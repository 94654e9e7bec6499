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

// e = exp(-z^2 / 2), and the upper tail of the normal distribution, Phi(-|z|) =
// erfc(x) / 2 with x = |z| / sqrt 2: erfc(x) = t H(t) exp(-x^2), t = 1 / (1 + x / 2).
// H is a degree-8 fit (relative error below 8.2e-8) of erfcx(x) / t over x in [0, 10],
// made for this file. With ex2.approx good to 2^-22 and rcp.approx to 2^-23 the tail
// errs by less than 4.1e-7 absolute, and by 1.4e-6 relative for |z| <= 4, 8e-6 for
// |z| <= 12 (the rounding of z^2 grows with it): what a bf16 result hides.
__device__ __forceinline__ void normal_tail2(float2 z, Pair& e, Pair& q) {
  const Pair zz = pair_of(z.x, z.y);
  const float2 m = floats_of(mul2(mul2(zz, zz), pair_of(-0.72134752044448170368f)));
  const float2 u = floats_of(fma2(pair_of(fabsf(z.x), fabsf(z.y)), pair_of(0.35355339059327376f),
                                  pair_of(1.f)));
  float ex, ey, tx, ty;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ex) : "f"(m.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ey) : "f"(m.y));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(tx) : "f"(u.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ty) : "f"(u.y));
  e = pair_of(ex, ey);
  const Pair t = pair_of(tx, ty);
  Pair h = pair_of(-0.05906904116272926f);
  h = fma2(h, t, pair_of(0.28457534313201904f));
  h = fma2(h, t, pair_of(-0.48720064759254456f));
  h = fma2(h, t, pair_of(0.2780679762363434f));
  h = fma2(h, t, pair_of(-0.026626206934452057f));
  h = fma2(h, t, pair_of(0.2026870846748352f));
  h = fma2(h, t, pair_of(0.24310371279716492f));
  h = fma2(h, t, pair_of(0.282375305891037f));
  h = fma2(h, t, pair_of(0.28208643198013306f));
  q = mul2(mul2(h, t), mul2(e, pair_of(0.5f)));
}

// The activation of two values, to the accuracy of the layer's element type T.
template <typename T, int kAct>
__device__ __forceinline__ float2 linear_act2(float2 z) {
  if (kAct == MOE_ACT_GELU) {
    if (sizeof(T) == 4) return make_float2(gelu_erf(z.x), gelu_erf(z.y));
    Pair e, q2;
    normal_tail2(z, e, q2);
    const float2 q = floats_of(q2);
    return make_float2(z.x * (z.x >= 0.f ? 1.f - q.x : q.x), z.y * (z.y >= 0.f ? 1.f - q.y : q.y));
  }
  // SiLU: exp of a large -z overflows to infinity and the quotient goes to -0
  if (kAct == MOE_ACT_SILU) {
    if (sizeof(T) == 4) return make_float2(z.x / (1.f + expf(-z.x)), z.y / (1.f + expf(-z.y)));
    return make_float2(__fdividef(z.x, 1.f + __expf(-z.x)), __fdividef(z.y, 1.f + __expf(-z.y)));
  }
  return z;
}
template <typename T, int kAct, int N>
__device__ __forceinline__ void linear_act(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 y = linear_act2<T, kAct>(make_float2(v[i], v[i + 1]));
    v[i] = y.x;
    v[i + 1] = y.y;
  }
}

// act'(z) of two values
template <typename T, int kAct>
__device__ __forceinline__ float2 linear_act_grad2(float2 z) {
  if (kAct == MOE_ACT_GELU) {   // Phi(z) + z phi(z)
    constexpr float kInvSqrt2Pi = 0.39894228040143267794f;
    if (sizeof(T) == 4) {
      auto one = [&](float x) {
        return 0.5f * (1.f + erff(x * 0.70710678118654752440f)) +
               x * (kInvSqrt2Pi * expf(-0.5f * x * x));
      };
      return make_float2(one(z.x), one(z.y));
    }
    Pair e, q2;
    normal_tail2(z, e, q2);
    const float2 q = floats_of(q2);
    return floats_of(fma2(pair_of(z.x, z.y), mul2(e, pair_of(kInvSqrt2Pi)),
                          pair_of(z.x >= 0.f ? 1.f - q.x : q.x, z.y >= 0.f ? 1.f - q.y : q.y)));
  }
  if (kAct == MOE_ACT_SILU) {
    auto one = [](float x) {
      const float s = sizeof(T) == 4 ? 1.f / (1.f + expf(-x)) : __fdividef(1.f, 1.f + __expf(-x));
      return s * fmaf(x, 1.f - s, 1.f);
    };
    return make_float2(one(z.x), one(z.y));
  }
  return make_float2(1.f, 1.f);
}

// Finishes N consecutive columns (one 16-byte vector of the element type) of
// one row: v holds the sums, o the element offset of the first column.
template <typename T, int kAct>
__device__ __forceinline__ void linear_finish(const LinearEpilogue& e, size_t o, int col,
                                              float (&v)[RowVec<T>::N]) {
  using V = RowVec<T>;
  float u[V::N];
  if (e.bias) {
    V::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(e.bias) + col), u);
#pragma unroll
    for (int i = 0; i < V::N; ++i) v[i] += u[i];
  }
  if (e.pre) *reinterpret_cast<uint4*>(static_cast<T*>(e.pre) + o) = V::pack(v);
  linear_act<T, kAct>(v);
  if (e.residual) {
    V::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(e.residual) + o), u);
#pragma unroll
    for (int i = 0; i < V::N; ++i) v[i] += u[i];
  }
  *reinterpret_cast<uint4*>(static_cast<T*>(e.out) + o) = V::pack(v);
}

}  // namespace moe
