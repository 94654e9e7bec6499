// 16-byte vectors of a row in the layer's element types, as fp32 values or pairs.
#pragma once

#include "common.cuh"

namespace moe {

// Pairs of floats: one instruction does two fp32 operations (fma.rn.f32x2).
struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair_of(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Pair pair_of(float a) { return pair_of(a, a); }
__device__ __forceinline__ float2 floats_of(Pair p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

__device__ __forceinline__ float sum_of(Pair p) {
  const float2 f = floats_of(p);
  return f.x + f.y;
}

template <typename T>
struct RowVec;
template <>
struct RowVec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void unpack(const uint4& v, float* f) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = __bfloat1622float2(h[i]);
      f[2 * i] = q.x;
      f[2 * i + 1] = q.y;
    }
  }
  __device__ __forceinline__ static uint4 pack(const float* f) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return v;
  }
};
template <>
struct RowVec<float> {
  static constexpr int N = 4;
  __device__ __forceinline__ static void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ __forceinline__ static uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& v, Pair (&p)[RowVec<T>::N / 2]) {
  float f[RowVec<T>::N];
  RowVec<T>::unpack(v, f);
#pragma unroll
  for (int i = 0; i < RowVec<T>::N / 2; ++i) p[i] = pair_of(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const Pair (&p)[RowVec<T>::N / 2]) {
  float f[RowVec<T>::N];
#pragma unroll
  for (int i = 0; i < RowVec<T>::N / 2; ++i) {
    const float2 q = floats_of(p[i]);
    f[2 * i] = q.x;
    f[2 * i + 1] = q.y;
  }
  return RowVec<T>::pack(f);
}

}  // namespace moe
