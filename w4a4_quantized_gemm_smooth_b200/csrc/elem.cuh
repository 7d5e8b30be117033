// Element types of the 16-bit operators: conversions between bf16, fp16 or
// fp32 storage and fp32 arithmetic, 16 bytes at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace svdq {

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float to_f(float v) { return v; }
  static __device__ __forceinline__ float from_f(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
};

// BYTES consecutive bytes as an aligned vector of T.
template <typename T, int BYTES>
struct alignas(BYTES) Pack {
  static constexpr int N = BYTES / (int)sizeof(T);
  T e[N];
};

// Elements [i0, i0 + V) of a row of `n` elements; zeros past n.  The row is
// 16-byte aligned and i0 a multiple of V, V * sizeof(T) a multiple of 16.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int i0, int n, float (&v)[V]) {
  constexpr int P = 16 / (int)sizeof(T);
  static_assert(V % P == 0, "whole 16-byte vectors");
  if (i0 + V <= n) {
#pragma unroll
    for (int j = 0; j < V; j += P) {
      const Pack<T, 16> x = *reinterpret_cast<const Pack<T, 16>*>(row + i0 + j);
#pragma unroll
      for (int e = 0; e < P; ++e) v[j + e] = Elem<T>::to_f(x.e[e]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = i0 + j < n ? Elem<T>::to_f(row[i0 + j]) : 0.0f;
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* row, int i0, int n, const float (&v)[V]) {
  constexpr int P = 16 / (int)sizeof(T);
  if (i0 + V <= n) {
#pragma unroll
    for (int j = 0; j < V; j += P) {
      Pack<T, 16> x;
#pragma unroll
      for (int e = 0; e < P; ++e) x.e[e] = Elem<T>::from_f(v[j + e]);
      *reinterpret_cast<Pack<T, 16>*>(row + i0 + j) = x;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (i0 + j < n) row[i0 + j] = Elem<T>::from_f(v[j]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

}  // namespace svdq
