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

// Pair j of a vector as two fp32 values, and back (rounded to nearest).
template <int BYTES>
__device__ __forceinline__ float2 get2(const Pack<__nv_bfloat16, BYTES>& v, int j) {
  const uint32_t u = reinterpret_cast<const uint32_t*>(&v)[j];
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
template <int BYTES>
__device__ __forceinline__ float2 get2(const Pack<__half, BYTES>& v, int j) {
  return __half22float2(reinterpret_cast<const __half2*>(&v)[j]);
}
template <int BYTES>
__device__ __forceinline__ float2 get2(const Pack<float, BYTES>& v, int j) {
  return make_float2(v.e[2 * j], v.e[2 * j + 1]);
}
template <int BYTES>
__device__ __forceinline__ void set2(Pack<__nv_bfloat16, BYTES>& v, int j, float2 f) {
  reinterpret_cast<__nv_bfloat162*>(&v)[j] = __float22bfloat162_rn(f);
}
template <int BYTES>
__device__ __forceinline__ void set2(Pack<__half, BYTES>& v, int j, float2 f) {
  reinterpret_cast<__half2*>(&v)[j] = __float22half2_rn(f);
}
template <int BYTES>
__device__ __forceinline__ void set2(Pack<float, BYTES>& v, int j, float2 f) {
  v.e[2 * j] = f.x;
  v.e[2 * j + 1] = f.y;
}

// V elements of a row as 16-byte vectors (V sizeof(T) = 16 or 32).
template <typename T, int V>
struct RowVec {
  static constexpr int P = 16 / (int)sizeof(T);
  static constexpr int N = V / P;
  Pack<T, 16> q[N];
  __device__ __forceinline__ float2 get(int j) const { return get2(q[j / (P / 2)], j % (P / 2)); }
  __device__ __forceinline__ void set(int j, float2 f) { set2(q[j / (P / 2)], j % (P / 2), f); }
};

template <typename T, int V>
__device__ __forceinline__ RowVec<T, V> read_vec(const uint4* src, int pitch) {
  RowVec<T, V> v;
#pragma unroll
  for (int k = 0; k < RowVec<T, V>::N; ++k) reinterpret_cast<uint4*>(v.q)[k] = src[k * pitch];
  return v;
}
// Elements [c, c + V) of a row of n (16-byte aligned rows, c a multiple of
// V); zeros past the row.
template <typename T, int V>
__device__ __forceinline__ RowVec<T, V> load_vec(const T* row, int c, int n) {
  RowVec<T, V> v;
  if (c + V <= n) {
#pragma unroll
    for (int k = 0; k < RowVec<T, V>::N; ++k) v.q[k] = reinterpret_cast<const Pack<T, 16>*>(row + c)[k];
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      v.q[e / RowVec<T, V>::P].e[e % RowVec<T, V>::P] = c + e < n ? row[c + e] : Elem<T>::from_f(0.0f);
  }
  return v;
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* row, int c, int n, const RowVec<T, V>& v) {
  if (c + V <= n) {
#pragma unroll
    for (int k = 0; k < RowVec<T, V>::N; ++k) reinterpret_cast<Pack<T, 16>*>(row + c)[k] = v.q[k];
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e < n) row[c + e] = v.q[e / RowVec<T, V>::P].e[e % RowVec<T, V>::P];
  }
}

// The kernel after this one in the stream may be brought up; and: everything
// before this kernel is done and visible (see launch_op).
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ float2 splat2(float v) { return make_float2(v, v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

}  // namespace svdq
