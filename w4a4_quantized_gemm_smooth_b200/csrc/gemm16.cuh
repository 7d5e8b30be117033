// Shared by the 16-bit product kernels: operands, descriptors, the epilogue's
// arithmetic.
#pragma once

#include "gemm_common.cuh"
#include "ops16.h"

#include <cuda_fp16.h>

namespace svdq {

// Sticky operator error word of the current device (defined in linear16.cu).
int* op_err_address();

constexpr int G_BK = 64;            // reduction elements per stage (128 bytes)

struct G16Args {
  const uint16_t* bias;    // [N] or null
  const uint16_t* res;     // [M][ldr] or null
  uint16_t* out;           // [M][ldo]
  uint16_t* pre;           // [M][ldp] or null
  long long ldr, ldo, ldp;
  int M, N;
  int kblocks;
  int tiles_m, tiles_n, num_tiles;
  int epilogue;
  int bf16;
  int* err;
};

// Shared-memory descriptor of a 128-byte-swizzled operand tile.
//   K-major: rows of 128 bytes (64 reduction elements), 8-row atoms of 1 KB
//     (stride 1 KB); 16 reduction elements further is 32 bytes further.
//   MN-major: 64-wide boxes of 64 reduction rows of 128 bytes, atoms of 8
//     reduction rows (stride 1 KB), the next 64 rows of the operand one box
//     (8 KB) on; 16 reduction elements further is 2 KB further.
template <bool MN>
__device__ __forceinline__ uint64_t g_sdesc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(MN ? 8192 >> 4 : 1) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
template <bool MN>
constexpr uint64_t G_KSTEP = MN ? 2048 >> 4 : 32 >> 4;    // 16 reduction elements

// kind::f16 instruction descriptor: fp16 or bf16 operands, fp32 D, majors.
__device__ __forceinline__ uint32_t g_idesc(int M, int N, bool bf16, bool a_mn, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
         ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ bool g_elect() {
  uint32_t pred = 0;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}\n"
      : "=r"(pred));
  return pred != 0;
}

__device__ __forceinline__ float g_act(float v, int epilogue) {
  if (epilogue == SVDQ_EPI_GELU) return gelu_f(v);
  if (epilogue == SVDQ_EPI_SILU) return v / (1.0f + __expf(-v));
  return v;
}

__device__ __forceinline__ float2 unpack2(uint32_t u, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint32_t pack2(float2 v, bool bf16) {
  if (bf16) return bf16x2_bits(v);
  const __half2 h = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight 16-bit elements [c, c + 8) of a row of n (16-byte aligned, c a
// multiple of 8): one vector, or element by element at the row's end.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int n) {
  if (c + 8 <= n) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < n) w[e >> 1] |= (uint32_t)row[c + e] << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(uint16_t* row, int c, int n, uint4 v) {
  if (c + 8 <= n) {
    *reinterpret_cast<uint4*>(row + c) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < n) row[c + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
}

// An operand as the product sees it: `rows` along its output axis, `red`
// along the reduction; mn: the output axis is the contiguous one.
struct Operand {
  const void* p;
  long long ld;
  int rows, red;
  bool mn;
};

inline bool operand_map(CUtensorMap* m, const Operand& o, int box_rows, bool bf16) {
  const auto dt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (o.mn)
    return make_map(m, o.p, dt, o.rows, o.red, (uint64_t)o.ld * 2, 64, G_BK,
                    CU_TENSOR_MAP_SWIZZLE_128B);
  return make_map(m, o.p, dt, o.red, o.rows, (uint64_t)o.ld * 2, G_BK, box_rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}


// The product kernels' launchers.  Y = epi(A B^T + bias) + R with the output
// M = A.rows by N = B.rows and the reduction A.red = B.red.
cudaError_t launch_gemm16_pair(const Operand& A, const Operand& B, const G16Args& a, cudaStream_t st);

}  // namespace svdq
