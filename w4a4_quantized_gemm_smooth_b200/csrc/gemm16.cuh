// Shared by the 16-bit product kernels: operands, descriptors, the epilogue's
// arithmetic.
#pragma once

#include "gemm_common.cuh"
#include "ops16.h"

#include <cuda_fp16.h>

#include <type_traits>

namespace svdq {

// Sticky operator error word of the current device (defined in linear16.cu).
int* op_err_address();

constexpr int G_BK = 64;            // reduction elements per stage (128 bytes)

// What a product does with its sums: out = epi(sums + bias) + res, and
// pre = sums + bias.
struct G16Out {
  const uint16_t* bias;    // [N] or null
  const uint16_t* res;     // [M][ldr] or null
  uint16_t* out;           // [M][ldo]
  uint16_t* pre;           // [M][ldp] or null
  long long ldr, ldo, ldp;
  int M, N;
  int epilogue;
  int bf16;
};

// One product as its kernel gets it.  A launch carries one, or the two
// gradients of a layer: their tiles fill the GPU together.
struct alignas(64) G16Problem {
  CUtensorMap a, b, y, r;
  G16Out o;
  int kblocks;
  int tiles_m, tiles_n, tiles;
  int a_bytes;             // bytes of A that arrive per stage
};

// Shared-memory descriptor of a 128-byte-swizzled operand tile.
//   K-major: rows of 128 bytes (64 reduction elements), 8-row atoms of 1 KB
//     (stride 1 KB); 16 reduction elements further is 32 bytes further.
//   MN-major: 64-wide boxes of 64 reduction rows of 128 bytes, atoms of 8
//     reduction rows (stride 1 KB), the next 64 rows of the operand one box
//     (8 KB) on; 16 reduction elements further is 2 KB further.
__device__ __forceinline__ uint64_t g_sdesc(uint32_t saddr, bool mn) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(mn ? 8192 >> 4 : 1) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// The descriptor's step for 16 reduction elements.
__device__ __forceinline__ uint64_t g_kstep(bool mn) { return mn ? 2048 >> 4 : 32 >> 4; }

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

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float ex2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Minimum and maximum that keep NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// For pairs: a = min(|x|, 32), e = exp(-x^2 / 2) and h = erfc(|x| / sqrt 2) / 2
// as e times a polynomial in t = 1 / (1 + z / 2), z = |x| / sqrt 2.  Its
// coefficients are a minimax fit (a linear program over z <= 9.4, where e
// leaves fp32) of the larger of the absolute error over 1e-7 and the relative
// one over 2e-5; in fp32 h is off by at most 2e-7 and by 1.5e-5 of itself, so
// that also the far negative side, where GELU is x h, is right to its own
// 16-bit step.  The epilogue's erff costs as much as the products of a short
// reduction; this form is a third of it.
struct GaussTail {
  float2 a, e, h;
};
__device__ __forceinline__ GaussTail gauss_tail(float2 x) {
  GaussTail g;
  g.a = make_float2(min_nan(fabsf(x.x), 32.0f), min_nan(fabsf(x.y), 32.0f));
  const float2 z = __fmul2_rn(g.a, make_float2(0.70710678f, 0.70710678f));
  const float2 d = __ffma2_rn(z, make_float2(0.5f, 0.5f), make_float2(1.0f, 1.0f));
  const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  const float2 q = __fmul2_rn(__fmul2_rn(g.a, make_float2(-0.72134752f, -0.72134752f)), g.a);
  g.e = make_float2(ex2_approx(q.x), ex2_approx(q.y));
  auto c = [](float v) { return make_float2(v, v); };
  float2 p = __ffma2_rn(t, c(0.0436265685f), c(-0.175381176f));
  p = __ffma2_rn(p, t, c(0.188301504f));
  p = __ffma2_rn(p, t, c(0.0251118732f));
  p = __ffma2_rn(p, t, c(0.13775973f));
  p = __ffma2_rn(p, t, c(0.139472375f));
  p = __ffma2_rn(p, t, c(0.141109165f));
  g.h = __fmul2_rn(__fmul2_rn(p, t), g.e);
  return g;
}

// For pairs: a = x clamped to +-128, t = exp(-|a|), at = a t and q = 1 / (1 + t),
// of which x / (1 + exp(-x)) is x q or, for x < 0, a t q.  1 + t lies in [1, 2],
// and t is the square of exp(-|a| / 2), by which `at` is formed without t, so
// nothing overflows and the far negative side keeps its digits down to the
// least number of the 16-bit type: a quotient by 1 + exp(-x) gave 0 from -87.4
// on.  The exponential's argument, up to 128, in fp32 makes t right to 2^-17.
struct LogisticTail {
  float2 t, at, q;
};
__device__ __forceinline__ LogisticTail logistic_tail(float2 x) {
  LogisticTail g;
  const float2 a = make_float2(max_nan(min_nan(x.x, 128.0f), -128.0f), max_nan(min_nan(x.y, 128.0f), -128.0f));
  const float2 z = __fmul2_rn(make_float2(fabsf(a.x), fabsf(a.y)), make_float2(-0.72134752f, -0.72134752f));
  const float2 h = make_float2(ex2_approx(z.x), ex2_approx(z.y));
  g.t = __fmul2_rn(h, h);
  g.at = __fmul2_rn(__fmul2_rn(a, h), h);
  const float2 d = __fadd2_rn(g.t, make_float2(1.0f, 1.0f));
  g.q = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  return g;
}

// The activation of two sums: GELU is x (1 - h) or, for x < 0, x h, that is
// max(x, 0) - |x| h (|x| clamped where h is 0, so that infinity stays); SiLU
// is x / (1 + exp(-x)).
__device__ __forceinline__ float2 g_act2(float2 x, int epilogue) {
  if (epilogue == SVDQ_EPI_GELU) {
    const GaussTail g = gauss_tail(x);
    return __ffma2_rn(make_float2(-g.a.x, -g.a.y), g.h, make_float2(max_nan(x.x, 0.0f), max_nan(x.y, 0.0f)));
  }
  if (epilogue == SVDQ_EPI_SILU) {
    const LogisticTail g = logistic_tail(x);
    return __fmul2_rn(make_float2(x.x >= 0.0f ? x.x : g.at.x, x.y >= 0.0f ? x.y : g.at.y), g.q);
  }
  return x;
}
// Its derivative: GELU's is Phi(x) + x phi(x), with Phi = 1 - h, or h for x < 0;
// SiLU's s + x s (1 - s) for s = 1 / (1 + exp(-x)), where s is q, or t q for
// x < 0, and s (1 - s) is t q^2 on both sides.
__device__ __forceinline__ float2 g_act_grad2(float2 x, int epilogue) {
  if (epilogue == SVDQ_EPI_GELU) {
    const GaussTail g = gauss_tail(x);
    const float2 u = __ffma2_rn(g.h, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
    const float2 up = make_float2(x.x < 0.0f ? g.h.x : u.x, x.y < 0.0f ? g.h.y : u.y);
    const float2 s = make_float2(copysignf(g.a.x, x.x), copysignf(g.a.y, x.y));
    return __ffma2_rn(__fmul2_rn(s, make_float2(0.39894228f, 0.39894228f)), g.e, up);
  }
  const LogisticTail g = logistic_tail(x);
  const float2 u = __fmul2_rn(g.t, g.q);
  const float2 s = make_float2(x.x < 0.0f ? u.x : g.q.x, x.y < 0.0f ? u.y : g.q.y);
  return __ffma2_rn(__fmul2_rn(g.at, g.q), g.q, s);
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

// Bounded wait of these kernels: polls (a sleeping wait wakes late, which a
// short product feels at every stage), looks at the clock now and then.
// Returns false once LIMIT_NS has passed or another thread of the CTA has
// given up.
__device__ __forceinline__ bool g_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u) {
      if (*abort_flag) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > LIMIT_NS) {
        *abort_flag = 1;
        atomicExch(err, SVDQ_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void prefetch_map(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(tmap) : "memory");
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

// ---- epilogue of one box: 32 rows (a lane each) by 32 columns from col0 ----
// r: the sums; bias: 32 floats in shared memory; place: the box's 2 KB in
// shared memory (64-byte rows, 64-byte swizzle), which holds the residual's
// box when there is one and receives the output.  boxed: the box leaves by a
// TMA store, which writes whole 16-byte pieces; a ragged last box is stored
// from here element by element instead.
__device__ __forceinline__ bool g_boxed(const G16Out& p, int col0) {
  return p.N % 8 == 0 || col0 + 32 <= p.N;
}
template <int EPI, bool BF16>
__device__ __forceinline__ void g_epilogue_box_as(const G16Out& p, const uint32_t (&r)[32],
                                                  const float* bias, uint8_t* place, int lane,
                                                  int row, int col0, bool boxed) {
  constexpr bool bf16 = BF16;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int col = col0 + 8 * u;
    float2 v[4];
    const float4 b0 = lds128(smem_u32(bias + 8 * u)), b1 = lds128(smem_u32(bias + 8 * u + 4));
    const float2 bv[4] = {{b0.x, b0.y}, {b0.z, b0.w}, {b1.x, b1.y}, {b1.z, b1.w}};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = __fadd2_rn(make_float2(__uint_as_float(r[8 * u + 2 * e]), __uint_as_float(r[8 * u + 2 * e + 1])),
                        bv[e]);
    uint32_t o[4];
    if (p.pre) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack2(v[e], bf16);
      if (row < p.M && col < p.N)
        store8(p.pre + (long long)row * p.ldp, col, p.N, make_uint4(o[0], o[1], o[2], o[3]));
    }
    if constexpr (EPI != SVDQ_EPI_NONE) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = g_act2(v[e], EPI);
    }
    uint4* at = reinterpret_cast<uint4*>(place + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4));
    if (p.res) {
      const uint4 rr = *at;
      const uint32_t rw[4] = {rr.x, rr.y, rr.z, rr.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __fadd2_rn(v[e], unpack2(rw[e], bf16));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack2(v[e], bf16);
    const uint4 o4 = make_uint4(o[0], o[1], o[2], o[3]);
    if (boxed)
      *at = o4;
    else if (row < p.M && col < p.N)
      store8(p.out + (long long)row * p.ldo, col, p.N, o4);
  }
}

__device__ __forceinline__ void g_epilogue_box(const G16Out& p, const uint32_t (&r)[32],
                                               const float* bias, uint8_t* place, int lane,
                                               int row, int col0, bool boxed) {
  auto as = [&](auto epi) {
    constexpr int EPI = decltype(epi)::value;
    if (p.bf16)
      g_epilogue_box_as<EPI, true>(p, r, bias, place, lane, row, col0, boxed);
    else
      g_epilogue_box_as<EPI, false>(p, r, bias, place, lane, row, col0, boxed);
  };
  if (p.epilogue == SVDQ_EPI_GELU)
    as(std::integral_constant<int, SVDQ_EPI_GELU>());
  else if (p.epilogue == SVDQ_EPI_SILU)
    as(std::integral_constant<int, SVDQ_EPI_SILU>());
  else
    as(std::integral_constant<int, SVDQ_EPI_NONE>());
}

// Eight sums of one row, columns [col, col + 8) (col a multiple of 8, row < M).
__device__ __forceinline__ void g_epilogue_row(const G16Out& p, float2 (&v)[4], int row, int col) {
  const bool bf16 = p.bf16 != 0;
  auto add8 = [&](uint4 q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __fadd2_rn(v[e], unpack2(w[e], bf16));
  };
  auto store = [&](uint16_t* base, long long ld) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack2(v[e], bf16);
    store8(base + (long long)row * ld, col, p.N, make_uint4(o[0], o[1], o[2], o[3]));
  };
  uint4 res = make_uint4(0, 0, 0, 0);
  if (p.res) res = load8(p.res + (long long)row * p.ldr, col, p.N);
  if (p.bias) add8(load8(p.bias, col, p.N));
  if (p.pre) store(p.pre, p.ldp);
  if (p.epilogue != SVDQ_EPI_NONE) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = g_act2(v[e], p.epilogue);
  }
  if (p.res) add8(res);
  store(p.out, p.ldo);
}

// Cluster helpers.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of the same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
__device__ __forceinline__ float lds32_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// Output tile of index t: bands of 8 row tiles, walked column by column, so
// that the tiles at work together share A and B in L2.
struct TilePos {
  int m, n;
};
__device__ __forceinline__ TilePos tile_pos(int t, int tiles_m, int tiles_n) {
  constexpr int BAND = 8;
  const int per = BAND * tiles_n;
  const int band = t / per, r = t - band * per;
  const int rows = min(BAND, tiles_m - band * BAND);
  return {band * BAND + r % rows, r / rows};
}

// What a launch computes.  The kernels know the operands' majors from the
// place of a problem: Forward has one, both operands K-major; Gradients has
// dX (A K-major, B MN-major) at 0 and dW (both MN-major) at 1, of which one
// may be missing (A.p null).  Descriptors of the MMAs are uniform this way,
// which their issue rate needs.
enum class G16Kind { Forward, Gradients };
struct G16Launch {
  G16Kind kind;
  Operand A[2], B[2];
  G16Out o[2];
  int bf16;
  int* err;
};

// Both problems of a launch; a missing one has no tiles.
template <typename F>
inline bool make_problems(G16Problem (&p)[2], const G16Launch& l, F&& make) {
  int have = -1;
  for (int i = 0; i < 2; ++i)
    if (l.A[i].p) {
      if (!make(&p[i], l.A[i], l.B[i], l.o[i])) return false;
      have = i;
    }
  if (have < 0) return false;
  for (int i = 0; i < 2; ++i)
    if (!l.A[i].p) {
      p[i] = p[have];
      p[i].tiles = 0;
    }
  return true;
}

// Fills one problem for tiles of bm x bn, of which a CTA loads box_m rows of
// A and box_n of B.  For an A of fewer rows than the box only those arrive
// (K-major: in groups of 8); the others are never used.
inline bool make_problem(G16Problem* p, const Operand& A, const Operand& B, const G16Out& o, int bm,
                         int bn, int box_m, int box_n, bool boxes) {
  const auto dt = o.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  int rows = box_m;
  if (!A.mn && A.rows < box_m) rows = (A.rows + 7) / 8 * 8;
  auto map = [&](CUtensorMap* m, const Operand& x, int box) {
    if (x.mn)
      return make_map(m, x.p, dt, x.rows, x.red, (uint64_t)x.ld * 2, 64, G_BK, CU_TENSOR_MAP_SWIZZLE_128B);
    return make_map(m, x.p, dt, x.red, x.rows, (uint64_t)x.ld * 2, G_BK, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!map(&p->a, A, rows) || !map(&p->b, B, box_n)) return false;
  p->y = p->r = p->a;          // unused without boxes
  if (boxes) {
    if (!make_map(&p->y, o.out, dt, B.rows, A.rows, (uint64_t)o.ldo * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
      return false;
    if (o.res && !make_map(&p->r, o.res, dt, B.rows, A.rows, (uint64_t)o.ldr * 2, 32, 32,
                           CU_TENSOR_MAP_SWIZZLE_64B))
      return false;
  }
  const long long tm = ((long long)A.rows + bm - 1) / bm, tn = ((long long)B.rows + bn - 1) / bn;
  if (tm * tn > 0x0FFFFFFF) return false;
  p->o = o;
  p->o.M = A.rows;
  p->o.N = B.rows;
  p->kblocks = (int)(((long long)A.red + G_BK - 1) / G_BK);
  p->tiles_m = (int)tm;
  p->tiles_n = (int)tn;
  p->tiles = (int)(tm * tn);
  p->a_bytes = A.mn ? box_m * 128 : rows * 128;
  return true;
}

// pair: 256 x bn tiles on CTA pairs; split: 128 x bn tiles, the reduction
// divided over a cluster of `splits` CTAs.
cudaError_t launch_gemm16_pair(const G16Launch& l, int bn, cudaStream_t st);
cudaError_t launch_gemm16_split(const G16Launch& l, int bn, int splits, cudaStream_t st);

// The forward product of up to THIN_ROWS rows, bound by reading W.
constexpr int THIN_ROWS = 16;
cudaError_t launch_thin16(const void* X, long long ldx, const void* W, long long ldw, int K,
                          const G16Out& o, cudaStream_t st);

// The gradients of up to THIN_BWD_ROWS rows: x and dw, w and dx are null together.
constexpr int THIN_BWD_ROWS = 8;
struct ThinBwdCall {
  const void *dy, *p, *x, *w;
  void *dx, *dw, *db, *workspace;
  long long lddy, ldp, ldx, ldw, lddx, lddw;
  int M, K, N, epilogue, bf16;
};
size_t thin16_bwd_workspace(int M, int K, int N);
cudaError_t launch_thin16_bwd(const ThinBwdCall& c, cudaStream_t st);

// out [rows][ldo] = the sums over `blocks` of part [block][rows][pitch], in order.
cudaError_t launch_join(const float* part, int blocks, int rows, int cols, int pitch, uint16_t* out,
                        long long ldo, int bf16, cudaStream_t st);

}  // namespace svdq
