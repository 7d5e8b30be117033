// Layer norm with a scale and a shift per group of rows, and its gradients.
//
// A row belongs to one team (a quarter of a warp for the shortest rows, a
// warp, or a block of 128, 256 or 512 threads for long ones), and a team walks
// over rows of one group, one to four at a time.  Each thread copies its own
// 16-byte vectors of the next rows to its own places in shared memory
// (cp.async, no barrier), so that the bytes in flight do not depend on the
// registers that a row needs; the group's scale (with its offset) and shift
// wait there too, in fp32, converted once per block.  Arithmetic runs on pairs
// (packed fp32 instructions), which keeps it below the memory time.
//
// Forward: the variance is the two-pass one, sum (x - mu)^2 in fp32 after the
// mean, from registers (no cancellation for rows with a large mean).  The mean
// is the sum times 1 / K in two floats, so that it is the quotient's nearest
// value: a step off it would stand in every difference, and rstd multiplies it
// (by up to 1000 with eps = 1e-6, in rows that hardly vary).  A division cost
// short rows 10 % (73941 x 65 fp32 15.0 to 16.5 us), this nothing; adding up the
// differences to mend also the sum's own rounding cost up to 47 %.
// 16384 x 1152 bf16 in four groups: 17.0 us, 4.4 TB/s (a plain copy: 13.7 us);
// bound by the chain sum - difference - sum - output of the few rows that fit
// an SM's registers at a time.
//
// Backward: a thread owns fixed columns; their sums of dy xhat and dy stay in
// its registers over all the rows of the team and are joined at the end:
// teams of a block in shared memory, blocks of a group through fp32 partials
// in the workspace, summed in block order by a second kernel.  X and dY are
// read once.  16384 x 1152 bf16: 28.3 us, 4.0 TB/s; 4608 x 4608 fp16: 32.9 us,
// 3.9 TB/s.  The columns' sums take the registers that more rows would need;
// two warps per row instead of one (48 sums a thread instead of 80) measured
// the same, so did one row at a time with three blocks per SM.
#include <climits>
#include <cmath>
#include <type_traits>

#include <math_constants.h>

#include "elem.cuh"
#include "gemm_common.cuh"
#include "ops16.h"

namespace svdq {
namespace {

struct NormArgs {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  long long ldx, ldw, ldb, ldy;
  int M, K, rows_per_group;  // rows_per_group >= 1 here
  int splits;                // blocks per group
  float w0, eps;
  float inv_k, inv_k_rest;   // 1 / K, and what its rounding left out
};

// The rows of a group that a block walks over.
struct RowSpan {
  long long g, r0, r1;
};
__device__ __forceinline__ RowSpan block_span(int M, int rows_per_group, int splits) {
  RowSpan s;
  s.g = blockIdx.x / (unsigned)splits;
  const int k = (int)(blockIdx.x - (unsigned)s.g * splits);
  const long long g0 = s.g * rows_per_group;
  const long long len = min((long long)rows_per_group, M - g0);
  s.r0 = g0 + len * k / splits;
  s.r1 = g0 + len * (k + 1) / splits;
  return s;
}

// How a row of up to G NV V elements (V = 16 / sizeof(T)) is held: threads of
// a block, teams of a block and of a warp, rows at a time and in flight per
// team, blocks per SM, and whether the scale and shift are kept in shared
// memory (wherever they fit; else every row reads them from the caches, with
// which 1500 x 12288 took 25.4 us instead of 18.9).
// Rows at a time: four of one vector a thread (60000 x 256: 16.1 us, 19.5 with
// two); in blocks of 256 threads two of three vectors (2250 x 5400: 11.8 us,
// 13.2 with one) and one of more (2250 x 7562: 16.4, 20.0 with two).
template <typename T, int G, int NV>
struct NormCfg {
  static constexpr int V = 16 / (int)sizeof(T), H = V / 2;
  static constexpr int THREADS = G > 128 ? G : 128;
  static constexpr int TEAMS = THREADS / G;
  static constexpr int TW = G < 32 ? 32 / G : 1;
  static constexpr int RF = NV == 1 ? 4 : G < 256 || (G == 256 && NV == 3) ? 2 : 1;   // rows at a time, forward
  static constexpr int DF = 2;                                 // and steps in flight
  static constexpr int RB = NV == 1 ? 4 : G < 512 ? 2 : 1;     // backward (x and dy): rows at a time
  static constexpr int DB = NV < 8 ? 2 : 1;                    // and steps in flight
  static constexpr int SM_F = NV == 1 ? 6 : G < 256 ? 4 : G == 256 ? 2 : 1;    // blocks per SM
  static constexpr int SM_B = NV == 1 ? 4 : G < 256 ? 2 : 1;
  static constexpr size_t ROW = (size_t)NV * G * V * 4;        // one fp32 parameter row
  static constexpr size_t RING_FWD = (size_t)DF * RF * NV * THREADS * 16;
  static constexpr size_t RING_BWD = (size_t)DB * RB * 2 * NV * THREADS * 16;
  static constexpr bool PSMEM_F = RING_FWD + 2 * ROW <= 227 * 1024;
  static constexpr bool PSMEM_B = RING_BWD + ROW <= 227 * 1024;
  static constexpr size_t FWD_SMEM = RING_FWD + (PSMEM_F ? 2 * ROW : 0);
  static constexpr size_t BWD_SMEM = RING_BWD + (PSMEM_B ? ROW : 0);
  static_assert(FWD_SMEM <= 227 * 1024 && BWD_SMEM <= 227 * 1024, "shared memory");
  static_assert(TEAMS == 1 || (size_t)2 * NV * THREADS * V * 4 <= RING_BWD, "the teams' sums fit the ring");
};

// A thread's share of a row: vectors at elements c(i) = (lane + i G) V, and
// how many bytes of the last one lie in the row of K elements (the others
// lie in it whole).
template <typename T, int G, int NV>
struct RowShare {
  static constexpr int V = 16 / (int)sizeof(T);
  int last;
  __device__ __forceinline__ RowShare(int lane, int K) {
    const int left = (K - (lane + (NV - 1) * G) * V) * (int)sizeof(T);
    last = left < 0 ? 0 : left < 16 ? left : 16;
  }
  // Asynchronous copy of the share to dst, dst + pitch, ...; zeros past the row.
  __device__ __forceinline__ void fetch(const T* row, int lane, uint32_t dst, uint32_t pitch) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const T* src = row + (i + 1 < NV || last ? (lane + i * G) * V : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                   ::"r"(dst + i * pitch), "l"(src), "r"(i + 1 < NV ? 16 : last) : "memory");
    }
  }
  // A row of zeros in the same place.
  __device__ __forceinline__ void clear(uint4* dst, uint32_t pitch) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) dst[i * pitch] = make_uint4(0, 0, 0, 0);
  }
};

// A parameter row as fp32 in shared memory: float4 k of vector i of lane l
// at (i V / 4 + k) G + l, so that a warp reads consecutive float4s.  Every
// thread of the block takes vectors in turn.
template <typename PT, int V, int G, int NV, int THREADS>
struct ParamStage {
  static constexpr int N = (NV * G + THREADS - 1) / THREADS;
  RowVec<PT, V> q[N];
  __device__ __forceinline__ void load(const PT* row, int K) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int u = threadIdx.x + n * THREADS;
      if (u < NV * G) q[n] = load_vec<PT, V>(row, u * V, K);
    }
  }
  __device__ __forceinline__ void store(float4* dst, float add) const {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int u = threadIdx.x + n * THREADS;
      if (u < NV * G) {
#pragma unroll
        for (int k = 0; k < V / 4; ++k) {
          const float2 a = q[n].get(2 * k), b = q[n].get(2 * k + 1);
          dst[(u / G * (V / 4) + k) * G + u % G] = make_float4(a.x + add, a.y + add, b.x + add, b.y + add);
        }
      }
    }
  }
};
// Pairs of a thread's vector i: from shared memory, or from the row itself.
template <typename PT, int V, int G, bool SMEM>
__device__ __forceinline__ void read_param(float2 (&out)[V / 2], const float4* staged, const PT* row,
                                           int K, int lane, int i, float add) {
  if constexpr (SMEM) {
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      const float4 f = staged[(i * (V / 4) + k) * G + lane];
      out[2 * k] = make_float2(f.x, f.y);
      out[2 * k + 1] = make_float2(f.z, f.w);
    }
  } else {
    const RowVec<PT, V> q = load_vec<PT, V>(row, (lane + i * G) * V, K);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) out[j] = __fadd2_rn(q.get(j), splat2(add));
  }
}

// Sums over a team of G threads (G <= 32: part of a warp, or the warp; else
// the whole block) of R values that every thread then has.  In a whole warp up
// to four values are scattered over the lanes while they are summed, which
// takes 4 to 6 exchanges instead of 5 R.  `red` has room for R G / 32 values;
// successive calls alternate between two of them, so that one barrier per
// call is enough.
template <int G, int R>
__device__ __forceinline__ void team_sum(float (&v)[R], float* red) {
  if constexpr (G < 32) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < R; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
  } else if constexpr (R == 8) {
    static_assert(G == 32, "rows of four at a time have one vector per thread");
    float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
    team_sum<G, 4>(a, red);
    team_sum<G, 4>(b, red);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = a[k];
      v[4 + k] = b[k];
    }
  } else {
    const int lane = threadIdx.x & 31;
    float c;
    if constexpr (R == 4) {
      const bool h = lane & 16;
      float a = h ? v[2] : v[0], b = h ? v[3] : v[1];
      a += __shfl_xor_sync(0xFFFFFFFFu, h ? v[0] : v[2], 16);
      b += __shfl_xor_sync(0xFFFFFFFFu, h ? v[1] : v[3], 16);
      const bool g = lane & 8;
      c = (g ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, g ? a : b, 8);
    } else if constexpr (R == 2) {
      const bool h = lane & 16;
      c = (h ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, h ? v[0] : v[1], 16);
      c += __shfl_xor_sync(0xFFFFFFFFu, c, 8);
    } else {
      c = v[0] + __shfl_xor_sync(0xFFFFFFFFu, v[0], 16);
      c += __shfl_xor_sync(0xFFFFFFFFu, c, 8);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
    constexpr int L = 32 / R;                  // lanes that hold one value
    if constexpr (G == 32) {
#pragma unroll
      for (int k = 0; k < R; ++k) v[k] = __shfl_sync(0xFFFFFFFFu, c, k * L);
    } else {
      constexpr int W = G / 32;
      if (lane % L == 0) red[(lane / L) * W + (threadIdx.x >> 5)] = c;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < R; ++k) {
        v[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) v[k] += red[k * W + i];
      }
    }
  }
}

template <int H>
__device__ __forceinline__ float sum_pairs(const float2 (&a)[H]) {
  float2 s = a[0];
#pragma unroll
  for (int j = 1; j < H; ++j) s = __fadd2_rn(s, a[j]);
  return s.x + s.y;
}

template <typename T, typename PT, int G, int NV>
__global__ void __launch_bounds__(NormCfg<T, G, NV>::THREADS, NormCfg<T, G, NV>::SM_F)
norm_kernel(const NormArgs p) {
  using C = NormCfg<T, G, NV>;
  constexpr int V = C::V, H = C::H, D = C::DF, TH = C::THREADS, R = C::RF;
  extern __shared__ uint4 smem[];
  __shared__ float red[2 * R * (G > 32 ? G / 32 : 1)];
  const int lane = threadIdx.x % G, team = threadIdx.x / G;
  grid_wait();
  const RowSpan span = block_span(p.M, p.rows_per_group, p.splits);
  const T* x = static_cast<const T*>(p.x);
  const uint4* ring = smem + threadIdx.x;              // vector (slot, row, i) at ((slot R + row) NV + i) TH
  const uint32_t ring_u = smem_u32(ring);
  float4* pw = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(smem) + C::RING_FWD);
  float4* pb = pw + C::ROW / 16;
  const PT* w = p.w ? static_cast<const PT*>(p.w) + span.g * p.ldw : nullptr;
  const PT* b = p.b ? static_cast<const PT*>(p.b) + span.g * p.ldb : nullptr;
  const RowShare<T, G, NV> share(lane, p.K);
  // the parameters' loads leave first, the rows' copies next to them
  ParamStage<PT, V, G, C::PSMEM_F ? NV : 1, TH> sw, sb;
  if constexpr (C::PSMEM_F) {
    if (w) sw.load(w, p.K);
    if (b) sb.load(b, p.K);
  }
  auto fetch = [&](long long row, int slot) {
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (row + k < span.r1)
        share.fetch(x + (row + k) * p.ldx, lane, ring_u + (slot * R + k) * NV * TH * 16, TH * 16);
    cp_async_commit();
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(span.r0 + (team + d * C::TEAMS) * R, d);
  if constexpr (C::PSMEM_F) {
    if (w) sw.store(pw, p.w0);
    if (b) sb.store(pb, 0.0f);
    __syncthreads();
  }
  const float inv_k = p.inv_k;
  const bool ragged = p.K % V != 0;
  int slot = 0;
  // R rows at a time: their sums overlap, and the parameters are read once.
  // The teams of a warp step together (they exchange sums), as long as the
  // first of them has a row.
  const int behind = (team % C::TW) * R;
  for (long long row = span.r0 + team * R; row - behind < span.r1; row += C::TEAMS * R) {
    cp_async_wait<D - 1>();
    float2 v[R][NV][H];
    float sum[R], rstd[R], mu[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float2 acc[H];                      // independent sums, short chains
#pragma unroll
      for (int j = 0; j < H; ++j) acc[j] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const RowVec<T, V> q = read_vec<T, V>(ring + ((slot * R + k) * NV + i) * TH, TH);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          v[k][i][j] = q.get(j);
          acc[j] = __fadd2_rn(acc[j], v[k][i][j]);
        }
      }
      sum[k] = sum_pairs(acc);
    }
    team_sum<G, R>(sum, red);
    // every value of the slot is in registers: the rows D steps on may land there
    fetch(row + (long long)D * C::TEAMS * R, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mu[k] = fmaf(sum[k], inv_k, sum[k] * p.inv_k_rest);    // sum / K, rounded once
      if (fabsf(sum[k]) == CUDART_INF_F) mu[k] = sum[k];
      float2 acc[H];
#pragma unroll
      for (int j = 0; j < H; ++j) acc[j] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * G) * V;
        const float2 m = splat2(i + 1 < NV || c < p.K ? -mu[k] : 0.0f);   // what lies past the row stays 0
#pragma unroll
        for (int j = 0; j < H; ++j) v[k][i][j] = __fadd2_rn(v[k][i][j], m);
        if (i + 1 == NV && ragged && c + V > p.K) {
#pragma unroll
          for (int j = 0; j < H; ++j) {
            if (c + 2 * j >= p.K) v[k][i][j].x = 0.0f;
            if (c + 2 * j + 1 >= p.K) v[k][i][j].y = 0.0f;
          }
        }
#pragma unroll
        for (int j = 0; j < H; ++j) acc[j] = __ffma2_rn(v[k][i][j], v[k][i][j], acc[j]);
      }
      sum[k] = sum_pairs(acc);
    }
    team_sum<G, R>(sum, red + R * (G > 32 ? G / 32 : 1));
#pragma unroll
    for (int k = 0; k < R; ++k) rstd[k] = 1.0f / sqrtf(sum[k] * inv_k + p.eps);
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (row + k < span.r1) {
          if (p.mean) p.mean[row + k] = mu[k];
          if (p.rstd) p.rstd[row + k] = rstd[k];
        }
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
      if (i + 1 < NV || c < p.K) {
        float2 fw[H], fb[H];
        if (w) read_param<PT, V, G, C::PSMEM_F>(fw, pw, w, p.K, lane, i, p.w0);
        if (b) read_param<PT, V, G, C::PSMEM_F>(fb, pb, b, p.K, lane, i, 0.0f);
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const float2 r2 = splat2(rstd[k]);
          RowVec<T, V> o;
#pragma unroll
          for (int j = 0; j < H; ++j) {
            const float2 t = w ? __fmul2_rn(r2, fw[j]) : r2;
            o.set(j, b ? __ffma2_rn(v[k][i][j], t, fb[j]) : __fmul2_rn(v[k][i][j], t));
          }
          if ((k == 0 && C::TW == 1) || row + k < span.r1)
            store_vec<T, V>(y + k * p.ldy, c, i + 1 < NV ? INT_MAX : p.K, o);
        }
      }
    }
  }
}

// Floats of a partial row.
__host__ __device__ constexpr int part_pitch(int K) { return (K + 7) / 8 * 8; }

struct NormBwdArgs {
  const void* dy;
  const void* x;
  const float* mean;
  const float* rstd;
  const void* w;
  void* dx;
  void* dw;
  void* db;
  float* part;               // [blocks][2][part_pitch(K)] when split, unused otherwise
  long long lddy, ldx, ldw, lddx, lddw, lddb;
  int M, K, rows_per_group;  // rows_per_group >= 1 here
  int splits;                // blocks per group
  float w0;
};

// PARAMS: dweight or dbias is wanted.
template <typename T, typename PT, int G, int NV, bool PARAMS>
__global__ void __launch_bounds__(NormCfg<T, G, NV>::THREADS, NormCfg<T, G, NV>::SM_B)
norm_bwd_kernel(const NormBwdArgs p) {
  using C = NormCfg<T, G, NV>;
  constexpr int V = C::V, H = C::H, D = C::DB, TH = C::THREADS, TEAMS = C::TEAMS, R = C::RB;
  extern __shared__ uint4 smem[];
  __shared__ float red[2 * (G > 32 ? 2 * R * (G / 32) : 1)];
  const int lane = threadIdx.x % G, team = threadIdx.x / G;
  grid_wait();
  const RowSpan span = block_span(p.M, p.rows_per_group, p.splits);
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  uint4* ring = smem + threadIdx.x;          // (slot, row): NV vectors of x, then NV of dy
  const uint32_t ring_u = smem_u32(ring);
  float4* pw = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(smem) + C::RING_BWD);
  const PT* w = p.w ? static_cast<const PT*>(p.w) + span.g * p.ldw : nullptr;
  const RowShare<T, G, NV> share(lane, p.K);
  ParamStage<PT, V, G, C::PSMEM_B ? NV : 1, TH> sw;
  if constexpr (C::PSMEM_B)
    if (w) sw.load(w, p.K);
  float nmu[D][R], nrs[D][R];                // the statistics of the rows in flight
  const int behind = (team % C::TW) * R;     // as in the forward kernel
  auto fetch = [&](long long row, int slot) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int at = (slot * R + k) * 2 * NV * TH;
      if (row + k < span.r1) {
        share.fetch(x + (row + k) * p.ldx, lane, ring_u + at * 16, TH * 16);
        share.fetch(dy + (row + k) * p.lddy, lane, ring_u + (at + NV * TH) * 16, TH * 16);
      } else if (row - behind < span.r1) {   // a step's missing row adds nothing
        share.clear(ring + at, TH);
        share.clear(ring + at + NV * TH, TH);
      }
    }
    cp_async_commit();
  };
  auto stats = [&](long long row, float (&mu)[R], float (&rs)[R]) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mu[k] = row + k < span.r1 ? p.mean[row + k] : 0.0f;
      rs[k] = row + k < span.r1 ? p.rstd[row + k] : 0.0f;
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const long long row = span.r0 + (team + d * TEAMS) * R;
    fetch(row, d);
    stats(row, nmu[d], nrs[d]);
  }
  const float inv_k = 1.0f / (float)p.K;
  float2 aw[PARAMS ? NV : 1][H], ab[PARAMS ? NV : 1][H];
  if constexpr (PARAMS) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j) aw[i][j] = ab[i][j] = make_float2(0.0f, 0.0f);
  }
  if constexpr (C::PSMEM_B) {
    if (w) sw.store(pw, p.w0);
    __syncthreads();
  }
  int slot = 0, phase = 0;
  // R rows at a time: their sums overlap, and the scale is read once
  for (long long row = span.r0 + team * R; row - behind < span.r1; row += TEAMS * R) {
    cp_async_wait<D - 1>();
    const uint4* q = ring + slot * R * 2 * NV * TH;
    float2 m[R], r[R], s1[R], s2[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      m[k] = splat2(-nmu[0][k]);
      r[k] = splat2(nrs[0][k]);
      s1[k] = s2[k] = make_float2(0.0f, 0.0f);
    }
    // the statistics of the rows D steps on, long before they are needed
    const long long ahead = row + (long long)D * TEAMS * R;
#pragma unroll
    for (int d = 0; d + 1 < D; ++d)
#pragma unroll
      for (int k = 0; k < R; ++k) {
        nmu[d][k] = nmu[d + 1][k];
        nrs[d][k] = nrs[d + 1][k];
      }
    stats(ahead, nmu[D - 1], nrs[D - 1]);
    // columns past K: x and dy read as 0 and add 0 to every sum
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float2 f[H];
      if (w) read_param<PT, V, G, C::PSMEM_B>(f, pw, w, p.K, lane, i, p.w0);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const RowVec<T, V> xr = read_vec<T, V>(q + (2 * k * NV + i) * TH, TH);
        const RowVec<T, V> dr = read_vec<T, V>(q + ((2 * k + 1) * NV + i) * TH, TH);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const float2 g = dr.get(j), d = __fadd2_rn(xr.get(j), m[k]);     // xhat = d r
          if constexpr (PARAMS) {
            aw[i][j] = __ffma2_rn(__fmul2_rn(g, r[k]), d, aw[i][j]);
            ab[i][j] = __fadd2_rn(ab[i][j], g);
          }
          const float2 t = w ? __fmul2_rn(g, f[j]) : g;
          s1[k] = __fadd2_rn(s1[k], t);
          s2[k] = __ffma2_rn(t, d, s2[k]);
        }
      }
    }
    if (p.dx) {
      float sum[2 * R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        sum[2 * k] = s1[k].x + s1[k].y;
        sum[2 * k + 1] = s2[k].x + s2[k].y;
      }
      team_sum<G, 2 * R>(sum, red + phase * (G > 32 ? 2 * R * (G / 32) : 0));
      phase ^= 1;
      // read the rows again rather than hold them: the registers are few
      asm volatile("" ::: "memory");
#pragma unroll
      for (int k = 0; k < R; ++k) {
        // dX = r t - r mean(t) - xhat r mean(t xhat)
        const float rs = r[k].x;
        s1[k] = splat2(-sum[2 * k] * inv_k * rs);
        s2[k] = splat2(-sum[2 * k + 1] * rs * inv_k * rs);
      }
      T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * G) * V;
        if (i + 1 < NV || c < p.K) {
          float2 f[H];
          if (w) read_param<PT, V, G, C::PSMEM_B>(f, pw, w, p.K, lane, i, p.w0);
#pragma unroll
          for (int k = 0; k < R; ++k) {
            const RowVec<T, V> xr = read_vec<T, V>(q + (2 * k * NV + i) * TH, TH);
            const RowVec<T, V> dr = read_vec<T, V>(q + ((2 * k + 1) * NV + i) * TH, TH);
            RowVec<T, V> o;
#pragma unroll
            for (int j = 0; j < H; ++j) {
              const float2 g = dr.get(j), d = __fadd2_rn(xr.get(j), m[k]);
              const float2 t = w ? __fmul2_rn(g, f[j]) : g;
              o.set(j, __ffma2_rn(t, r[k], __ffma2_rn(__fmul2_rn(d, r[k]), s2[k], s1[k])));
            }
            if ((k == 0 && C::TW == 1) || row + k < span.r1)
              store_vec<T, V>(dx + k * p.lddx, c, i + 1 < NV ? INT_MAX : p.K, o);
          }
        }
      }
    }
    fetch(ahead, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  if constexpr (PARAMS) {
    const bool whole = p.splits == 1;
    // an own row of the gradients, or this block's partial row (of whole vectors)
    PT* dw = whole && p.dw ? static_cast<PT*>(p.dw) + span.g * p.lddw : nullptr;
    PT* db = whole && p.db ? static_cast<PT*>(p.db) + span.g * p.lddb : nullptr;
    float* part = p.part + (whole ? 0 : (size_t)blockIdx.x * 2 * part_pitch(p.K));
    if constexpr (TEAMS == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * G) * V;
        if (c >= p.K) continue;
        if (whole) {
          RowVec<PT, V> ow, ob;
#pragma unroll
          for (int j = 0; j < H; ++j) {
            ow.set(j, aw[i][j]);
            ob.set(j, ab[i][j]);
          }
          if (dw) store_vec<PT, V>(dw, c, p.K, ow);
          if (db) store_vec<PT, V>(db, c, p.K, ob);
        } else {
          float4* dst_w = reinterpret_cast<float4*>(part + c);
          float4* dst_b = reinterpret_cast<float4*>(part + part_pitch(p.K) + c);
#pragma unroll
          for (int j = 0; j < H; j += 2) {
            dst_w[j / 2] = make_float4(aw[i][j].x, aw[i][j].y, aw[i][j + 1].x, aw[i][j + 1].y);
            dst_b[j / 2] = make_float4(ab[i][j].x, ab[i][j].y, ab[i][j + 1].x, ab[i][j + 1].y);
          }
        }
      }
    } else {
      // the teams' sums meet where the rows were (none is in flight), and
      // every thread adds up some columns over the teams, in order
      constexpr int COLS = NV * G * V;
      float* meet = reinterpret_cast<float*>(smem);       // [team][2][COLS]
      cp_async_wait<0>();
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < H; j += 2) {
          const int c = (lane + i * G) * V + 2 * j;
          float* at = meet + team * 2 * COLS + c;
          *reinterpret_cast<float4*>(at) = make_float4(aw[i][j].x, aw[i][j].y, aw[i][j + 1].x, aw[i][j + 1].y);
          *reinterpret_cast<float4*>(at + COLS) = make_float4(ab[i][j].x, ab[i][j].y, ab[i][j + 1].x, ab[i][j + 1].y);
        }
      __syncthreads();
      for (int u = threadIdx.x; u < 2 * COLS / 4; u += TH) {
        const int which = u >= COLS / 4, c = 4 * u - which * COLS;
        if (c >= p.K) continue;
        float4 s = *reinterpret_cast<const float4*>(meet + 4 * u);
#pragma unroll
        for (int t = 1; t < TEAMS; ++t) {
          const float4 v = *reinterpret_cast<const float4*>(meet + t * 2 * COLS + 4 * u);
          s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        if (whole) {
          PT* out = which ? db : dw;
          const float e[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (out && c + k < p.K) out[c + k] = Elem<PT>::from_f(e[k]);
        } else {
          *reinterpret_cast<float4*>(part + (which ? part_pitch(p.K) : 0) + c) = s;
        }
      }
    }
  }
}

// Sums the blocks' partials of every group and column in block order: 32
// columns (a float4 a thread) by 32 threads that each take a contiguous share
// of the blocks, then the shares in order.
template <typename PT>
__global__ void __launch_bounds__(256)
norm_bwd_join_kernel(const float* part, int splits, int K, PT* dw, long long lddw, PT* db,
                     long long lddb) {
  __shared__ float4 sh[32][8];
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + tx * 4;
  const int which = blockIdx.y & 1;
  const long long g = blockIdx.z;
  grid_wait();
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const size_t pitch = part_pitch(K);
  if (c < K) {
    const int s0 = splits * ty / 32, s1 = splits * (ty + 1) / 32;
    const float* q = part + (((size_t)g * splits + s0) * 2 + which) * pitch + c;
#pragma unroll 8
    for (int s = s0; s < s1; ++s, q += 2 * pitch) {
      const float4 v = *reinterpret_cast<const float4*>(q);
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  sh[ty][tx] = acc;
  __syncthreads();
  const int col = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && col < K) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += reinterpret_cast<const float*>(sh[i])[threadIdx.x];
    PT* out = which ? db : dw;
    if (out) out[g * (which ? lddb : lddw) + col] = Elem<PT>::from_f(s);
  }
}

// Blocks per group: `per_sm` blocks per SM over all groups (what fits there
// at once), with at least `rows` rows each.
int split_rows(int M, int rows_per_group, int per_sm, int rows) {
  const long long groups = ((long long)M + rows_per_group - 1) / rows_per_group;
  const long long len = rows_per_group < M ? rows_per_group : M;
  long long s = (long long)per_sm * 148 / groups;
  const long long most = (len + rows - 1) / rows;
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s);
}
// Backward: rows of up to 1280 elements, of which a block has several teams,
// in blocks of at least eight (300 x 1152: 6.1 us, 7.0 with four), a group of
// up to 16 in one, whose sums are final (16 x 200: 3.1 us, 4.4 with a second
// launch).  Longer rows, at which the whole block works, in blocks of at least
// two (64 x 4608: 7.1 us, 10.9 with eight; 16 x 12288: 12, 37 in one), a group
// of up to four in one.  The split does not depend on the element type (the
// workspace's size does not know it): rows of up to 256 elements have four
// blocks per SM (60000 x 256: 23 us, 33 with two).
int bwd_splits(int M, int K, int rows_per_group) {
  const int len = M < rows_per_group ? M : rows_per_group;
  if (len <= (K <= 1280 ? 16 : 4)) return 1;
  return split_rows(M, rows_per_group, K <= 256 ? 4 : 2, K <= 1280 ? 8 : 2);
}

// Raises the kernel's dynamic shared-memory limit once per device.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, bool* done) {
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

template <typename T, typename PT, int G, int NV>
cudaError_t fwd_launch(NormArgs a, cudaStream_t st) {
  using C = NormCfg<T, G, NV>;
  static bool done[kMaxDevices] = {};
  const cudaError_t e = allow_smem(norm_kernel<T, PT, G, NV>, C::FWD_SMEM, done);
  if (e != cudaSuccess) return e;
  const long long groups = ((long long)a.M + a.rows_per_group - 1) / a.rows_per_group;
  a.splits = split_rows(a.M, a.rows_per_group, C::PSMEM_F ? C::SM_F : 2, C::TEAMS);
  return launch_op(norm_kernel<T, PT, G, NV>, dim3((unsigned)(groups * a.splits)), C::THREADS,
                   C::FWD_SMEM, 1, st, a);
}

// Team and vectors per thread for a row of `vecs` 16-byte vectors of V
// elements (SVDQ_NORM_MAX_K elements at most): the fewest that hold the row,
// so that only a thread's last vector can lie past it.  A warp per row while
// it fits (16384 x 1152: 14.3 us, 21.3 with 128 threads), 256 threads rather
// than 512 (2250 x 7562: 16.4, 28.3), which forward are also better than 128
// with five vectors (2250 x 4608: 10.8, 14.0) and backward are not (a block of
// 256 has the SM for itself: 2250 x 5400 27 us, 2250 x 4608 19.6 with two of
// 128).
template <int V, bool FWD, typename F>
cudaError_t dispatch_row(int vecs, F&& f) {
  if (vecs <= 8 * 1) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  if (vecs <= 16 * 1) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  if (vecs <= 32 * 1) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  if (vecs <= 32 * 2) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
  if (vecs <= 32 * 3) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 3>());
  if (vecs <= 32 * 4) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 4>());
  if (vecs <= 32 * 5) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 5>());
  if (vecs <= 128 * 2) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
  if (vecs <= 128 * 3) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 3>());
  if (vecs <= 128 * 4) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 4>());
  if constexpr (!FWD)
    if (vecs <= 128 * 5) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 5>());
  if (vecs <= 256 * 3) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 3>());
  if (vecs <= 256 * 4) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
  if (vecs <= 256 * 5) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 5>());
  if (vecs <= 512 * 3) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 3>());
  if constexpr (V == 4) {
    if (vecs <= 512 * 4) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
    if (vecs <= 512 * 5) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 5>());
    if (vecs <= 512 * 6) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 6>());
    if (vecs <= 512 * 7) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 7>());
    return f(std::integral_constant<int, 512>(), std::integral_constant<int, 8>());
  }
  return f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
}

template <typename T, typename PT>
cudaError_t fwd(const NormArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  return dispatch_row<V, true>((a.K + V - 1) / V, [&](auto g, auto nv) {
    return fwd_launch<T, PT, decltype(g)::value, decltype(nv)::value>(a, st);
  });
}

template <typename T, typename PT, int G, int NV>
cudaError_t bwd_launch(const NormBwdArgs& a, long long groups, cudaStream_t st) {
  using C = NormCfg<T, G, NV>;
  const unsigned blocks = (unsigned)(groups * a.splits);
  static bool done[2][kMaxDevices] = {};
  cudaError_t e;
  if (a.dw || a.db) {
    e = allow_smem(norm_bwd_kernel<T, PT, G, NV, true>, C::BWD_SMEM, done[0]);
    if (e != cudaSuccess) return e;
    return launch_op(norm_bwd_kernel<T, PT, G, NV, true>, dim3(blocks), C::THREADS, C::BWD_SMEM, 1, st, a);
  } else {
    e = allow_smem(norm_bwd_kernel<T, PT, G, NV, false>, C::BWD_SMEM, done[1]);
    if (e != cudaSuccess) return e;
    return launch_op(norm_bwd_kernel<T, PT, G, NV, false>, dim3(blocks), C::THREADS, C::BWD_SMEM, 1, st, a);
  }
}

template <typename T, typename PT>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  const long long groups = ((long long)a.M + a.rows_per_group - 1) / a.rows_per_group;
  cudaError_t e = dispatch_row<V, false>((a.K + V - 1) / V, [&](auto g, auto nv) {
    return bwd_launch<T, PT, decltype(g)::value, decltype(nv)::value>(a, groups, st);
  });
  if (e != cudaSuccess || a.splits == 1 || (!a.dw && !a.db)) return e;
  const dim3 grid((unsigned)((a.K + 31) / 32), 2, (unsigned)groups);
  return launch_op(norm_bwd_join_kernel<PT>, grid, 256, 0, 1, st, a.part, a.splits, a.K,
                   static_cast<PT*>(a.dw), a.lddw, static_cast<PT*>(a.db), a.lddb);
}

// f(T{}, PT{}) for the element and parameter types.
template <typename F>
cudaError_t dispatch_types(int dtype, int param_dtype, F&& f) {
  const bool pf = param_dtype == SVDQ_DTYPE_F32;
  if (dtype == SVDQ_DTYPE_BF16)
    return pf ? f(__nv_bfloat16(), float()) : f(__nv_bfloat16(), __nv_bfloat16());
  if (dtype == SVDQ_DTYPE_F16) return pf ? f(__half(), float()) : f(__half(), __half());
  return f(float(), float());
}

bool ok_types(int dtype, int param_dtype) {
  return dtype >= SVDQ_DTYPE_BF16 && dtype <= SVDQ_DTYPE_F32 &&
         (param_dtype == dtype || param_dtype == SVDQ_DTYPE_F32);
}

}  // namespace
}  // namespace svdq

using svdq::dtype_size;
using svdq::rows_aligned16;

extern "C" {

svdq_status svdq_layer_norm(int dtype, int param_dtype, int M, int K, const void* X, int ldx,
                            const void* weight, int ldw, const void* bias, int ldb,
                            float weight_offset, int rows_per_group, float eps, void* Y, int ldy,
                            float* mean, float* rstd, cudaStream_t stream) {
  if (!svdq::ok_types(dtype, param_dtype) || !(eps >= 0.0f) || !std::isfinite(eps) ||
      !std::isfinite(weight_offset))
    return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || K < 1 || rows_per_group < 0 || ldx < K || ldy < K ||
      (weight && ldw != 0 && ldw < K) || (bias && ldb != 0 && ldb < K))
    return SVDQ_ERR_SHAPE;
  if (K > SVDQ_NORM_MAX_K) return SVDQ_ERR_UNSUPPORTED;
  if (M == 0) return SVDQ_OK;
  if (!X || !Y || (X == Y && ldx != ldy)) return SVDQ_ERR_INVALID_ARG;
  const int es = dtype_size(dtype), ps = dtype_size(param_dtype);
  if (!rows_aligned16(X, ldx, es) || !rows_aligned16(Y, ldy, es) ||
      (weight && !rows_aligned16(weight, ldw, ps)) || (bias && !rows_aligned16(bias, ldb, ps)) ||
      (reinterpret_cast<uintptr_t>(mean) & 3) || (reinterpret_cast<uintptr_t>(rstd) & 3))
    return SVDQ_ERR_ALIGNMENT;
  {
    using svdq::extent_flat;
    using svdq::extent_rows;
    const long long groups = rows_per_group ? ((long long)M + rows_per_group - 1) / rows_per_group : 1;
    const svdq::Extent x = extent_rows(X, M, K, ldx, es), y = extent_rows(Y, M, K, ldy, es),
                       w = extent_rows(weight, groups, K, ldw, ps), b = extent_rows(bias, groups, K, ldb, ps),
                       mu = extent_flat(mean, 4ll * M), rs = extent_flat(rstd, 4ll * M);
    if ((Y != X && svdq::overlap(y, x)) || svdq::overlaps_any(y, {w, b, mu, rs}) ||
        svdq::overlaps_any(mu, {x, w, b, rs}) || svdq::overlaps_any(rs, {x, w, b}))
      return SVDQ_ERR_INVALID_ARG;
  }
  svdq::NormArgs a{};
  a.x = X; a.w = weight; a.b = bias; a.y = Y; a.mean = mean; a.rstd = rstd;
  a.ldx = ldx; a.ldw = ldw; a.ldb = ldb; a.ldy = ldy;
  a.M = M; a.K = K; a.rows_per_group = rows_per_group ? rows_per_group : M;
  a.w0 = weight_offset; a.eps = eps;
  a.inv_k = (float)(1.0 / K);
  a.inv_k_rest = (float)(1.0 / K - (double)a.inv_k);
  const cudaError_t e = svdq::dispatch_types(dtype, param_dtype, [&](auto t, auto pt) {
    return svdq::fwd<decltype(t), decltype(pt)>(a, stream);
  });
  return svdq::status_of(e);
}

size_t svdq_layer_norm_backward_workspace(int M, int K, int rows_per_group) {
  if (M <= 0 || K < 1 || K > SVDQ_NORM_MAX_K || rows_per_group < 0) return 0;
  const int rpg = rows_per_group ? rows_per_group : M;
  const size_t groups = ((size_t)M + rpg - 1) / rpg;
  const int s = svdq::bwd_splits(M, K, rpg);
  return s == 1 ? 0 : groups * s * 2 * (size_t)svdq::part_pitch(K) * sizeof(float);
}

svdq_status svdq_layer_norm_backward(int dtype, int param_dtype, int M, int K, const void* dY,
                                     int lddy, const void* X, int ldx, const float* mean,
                                     const float* rstd, const void* weight, int ldw,
                                     float weight_offset, int rows_per_group, void* dX, int lddx,
                                     void* dweight, int lddw, void* dbias, int lddb,
                                     void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  if (!svdq::ok_types(dtype, param_dtype) || !std::isfinite(weight_offset))
    return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || K < 1 || rows_per_group < 0 || lddy < K || ldx < K || (dX && lddx < K) ||
      (weight && ldw != 0 && ldw < K) || (dweight && lddw < K) || (dbias && lddb < K))
    return SVDQ_ERR_SHAPE;
  if (K > SVDQ_NORM_MAX_K) return SVDQ_ERR_UNSUPPORTED;
  const int es = dtype_size(dtype), ps = dtype_size(param_dtype);
  if ((dweight && !rows_aligned16(dweight, lddw, ps)) || (dbias && !rows_aligned16(dbias, lddb, ps)))
    return SVDQ_ERR_ALIGNMENT;
  if (M == 0) {
    if (rows_per_group) return SVDQ_OK;
    cudaError_t e = dweight ? cudaMemsetAsync(dweight, 0, (size_t)K * ps, stream) : cudaSuccess;
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)K * ps, stream);
    return svdq::status_of(e);
  }
  if (!dY || !X || !mean || !rstd || (dX == dY && lddx != lddy) || (dX == X && lddx != ldx))
    return SVDQ_ERR_INVALID_ARG;
  if (!rows_aligned16(dY, lddy, es) || !rows_aligned16(X, ldx, es) ||
      (dX && !rows_aligned16(dX, lddx, es)) || (weight && !rows_aligned16(weight, ldw, ps)) ||
      (reinterpret_cast<uintptr_t>(mean) & 3) || (reinterpret_cast<uintptr_t>(rstd) & 3))
    return SVDQ_ERR_ALIGNMENT;
  if (!dX && !dweight && !dbias) return SVDQ_OK;
  svdq::NormBwdArgs a{};
  a.rows_per_group = rows_per_group ? rows_per_group : M;
  a.splits = svdq::bwd_splits(M, K, a.rows_per_group);
  const size_t need = (dweight || dbias) ? svdq_layer_norm_backward_workspace(M, K, rows_per_group) : 0;
  if (need) {
    if (!workspace) return SVDQ_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return SVDQ_ERR_ALIGNMENT;
    if (workspace_bytes < need) return SVDQ_ERR_SHAPE;
  }
  {
    using svdq::extent_flat;
    using svdq::extent_rows;
    const long long groups = ((long long)M + a.rows_per_group - 1) / a.rows_per_group;
    const svdq::Extent dy = extent_rows(dY, M, K, lddy, es), x = extent_rows(X, M, K, ldx, es),
                       w = extent_rows(weight, groups, K, ldw, ps), mu = extent_flat(mean, 4ll * M),
                       rs = extent_flat(rstd, 4ll * M), gx = extent_rows(dX, M, K, lddx, es),
                       gw = extent_rows(dweight, groups, K, lddw, ps), gb = extent_rows(dbias, groups, K, lddb, ps),
                       ws = extent_flat(need ? workspace : nullptr, (long long)need);
    if ((dX != dY && svdq::overlap(gx, dy)) || (dX != X && svdq::overlap(gx, x)) ||
        svdq::overlaps_any(gx, {w, mu, rs, gw, gb, ws}) || svdq::overlaps_any(gw, {dy, x, w, mu, rs, gb, ws}) ||
        svdq::overlaps_any(gb, {dy, x, w, mu, rs, ws}) || svdq::overlaps_any(ws, {dy, x, w, mu, rs}))
      return SVDQ_ERR_INVALID_ARG;
  }
  a.dy = dY; a.x = X; a.mean = mean; a.rstd = rstd; a.w = weight;
  a.dx = dX; a.dw = dweight; a.db = dbias; a.part = static_cast<float*>(workspace);
  a.lddy = lddy; a.ldx = ldx; a.ldw = ldw; a.lddx = lddx; a.lddw = lddw; a.lddb = lddb;
  a.M = M; a.K = K; a.w0 = weight_offset;
  const cudaError_t e = svdq::dispatch_types(dtype, param_dtype, [&](auto t, auto pt) {
    return svdq::bwd<decltype(t), decltype(pt)>(a, stream);
  });
  return svdq::status_of(e);
}

}  // extern "C"
