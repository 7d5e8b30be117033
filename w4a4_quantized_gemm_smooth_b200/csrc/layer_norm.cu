// Layer norm with a scale and a shift per group of rows, and its gradients.
//
// Forward: a row is held in the registers of one team (a warp, or a block of
// 128 or 512 threads for long rows), so that X is read once although the
// variance is the two-pass one, sum (x - mu)^2 in fp32 after the mean (no
// cancellation for rows with a large mean).  Bound by memory.
//
// Backward: a team owns fixed columns and walks over rows of one group.  Per
// row it forms the two row sums and dX from registers; the columns' sums of
// dy xhat and dy stay in registers over all the rows of the team and are
// joined at the end: teams of a block in shared memory in order, blocks of a
// group through fp32 partials in the workspace, summed in block order by a
// second kernel.  X and dY are read once.
#include <cmath>
#include <type_traits>

#include "elem.cuh"
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
  int M, K, rows_per_group;
  float w0, eps;
};

// Sum over a team of G threads (G = 32: the warp; else the whole block).
// `red` has room for 2 x G / 32 values; two calls in a row use `phase` 0 and 1.
template <int G>
__device__ __forceinline__ float team_sum(float v, float* red, int phase) {
  v = warp_sum(v);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    float* r = red + phase * W;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += r[i];
  }
  return v;
}

// V elements per vector (16 bytes of T), NV vectors per thread.
template <typename T, typename PT, int G, int NV>
__global__ void __launch_bounds__(G > 128 ? G : 128)
norm_kernel(const NormArgs p) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int TEAMS = G >= 128 ? 1 : 128 / G;
  __shared__ float red[2 * (G > 32 ? G / 32 : 1)];
  const int lane = threadIdx.x % G;
  const long long row = (long long)blockIdx.x * TEAMS + threadIdx.x / G;
  if (row >= p.M) return;                 // whole teams only
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  float v[NV][V];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * G) * V;
    if (c < p.K) {
      load_row<T, V>(x, c, p.K, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sum += v[i][e];
  }
  const float inv_k = 1.0f / (float)p.K;
  const float mu = team_sum<G>(sum, red, 0) * inv_k;
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * G) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = v[i][e] - mu;
      if (c + e < p.K) sq += d * d;
    }
  }
  const float rstd = 1.0f / sqrtf(team_sum<G>(sq, red, 1) * inv_k + p.eps);
  if (lane == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = rstd;
  }
  const long long g = p.rows_per_group ? row / p.rows_per_group : 0;
  const PT* w = p.w ? static_cast<const PT*>(p.w) + g * p.ldw : nullptr;
  const PT* b = p.b ? static_cast<const PT*>(p.b) + g * p.ldb : nullptr;
  T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * G) * V;
    if (c >= p.K) break;
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] = (v[i][e] - mu) * rstd;
    if (w) {
      float t[V];
      load_row<PT, V>(w, c, p.K, t);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] *= t[e] + p.w0;
    }
    if (b) {
      float t[V];
      load_row<PT, V>(b, c, p.K, t);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] += t[e];
    }
    store_row<T, V>(y, c, p.K, v[i]);
  }
}

// 16 bytes of a row from element c on; zeros past n.
template <typename T>
__device__ __forceinline__ Pack<T, 16> load_pack(const T* row, int c, int n) {
  constexpr int V = 16 / (int)sizeof(T);
  if (c + V <= n) return *reinterpret_cast<const Pack<T, 16>*>(row + c);
  Pack<T, 16> v;
#pragma unroll
  for (int e = 0; e < V; ++e) v.e[e] = c + e < n ? row[c + e] : Elem<T>::from_f(0.0f);
  return v;
}

struct NormBwdArgs {
  const void* dy;
  const void* x;
  const float* mean;
  const float* rstd;
  const void* w;
  void* dx;
  void* dw;
  void* db;
  float* part;               // [items][2][K] when split, unused otherwise
  long long lddy, ldx, ldw, lddx, lddw, lddb;
  int M, K, rows_per_group;  // rows_per_group >= 1 here
  int splits;                // blocks per group
  float w0;
};

// PARAMS: dweight or dbias is wanted.
template <typename T, typename PT, int G, int NV, bool PARAMS>
__global__ void __launch_bounds__(G > 128 ? G : 128)
norm_bwd_kernel(const NormBwdArgs p) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int TEAMS = G >= 128 ? 1 : 128 / G;
  __shared__ float red[2 * (G > 32 ? 2 * (G / 32) : 1)];
  extern __shared__ float colsum[];       // TEAMS > 1: [2][NV * G * V]
  const int lane = threadIdx.x % G, team = threadIdx.x / G;
  const long long g = blockIdx.x / p.splits;
  const int s = (int)(blockIdx.x - g * p.splits);
  const long long g0 = g * p.rows_per_group;
  const long long glen = min((long long)p.rows_per_group, p.M - g0);
  const long long r0 = g0 + glen * s / p.splits, r1 = g0 + glen * (s + 1) / p.splits;
  const PT* w = p.w ? static_cast<const PT*>(p.w) + g * p.ldw : nullptr;
  const float inv_k = 1.0f / (float)p.K;
  float aw[PARAMS ? NV : 1][V], ab[PARAMS ? NV : 1][V];
  if constexpr (PARAMS) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) aw[i][e] = ab[i][e] = 0.0f;
  }
  int phase = 0;
  for (long long row = r0 + team; row < r1; row += TEAMS) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mu = p.mean[row], rstd = p.rstd[row];
    // the row stays packed in registers: the columns' sums need the room
    Pack<T, 16> xr[NV], dr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
      xr[i] = load_pack(x, c, p.K);
      dr[i] = load_pack(dy, c, p.K);
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
      float wv[V];
      if (w && c < p.K) load_row<PT, V>(w, c, p.K, wv);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float dv = Elem<T>::to_f(dr[i].e[e]);
        // columns past K: dy is 0, and xhat is set to 0
        const float h = c + e < p.K ? (Elem<T>::to_f(xr[i].e[e]) - mu) * rstd : 0.0f;
        if constexpr (PARAMS) {
          aw[i][e] += dv * h;
          ab[i][e] += dv;
        }
        const float t = w ? (c + e < p.K ? dv * (wv[e] + p.w0) : 0.0f) : dv;
        s1 += t;
        s2 += t * h;
      }
    }
    if (!p.dx) continue;
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (G > 32) {
      constexpr int W = G / 32;
      float* r = red + phase * 2 * W;     // two buffers: one barrier per row
      if ((threadIdx.x & 31) == 0) {
        r[threadIdx.x >> 5] = s1;
        r[W + (threadIdx.x >> 5)] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        s1 += r[i];
        s2 += r[W + i];
      }
      phase ^= 1;
    }
    s1 *= inv_k;
    s2 *= inv_k;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
      if (c >= p.K) break;
      float wv[V], o[V];
      if (w) load_row<PT, V>(w, c, p.K, wv);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float dv = Elem<T>::to_f(dr[i].e[e]);
        const float h = (Elem<T>::to_f(xr[i].e[e]) - mu) * rstd;
        o[e] = rstd * ((w ? dv * (wv[e] + p.w0) : dv) - s1 - h * s2);
      }
      store_row<T, V>(dx, c, p.K, o);
    }
  }
  if constexpr (PARAMS) {
    if constexpr (TEAMS > 1) {
      // join the teams in order
      constexpr int COLS = NV * G * V;
      for (int k = 0; k < TEAMS; ++k) {
        if (team == k) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const int c = (lane + i * G) * V + e;
              if (k > 0) {
                aw[i][e] += colsum[c];
                ab[i][e] += colsum[COLS + c];
              }
              if (k < TEAMS - 1) {
                colsum[c] = aw[i][e];
                colsum[COLS + c] = ab[i][e];
              }
            }
        }
        __syncthreads();
      }
      if (team != TEAMS - 1) return;
    }
    if (p.splits == 1) {
      PT* dw = p.dw ? static_cast<PT*>(p.dw) + g * p.lddw : nullptr;
      PT* db = p.db ? static_cast<PT*>(p.db) + g * p.lddb : nullptr;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * G) * V;
        if (c >= p.K) break;
        if (dw) store_row<PT, V>(dw, c, p.K, aw[i]);
        if (db) store_row<PT, V>(db, c, p.K, ab[i]);
      }
    } else {
      float* pw = p.part + (size_t)blockIdx.x * 2 * p.K;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int c = (lane + i * G) * V + e;
          if (c < p.K) {
            pw[c] = aw[i][e];
            pw[p.K + c] = ab[i][e];
          }
        }
    }
  }
}

// Sums the blocks' partials of every group and column in block order: 32
// columns by 8 rows of threads, each row summing a contiguous eighth of the
// blocks, then the eighths in order.
template <typename PT>
__global__ void __launch_bounds__(256)
norm_bwd_join_kernel(const float* part, int splits, int K, PT* dw, long long lddw, PT* db,
                     long long lddb) {
  __shared__ float sh[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  const int which = blockIdx.y & 1;
  const long long g = blockIdx.z;
  float acc = 0.0f;
  if (c < K) {
    const int s0 = splits * ty / 8, s1 = splits * (ty + 1) / 8;
    const float* q = part + ((size_t)g * splits + s0) * 2 * K + (size_t)which * K + c;
#pragma unroll 8
    for (int s = s0; s < s1; ++s, q += 2 * (size_t)K) acc += *q;
  }
  sh[ty][tx] = acc;
  __syncthreads();
  if (ty == 0 && c < K) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += sh[i][tx];
    PT* out = which ? db : dw;
    if (out) out[g * (which ? lddb : lddw) + c] = Elem<PT>::from_f(acc);
  }
}

// Blocks per group of the backward pass: about four per SM over all groups,
// with at least eight rows per block (two per warp of a four-warp block), so
// that the partials stay a small share of the traffic.
int bwd_splits(int M, int rows_per_group) {
  const long long groups = ((long long)M + rows_per_group - 1) / rows_per_group;
  const long long len = rows_per_group < M ? rows_per_group : M;
  long long s = (4 * 148 + groups - 1) / groups;
  const long long most = (len + 7) / 8;
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s);
}

template <typename T, typename PT, int G, int NV>
cudaError_t fwd_launch(const NormArgs& a, cudaStream_t st) {
  constexpr int TEAMS = G >= 128 ? 1 : 128 / G;
  const long long blocks = ((long long)a.M + TEAMS - 1) / TEAMS;
  norm_kernel<T, PT, G, NV><<<(unsigned)blocks, G > 128 ? G : 128, 0, st>>>(a);
  return cudaGetLastError();
}

// Team and vectors per thread for a row of `vecs` 16-byte vectors of V
// elements (SVDQ_NORM_MAX_K elements at most).
template <int V, typename F>
cudaError_t dispatch_row(int vecs, F&& f) {
  if (vecs <= 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  if (vecs <= 64) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
  if (vecs <= 96) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 3>());
  if (vecs <= 160) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 5>());
  if (vecs <= 256) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
  if (vecs <= 384) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 3>());
  if (vecs <= 640) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 5>());
  if (vecs <= 1024) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
  if constexpr (V == 4)
    if (vecs > 2048) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
}

template <typename T, typename PT>
cudaError_t fwd(const NormArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  return dispatch_row<V>((a.K + V - 1) / V, [&](auto g, auto nv) {
    return fwd_launch<T, PT, decltype(g)::value, decltype(nv)::value>(a, st);
  });
}

template <typename T, typename PT, int G, int NV>
cudaError_t bwd_launch(const NormBwdArgs& a, long long groups, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int TEAMS = G >= 128 ? 1 : 128 / G;
  const unsigned blocks = (unsigned)(groups * a.splits);
  const int threads = G > 128 ? G : 128;
  if (a.dw || a.db) {
    const size_t sh = TEAMS > 1 ? sizeof(float) * 2 * NV * G * V : 0;
    norm_bwd_kernel<T, PT, G, NV, true><<<blocks, threads, sh, st>>>(a);
  } else {
    norm_bwd_kernel<T, PT, G, NV, false><<<blocks, threads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T, typename PT>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  const long long groups = ((long long)a.M + a.rows_per_group - 1) / a.rows_per_group;
  cudaError_t e = dispatch_row<V>((a.K + V - 1) / V, [&](auto g, auto nv) {
    return bwd_launch<T, PT, decltype(g)::value, decltype(nv)::value>(a, groups, st);
  });
  if (e != cudaSuccess || a.splits == 1 || (!a.dw && !a.db)) return e;
  const dim3 grid((unsigned)((a.K + 31) / 32), 2, (unsigned)groups);
  norm_bwd_join_kernel<PT><<<grid, 256, 0, st>>>(a.part, a.splits, a.K, static_cast<PT*>(a.dw),
                                                 a.lddw, static_cast<PT*>(a.db), a.lddb);
  return cudaGetLastError();
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
  svdq::NormArgs a{};
  a.x = X; a.w = weight; a.b = bias; a.y = Y; a.mean = mean; a.rstd = rstd;
  a.ldx = ldx; a.ldw = ldw; a.ldb = ldb; a.ldy = ldy;
  a.M = M; a.K = K; a.rows_per_group = rows_per_group;
  a.w0 = weight_offset; a.eps = eps;
  const cudaError_t e = svdq::dispatch_types(dtype, param_dtype, [&](auto t, auto pt) {
    return svdq::fwd<decltype(t), decltype(pt)>(a, stream);
  });
  return e == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

size_t svdq_layer_norm_backward_workspace(int M, int K, int rows_per_group) {
  if (M <= 0 || K < 1 || K > SVDQ_NORM_MAX_K || rows_per_group < 0) return 0;
  const int rpg = rows_per_group ? rows_per_group : M;
  const size_t groups = ((size_t)M + rpg - 1) / rpg;
  const int s = svdq::bwd_splits(M, rpg);
  return s == 1 ? 0 : groups * s * 2 * (size_t)K * sizeof(float);
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
    if ((dweight && cudaMemsetAsync(dweight, 0, (size_t)K * ps, stream) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, (size_t)K * ps, stream) != cudaSuccess))
      return SVDQ_ERR_CUDA;
    return SVDQ_OK;
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
  a.splits = svdq::bwd_splits(M, a.rows_per_group);
  const size_t need = (dweight || dbias) ? svdq_layer_norm_backward_workspace(M, K, rows_per_group) : 0;
  if (need) {
    if (!workspace) return SVDQ_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return SVDQ_ERR_ALIGNMENT;
    if (workspace_bytes < need) return SVDQ_ERR_SHAPE;
  }
  a.dy = dY; a.x = X; a.mean = mean; a.rstd = rstd; a.w = weight;
  a.dx = dX; a.dw = dweight; a.db = dbias; a.part = static_cast<float*>(workspace);
  a.lddy = lddy; a.ldx = ldx; a.ldw = ldw; a.lddx = lddx; a.lddw = lddw; a.lddb = lddb;
  a.M = M; a.K = K; a.w0 = weight_offset;
  const cudaError_t e = svdq::dispatch_types(dtype, param_dtype, [&](auto t, auto pt) {
    return svdq::bwd<decltype(t), decltype(pt)>(a, stream);
  });
  return e == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

}  // extern "C"
