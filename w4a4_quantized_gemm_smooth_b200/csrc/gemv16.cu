// 16-bit linear layer for a few rows (single tokens, the conditioning vector
// of a modulation layer): Y = epi(X W^T + b) + R for M <= 4.
//
// Bound by reading W once.  A warp owns NR rows of W (output columns) and
// walks along them with 16-byte loads, several of each row in flight; the rows
// of X wait in shared memory as they are, and each of their vectors serves NR
// rows of W.  Products and sums are fp32 on pairs; a warp's sums meet by
// exchange, and its lanes store an output each.  One row of 12288 to 4608: 21 us, 5.3
// TB/s; of 4608 to 21504: 36 us, 5.5 TB/s; of 1152 to 6912: 5.5 us.
#include "elem.cuh"
#include "gemm16.cuh"

namespace svdq {
namespace {

constexpr int V_THREADS = 256, V_WARPS = V_THREADS / 32;
constexpr int V_TILE = 4096;        // elements of a row of X in shared memory at a time

struct GemvArgs {
  const uint16_t* x;
  const uint16_t* w;
  long long ldx, ldw;
  int K;
  G16Out o;
};

template <bool BF16, int MR, int NR>
__global__ void __launch_bounds__(V_THREADS)
gemv16_kernel(const GemvArgs a) {
  __shared__ uint4 xs[MR][V_TILE / 8];
  grid_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * V_WARPS + warp) * NR;
  const int M = a.o.M, N = a.o.N;
  float2 acc[MR][NR];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[m][r] = make_float2(0.0f, 0.0f);
  const uint16_t* w[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) w[r] = a.w + (long long)min(n0 + r, N - 1) * a.ldw;
  for (int k0 = 0; k0 < a.K; k0 += V_TILE) {
    const int kt = min(V_TILE, a.K - k0);
    if (k0) __syncthreads();                       // the previous tile has been read
#pragma unroll
    for (int m = 0; m < MR; ++m)
      for (int v = threadIdx.x; v * 8 < kt; v += V_THREADS)
        xs[m][v] = m < M ? load8(a.x + m * a.ldx + k0, v * 8, kt) : make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (n0 >= N) continue;
    auto products = [&](int v, const uint4 (&q)[NR]) {
      float2 f[NR][4];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const uint32_t u[4] = {q[r].x, q[r].y, q[r].z, q[r].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) f[r][e] = unpack2(u[e], BF16);
      }
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        const uint4 xq = xs[m][v];
        const uint32_t u[4] = {xq.x, xq.y, xq.z, xq.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack2(u[e], BF16);
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[m][r] = __ffma2_rn(x, f[r][e], acc[m][r]);
        }
      }
    };
    constexpr int U = NR == 1 ? 8 : 4;             // vectors of each row in flight
    const int whole = kt / 8;                      // whole vectors; a ragged one follows
    int v = lane;
    for (; v + 32 * (U - 1) < whole; v += 32 * U) {
      uint4 q[U][NR];
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int r = 0; r < NR; ++r)
          q[j][r] = __ldg(reinterpret_cast<const uint4*>(w[r] + k0) + v + 32 * j);
#pragma unroll
      for (int j = 0; j < U; ++j) products(v + 32 * j, q[j]);
    }
    {
      uint4 q[U][NR];
#pragma unroll
      for (int j = 0; j < U - 1; ++j)              // what is left, at once as well
#pragma unroll
        for (int r = 0; r < NR; ++r)
          q[j][r] = v + 32 * j < whole ? __ldg(reinterpret_cast<const uint4*>(w[r] + k0) + v + 32 * j)
                                       : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < U - 1; ++j)
        if (v + 32 * j < whole) products(v + 32 * j, q[j]);
    }
    if (kt % 8 != 0 && lane == 0) {
      uint4 q[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) q[r] = load8(w[r] + k0, whole * 8, kt);
      products(whole, q);
    }
  }
  if (n0 >= N) return;
  // lane m NR + r takes the sum of (m, r)
  float mine = 0.0f;
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float s = warp_sum(acc[m][r].x + acc[m][r].y);
      if (lane == m * NR + r) mine = s;
    }
  const int m = lane / NR, n = n0 + lane % NR;
  if (m >= MR || m >= M || n >= N) return;
  const G16Out& o = a.o;
  if (o.bias) mine += unpack2(o.bias[n], BF16).x;
  if (o.pre) o.pre[m * o.ldp + n] = (uint16_t)pack2(make_float2(mine, 0.0f), BF16);
  if (o.epilogue != SVDQ_EPI_NONE) mine = g_act2(make_float2(mine, mine), o.epilogue).x;
  if (o.res) mine += unpack2(o.res[m * o.ldr + n], BF16).x;
  o.out[m * o.ldo + n] = (uint16_t)pack2(make_float2(mine, 0.0f), BF16);
}

template <bool BF16, int MR, int NR>
cudaError_t launch(const GemvArgs& a, cudaStream_t st) {
  const int per = V_WARPS * NR;
  return launch_op(gemv16_kernel<BF16, MR, NR>, dim3((unsigned)(((long long)a.o.N + per - 1) / per)),
                   V_THREADS, 0, 1, st, a);
}

// Rows of W a warp: one, or with one or two rows of X four where that still
// gives every SM a block (64 to 12288: 3.3 us with four, 4.7 with one; 1152 to
// 1152: 2.5 with one, 3.0 with four).  With three or four rows of X the sums
// of four would take the registers that keep loads in flight.
template <bool BF16>
cudaError_t launch_type(const GemvArgs& a, cudaStream_t st) {
  const bool wide = a.o.N >= 4 * V_WARPS * num_sms();
  if (a.o.M == 1) return wide ? launch<BF16, 1, 4>(a, st) : launch<BF16, 1, 1>(a, st);
  if (a.o.M == 2) return wide ? launch<BF16, 2, 4>(a, st) : launch<BF16, 2, 1>(a, st);
  return launch<BF16, 4, 1>(a, st);
}

}  // namespace

// One or two rows always come out ahead of the tensor-core kernels (1152 to
// 6912: 5.5 against 8.7 us, 4096 to 4096: 8.4 against 19.9); three or four
// unless the rows of W are many and short (1152 to 6912: 10.0 against 8.7,
// 12288 to 4608: 32 against 41).
bool gemv16_fits(int M, int K, int N) {
  return M <= 2 || (M <= 4 && (K > 2048 || N < 4 * V_WARPS * num_sms()));
}

cudaError_t launch_gemv16(const void* X, long long ldx, const void* W, long long ldw, int K,
                          const G16Out& o, cudaStream_t st) {
  const GemvArgs a{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(W), ldx, ldw, K, o};
  return o.bf16 ? launch_type<true>(a, st) : launch_type<false>(a, st);
}

}  // namespace svdq
