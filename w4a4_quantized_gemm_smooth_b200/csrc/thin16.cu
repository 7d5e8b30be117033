// 16-bit linear layer for up to 16 rows of X (single tokens, small batches,
// the conditioning vector of a modulation layer): Y = epi(X W^T + b) + R.
//
// Bound by reading W once, so nothing is staged: a block owns 8 rows of W
// (output columns), its eight warps share out the reduction, and every thread
// loads 16 bytes of its rows of W and of X straight into the fragments of
// mma.sync m16n8k16 (X as the 16-row operand, eight rows of W as the other).  A
// thread's eight consecutive elements go to two products as (0, 1, 2, 3) and
// (4, 5, 6, 7), in W and X alike: the order of the reduction inside a run does
// not matter, and both operands keep it.  The warps' sums meet in shared memory,
// in order.
//
// The fifth-generation tensor cores would take 128 rows for one, and a tile's
// way through TMA, shared memory and TMEM costs 4 us before the first byte of
// the result leaves.
//
// One row of 12288 to 4608: 19.3 us, 5.9 TB/s; 8 rows 20.2, 16 rows 35 us (the
// tcgen05 kernels: 41).  One row of 4608 to 21504: 35 us, 5.7 TB/s; of 1152 to
// 6912: 5.9 us (8.7).  Four runs in flight measured best (three 20.8 us, five
// 20.0, eight 24.7 for the first size: more loads per thread, fewer threads);
// 16 or 32 rows of W a block were slower (22.8 us and more).
#include "elem.cuh"
#include "gemm16.cuh"

namespace svdq {
namespace {

constexpr int T_THREADS = 256, T_WARPS = T_THREADS / 32;

struct ThinArgs {
  const uint16_t* x;
  const uint16_t* w;
  long long ldx, ldw;
  int K;
  G16Out o;
};

template <bool BF16>
__device__ __forceinline__ void mma_thin(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An ordinary, coherent load of 16 bytes that stays where it stands, in a batch
// of U: with loads that the compiler may move the batch comes apart (one row of
// 12288 to 4608 26.3 us, 19.3 with this one).  Past the first-level cache that
// size takes 19.0 us, but 1152 to 6912, call by call from L2, 5.4 instead of 4.7.
__device__ __forceinline__ uint4 load_here(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// XT x 8 rows of X (1 or 2; with 1 the lower half of their operand is 0).
template <bool BF16, int XT>
__global__ void __launch_bounds__(T_THREADS)
thin16_kernel(const ThinArgs a) {
  constexpr int U = 4;                             // runs of 32 elements in flight
  constexpr int ROWS = 8, COLS = 8 * XT;
  __shared__ float part[T_WARPS][COLS][ROWS + 1];
  grid_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * ROWS, M = a.o.M, N = a.o.N;
  // rows past the end repeat the last one; their sums are not stored
  const uint16_t* w = a.w + (long long)min(n0 + g, N - 1) * a.ldw + 8 * t;
  const uint16_t* x[XT];
#pragma unroll
  for (int j = 0; j < XT; ++j) x[j] = a.x + (long long)min(8 * j + g, M - 1) * a.ldx + 8 * t;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto products = [&](const uint4& wq, const uint4 (&xq)[XT]) {
    const uint4 lo = xq[0], hi = XT > 1 ? xq[XT - 1] : make_uint4(0, 0, 0, 0);
    mma_thin<BF16>(acc, lo.x, hi.x, lo.y, hi.y, wq.x, wq.y);
    mma_thin<BF16>(acc, lo.z, hi.z, lo.w, hi.w, wq.z, wq.w);
  };
  const int runs = a.K / 32;                       // whole ones; a ragged one follows
  const int end = (int)((long long)runs * (warp + 1) / T_WARPS);
  for (int r0 = (int)((long long)runs * warp / T_WARPS); r0 < end; r0 += U) {
    uint4 wq[U], xq[U][XT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = 32 * (r0 + u);
      if (r0 + u < end) {
        wq[u] = load_here(w + k);
#pragma unroll
        for (int j = 0; j < XT; ++j) xq[u][j] = *reinterpret_cast<const uint4*>(x[j] + k);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r0 + u < end) products(wq[u], xq[u]);
  }
  if (a.K % 32 != 0 && warp == 0) {
    const int k = 32 * runs, n = a.K - k - 8 * t;  // n: elements of the thread's eight that exist
    uint4 wq = make_uint4(0, 0, 0, 0), xq[XT] = {};
    if (n > 0) {
      wq = load8(w + k, 0, n);
#pragma unroll
      for (int j = 0; j < XT; ++j) xq[j] = load8(x[j] + k, 0, n);
    }
    products(wq, xq);
  }
#pragma unroll
  for (int e = 0; e < 2 * XT; ++e) part[warp][g + 8 * (e >> 1)][2 * t + (e & 1)] = acc[e];
  __syncthreads();
  const G16Out& o = a.o;
  if (threadIdx.x >= ROWS * COLS) return;
  const int m = threadIdx.x / ROWS, r = threadIdx.x % ROWS, n = n0 + r;
  if (m >= M || n >= N) return;
  float v = part[0][m][r];
#pragma unroll
  for (int q = 1; q < T_WARPS; ++q) v += part[q][m][r];
  if (o.bias) v += unpack2(o.bias[n], BF16).x;
  if (o.pre) o.pre[m * o.ldp + n] = (uint16_t)pack2(make_float2(v, 0.0f), BF16);
  if (o.epilogue != SVDQ_EPI_NONE) v = g_act2(make_float2(v, v), o.epilogue).x;
  if (o.res) v += unpack2(o.res[m * o.ldr + n], BF16).x;
  o.out[m * o.ldo + n] = (uint16_t)pack2(make_float2(v, 0.0f), BF16);
}

template <bool BF16, int XT>
cudaError_t launch(const ThinArgs& a, cudaStream_t st) {
  return launch_op(thin16_kernel<BF16, XT>, dim3((unsigned)(((long long)a.o.N + 7) / 8)), T_THREADS, 0, 1, st, a);
}

template <bool BF16>
cudaError_t launch_type(const ThinArgs& a, cudaStream_t st) {
  return a.o.M <= 8 ? launch<BF16, 1>(a, st) : launch<BF16, 2>(a, st);
}

}  // namespace

cudaError_t launch_thin16(const void* X, long long ldx, const void* W, long long ldw, int K,
                          const G16Out& o, cudaStream_t st) {
  const ThinArgs a{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(W), ldx, ldw, K, o};
  return o.bf16 ? launch_type<true>(a, st) : launch_type<false>(a, st);
}

}  // namespace svdq
