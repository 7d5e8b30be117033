// Gradients of the 16-bit linear layer for up to 8 rows (the conditioning
// vectors of modulation layers, small batches): with dP = dY epi'(P), in fp32
// here, since no product takes 16-bit operands,
//   dX [M][K] = dP W,   dW [N][K] = dP^T X,   db [N] = sum_m dP.
//
// Both products walk the same N x K places, one reading W, the other writing
// dW, so one kernel does both: a thread owns C columns k of all rows of X
// and dX and goes down rows n of W, for each of which dX[m] += dP[m][n] W[n]
// and dW[n] = sum_m dP[m][n] X[m], in packed fp32.  A block's eight warps
// take every eighth row, their dX meet in shared memory, and the blocks' in
// the workspace, in order.  The activation's gradient is formed at the head
// of the block, for its own rows.
//
// Bound by reading W and writing dW once, and from four rows on by the packed
// products (2 M for every pair of places).  With the join of dX, GELU:
//   12288 to 4608   1 row 41 us (226 MB, 5.5 TB/s), 4 rows 54, 8 rows 84
//   1152 to 4608    1 row 8.7 us, 4 rows 10.5, 8 rows 13
// where the tensor-core kernels take 106 and 28 us for any of them.  With 16
// rows this way takes 213 and 20 us, those kernels 106 and 23, so 8 is the limit.
// (Branches between the loads cost up to a third of it: none is left but in an
// odd K's last block.)
#include "elem.cuh"
#include "gemm16.cuh"

namespace svdq {
namespace {

constexpr int B_THREADS = 256, B_WARPS = B_THREADS / 32;

struct ThinBwdArgs {
  const uint16_t* dy;
  const uint16_t* p;         // pre-activation, null without an activation
  const uint16_t* x;         // null without dW
  const uint16_t* w;         // null without dX
  uint16_t* dx;              // null, or not split
  uint16_t* dw;
  uint16_t* db;
  float* part;               // [splits][M][pitch] sums of dX when split
  long long lddy, ldp, ldx, ldw, lddx, lddw;
  int M, K, N, pitch, epilogue;
};

// MT: rows that M is rounded up to (the others are zeros); C: columns per
// thread (a vector of 16 or 8 bytes), so that the sums and X fit the registers.
template <int MT>
struct ThinBwd {
  static constexpr int C = MT <= 4 ? 8 : 4;
  static constexpr int U = 32 / C;               // rows of W in flight per warp
  static constexpr int COLS = 32 * C;            // columns of a block
  static constexpr int PER_SM = MT <= 2 ? 3 : 2;   // blocks per SM
  static constexpr int MG = MT < 16 / C ? MT : 16 / C;   // rows of dX that meet at a time
};

template <int C>
struct Cols16 {
  uint32_t q[C / 2];
};
// C 16-bit elements of which n exist (C: all, aligned).
template <int C>
__device__ __forceinline__ Cols16<C> load_cols(const uint16_t* at, int n) {
  Cols16<C> v;
  if (n >= C) {
    if constexpr (C == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(at);
      v.q[0] = u.x; v.q[1] = u.y; v.q[2] = u.z; v.q[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(at);
      v.q[0] = u.x; v.q[1] = u.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C / 2; ++j) v.q[j] = 0;
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < n) v.q[e >> 1] |= (uint32_t)at[e] << (16 * (e & 1));
  }
  return v;
}
template <int C>
__device__ __forceinline__ void store_cols(uint16_t* at, int n, const Cols16<C>& v) {
  if (n >= C) {
    if constexpr (C == 8)
      *reinterpret_cast<uint4*>(at) = make_uint4(v.q[0], v.q[1], v.q[2], v.q[3]);
    else
      *reinterpret_cast<uint2*>(at) = make_uint2(v.q[0], v.q[1]);
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < n) at[e] = (uint16_t)(v.q[e >> 1] >> (16 * (e & 1)));
  }
}

template <bool BF16, int MT>
__global__ void __launch_bounds__(B_THREADS, ThinBwd<MT>::PER_SM)
thin16_bwd_kernel(const ThinBwdArgs a) {
  using L = ThinBwd<MT>;
  constexpr int C = L::C, H = C / 2, U = L::U, MG = L::MG;
  __shared__ float2 grad[B_THREADS][MT];         // dP of up to 256 rows n, doubled for packed products
  __shared__ float meet[B_WARPS][MG][L::COLS];
  grid_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col0 = blockIdx.x * L::COLS, col = col0 + lane * C, left = a.K - col;
  const int n0 = (int)((long long)a.N * blockIdx.y / gridDim.y);
  const int n1 = (int)((long long)a.N * (blockIdx.y + 1) / gridDim.y);
  float2 xf[MT][H], acc[MT][H];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const Cols16<C> xq = load_cols<C>(a.x + m * a.ldx + col, a.x && m < a.M ? left : 0);
#pragma unroll
    for (int j = 0; j < H; ++j) {
      xf[m][j] = unpack2(xq.q[j], BF16);
      acc[m][j] = make_float2(0.0f, 0.0f);
    }
  }
  // Only the last block of an odd K has a vector that the row ends in; where
  // none can, lanes past the row load its start and store nothing, so that no
  // branch stands between the loads.
  const bool ragged = a.K % C != 0 && col0 + L::COLS > a.K;
  const int at = ragged || left > 0 ? col : 0;
  auto walk = [&](auto odd, int c0, int rows) {
    constexpr bool ODD = decltype(odd)::value;
    const uint16_t* w = a.w + (long long)c0 * a.ldw + at;
    uint16_t* dw = a.dw + (long long)c0 * a.lddw + at;
    for (int r0 = warp; r0 < rows; r0 += B_WARPS * U) {
      Cols16<C> wq[U] = {};
      if (a.w)
#pragma unroll
        for (int u = 0; u < U; ++u)
          wq[u] = load_cols<C>(w + (long long)min(r0 + B_WARPS * u, rows - 1) * a.ldw, ODD ? left : C);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + B_WARPS * u;
        if (r >= rows) break;
        float2 wf[H], o[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
          wf[j] = unpack2(wq[u].q[j], BF16);
          o[j] = make_float2(0.0f, 0.0f);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float2 d = grad[r][m];
#pragma unroll
          for (int j = 0; j < H; ++j) {
            acc[m][j] = __ffma2_rn(d, wf[j], acc[m][j]);
            o[j] = __ffma2_rn(d, xf[m][j], o[j]);
          }
        }
        if (a.dw && left > 0) {
          Cols16<C> q;
#pragma unroll
          for (int j = 0; j < H; ++j) q.q[j] = pack2(o[j], BF16);
          store_cols<C>(dw + (long long)r * a.lddw, ODD ? left : C, q);
        }
      }
    }
  };
  for (int c0 = n0; c0 < n1; c0 += B_THREADS) {
    const int rows = min(B_THREADS, n1 - c0);
    if (c0 > n0) __syncthreads();
    if ((int)threadIdx.x < rows) {
      const int n = c0 + threadIdx.x;
      // every load is out before the first is used; rows past M repeat the
      // last one and count as 0
      uint32_t dq[MT], pq[MT] = {};
#pragma unroll
      for (int m = 0; m < MT; ++m) dq[m] = a.dy[min(m, a.M - 1) * a.lddy + n];
      if (a.p)
#pragma unroll
        for (int m = 0; m < MT; ++m) pq[m] = a.p[min(m, a.M - 1) * a.ldp + n];
      float sum = 0.0f;
#pragma unroll
      for (int m = 0; m < MT; m += 2) {
        float2 d = unpack2(dq[m] | dq[m + 1] << 16, BF16);
        if (a.p) d = __fmul2_rn(d, g_act_grad2(unpack2(pq[m] | pq[m + 1] << 16, BF16), a.epilogue));
        if (m >= a.M) d.x = 0.0f;
        if (m + 1 >= a.M) d.y = 0.0f;
        sum = sum + d.x + d.y;
        grad[threadIdx.x][m] = make_float2(d.x, d.x);
        grad[threadIdx.x][m + 1] = make_float2(d.y, d.y);
      }
      if (a.db && blockIdx.x == 0) a.db[n] = (uint16_t)pack2(make_float2(sum, 0.0f), BF16);
    }
    __syncthreads();
    if (ragged)
      walk(std::true_type(), c0, rows);
    else
      walk(std::false_type(), c0, rows);
  }
  if (!a.w) return;
#pragma unroll
  for (int m0 = 0; m0 < MT; m0 += MG) {          // MG rows of dX at a time, the warps' sums in order
    if (m0 >= a.M) break;
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
      for (int j = 0; j < H; ++j)
        *reinterpret_cast<float2*>(&meet[warp][m][lane * C + 2 * j]) = acc[m0 + m][j];
    __syncthreads();
    for (int i = threadIdx.x; i < MG * L::COLS; i += B_THREADS) {
      const int m = i / L::COLS, c = i % L::COLS;
      if (m0 + m >= a.M || col0 + c >= a.K) continue;
      float s = meet[0][m][c];
#pragma unroll
      for (int q = 1; q < B_WARPS; ++q) s += meet[q][m][c];
      if (a.part)
        a.part[((size_t)blockIdx.y * a.M + m0 + m) * a.pitch + col0 + c] = s;
      else
        a.dx[(m0 + m) * a.lddx + col0 + c] = (uint16_t)pack2(make_float2(s, 0.0f), BF16);
    }
  }
}

template <int MT>
int splits_of(int M, int K, int N) {
  using L = ThinBwd<MT>;
  const int cols = (int)(((long long)K + L::COLS - 1) / L::COLS);
  // the blocks that fit at once, of at least 2 M rows each (8 for M < 4), so
  // that the partial sums stay below the traffic of W and dW
  long long s = (long long)L::PER_SM * 148 / cols;
  const int rows = 2 * (M < 4 ? 4 : M);
  const long long most = ((long long)N + rows - 1) / rows;
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s);
}

// f of the rows that M is rounded up to.
template <typename F>
auto with_rows(int M, F&& f) {
  if (M <= 2) return f(std::integral_constant<int, 2>());
  if (M <= 4) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 8>());
}

int pitch_of(int K) { return (int)(((long long)K + 7) / 8 * 8); }

}  // namespace

size_t thin16_bwd_workspace(int M, int K, int N) {
  const int s = with_rows(M, [&](auto mt) { return splits_of<decltype(mt)::value>(M, K, N); });
  return s == 1 ? 0 : (size_t)s * M * pitch_of(K) * sizeof(float);
}

cudaError_t launch_thin16_bwd(const ThinBwdCall& c, cudaStream_t st) {
  return with_rows(c.M, [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    using L = ThinBwd<MT>;
    const int splits = splits_of<MT>(c.M, c.K, c.N);
    ThinBwdArgs a{};
    a.dy = static_cast<const uint16_t*>(c.dy);
    a.p = static_cast<const uint16_t*>(c.p);
    a.x = static_cast<const uint16_t*>(c.x);
    a.w = static_cast<const uint16_t*>(c.w);
    a.dx = static_cast<uint16_t*>(c.dx);
    a.dw = static_cast<uint16_t*>(c.dw);
    a.db = static_cast<uint16_t*>(c.db);
    a.lddy = c.lddy; a.ldp = c.ldp; a.ldx = c.ldx; a.ldw = c.ldw; a.lddx = c.lddx; a.lddw = c.lddw;
    a.M = c.M; a.K = c.K; a.N = c.N; a.pitch = pitch_of(c.K); a.epilogue = c.epilogue;
    const bool joined = c.w && splits > 1;
    if (joined) a.part = static_cast<float*>(c.workspace);
    const dim3 grid((unsigned)(((long long)c.K + L::COLS - 1) / L::COLS), (unsigned)splits);
    cudaError_t e = c.bf16 ? launch_op(thin16_bwd_kernel<true, MT>, grid, B_THREADS, 0, 1, st, a)
                           : launch_op(thin16_bwd_kernel<false, MT>, grid, B_THREADS, 0, 1, st, a);
    if (e != cudaSuccess || !joined) return e;
    return launch_join(a.part, splits, c.M, c.K, a.pitch, a.dx, c.lddx, c.bf16, st);
  });
}

}  // namespace svdq
