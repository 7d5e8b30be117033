// 16-bit linear layer (bf16 or fp16 operands, fp32 accumulation on the
// tensor cores) and its gradients: three products of one kernel,
//   Y  = epi(X W^T + b) + R      A = X   (K-major), B = W (K-major)
//   dX = dP W                    A = dP  (K-major), B = W^T (MN-major)
//   dW = dP^T X                  A = dP^T, B = X^T  (both MN-major)
// where "K" is the product's reduction axis.  An operand whose reduction
// axis is contiguous in memory is K-major; one whose other axis is, is
// MN-major: TMA brings both as 128-byte-swizzled boxes, and the MMA's
// descriptors say which way they lie, so no transposed copy is ever made.
//
// Warp-specialised persistent CTAs, one per SM: warp 0 issues TMA, warp 1
// the tcgen05.mma kind::f16, warps 4-7 the epilogue; two TMEM accumulators
// let a tile accumulate while the previous one is stored.  Every wait is
// bounded (the device's operator error word is raised on expiry).
#include "elem.cuh"
#include "gemm16.cuh"

namespace svdq {

__device__ int g_op_err;      // sticky operator error word, one per device

int* op_err_address() {
  static int* at[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return nullptr;
  if (!at[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_op_err) != cudaSuccess) return nullptr;
    at[dev] = static_cast<int*>(p);
  }
  return at[dev];
}

namespace {

constexpr int G_THREADS = 256;
constexpr int G_EPI0 = 4;           // epilogue warps 4-7

template <int BN>
struct GLay {
  static constexpr int BM = 128;
  static constexpr int ST_A = BM * 128, ST_B = BN * 128;
  static constexpr int STAGE = ST_A + ST_B;
  static constexpr int NST = 4;
  static constexpr int OFF_BAR = NST * STAGE;
  static constexpr int N_BARS = 2 * NST + 5;      // the last one: drain after an expired wait
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static_assert(ALLOC <= 227 * 1024, "shared memory");
};

template <int BN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(G_THREADS, 1)
gemm16_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const G16Args p) {
  using L = GLay<BN>;
  constexpr int BM = L::BM, NST = L::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::OFF_BAR;
  auto st_full = [&](int s) { return bar0 + 8u * s; };
  auto st_empty = [&](int s) { return bar0 + 8u * (NST + s); };
  auto tm_full = [&](int b) { return bar0 + 8u * (2 * NST + b); };
  auto tm_empty = [&](int b) { return bar0 + 8u * (2 * NST + 2 + b); };
  const uint32_t drain = bar0 + 8u * (2 * NST + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  int* err = p.err;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NST; ++s) { mbar_init(st_full(s), 1); mbar_init(st_empty(s), 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(tm_full(b), 1); mbar_init(tm_empty(b), 4); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 2 * BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool alive = true;
      for (int t = blockIdx.x; t < p.num_tiles && alive; t += gridDim.x) {
        const int m0 = (t % p.tiles_m) * BM, n0 = (t / p.tiles_m) * BN;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int st = it % NST;
          if (!wait_or_abort(st_empty(st), ((it / NST) & 1) ^ 1, abort_flag, err)) { alive = false; break; }
          mbar_arrive_expect_tx(st_full(st), L::STAGE);
          const uint32_t da = sbase + st * L::STAGE, db = da + L::ST_A;
          if constexpr (A_MN) {
#pragma unroll
            for (int j = 0; j < BM / 64; ++j)
              tma_load_2d(da + j * 8192, &tm_a, m0 + 64 * j, kb * G_BK, st_full(st));
          } else {
            tma_load_2d(da, &tm_a, kb * G_BK, m0, st_full(st));
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int j = 0; j < BN / 64; ++j)
              tma_load_2d(db + j * 8192, &tm_b, n0 + 64 * j, kb * G_BK, st_full(st));
          } else {
            tma_load_2d(db, &tm_b, kb * G_BK, n0, st_full(st));
          }
        }
      }
      // no copy is in flight when the CTA ends
      for (uint32_t k = (it > NST ? it - NST : 0); k < it; ++k)
        mbar_wait_bounded(st_full(k % NST), (k / NST) & 1, LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = g_idesc(BM, BN, p.bf16 != 0, A_MN, B_MN);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    auto wait_warp = [&](uint32_t bar, uint32_t parity) -> bool {
      int ok = 1;
      if (lane == 0) ok = wait_or_abort(bar, parity, abort_flag, err) ? 1 : 0;
      return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
    };
    uint32_t it = 0, tb = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < p.num_tiles; t += gridDim.x, ++tb) {
      const int b = tb & 1;
      if (!wait_warp(tm_empty(b), ((tb >> 1) & 1) ^ 1)) { ok = false; break; }
      tc_fence_after();
      const uint32_t d = tm + b * BN;
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        const int st = it % NST;
        if (!wait_warp(st_full(st), (it / NST) & 1)) { ok = false; break; }
        tc_fence_after();
        if (g_elect()) {
          const uint64_t ad = g_sdesc<A_MN>(sbase + st * L::STAGE);
          const uint64_t bd = g_sdesc<B_MN>(sbase + st * L::STAGE + L::ST_A);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_bf16(d, ad + j * G_KSTEP<A_MN>, bd + j * G_KSTEP<B_MN>, idesc,
                     (kb > 0 || j > 0) ? 1u : 0u);
          mma_commit(st_empty(st));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (g_elect()) mma_commit(tm_full(b));
      __syncwarp();
    }
    // after an expired wait, TMEM is freed only once the issued MMAs are done
    if (!ok && g_elect()) {
      mma_commit(drain);
      mbar_wait_bounded(drain, 0, LIMIT_NS);
    }
    __syncwarp();
  } else if (warp >= G_EPI0) {
    const int q = warp & 3;
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    const bool bf16 = p.bf16 != 0;
    uint32_t tb = 0;
    for (int t = blockIdx.x; t < p.num_tiles; t += gridDim.x, ++tb) {
      const int m0 = (t % p.tiles_m) * BM, n0 = (t / p.tiles_m) * BN;
      const int row = m0 + 32 * q + lane;
      const int b = tb & 1;
      if (!wait_or_abort(tm_full(b), (tb >> 1) & 1, abort_flag, err)) break;
      tc_fence_after();
      __syncwarp();
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(tmem + b * BN + 32 * c + lane_off, r);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int col = n0 + 32 * c + 8 * u;
          if (row < p.M && col < p.N) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r[8 * u + e]);
            if (p.bias) {
              const uint4 bb = load8(p.bias, col, p.N);
              const uint32_t w[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2(w[e], bf16);
                v[2 * e] += f.x;
                v[2 * e + 1] += f.y;
              }
            }
            if (p.pre) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = pack2(make_float2(v[2 * e], v[2 * e + 1]), bf16);
              store8(p.pre + (long long)row * p.ldp, col, p.N, make_uint4(w[0], w[1], w[2], w[3]));
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = g_act(v[e], p.epilogue);
            if (p.res) {
              const uint4 bb = load8(p.res + (long long)row * p.ldr, col, p.N);
              const uint32_t w[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2(w[e], bf16);
                v[2 * e] += f.x;
                v[2 * e + 1] += f.y;
              }
            }
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack2(make_float2(v[2 * e], v[2 * e + 1]), bf16);
            store8(p.out + (long long)row * p.ldo, col, p.N, make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tm_empty(b));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * BN);
  }
}

// ------------------------------------------------ activation's gradient
// dP = dY epi'(P) rounded to 16 bits, and the column sums of its fp32 values.
__device__ __forceinline__ float g_act_grad(float x, int epilogue) {
  if (epilogue == SVDQ_EPI_GELU) {
    const float phi = 0.3989422804014327f * __expf(-0.5f * x * x);
    return 0.5f * (1.0f + erff(x * 0.70710678118654752f)) + x * phi;
  }
  const float s = 1.0f / (1.0f + __expf(-x));
  return s * (1.0f + x * (1.0f - s));
}

struct DpArgs {
  const uint16_t* dy;
  const uint16_t* p;       // pre-activation, null without an activation
  uint16_t* dp;            // null without an activation
  float* part;             // [row blocks][N8] column sums, or null
  long long lddy, ldp, lddp;
  int M, N, rows_per_block;
  int epilogue, bf16;
};

// 32 columns x 8 per thread by 8 rows of threads.
constexpr int DP_COLS = 256;
__global__ void __launch_bounds__(256)
dp_kernel(const DpArgs a) {
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * DP_COLS + tx * 8;
  const bool bf16 = a.bf16 != 0;
  const long long r0 = (long long)blockIdx.y * a.rows_per_block;
  const long long r1 = min((long long)a.M, r0 + a.rows_per_block);
  float acc[8] = {};
  if (c < a.N) {
    for (long long r = r0 + ty; r < r1; r += 8) {
      const uint4 d4 = load8(a.dy + r * a.lddy, c, a.N);
      uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w};
      if (a.p) {
        const uint4 p4 = load8(a.p + r * a.ldp, c, a.N);
        const uint32_t pw[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 d = unpack2(dw[e], bf16);
          const float2 x = unpack2(pw[e], bf16);
          d.x *= g_act_grad(x.x, a.epilogue);
          d.y *= g_act_grad(x.y, a.epilogue);
          acc[2 * e] += d.x;
          acc[2 * e + 1] += d.y;
          dw[e] = pack2(d, bf16);
        }
        store8(a.dp + r * a.lddp, c, a.N, make_uint4(dw[0], dw[1], dw[2], dw[3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 d = unpack2(dw[e], bf16);
          acc[2 * e] += d.x;
          acc[2 * e + 1] += d.y;
        }
      }
    }
  }
  if (!a.part) return;
  __shared__ float sh[8][DP_COLS + 8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sh[ty][tx * 8 + e] = acc[e];
  __syncthreads();
  const int col = blockIdx.x * DP_COLS + threadIdx.x;
  if (col < a.N) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sh[i][threadIdx.x];
    a.part[(size_t)blockIdx.y * a.N + col] = s;
  }
}

// db = the row blocks' sums in order: 32 columns by 8 rows of threads.
__global__ void __launch_bounds__(256)
db_join_kernel(const float* part, int blocks, int N, uint16_t* db, int bf16) {
  __shared__ float sh[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float acc = 0.0f;
  if (c < N) {
    const int b0 = blocks * ty / 8, b1 = blocks * (ty + 1) / 8;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) acc += part[(size_t)b * N + c];
  }
  sh[ty][tx] = acc;
  __syncthreads();
  if (ty == 0 && c < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += sh[i][tx];
    db[c] = (uint16_t)pack2(make_float2(acc, 0.0f), bf16 != 0);
  }
}

// Row blocks of dp_kernel: about four blocks per SM in all, of at least 32
// rows, so that the partial sums stay small beside the rows themselves.
int dp_row_blocks(int M, int N) {
  const int col_blocks = (int)(((long long)N + DP_COLS - 1) / DP_COLS);
  long long b = (4 * 148 + col_blocks - 1) / col_blocks;
  const long long most = ((long long)M + 31) / 32;
  if (b > most) b = most;
  return (int)(b < 1 ? 1 : b);
}

// --------------------------------------------------------------- launches
template <int BN, bool A_MN, bool B_MN>
cudaError_t launch_gemm_bn(const Operand& A, const Operand& B, G16Args a, cudaStream_t st) {
  using L = GLay<BN>;
  static bool attr[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(gemm16_kernel<BN, A_MN, B_MN>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    attr[dev] = true;
  }
  CUtensorMap ta, tb;
  if (!operand_map(&ta, A, L::BM, a.bf16 != 0) || !operand_map(&tb, B, BN, a.bf16 != 0))
    return cudaErrorInvalidValue;
  const long long tm = ((long long)A.rows + L::BM - 1) / L::BM, tn = ((long long)B.rows + BN - 1) / BN;
  if (tm * tn > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
  a.M = A.rows;
  a.N = B.rows;
  a.kblocks = (int)(((long long)A.red + G_BK - 1) / G_BK);
  a.tiles_m = (int)tm;
  a.tiles_n = (int)tn;
  a.num_tiles = (int)(tm * tn);
  const int grid = a.num_tiles < num_sms() ? a.num_tiles : num_sms();
  gemm16_kernel<BN, A_MN, B_MN><<<grid, G_THREADS, L::ALLOC, st>>>(ta, tb, a);
  return cudaGetLastError();
}

cudaError_t launch_gemm(const Operand& A, const Operand& B, G16Args a, cudaStream_t st) {
  a.err = op_err_address();
  if (!a.err) return cudaErrorInvalidDevice;
  if (A.rows > 256) return launch_gemm16_pair(A, B, a, st);
  if (A.mn) return launch_gemm_bn<128, true, true>(A, B, a, st);
  if (B.mn) return launch_gemm_bn<128, false, true>(A, B, a, st);
  return launch_gemm_bn<128, false, false>(A, B, a, st);
}

// Workspace of the backward call: dP, then the column sums' partials.
struct BwdLayout {
  size_t dp, part, total;
  long long lddp;
};
BwdLayout bwd_layout(int M, int N, int epilogue) {
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  BwdLayout L{};
  L.lddp = ((long long)N + 7) / 8 * 8;
  L.dp = 0;
  L.part = epilogue == SVDQ_EPI_NONE ? 0 : up((size_t)M * L.lddp * 2);
  L.total = L.part + up((size_t)dp_row_blocks(M, N) * N * sizeof(float));
  return L;
}

// Row and column indexes of a last, partial tile stay below 2^31.
bool sizes_fit(int M, int K, int N) {
  constexpr int most = 0x7FFFFC00;
  return M <= most && K <= most && N <= most;
}

bool ok_call(int dtype, int epilogue) {
  return (dtype == SVDQ_DTYPE_BF16 || dtype == SVDQ_DTYPE_F16) &&
         (epilogue == SVDQ_EPI_NONE || epilogue == SVDQ_EPI_GELU || epilogue == SVDQ_EPI_SILU);
}

}  // namespace
}  // namespace svdq

using svdq::rows_aligned16;

extern "C" {

svdq_status svdq_linear16(int dtype, int M, int K, int N, const void* X, int ldx, const void* W,
                          int ldw, const void* bias, const void* R, int ldr, int epilogue, void* Y,
                          int ldy, void* P, int ldp, cudaStream_t stream) {
  if (!svdq::ok_call(dtype, epilogue)) return SVDQ_ERR_INVALID_ARG;
  if (M < 0 || K < 1 || N < 1 || ldx < K || ldw < K || ldy < N || (R && ldr < N) || (P && ldp < N))
    return SVDQ_ERR_SHAPE;
  if (!svdq::sizes_fit(M, K, N)) return SVDQ_ERR_UNSUPPORTED;
  if (M == 0) return SVDQ_OK;
  if (!X || !W || !Y || Y == P || (R && (R == P || (R == Y && ldr != ldy)))) return SVDQ_ERR_INVALID_ARG;
  if (!rows_aligned16(X, ldx, 2) || !rows_aligned16(W, ldw, 2) || !rows_aligned16(Y, ldy, 2) ||
      (bias && !svdq::is_aligned16(bias)) || (R && !rows_aligned16(R, ldr, 2)) ||
      (P && !rows_aligned16(P, ldp, 2)))
    return SVDQ_ERR_ALIGNMENT;
  svdq::G16Args a{};
  a.bias = static_cast<const uint16_t*>(bias);
  a.res = static_cast<const uint16_t*>(R);
  a.out = static_cast<uint16_t*>(Y);
  a.pre = static_cast<uint16_t*>(P);
  a.ldr = ldr; a.ldo = ldy; a.ldp = ldp;
  a.epilogue = epilogue;
  a.bf16 = dtype == SVDQ_DTYPE_BF16;
  const svdq::Operand A{X, ldx, M, K, false}, B{W, ldw, N, K, false};
  return svdq::launch_gemm(A, B, a, stream) == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

size_t svdq_linear16_backward_workspace(int M, int K, int N, int epilogue) {
  if (M <= 0 || K < 1 || N < 1 || !svdq::ok_call(SVDQ_DTYPE_BF16, epilogue)) return 0;
  return svdq::bwd_layout(M, N, epilogue).total;
}

svdq_status svdq_linear16_backward(int dtype, int M, int K, int N, const void* dY, int lddy,
                                   const void* X, int ldx, const void* W, int ldw, const void* P,
                                   int ldp, int epilogue, void* dX, int lddx, void* dW, int lddw,
                                   void* db, void* workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  if (!svdq::ok_call(dtype, epilogue)) return SVDQ_ERR_INVALID_ARG;
  const bool act = epilogue != SVDQ_EPI_NONE;
  if (M < 0 || K < 1 || N < 1 || lddy < N || (dW && (ldx < K || lddw < K)) ||
      (dX && (ldw < K || lddx < K)) || (act && ldp < N))
    return SVDQ_ERR_SHAPE;
  if (!svdq::sizes_fit(M, K, N)) return SVDQ_ERR_UNSUPPORTED;
  if ((dW && !rows_aligned16(dW, lddw, 2)) || (db && (reinterpret_cast<uintptr_t>(db) & 1)))
    return SVDQ_ERR_ALIGNMENT;
  if (M == 0) {
    if ((dW && cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)K * 2, N, stream) != cudaSuccess) ||
        (db && cudaMemsetAsync(db, 0, (size_t)N * 2, stream) != cudaSuccess))
      return SVDQ_ERR_CUDA;
    return SVDQ_OK;
  }
  if (!dX && !dW && !db) return SVDQ_OK;
  if (!dY || (dW && !X) || (dX && !W) || (act && !P) || ((act || db) && !workspace))
    return SVDQ_ERR_INVALID_ARG;
  if (!rows_aligned16(dY, lddy, 2) || (dW && !rows_aligned16(X, ldx, 2)) ||
      (dX && (!rows_aligned16(W, ldw, 2) || !rows_aligned16(dX, lddx, 2))) ||
      (act && !rows_aligned16(P, ldp, 2)) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SVDQ_ERR_ALIGNMENT;
  const svdq::BwdLayout L = svdq::bwd_layout(M, N, epilogue);
  if ((act || db) && workspace_bytes < L.total) return SVDQ_ERR_SHAPE;
  const int bf16 = dtype == SVDQ_DTYPE_BF16;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const void* dP = dY;
  long long lddp = lddy;
  if (act || db) {
    svdq::DpArgs d{};
    d.dy = static_cast<const uint16_t*>(dY);
    d.lddy = lddy;
    d.M = M; d.N = N; d.epilogue = epilogue; d.bf16 = bf16;
    if (act) {
      d.p = static_cast<const uint16_t*>(P);
      d.ldp = ldp;
      d.dp = reinterpret_cast<uint16_t*>(base + L.dp);
      d.lddp = L.lddp;
      dP = d.dp;
      lddp = L.lddp;
    }
    if (db) d.part = reinterpret_cast<float*>(base + L.part);
    const int want = svdq::dp_row_blocks(M, N);
    d.rows_per_block = (int)(((long long)M + want - 1) / want);
    const int blocks = (int)(((long long)M + d.rows_per_block - 1) / d.rows_per_block);
    const dim3 grid((unsigned)(((long long)N + svdq::DP_COLS - 1) / svdq::DP_COLS), (unsigned)blocks);
    svdq::dp_kernel<<<grid, 256, 0, stream>>>(d);
    if (cudaGetLastError() != cudaSuccess) return SVDQ_ERR_CUDA;
    if (db) {
      svdq::db_join_kernel<<<(unsigned)(((long long)N + 31) / 32), 256, 0, stream>>>(
          d.part, blocks, N, static_cast<uint16_t*>(db), bf16);
      if (cudaGetLastError() != cudaSuccess) return SVDQ_ERR_CUDA;
    }
  }
  svdq::G16Args a{};
  a.epilogue = SVDQ_EPI_NONE;
  a.bf16 = bf16;
  if (dX) {
    a.out = static_cast<uint16_t*>(dX);
    a.ldo = lddx;
    const svdq::Operand A{dP, lddp, M, N, false}, B{W, ldw, K, N, true};
    if (svdq::launch_gemm(A, B, a, stream) != cudaSuccess) return SVDQ_ERR_CUDA;
  }
  if (dW) {
    a.out = static_cast<uint16_t*>(dW);
    a.ldo = lddw;
    const svdq::Operand A{dP, lddp, N, M, true}, B{X, ldx, K, M, true};
    if (svdq::launch_gemm(A, B, a, stream) != cudaSuccess) return SVDQ_ERR_CUDA;
  }
  return SVDQ_OK;
}

svdq_status svdq_get_op_error(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return SVDQ_ERR_CUDA;
  int v = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, svdq::g_op_err, sizeof(int), 0, cudaMemcpyDeviceToHost,
                                stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return SVDQ_ERR_CUDA;
  if (v == SVDQ_DEVERR_NONE) return SVDQ_OK;
  if (cudaMemcpyToSymbolAsync(svdq::g_op_err, &zero, sizeof(int), 0, cudaMemcpyHostToDevice,
                              stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return SVDQ_ERR_CUDA;
  return SVDQ_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
