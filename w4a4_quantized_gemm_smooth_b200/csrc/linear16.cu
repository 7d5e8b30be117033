// 16-bit linear layer (bf16 or fp16 operands, fp32 accumulation on the
// tensor cores) and its gradients: the entry points, the activation's
// gradient, and the choice among the product kernels.  Three products:
//   Y  = epi(X W^T + b) + R      A = X   (K-major), B = W (K-major)
//   dX = dP W                    A = dP  (K-major), B = W^T (MN-major)
//   dW = dP^T X                  A = dP^T, B = X^T  (both MN-major)
// where "K" is the product's reduction axis.  An operand whose reduction
// axis is contiguous in memory is K-major; one whose other axis is, is
// MN-major: TMA brings both as 128-byte-swizzled boxes, and the MMA's
// descriptors say which way they lie, so no transposed copy is ever made.
// Both gradients go out in one launch where one form suits both.  Few rows go
// another way (thin16.cu, thin16_bwd.cu).
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

// ------------------------------------------------ activation's gradient
// dP = dY epi'(P) rounded to 16 bits, and the column sums of its fp32 values.
// The rounding is the tensor cores' operand type: it adds half a step to each
// term of dX and dW, which makes their error against 64 bits 0.0023 of their
// size in bf16 (fp16 0.00029) where the outputs' own rounding is 0.0017
// (0.00021).  Two 16-bit parts of dP would take it away and double the products
// (75 us of 113 at 4096, 1152 to 4608).  Up to THIN_BWD_ROWS rows, whose
// products run in fp32, nothing is rounded, so that the error steps up with the
// next row.  Bound by memory: 4096 x 4608 with GELU 23 us with its join, 4.9 TB/s.
struct DpArgs {
  const uint16_t* dy;
  const uint16_t* p;       // pre-activation, null without an activation
  uint16_t* dp;            // null without an activation
  float* part;             // [row blocks][N] column sums, or null
  uint16_t* db;            // [N], for a single row block, or null
  long long lddy, ldp, lddp;
  int M, N, rows_per_block;
  int bf16;
};

// 32 columns x 8 per thread by 8 rows of threads.
constexpr int DP_COLS = 256;
template <int EPI>
__global__ void __launch_bounds__(256, 4)
dp_kernel(const DpArgs a) {
  grid_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * DP_COLS + tx * 8;
  const bool bf16 = a.bf16 != 0;
  const long long r0 = (long long)blockIdx.y * a.rows_per_block;
  const long long r1 = min((long long)a.M, r0 + a.rows_per_block);
  float2 acc[4] = {};
  auto walk = [&](auto whole) {
    // whole: the thread's eight columns lie in the row (vector accesses)
    const int n = decltype(whole)::value ? 8 : a.N - c;
    for (long long r = r0 + ty; r < r1; r += 8) {
      const uint4 d4 = load8(a.dy + c + r * a.lddy, 0, n);
      uint4 p4 = make_uint4(0, 0, 0, 0);
      if (EPI != SVDQ_EPI_NONE) p4 = load8(a.p + c + r * a.ldp, 0, n);
      uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w};
      const uint32_t pw[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 d = unpack2(dw[e], bf16);
        if (EPI != SVDQ_EPI_NONE) d = __fmul2_rn(d, g_act_grad2(unpack2(pw[e], bf16), EPI));
        acc[e] = __fadd2_rn(acc[e], d);
        dw[e] = pack2(d, bf16);
      }
      if (EPI != SVDQ_EPI_NONE) store8(a.dp + c + r * a.lddp, 0, n, make_uint4(dw[0], dw[1], dw[2], dw[3]));
    }
  };
  if (c + 8 <= a.N)
    walk(std::true_type());
  else if (c < a.N)
    walk(std::false_type());
  if (!a.part && !a.db) return;
  __shared__ float sh[8][DP_COLS + 8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    sh[ty][tx * 8 + 2 * e] = acc[e].x;
    sh[ty][tx * 8 + 2 * e + 1] = acc[e].y;
  }
  __syncthreads();
  const int col = blockIdx.x * DP_COLS + threadIdx.x;
  if (col < a.N) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sh[i][threadIdx.x];
    if (a.part)
      a.part[(size_t)blockIdx.y * a.N + col] = s;
    else
      a.db[col] = (uint16_t)pack2(make_float2(s, 0.0f), bf16);
  }
}

// The blocks' sums in order: 32 columns of a row by up to 32 rows of threads,
// each summing a contiguous share of the blocks, then the shares in order.
__global__ void __launch_bounds__(1024)
join_kernel(const float* part, int blocks, int cols, int pitch, uint16_t* out, long long ldo, int bf16) {
  __shared__ float sh[32][33];
  grid_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, rows = blockDim.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  const size_t block = (size_t)gridDim.y * pitch, at = (size_t)blockIdx.y * pitch + c;
  float acc = 0.0f;
  if (c < cols) {
    const int shift = __ffs(rows) - 1;         // a power of two
    const int b0 = (blocks * ty) >> shift, b1 = (blocks * (ty + 1)) >> shift;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) acc += part[b * block + at];
  }
  sh[ty][tx] = acc;
  __syncthreads();
  if (ty == 0 && c < cols) {
    acc = 0.0f;
    for (int i = 0; i < rows; i += 4) {
      const float v[4] = {sh[i][tx], sh[i + 1][tx], sh[i + 2][tx], sh[i + 3][tx]};
      acc = acc + v[0] + v[1] + v[2] + v[3];
    }
    out[blockIdx.y * ldo + c] = (uint16_t)pack2(make_float2(acc, 0.0f), bf16 != 0);
  }
}

// Row blocks of dp_kernel: no more than the four blocks per SM that fit at
// once (two more would take another round, 30 us instead of 22), of at least
// eight rows (gradients of 128 x 1152 to 4608: 29.4 us, 30.4 with 16, 36 with
// 64); a batch of up to 32 rows is one block, whose sums are db itself (no
// second launch: 32 x 512 to 512 7.8 us, 8.0 with two; 64 x 1152 to 4608 34 us
// in one block, 28.9 in eight).
int dp_row_blocks(int M, int N) {
  if (M <= 32) return 1;
  const int col_blocks = (int)(((long long)N + DP_COLS - 1) / DP_COLS);
  long long b = 4 * 148 / col_blocks;
  const long long most = ((long long)M + 7) / 8;
  if (b > most) b = most;
  return (int)(b < 1 ? 1 : b);
}

// --------------------------------------------------------------- launches
// ---- which kernel, tile width and split -------------------------------
// The launch takes the form whose time a small model puts lowest.  In it, a
// worker (a CTA pair, or a CTA) takes `step` us per stage of 64 reduction
// elements and `tile` us more per tile, and a launch takes `launch` us; the
// worker that has the first tile has the most of them.  The constants are
// fitted to measured launches (us, model / measured):
//   pair 256   4096 x 1152 to 4608          35 / 35    both gradients  75 / 75
//   pair 192   4096 x 1152 to 1152          20 / 21    777 x 1152 to 2304  15 / 16
//   pair 128   4096 x 1152 to 1152          17 / 18    both gradients of 777  21 / 22
//   split 128  777 x 1152 to 2304           13 / 13    128 x 12288 to 1152 by 8  16 / 16
//   split 64   333 x 1152 to 2304           10 / 10    1024 x 1152 to 1152  10 / 10
// The choice matters where the forms differ: 128 x 12288 to 1152 takes 16 us
// split by 8 and 67 on pairs, 4608 x 12288 to 4608 takes 370 us on pairs and
// 600 on single CTAs.
struct G16Choice {
  bool pair;
  int bn, splits;
  double us;
};

double model_us(const G16Launch& l, int bm, int bn, int splits, int workers, double launch, double tile,
                double step) {
  long long tiles[2] = {0, 0};
  int kb[2] = {0, 0};
  for (int i = 0; i < 2; ++i)
    if (l.A[i].p) {
      tiles[i] = (((long long)l.A[i].rows + bm - 1) / bm) * (((long long)l.B[i].rows + bn - 1) / bn);
      kb[i] = (int)(((long long)l.A[i].red + G_BK - 1) / G_BK);
    }
  // the first worker's tiles of each problem, workers apart
  const long long n0 = (tiles[0] + workers - 1) / workers;
  const long long all = (tiles[0] + tiles[1] + workers - 1) / workers;
  const long long n1 = all - n0;
  auto part = [&](long long n, int k) { return n * (((k + splits - 1) / splits) * step + tile); };
  return launch + part(n0, kb[0]) + part(n1, kb[1]);
}

G16Choice choose_gemm16(const G16Launch& l) {
  const bool grad = l.kind == G16Kind::Gradients;
  const int sms = num_sms();
  G16Choice best{true, 256, 1, 1e30};
  auto offer = [&](bool pair, int bn, int splits, double us) {
    if (us < best.us) best = {pair, bn, splits, us};
  };
  offer(true, 256, 1, model_us(l, 256, 256, 1, sms / 2, 10.5, 0.8, 0.30));
  if (!grad) offer(true, 192, 1, model_us(l, 256, 192, 1, sms / 2, 9.5, 0.7, 0.26));
  offer(true, 128, 1, model_us(l, 256, 128, 1, sms / 2, 8.0, 0.7, 0.24));
  int kb = 1 << 30, rows = 128;
  for (int i = 0; i < 2; ++i)
    if (l.A[i].p) {
      const int k = (int)(((long long)l.A[i].red + G_BK - 1) / G_BK);
      if (k < kb) kb = k;
      if (!l.A[i].mn && l.A[i].rows < rows) rows = l.A[i].rows;
    }
  for (int bn = 128; bn >= (grad ? 64 : 32); bn >>= 1)
    for (int s = 1; s <= 8 && s <= kb && bn / s >= 8; s <<= 1) {
      // clusters of 4 and 8 do not fill every SM
      const int ctas = s == 8 ? sms - 20 : s == 4 ? sms - 4 : sms;
      const double step = 0.05 + 0.25 * (rows + bn) / 256.0;
      offer(false, bn, s, model_us(l, 128, bn, s, ctas / s, 1.5 + bn / 85.0, 3.0 + bn / 85.0 + (s > 1 ? 1.5 : 0.0), step));
    }
  return best;
}

// The launches of a call and their forms.
struct G16Plan {
  int launches;
  G16Launch l[2];
  G16Choice c[2];
};

G16Plan plan_gemm(const G16Launch& l) {
  // Two launches where the two gradients want different forms (16 x 64 to
  // 12288: 16.5 us, 52 in one launch; 16 x 1152 to 4608: 23, 28) and the model
  // puts their sum a tenth lower: one launch fills the GPU better and saves the
  // second start (16 x 512 to 512: 6.9 us, 10.6 in two launches).
  const G16Choice both = choose_gemm16(l);
  if (l.A[0].p && l.A[1].p) {
    G16Plan two{2, {l, l}, {}};
    two.l[0].A[1].p = two.l[1].A[0].p = nullptr;
    for (int i = 0; i < 2; ++i) two.c[i] = choose_gemm16(two.l[i]);
    if (two.c[0].us + two.c[1].us < 0.9 * both.us) return two;
  }
  return {1, {l, l}, {both, both}};
}

cudaError_t launch_gemm(G16Launch& l, cudaStream_t st) {
  l.err = op_err_address();
  if (!l.err) return cudaErrorInvalidDevice;
  const G16Plan plan = plan_gemm(l);
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < plan.launches && e == cudaSuccess; ++i) {
    const G16Choice& c = plan.c[i];
    e = c.pair ? launch_gemm16_pair(plan.l[i], c.bn, st) : launch_gemm16_split(plan.l[i], c.bn, c.splits, st);
  }
  return e;
}

// The operands of the gradients' products, dX at 0 and dW at 1.
void set_gradient(G16Launch& l, int i, const void* dP, long long lddp, const void* other, long long ldo, int M,
                  int K, int N) {
  if (i == 0) {
    l.A[0] = {dP, lddp, M, N, false};
    l.B[0] = {other, ldo, K, N, true};
  } else {
    l.A[1] = {dP, lddp, N, M, true};
    l.B[1] = {other, ldo, K, M, true};
  }
}

// Workspace of a backward call: dP of an activation, then the partial column
// sums of db; or, for few rows, the partial sums of dX.  What a call does not
// ask for takes no room, so that `need` of a call is at most that of the call
// for all three gradients, whatever K stands in the call for db alone.
struct BwdLayout {
  size_t dp, part, need;
  long long lddp;
  bool thin;
  int row_blocks;              // of dp_kernel
};
BwdLayout bwd_layout(int M, int K, int N, int epilogue, bool dX, bool dW, bool db) {
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  BwdLayout L{};
  L.thin = M <= THIN_BWD_ROWS && (dX || dW);
  if (L.thin) {
    L.need = dX ? up(thin16_bwd_workspace(M, K, N)) : 0;
    return L;
  }
  L.lddp = ((long long)N + 7) / 8 * 8;
  L.part = epilogue == SVDQ_EPI_NONE ? 0 : up((size_t)M * L.lddp * 2);
  L.row_blocks = dp_row_blocks(M, N);
  L.need = L.part + (db && L.row_blocks > 1 ? up((size_t)L.row_blocks * N * sizeof(float)) : 0);
  return L;
}

// Indexes of a last, partial tile (of up to 4096 elements) stay below 2^31.
bool sizes_fit(int M, int K, int N) {
  constexpr int most = 0x7FFF0000;
  return M <= most && K <= most && N <= most;
}

bool ok_call(int dtype, int epilogue) {
  return (dtype == SVDQ_DTYPE_BF16 || dtype == SVDQ_DTYPE_F16) &&
         (epilogue == SVDQ_EPI_NONE || epilogue == SVDQ_EPI_GELU || epilogue == SVDQ_EPI_SILU);
}

}  // namespace

cudaError_t launch_join(const float* part, int blocks, int rows, int cols, int pitch, uint16_t* out,
                        long long ldo, int bf16, cudaStream_t st) {
  const dim3 grid((unsigned)(((long long)cols + 31) / 32), (unsigned)rows);
  int ty = 4;                 // rows of threads: no more than there are blocks to sum
  while (ty < 32 && ty < blocks) ty *= 2;
  return launch_op(join_kernel, grid, 32 * ty, 0, 1, st, part, blocks, cols, pitch, out, ldo, bf16);
}

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
  {
    using svdq::extent_rows;
    const bool in_place = R == Y;
    const svdq::Extent x = extent_rows(X, M, K, ldx, 2), w = extent_rows(W, N, K, ldw, 2),
                       b = svdq::extent_flat(bias, 2ll * N), r = extent_rows(R, M, N, ldr, 2),
                       y = extent_rows(Y, M, N, ldy, 2), p = extent_rows(P, M, N, ldp, 2);
    if (svdq::overlaps_any(y, {x, w, b, in_place ? p : r, p}) || svdq::overlaps_any(p, {x, w, b, r}))
      return SVDQ_ERR_INVALID_ARG;
  }
  svdq::G16Launch l{};
  l.kind = svdq::G16Kind::Forward;
  l.bf16 = dtype == SVDQ_DTYPE_BF16;
  l.A[0] = {X, ldx, M, K, false};
  l.B[0] = {W, ldw, N, K, false};
  svdq::G16Out& o = l.o[0];
  o.bias = static_cast<const uint16_t*>(bias);
  o.res = static_cast<const uint16_t*>(R);
  o.out = static_cast<uint16_t*>(Y);
  o.pre = static_cast<uint16_t*>(P);
  o.ldr = ldr; o.ldo = ldy; o.ldp = ldp;
  o.epilogue = epilogue;
  o.bf16 = l.bf16;
  o.M = M;
  o.N = N;
  if (M <= svdq::THIN_ROWS)
    return svdq::status_of(svdq::launch_thin16(X, ldx, W, ldw, K, o, stream));
  return svdq::status_of(svdq::launch_gemm(l, stream));
}

size_t svdq_linear16_backward_workspace(int M, int K, int N, int epilogue) {
  if (M <= 0 || K < 1 || N < 1 || !svdq::ok_call(SVDQ_DTYPE_BF16, epilogue)) return 0;
  // the most that any choice of gradients needs: few rows go another way for db alone
  const size_t all = svdq::bwd_layout(M, K, N, epilogue, true, true, true).need;
  const size_t db = svdq::bwd_layout(M, K, N, epilogue, false, false, true).need;
  return all > db ? all : db;
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
    cudaError_t e = dW ? cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)K * 2, N, stream) : cudaSuccess;
    if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, (size_t)N * 2, stream);
    return svdq::status_of(e);
  }
  if (!dX && !dW && !db) return SVDQ_OK;
  const svdq::BwdLayout L = svdq::bwd_layout(M, K, N, epilogue, dX, dW, db);
  if (!dY || (dW && !X) || (dX && !W) || (act && !P) || (L.need && !workspace)) return SVDQ_ERR_INVALID_ARG;
  if (!rows_aligned16(dY, lddy, 2) || (dW && !rows_aligned16(X, ldx, 2)) ||
      (dX && (!rows_aligned16(W, ldw, 2) || !rows_aligned16(dX, lddx, 2))) ||
      (act && !rows_aligned16(P, ldp, 2)) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SVDQ_ERR_ALIGNMENT;
  if (L.need && workspace_bytes < L.need) return SVDQ_ERR_SHAPE;
  {
    using svdq::extent_rows;
    const svdq::Extent dy = extent_rows(dY, M, N, lddy, 2), x = extent_rows(dW ? X : nullptr, M, K, ldx, 2),
                       w = extent_rows(dX ? W : nullptr, N, K, ldw, 2),
                       p = extent_rows(act ? P : nullptr, M, N, ldp, 2),
                       ws = svdq::extent_flat(workspace, (long long)L.need),
                       gx = extent_rows(dX, M, K, lddx, 2), gw = extent_rows(dW, N, K, lddw, 2),
                       gb = svdq::extent_flat(db, 2ll * N);
    if (svdq::overlaps_any(gx, {dy, x, w, p, ws, gw, gb}) || svdq::overlaps_any(gw, {dy, x, w, p, ws, gb}) ||
        svdq::overlaps_any(gb, {dy, x, w, p, ws}) || svdq::overlaps_any(ws, {dy, x, w, p}))
      return SVDQ_ERR_INVALID_ARG;
  }
  const int bf16 = dtype == SVDQ_DTYPE_BF16;
  if (L.thin) {
    const svdq::ThinBwdCall c{dY, act ? P : nullptr, dW ? X : nullptr, dX ? W : nullptr, dX, dW, db, workspace,
                              lddy, ldp, ldx, ldw, lddx, lddw, M, K, N, epilogue, bf16};
    return svdq::status_of(svdq::launch_thin16_bwd(c, stream));
  }
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const void* dP = dY;
  long long lddp = lddy;
  if (act || db) {
    svdq::DpArgs d{};
    d.dy = static_cast<const uint16_t*>(dY);
    d.lddy = lddy;
    d.M = M; d.N = N; d.bf16 = bf16;
    if (act) {
      d.p = static_cast<const uint16_t*>(P);
      d.ldp = ldp;
      d.dp = reinterpret_cast<uint16_t*>(base + L.dp);
      d.lddp = L.lddp;
      dP = d.dp;
      lddp = L.lddp;
    }
    d.rows_per_block = (int)(((long long)M + L.row_blocks - 1) / L.row_blocks);
    const int blocks = (int)(((long long)M + d.rows_per_block - 1) / d.rows_per_block);
    const dim3 grid((unsigned)(((long long)N + svdq::DP_COLS - 1) / svdq::DP_COLS), (unsigned)blocks);
    if (db && blocks == 1)
      d.db = static_cast<uint16_t*>(db);
    else if (db)
      d.part = reinterpret_cast<float*>(base + L.part);
    auto kernel = epilogue == SVDQ_EPI_GELU   ? svdq::dp_kernel<SVDQ_EPI_GELU>
                  : epilogue == SVDQ_EPI_SILU ? svdq::dp_kernel<SVDQ_EPI_SILU>
                                              : svdq::dp_kernel<SVDQ_EPI_NONE>;
    cudaError_t e = svdq::launch_op(kernel, grid, 256, 0, 1, stream, d);
    if (e == cudaSuccess && d.part)
      e = svdq::launch_join(d.part, blocks, 1, N, N, static_cast<uint16_t*>(db), 0, bf16, stream);
    if (e != cudaSuccess) return svdq::status_of(e);
  }
  svdq::G16Launch l{};
  l.kind = svdq::G16Kind::Gradients;
  l.bf16 = bf16;
  auto set = [&](int i, const void* other, int ldo, void* out, int ld) {
    svdq::set_gradient(l, i, dP, lddp, other, ldo, M, K, N);
    l.o[i].out = static_cast<uint16_t*>(out);
    l.o[i].ldo = ld;
    l.o[i].epilogue = SVDQ_EPI_NONE;
    l.o[i].bf16 = bf16;
  };
  if (dX) set(0, W, ldw, dX, lddx);
  if (dW) set(1, X, ldx, dW, lddw);
  return svdq::status_of(dX || dW ? svdq::launch_gemm(l, stream) : cudaSuccess);
}

int svdq_debug_linear16_forms(int M, int K, int N, int gradients, int forms[2][3]) {
  if (M < 1 || K < 1 || N < 1 || !svdq::sizes_fit(M, K, N) || gradients < 0 || gradients > 3 || !forms) return 0;
  if (M <= (gradients ? svdq::THIN_BWD_ROWS : svdq::THIN_ROWS)) return 0;
  svdq::G16Launch l{};
  const void* there = &l;      // the choice goes by sizes, and by which operands there are
  if (gradients) {
    l.kind = svdq::G16Kind::Gradients;
    for (int i = 0; i < 2; ++i)
      if (gradients >> i & 1) svdq::set_gradient(l, i, there, N, there, K, M, K, N);
  } else {
    l.kind = svdq::G16Kind::Forward;
    l.A[0] = {there, K, M, K, false};
    l.B[0] = {there, K, N, K, false};
  }
  const svdq::G16Plan plan = svdq::plan_gemm(l);
  for (int i = 0; i < plan.launches; ++i) {
    forms[i][0] = plan.c[i].pair;
    forms[i][1] = plan.c[i].bn;
    forms[i][2] = plan.c[i].splits;
  }
  return plan.launches;
}

svdq_status svdq_get_op_error(cudaStream_t stream) {
  cudaError_t e = cudaStreamSynchronize(stream);
  int v = 0;
  const int zero = 0;
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(&v, svdq::g_op_err, sizeof(int), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess || v == SVDQ_DEVERR_NONE) return svdq::status_of(e);
  e = cudaMemcpyToSymbolAsync(svdq::g_op_err, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e == cudaSuccess ? SVDQ_ERR_DEVICE_TIMEOUT : svdq::status_of(e);
}

}  // extern "C"
