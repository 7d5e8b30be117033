// 16-bit product for outputs too small to fill the GPU with 256-row tiles:
// 128 x BN tiles, one CTA each, or one cluster of up to 8 CTAs that divide
// the reduction.
//
// A small product is bound by latency (launch, the first copies, the chain of
// stages), so it is spread over as many SMs as there are: narrower tiles
// first, then the reduction over a cluster.  The parts meet in shared memory:
// each CTA leaves its fp32 sums there, and after a cluster barrier each adds
// up its share of the columns over the CTAs, in rank order, and runs the
// epilogue on it.  No workspace, no atomics, one launch.
//
// An SM takes 64 bytes a cycle from L2, so a 128 x 128 tile's stage (32 KB)
// lasts 0.26 us whatever the tensor cores do, and a launch with one stage 4 to
// 6 us.  333 x 1153 to 2307 (fp16, GELU, residual, pre-activation): 9.8 us as
// 111 tiles of 128 x 64; 128 x 12288 to 1152: 16 us split by 8, 58 unsplit.
//
// 10 warps: TMA, MMA (and TMEM), eight epilogue warps.
#include "elem.cuh"
#include "gemm16.cuh"

namespace svdq {
namespace {

constexpr int S_THREADS = 320;
constexpr int S_EPI0 = 2, S_EPI = 8;

template <int BN>
struct SLay {
  static constexpr int ST_A = 128 * 128, ST_B = BN * 128;
  static constexpr int STAGE = ST_A + ST_B;
  static constexpr int NST = BN == 128 ? 5 : 8;
  static constexpr int BOX = 32 * 64;
  static constexpr int EW = BN >= 64 ? 2 : 1;                     // epilogue warps per lane quarter
  static constexpr int CH = BN / (32 * EW);                       // boxes per warp
  static constexpr int OFF_Y = NST * STAGE;                       // each warp's boxes
  static constexpr int OFF_BIAS = OFF_Y + S_EPI * CH * BOX;       // and their 32 floats each
  static constexpr int OFF_BAR = OFF_BIAS + S_EPI * CH * 128;
  static constexpr int N_BARS = 2 * NST + 1 + S_EPI + 1;          // full, empty, tm_full, residual, drain
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static constexpr int TM = BN < 32 ? 32 : BN;
  static_assert(128 * BN * 4 <= NST * STAGE, "the sums fit where the stages were");
  static_assert(ALLOC <= 227 * 1024, "shared memory");
};

template <int BN, bool GRAD>
__global__ void __launch_bounds__(S_THREADS, 1)
gemm16_split_kernel(const __grid_constant__ G16Problem p0, const __grid_constant__ G16Problem p1,
                    const int splits, const int bf16, int* err) {
  using L = SLay<BN>;
  constexpr int NST = L::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::OFF_BAR;
  auto st_full = [&](int s) { return bar0 + 8u * s; };
  auto st_empty = [&](int s) { return bar0 + 8u * (NST + s); };
  const uint32_t tm_full = bar0 + 8u * (2 * NST);
  auto r_full = [&](int w) { return bar0 + 8u * (2 * NST + 1 + w); };
  const uint32_t drain = bar0 + 8u * (2 * NST + 1 + S_EPI);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = splits > 1 ? (int)cluster_rank() : 0;
  const int tile = (int)blockIdx.x / splits;
  const bool first = tile < p0.tiles;
  const G16Problem& pr = first ? p0 : p1;
  const G16Out p = pr.o;
  const TilePos pos = tile_pos(first ? tile : tile - p0.tiles, pr.tiles_m, pr.tiles_n);
  const int m0 = pos.m * 128, n0 = pos.n * BN;
  // read from the parameters themselves: uniform, as the MMAs' operands have to be
  const int kblocks = first ? p0.kblocks : p1.kblocks;
  const int kb0 = (int)((long long)kblocks * rank / splits);
  const int kb1 = (int)((long long)kblocks * (rank + 1) / splits);
  const bool a_mn = GRAD && !first;
  constexpr bool b_mn = GRAD;

  if (tid == 32) {
    prefetch_map(&pr.a);
    prefetch_map(&pr.b);
  }
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) { mbar_init(st_full(s), 1); mbar_init(st_empty(s), 1); }
    mbar_init(tm_full, 1);
    for (int w = 0; w < S_EPI; ++w) mbar_init(r_full(w), 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), L::TM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_wait();
  const uint32_t tmem = *tmem_slot;

  const int w = warp - S_EPI0, q = warp & 3, half = w >> 2;
  const int row = m0 + 32 * q + lane;
  float* part = reinterpret_cast<float*>(smem);             // [column][128 rows], after the stages
  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int st = it % NST;
        if (!g_wait(st_empty(st), ((it / NST) & 1) ^ 1, abort_flag, err)) break;
        mbar_arrive_expect_tx(st_full(st), pr.a_bytes + L::ST_B);
        const uint32_t da = sbase + st * L::STAGE, db = da + L::ST_A;
        if (a_mn) {
#pragma unroll
          for (int j = 0; j < 2; ++j) tma_load_2d(da + j * 8192, &pr.a, m0 + 64 * j, kb * G_BK, st_full(st));
        } else {
          tma_load_2d(da, &pr.a, kb * G_BK, m0, st_full(st));
        }
        if (b_mn) {
#pragma unroll
          for (int j = 0; j < BN / 64; ++j) tma_load_2d(db + j * 8192, &pr.b, n0 + 64 * j, kb * G_BK, st_full(st));
        } else {
          tma_load_2d(db, &pr.b, kb * G_BK, n0, st_full(st));
        }
      }
      // no copy is in flight when the stages are given to the sums
      for (uint32_t k = (it > NST ? it - NST : 0); k < it; ++k)
        mbar_wait_bounded(st_full(k % NST), (k / NST) & 1, LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = g_idesc(128, BN, bf16 != 0, a_mn, b_mn);
    const uint64_t ak = g_kstep(a_mn), bk = g_kstep(b_mn);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    uint32_t it = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int st = it % NST;
      int got = 1;
      if (lane == 0) got = g_wait(st_full(st), (it / NST) & 1, abort_flag, err) ? 1 : 0;
      if (!__shfl_sync(0xFFFFFFFFu, got, 0)) { ok = false; break; }
      tc_fence_after();
      if (g_elect()) {
        const uint64_t ad = g_sdesc(sbase + st * L::STAGE, a_mn);
        const uint64_t bd = g_sdesc(sbase + st * L::STAGE + L::ST_A, b_mn);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_bf16(tm, ad + j * ak, bd + j * bk, idesc,
                   (kb > kb0 || j > 0) ? 1u : 0u);
        mma_commit(st_empty(st));
      }
      __syncwarp();
    }
    // the sums are ready; or, after an expired wait, the issued MMAs are done
    if (g_elect()) {
      mma_commit(ok ? tm_full : drain);
      if (!ok) mbar_wait_bounded(drain, 0, LIMIT_NS);
    }
    __syncwarp();
  } else {
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    const bool live = half < L::EW;
    uint8_t* stage = smem + L::OFF_Y + w * L::CH * L::BOX;
    const uint32_t stage_u = smem_u32(stage);
    float* bias_s = reinterpret_cast<float*>(smem + L::OFF_BIAS + w * L::CH * 128);
    const bool has_r = p.res != nullptr && splits == 1;
    const int c0 = half * L::CH;
    if (live && splits == 1) {
      if (has_r && lane == 0) {                     // all of the warp's residual boxes
        mbar_arrive_expect_tx(r_full(w), L::CH * L::BOX);
#pragma unroll
        for (int c = 0; c < L::CH; ++c)
          tma_load_2d(stage_u + c * L::BOX, &pr.r, n0 + 32 * (c0 + c), m0 + 32 * q, r_full(w));
      }
#pragma unroll
      for (int c = 0; c < L::CH; ++c) {
        const int col = n0 + 32 * (c0 + c) + lane;
        bias_s[32 * c + lane] = p.bias && col < p.N ? unpack2(p.bias[col], p.bf16 != 0).x : 0.0f;
      }
      __syncwarp();
    }
    bool alive = g_wait(tm_full, 0, abort_flag, err);
    // also after an expired wait: the residual's boxes land before the CTA ends
    if (live && has_r) alive = mbar_wait_bounded(r_full(w), 0, LIMIT_NS) && alive;
    alive = __all_sync(0xFFFFFFFFu, alive);
    tc_fence_after();
    if (live && alive) {
      uint32_t r[L::CH][32];
#pragma unroll
      for (int c = 0; c < L::CH; ++c) tmem_ld32(tmem + 32 * (c0 + c) + lane_off, r[c]);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < L::CH; ++c) {
        if (splits > 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            part[(32 * (c0 + c) + j) * 128 + 32 * q + lane] = __uint_as_float(r[c][j]);
        } else {
          const int col0 = n0 + 32 * (c0 + c);
          const bool boxed = g_boxed(p, col0);
          g_epilogue_box(p, r[c], bias_s + 32 * c, stage + c * L::BOX, lane, row, col0, boxed);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && boxed) {
            tma_store_2d(&pr.y, col0, m0 + 32 * q, stage_u + c * L::BOX);
            tma_store_commit();
          }
        }
      }
    }
    if (lane == 0) tma_store_wait_read0();          // the boxes have left; the grid's end orders the writes
    __syncwarp();
  }

  tc_fence_before();
  if (splits > 1) {
    cluster_sync();               // every CTA's sums are in its shared memory
    if (warp >= S_EPI0 && row < p.M) {
      const int cols = BN / splits;           // a multiple of 8
      for (int u = 8 * half; u < cols; u += 16) {
        const int cl = rank * cols + u, col = n0 + cl;
        if (col >= p.N) break;
        float2 v[4] = {};
        for (int s = 0; s < splits; ++s) {
          const uint32_t at = map_rank(sbase + (uint32_t)(cl * 128 + 32 * q + lane) * 4, s);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = __fadd2_rn(v[e], make_float2(lds32_cluster(at + e * 1024), lds32_cluster(at + e * 1024 + 512)));
        }
        g_epilogue_row(p, v, row, col);
      }
    }
    cluster_sync();               // no CTA leaves while its sums are read
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TM);
  }
}

template <int BN, bool GRAD>
cudaError_t launch_bn(const G16Launch& l, int splits, cudaStream_t st) {
  using L = SLay<BN>;
  static bool attr[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(gemm16_split_kernel<BN, GRAD>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    attr[dev] = true;
  }
  G16Problem p[2];
  if (!make_problems(p, l, [&](G16Problem* q, const Operand& A, const Operand& B, const G16Out& o) {
        return make_problem(q, A, B, o, 128, BN, 128, BN, splits == 1);
      }))
    return cudaErrorInvalidValue;
  return launch_op(gemm16_split_kernel<BN, GRAD>, dim3((unsigned)((p[0].tiles + p[1].tiles) * splits)),
                   S_THREADS, L::ALLOC, splits, st, p[0], p[1], splits, l.bf16, l.err);
}

}  // namespace

cudaError_t launch_gemm16_split(const G16Launch& l, int bn, int splits, cudaStream_t st) {
  if (l.kind == G16Kind::Gradients)      // MN-major boxes are 64 wide
    return bn == 64 ? launch_bn<64, true>(l, splits, st) : launch_bn<128, true>(l, splits, st);
  if (bn == 32) return launch_bn<32, false>(l, splits, st);
  if (bn == 64) return launch_bn<64, false>(l, splits, st);
  return launch_bn<128, false>(l, splits, st);
}

}  // namespace svdq
