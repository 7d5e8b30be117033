// 16-bit product on CTA pairs: 256 x BN output tiles, one tcgen05.mma
// (cta_group::2, M = 256) over both SMs of a cluster of two.
//
// Each CTA brings its 128 rows of A and its half of B's rows, so that an SM's
// shared memory takes and gives 64 bytes a cycle each at the tensor cores'
// full rate; a single CTA's 128 x 256 tile needs 96 + 96 of the 128 there
// are.  The even CTA issues the MMAs; both load and both store their half of
// the rows.
//
// Persistent, static round-robin over the tiles; 12 warps:
//   warp 0       TMA producer: stages of 64 reduction elements; the pair's
//                bytes complete on the even CTA's barrier;
//   warp 1       MMA issuer (even CTA); its commits reach both CTAs;
//   warp 2       TMEM owner: two accumulators of BN <= 256 columns;
//   warps 4-11   epilogue: warp w owns TMEM lanes 32 (w % 4).. and one half
//                of the columns, in boxes of 32 x 32 that leave by TMA.  The
//                residual's boxes come by TMA into the same place before.
//
// 4608 x 12288 to 4608 (bf16, bias and residual): 361 us alone (1445 TFLOP/s,
// tensor pipe 77 % of the time: 324 tiles are 4.4 rounds of 74 pairs), 430 us
// back to back, where the power limit sets the clock (1.2 GHz).  8192^3: 718
// us, 1531 TFLOP/s.  Not kept: 192 columns for the first size (six full
// rounds; 450 us back to back: more operand traffic per product costs power),
// sleeping waits (no change), bands of equal height (no change).
#include "elem.cuh"
#include "gemm16.cuh"

namespace svdq {
namespace {

constexpr int P_THREADS = 384;
constexpr int P_EPI0 = 4, P_EPI = 8;        // epilogue warps 4-11

template <int BN>
struct PLay {
  static constexpr int ST_A = 128 * 128, ST_B = BN / 2 * 128;     // one CTA's share
  static constexpr int STAGE = ST_A + ST_B;
  static constexpr int NST = BN == 256 ? 5 : BN == 192 ? 6 : 8;
  static constexpr int BOX = 32 * 64;                             // 32 rows x 32 elements
  static constexpr int CH = BN / 64;                              // boxes per epilogue warp and tile
  static constexpr int OFF_Y = NST * STAGE;                       // a place for each box
  static constexpr int OFF_BIAS = OFF_Y + P_EPI * CH * BOX;       // 32 floats per epilogue warp
  static constexpr int OFF_BAR = OFF_BIAS + P_EPI * 128;
  // full[NST], empty[NST], tm_full[2], tm_empty[2], residual[8], drain
  static constexpr int N_BARS = 2 * NST + 4 + P_EPI + 1;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static_assert(STAGE % 1024 == 0 && ST_A % 1024 == 0, "swizzle atoms");
  static_assert(ALLOC <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Tiled load into this CTA's shared memory, completing on a barrier of the
// pair's even CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* tmap, int x, int y,
                                              uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once every prior MMA of
// this thread has completed.
__device__ __forceinline__ void commit_pair(uint32_t mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(mbar), "h"((uint16_t)3) : "memory");
}

template <int BN, bool GRAD>
__global__ void __launch_bounds__(P_THREADS, 1)
gemm16_pair_kernel(const __grid_constant__ G16Problem p0, const __grid_constant__ G16Problem p1,
                   const int total, const int bf16, int* err) {
  using L = PLay<BN>;
  constexpr int NST = L::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::OFF_BAR;
  auto st_full = [&](int s) { return bar0 + 8u * s; };
  auto st_empty = [&](int s) { return bar0 + 8u * (NST + s); };
  auto tm_full = [&](int b) { return bar0 + 8u * (2 * NST + b); };
  auto tm_empty = [&](int b) { return bar0 + 8u * (2 * NST + 2 + b); };
  auto r_full = [&](int w) { return bar0 + 8u * (2 * NST + 4 + w); };
  const uint32_t drain = bar0 + 8u * (2 * NST + 4 + P_EPI);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (tid == 32) {
    prefetch_map(&p0.a);
    prefetch_map(&p0.b);
    prefetch_map(&p0.y);
  }
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) { mbar_init(st_full(s), 1); mbar_init(st_empty(s), 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(tm_full(b), 1); mbar_init(tm_empty(b), 2 * P_EPI); }
    for (int w = 0; w < P_EPI; ++w) mbar_init(r_full(w), 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                 // the peer's barriers are ready
  tc_fence_after();
  grid_wait();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------- TMA producer
      uint32_t it = 0;
      bool alive = true;
      for (int t = pair; t < total && alive; t += pairs) {
        const bool first = t < p0.tiles;
        const G16Problem& p = first ? p0 : p1;
        const TilePos pos = tile_pos(first ? t : t - p0.tiles, p.tiles_m, p.tiles_n);
        const int m0 = pos.m * 256 + 128 * rank, n0 = pos.n * BN + BN / 2 * rank;
        const int kblocks = p.kblocks;
        const bool a_mn = GRAD && !first;
        constexpr bool b_mn = GRAD;
        const uint32_t bytes = 2 * (p.a_bytes + L::ST_B);
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int st = it % NST;
          if (!g_wait(st_empty(st), ((it / NST) & 1) ^ 1, abort_flag, err)) { alive = false; break; }
          const uint32_t full = map_rank(st_full(st), 0);
          if (rank == 0) mbar_arrive_expect_tx(st_full(st), bytes);
          const uint32_t da = sbase + st * L::STAGE, db = da + L::ST_A;
          if (a_mn) {
#pragma unroll
            for (int j = 0; j < 2; ++j) tma_load_pair(da + j * 8192, &p.a, m0 + 64 * j, kb * G_BK, full);
          } else {
            tma_load_pair(da, &p.a, kb * G_BK, m0, full);
          }
          if (b_mn) {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j) tma_load_pair(db + j * 8192, &p.b, n0 + 64 * j, kb * G_BK, full);
          } else {
            tma_load_pair(db, &p.b, kb * G_BK, n0, full);
          }
        }
      }
      // no copy is in flight when the CTA ends: every stage has been consumed
      // (after an expired wait elsewhere, the bounded wait outlasts the copies)
      for (uint32_t k = (it > NST ? it - NST : 0); k < it; ++k)
        if (!mbar_wait_bounded(st_empty(k % NST), (k / NST) & 1, LIMIT_NS)) break;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------ MMA issuer
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      auto wait_warp = [&](uint32_t bar, uint32_t parity) -> bool {
        int ok = 1;
        if (lane == 0) ok = g_wait(bar, parity, abort_flag, err) ? 1 : 0;
        return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
      };
      uint32_t it = 0, tb = 0;
      bool ok = true;
      for (int t = pair; t < total; t += pairs, ++tb) {
        const int b = tb & 1;
        if (!wait_warp(tm_empty(b), ((tb >> 1) & 1) ^ 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tm + b * 256;
        // read from the parameters themselves: uniform
        const bool first = t < p0.tiles;
        const bool a_mn = GRAD && !first;
        constexpr bool b_mn = GRAD;
        const uint32_t idesc = g_idesc(256, BN, bf16 != 0, a_mn, b_mn);
        const uint64_t ak = g_kstep(a_mn), bk = g_kstep(b_mn);
        const int kblocks = first ? p0.kblocks : p1.kblocks;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int st = it % NST;
          if (!wait_warp(st_full(st), (it / NST) & 1)) { ok = false; break; }
          tc_fence_after();
          if (g_elect()) {
            const uint64_t ad = g_sdesc(sbase + st * L::STAGE, a_mn);
            const uint64_t bd = g_sdesc(sbase + st * L::STAGE + L::ST_A, b_mn);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_pair(d, ad + j * ak, bd + j * bk, idesc,
                       (kb > 0 || j > 0) ? 1u : 0u);
            commit_pair(st_empty(st));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (g_elect()) commit_pair(tm_full(b));
        __syncwarp();
      }
      // after an expired wait, TMEM is freed only once the issued MMAs are done
      if (!ok && g_elect()) {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(drain) : "memory");
        mbar_wait_bounded(drain, 0, LIMIT_NS);
      }
      __syncwarp();
    }
  } else if (warp >= P_EPI0) {
    // ------------------------------------------------------ epilogue
    const int w = warp - P_EPI0, q = warp & 3, half = w >> 2;
    constexpr int CH = L::CH;                         // 32-column boxes of this warp
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    uint8_t* stage = smem + L::OFF_Y + w * CH * L::BOX;
    const uint32_t stage_u = smem_u32(stage);
    float* bias_s = reinterpret_cast<float*>(smem + L::OFF_BIAS + w * 128);
    const uint32_t tm_empty0[2] = {map_rank(tm_empty(0), 0), map_rank(tm_empty(1), 0)};
    uint32_t tb = 0, rb = 0;                          // tiles so far, and those with a residual
    for (int t = pair; t < total; t += pairs, ++tb) {
      const bool first = t < p0.tiles;
      const G16Problem& pr = first ? p0 : p1;
      const G16Out p = pr.o;
      const bool has_r = p.res != nullptr;
      const TilePos pos = tile_pos(first ? t : t - p0.tiles, pr.tiles_m, pr.tiles_n);
      const int m0 = pos.m * 256 + 128 * rank + 32 * q, n0 = pos.n * BN + BN / 2 * half;
      const int b = tb & 1;
      const int row = m0 + lane;
      float bias[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = n0 + 32 * c + lane;
        bias[c] = p.bias && col < p.N ? unpack2(p.bias[col], p.bf16 != 0).x : 0.0f;
      }
      if (lane == 0) {
        tma_store_wait_read0();                       // the previous tile's boxes have left
        if (has_r) {
          mbar_arrive_expect_tx(r_full(w), CH * L::BOX);
#pragma unroll
          for (int c = 0; c < CH; ++c)
            tma_load_2d(stage_u + c * L::BOX, &pr.r, n0 + 32 * c, m0, r_full(w));
        }
      }
      bool alive = g_wait(tm_full(b), (tb >> 1) & 1, abort_flag, err);
      if (has_r) {
        // also after an expired wait: the boxes land before the CTA ends
        alive = mbar_wait_bounded(r_full(w), rb & 1, LIMIT_NS) && alive;
        ++rb;
      }
      if (!__all_sync(0xFFFFFFFFu, alive)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < CH; c += 2) {
        constexpr int TWO = 2;
        uint32_t r[TWO][32];
        const int n = CH - c < TWO ? CH - c : TWO;    // known at compile time
#pragma unroll
        for (int k = 0; k < n; ++k) tmem_ld32(tmem + b * 256 + BN / 2 * half + 32 * (c + k) + lane_off, r[k]);
        tmem_wait_ld();
        if (c + TWO >= CH) {                          // the accumulator may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(tm_empty0[b]);
        }
#pragma unroll
        for (int k = 0; k < n; ++k) {
          const int col0 = n0 + 32 * (c + k);
          __syncwarp();
          bias_s[lane] = bias[c + k];
          __syncwarp();
          const bool boxed = g_boxed(p, col0);
          g_epilogue_box(p, r[k], bias_s, stage + (c + k) * L::BOX, lane, row, col0, boxed);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && boxed) {
            tma_store_2d(&pr.y, col0, m0, stage_u + (c + k) * L::BOX);
            tma_store_commit();
          }
        }
      }
    }
    if (lane == 0) tma_store_wait_read0();      // the boxes have left; the grid's end orders the writes
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                 // no MMA reads the peer's memory, no arrival is under way
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int BN, bool GRAD>
cudaError_t launch_bn(const G16Launch& l, cudaStream_t st) {
  using L = PLay<BN>;
  static bool attr[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(gemm16_pair_kernel<BN, GRAD>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    attr[dev] = true;
  }
  G16Problem p[2];
  if (!make_problems(p, l, [](G16Problem* q, const Operand& A, const Operand& B, const G16Out& o) {
        return make_problem(q, A, B, o, 256, BN, 128, BN / 2, true);
      }))
    return cudaErrorInvalidValue;
  const int total = p[0].tiles + p[1].tiles;
  const int pairs = total < num_sms() / 2 ? total : num_sms() / 2;
  return launch_op(gemm16_pair_kernel<BN, GRAD>, dim3(2 * pairs), P_THREADS, L::ALLOC, 2, st, p[0], p[1],
                   total, l.bf16, l.err);
}

}  // namespace

cudaError_t launch_gemm16_pair(const G16Launch& l, int bn, cudaStream_t st) {
  if (l.kind == G16Kind::Gradients)      // half of 192 MN-major columns is no whole number of boxes
    return bn == 128 ? launch_bn<128, true>(l, st) : launch_bn<256, true>(l, st);
  if (bn == 128) return launch_bn<128, false>(l, st);
  if (bn == 192) return launch_bn<192, false>(l, st);
  return launch_bn<256, false>(l, st);
}

}  // namespace svdq
