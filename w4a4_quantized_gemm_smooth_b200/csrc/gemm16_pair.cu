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
#include "gemm16.cuh"

namespace svdq {
namespace {

constexpr int P_THREADS = 384;
constexpr int P_EPI0 = 4, P_EPI = 8;        // epilogue warps 4-11

template <int BN>
struct PLay {
  static constexpr int ST_A = 128 * 128, ST_B = BN / 2 * 128;     // one CTA's share
  static constexpr int STAGE = ST_A + ST_B;
  static constexpr int NST = BN == 256 ? 6 : BN == 192 ? 6 : 7;
  static constexpr int BOX = 32 * 64;                             // 32 rows x 32 elements
  static constexpr int OFF_Y = NST * STAGE;                       // two boxes per epilogue warp
  static constexpr int OFF_BIAS = OFF_Y + P_EPI * 2 * BOX;        // 32 floats per epilogue warp
  static constexpr int OFF_BAR = OFF_BIAS + P_EPI * 128;
  // full[NST], empty[NST], tm_full[2], tm_empty[2], residual[8][2], drain
  static constexpr int N_BARS = 2 * NST + 4 + 2 * P_EPI + 1;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int ALLOC = OFF_MISC + 16 + 1024;
  static_assert(STAGE % 1024 == 0 && ST_A % 1024 == 0, "swizzle atoms");
  static_assert(ALLOC <= 227 * 1024, "shared memory");
};

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

// Output tile of index t: bands of 8 row tiles, walked column by column, so
// that the pairs at work together share A and B in L2.
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

template <int BN, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1)
gemm16_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_r,
                   const G16Args p) {
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
  auto r_full = [&](int w, int b) { return bar0 + 8u * (2 * NST + 4 + 2 * w + b); };
  const uint32_t drain = bar0 + 8u * (2 * NST + 4 + 2 * P_EPI);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (tid == 0) {
    for (int s = 0; s < NST; ++s) { mbar_init(st_full(s), 1); mbar_init(st_empty(s), 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(tm_full(b), 1); mbar_init(tm_empty(b), 2 * P_EPI); }
    for (int w = 0; w < P_EPI; ++w) { mbar_init(r_full(w, 0), 1); mbar_init(r_full(w, 1), 1); }
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
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------- TMA producer
      uint32_t it = 0;
      bool alive = true;
      for (int t = pair; t < p.num_tiles && alive; t += pairs) {
        const TilePos pos = tile_pos(t, p.tiles_m, p.tiles_n);
        const int m0 = pos.m * 256 + 128 * rank, n0 = pos.n * BN + BN / 2 * rank;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int st = it % NST;
          if (!wait_or_abort(st_empty(st), ((it / NST) & 1) ^ 1, abort_flag, p.err)) { alive = false; break; }
          const uint32_t full = map_rank(st_full(st), 0);
          if (rank == 0) mbar_arrive_expect_tx(st_full(st), 2 * L::STAGE);
          const uint32_t da = sbase + st * L::STAGE, db = da + L::ST_A;
          if constexpr (A_MN) {
#pragma unroll
            for (int j = 0; j < 2; ++j) tma_load_pair(da + j * 8192, &tm_a, m0 + 64 * j, kb * G_BK, full);
          } else {
            tma_load_pair(da, &tm_a, kb * G_BK, m0, full);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j) tma_load_pair(db + j * 8192, &tm_b, n0 + 64 * j, kb * G_BK, full);
          } else {
            tma_load_pair(db, &tm_b, kb * G_BK, n0, full);
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
      const uint32_t idesc = g_idesc(256, BN, p.bf16 != 0, A_MN, B_MN);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      auto wait_warp = [&](uint32_t bar, uint32_t parity) -> bool {
        int ok = 1;
        if (lane == 0) ok = wait_or_abort(bar, parity, abort_flag, p.err) ? 1 : 0;
        return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
      };
      uint32_t it = 0, tb = 0;
      bool ok = true;
      for (int t = pair; t < p.num_tiles; t += pairs, ++tb) {
        const int b = tb & 1;
        if (!wait_warp(tm_empty(b), ((tb >> 1) & 1) ^ 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tm + b * 256;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int st = it % NST;
          if (!wait_warp(st_full(st), (it / NST) & 1)) { ok = false; break; }
          tc_fence_after();
          if (g_elect()) {
            const uint64_t ad = g_sdesc<A_MN>(sbase + st * L::STAGE);
            const uint64_t bd = g_sdesc<B_MN>(sbase + st * L::STAGE + L::ST_A);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_pair(d, ad + j * G_KSTEP<A_MN>, bd + j * G_KSTEP<B_MN>, idesc,
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
    constexpr int CH = BN / 64;                       // 32-column boxes of this warp
    const uint32_t lane_off = (uint32_t)(32 * q) << 16;
    uint8_t* stage = smem + L::OFF_Y + w * 2 * L::BOX;
    const uint32_t stage_u = smem_u32(stage);
    float* bias_s = reinterpret_cast<float*>(smem + L::OFF_BIAS + w * 128);
    const bool bf16 = p.bf16 != 0, has_r = p.res != nullptr;
    const uint32_t tm_empty0[2] = {map_rank(tm_empty(0), 0), map_rank(tm_empty(1), 0)};
    uint32_t tb = 0, cc = 0;                          // tiles and boxes so far
    bool alive = true;
    for (int t = pair; t < p.num_tiles && alive; t += pairs, ++tb) {
      const TilePos pos = tile_pos(t, p.tiles_m, p.tiles_n);
      const int m0 = pos.m * 256 + 128 * rank + 32 * q, n0 = pos.n * BN + BN / 2 * half;
      const int b = tb & 1;
      const int row = m0 + lane;
      float bias[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = n0 + 32 * c + lane;
        bias[c] = p.bias && col < p.N ? unpack2(__ldg(p.bias + col), bf16).x : 0.0f;
      }
      auto load_r = [&](int c, uint32_t buf) {        // lane 0: the residual's box c
        tma_store_wait_read0();
        mbar_arrive_expect_tx(r_full(w, buf), L::BOX);
        tma_load_2d(stage_u + buf * L::BOX, &tm_r, n0 + 32 * c, m0, r_full(w, buf));
      };
      if (has_r && lane == 0) load_r(0, cc & 1);
      if (!wait_or_abort(tm_full(b), (tb >> 1) & 1, abort_flag, p.err)) alive = false;
      alive = __all_sync(0xFFFFFFFFu, alive);
      if (!alive) {
        // the residual's box in flight lands before the CTA ends
        if (has_r) mbar_wait_bounded(r_full(w, cc & 1), (cc >> 1) & 1, LIMIT_NS);
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < CH; ++c, ++cc) {
        const uint32_t buf = cc & 1;
        if (lane == 0) {
          if (has_r) {
            if (c + 1 < CH) load_r(c + 1, buf ^ 1);
          } else {
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          }
        }
        uint32_t r[32];
        tmem_ld32(tmem + b * 256 + BN / 2 * half + 32 * c + lane_off, r);
        bias_s[lane] = bias[c];
        tmem_wait_ld();
        if (c + 1 == CH) {                            // the accumulator may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(tm_empty0[b]);
        }
        __syncwarp();
        if (has_r && !wait_or_abort(r_full(w, buf), (cc >> 1) & 1, abort_flag, p.err)) alive = false;
        uint8_t* yrow = stage + buf * L::BOX + lane * 64;
        // a TMA store writes whole 16-byte pieces: a ragged last box leaves
        // by element stores instead
        const bool boxed = p.N % 8 == 0 || n0 + 32 * c + 32 <= p.N;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float v[8];
          const float4 b0 = lds128(smem_u32(bias_s + 8 * u)), b1 = lds128(smem_u32(bias_s + 8 * u + 4));
          const float bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r[8 * u + e]) + bv[e];
          if (p.pre) {
            const int col = n0 + 32 * c + 8 * u;
            if (row < p.M && col < p.N) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = pack2(make_float2(v[2 * e], v[2 * e + 1]), bf16);
              store8(p.pre + (long long)row * p.ldp, col, p.N, make_uint4(o[0], o[1], o[2], o[3]));
            }
          }
          if (p.epilogue != SVDQ_EPI_NONE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = g_act(v[e], p.epilogue);
          }
          uint4* place = reinterpret_cast<uint4*>(yrow + ((u ^ ((lane >> 1) & 3)) << 4));
          if (has_r) {
            const uint4 rr = *place;
            const uint32_t rw[4] = {rr.x, rr.y, rr.z, rr.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack2(rw[e], bf16);
              v[2 * e] += f.x;
              v[2 * e + 1] += f.y;
            }
          }
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = pack2(make_float2(v[2 * e], v[2 * e + 1]), bf16);
          const uint4 o4 = make_uint4(o[0], o[1], o[2], o[3]);
          const int col = n0 + 32 * c + 8 * u;
          if (boxed)
            *place = o4;
          else if (row < p.M && col < p.N)
            store8(p.out + (long long)row * p.ldo, col, p.N, o4);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (boxed) tma_store_2d(&tm_y, n0 + 32 * c, m0, stage_u + buf * L::BOX);
          tma_store_commit();         // an empty group keeps the count of groups
        }
      }
      alive = __all_sync(0xFFFFFFFFu, alive);
    }
    if (lane == 0) tma_store_wait0();
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

template <int BN, bool A_MN, bool B_MN>
cudaError_t launch_bn(const Operand& A, const Operand& B, G16Args a, cudaStream_t st) {
  using L = PLay<BN>;
  static bool attr[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(gemm16_pair_kernel<BN, A_MN, B_MN>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    attr[dev] = true;
  }
  const bool bf16 = a.bf16 != 0;
  const auto dt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap ta, tb, ty, tr;
  if (!operand_map(&ta, A, 128, bf16) || !operand_map(&tb, B, BN / 2, bf16) ||
      !make_map(&ty, a.out, dt, B.rows, A.rows, (uint64_t)a.ldo * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  tr = ty;
  if (a.res && !make_map(&tr, a.res, dt, B.rows, A.rows, (uint64_t)a.ldr * 2, 32, 32,
                         CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const long long tm = ((long long)A.rows + 255) / 256, tn = ((long long)B.rows + BN - 1) / BN;
  if (tm * tn > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
  a.M = A.rows;
  a.N = B.rows;
  a.kblocks = (int)(((long long)A.red + G_BK - 1) / G_BK);
  a.tiles_m = (int)tm;
  a.tiles_n = (int)tn;
  a.num_tiles = (int)(tm * tn);
  const int pairs = a.num_tiles < num_sms() / 2 ? a.num_tiles : num_sms() / 2;
  gemm16_pair_kernel<BN, A_MN, B_MN><<<2 * pairs, P_THREADS, L::ALLOC, st>>>(ta, tb, ty, tr, a);
  return cudaGetLastError();
}

template <bool A_MN, bool B_MN>
cudaError_t launch_major(const Operand& A, const Operand& B, const G16Args& a, cudaStream_t st) {
  return launch_bn<256, A_MN, B_MN>(A, B, a, st);
}

}  // namespace

cudaError_t launch_gemm16_pair(const Operand& A, const Operand& B, const G16Args& a, cudaStream_t st) {
  if (A.mn) return launch_major<true, true>(A, B, a, st);
  if (B.mn) return launch_major<false, true>(A, B, a, st);
  return launch_major<false, false>(A, B, a, st);
}

}  // namespace svdq
