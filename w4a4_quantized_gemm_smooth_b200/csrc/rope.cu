// Rotary positions with several axes (svdq_rope): every pair of a head is
// turned by position[axis] * frequency, shared by all heads of a token.
//
// The angle is formed modulo one turn without rounding: a frequency is held
// as a 64-bit fraction of a turn, the low 64 bits of its product with the
// 32-bit position are the angle's fraction of a turn, and their top 32 bits
// (2^-32 turn) go through sincospi.  A far position thus costs no accuracy.
//
// Bound by memory: one read and one write of T H D elements.  A thread holds
// the sines and cosines of one vector's pairs and walks the heads, four loads
// at a time, so the trigonometry is paid once per heads_per_thread heads.
// 4608 tokens x 64 heads x 128 (bf16, in rows of 12288): 28.4 us, 5.3 TB/s;
// 16640 x 32 x 72 in halves (fp16, 8-byte vectors): 29.8 us, 5.2 TB/s; a plain
// copy of as many bytes takes 25 us.
#include <cmath>
#include <new>

#include "elem.cuh"
#include "ops16.h"

struct svdq_rope_plan {
  svdq::RopeTurns t;
  int pairing;
};

namespace svdq {
namespace {

struct RopeArgs {
  const int32_t* pos;
  const void* x;
  void* y;
  long long ldxt, ldxh, ldyt, ldyh;
  long long work;            // tokens * units
  int pos_rows, ld_pos;
  int heads, heads_per_thread;
  int units;                 // vectors (interleaved) or rotating vector pairs + tail vectors (halves)
  int pairs, rot_units;      // halves: the first rot_units units hold pairs
  int inverse, in_place;
};

__device__ __forceinline__ void sincos_turn(int32_t pos, uint64_t turn, bool inverse, float& c,
                                            float& s) {
  const uint64_t a = (uint64_t)(int64_t)pos * turn;
  const float half_turns = (float)(int32_t)(a >> 32) * 4.656612873077393e-10f;   // 2^-31
  sincospif(half_turns, &s, &c);
  if (inverse) s = -s;
}

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_BATCH = 4;      // heads whose loads are in flight together

// V elements of a head, of any alignment; pairs of them as fp32.
template <typename T, int V, int ALIGN>
struct alignas(ALIGN) RopeVec {
  T e[V];
};
__device__ __forceinline__ float2 rope_get(const __nv_bfloat16* e) {
  return make_float2(__bfloat162float(e[0]), __bfloat162float(e[1]));
}
__device__ __forceinline__ float2 rope_get(const __half* e) {
  return make_float2(__half2float(e[0]), __half2float(e[1]));
}
__device__ __forceinline__ float2 rope_get(const float* e) { return make_float2(e[0], e[1]); }
__device__ __forceinline__ void rope_set(__nv_bfloat16* e, float2 f) {
  const __nv_bfloat162 h = __float22bfloat162_rn(f);
  e[0] = h.x;
  e[1] = h.y;
}
__device__ __forceinline__ void rope_set(__half* e, float2 f) {
  const __half2 h = __float22half2_rn(f);
  e[0] = h.x;
  e[1] = h.y;
}
__device__ __forceinline__ void rope_set(float* e, float2 f) {
  e[0] = f.x;
  e[1] = f.y;
}

// V elements per vector.  HALVES: a unit below rot_units holds pairs
// [V unit, V unit + V) as two vectors P elements apart, a later unit one
// vector past the pairs; interleaved: a unit is one vector.  Arithmetic runs
// on packed fp32 pairs.
template <typename T, int V, bool HALVES, int ALIGN>
__global__ void __launch_bounds__(ROPE_THREADS, HALVES && V * (int)sizeof(T) == 16 ? 3 : 5)
rope_kernel(const __grid_constant__ RopeTurns turns, const RopeArgs p) {
  using VT = RopeVec<T, V, ALIGN>;
  grid_wait();
  const long long i = (long long)blockIdx.x * ROPE_THREADS + threadIdx.x;
  if (i >= p.work) return;
  const long long tok = p.work <= 0x7FFFFFFF ? (int)i / p.units : i / p.units;
  const int u = (int)(i - tok * p.units);
  const int h0 = blockIdx.y * p.heads_per_thread;
  const int h1 = min(p.heads, h0 + p.heads_per_thread);
  const T* x = static_cast<const T*>(p.x) + tok * p.ldxt + h0 * p.ldxh;
  T* y = static_cast<T*>(p.y) + tok * p.ldyt + h0 * p.ldyh;
  constexpr int NP = HALVES ? V : V / 2;          // pairs of a unit
  const bool rot = HALVES ? u < p.rot_units : u * NP < p.pairs;
  if (!rot) {
    if (p.in_place) return;
    const int d = HALVES ? 2 * p.pairs + (u - p.rot_units) * V : u * V;
    for (int h = h0; h < h1; ++h, x += p.ldxh, y += p.ldyh)
      *reinterpret_cast<VT*>(y + d) = *reinterpret_cast<const VT*>(x + d);
    return;
  }
  const int32_t* pos = p.pos + (long long)((int)tok % p.pos_rows) * p.ld_pos;
  float c[NP], s[NP];
  {
    // the unit's frequencies in one run: lanes read different places of the
    // parameters, which costs a pass per place, so wide reads are few passes
    uint64_t turn[NP];
    uint8_t axis[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      turn[j] = turns.turn[u * NP + j];           // zeros past the pairs
      axis[j] = turns.axis[u * NP + j];
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) sincos_turn(pos[axis[j]], turn[j], p.inverse != 0, c[j], s[j]);
  }
  x += u * V;
  y += u * V;
  const int pairs = p.pairs;
  // a vector may straddle the last pair: what follows is copied as it is
  const int live = HALVES ? NP : min(NP, pairs - u * NP);
  auto turn_head = [&](VT& a, VT& b) {
    if constexpr (!HALVES) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float2 v = rope_get(&a.e[2 * j]);
        const float2 r = __ffma2_rn(make_float2(v.y, v.x), make_float2(-s[j], s[j]),
                                    __fmul2_rn(v, make_float2(c[j], c[j])));
        if (j < live) rope_set(&a.e[2 * j], r);
      }
    } else if constexpr (V == 1) {
      const float fa = Elem<T>::to_f(a.e[0]), fb = Elem<T>::to_f(b.e[0]);
      a.e[0] = Elem<T>::from_f(fa * c[0] - fb * s[0]);
      b.e[0] = Elem<T>::from_f(fa * s[0] + fb * c[0]);
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 fa = rope_get(&a.e[j]), fb = rope_get(&b.e[j]);
        const float2 c2 = make_float2(c[j], c[j + 1]), s2 = make_float2(s[j], s[j + 1]);
        rope_set(&a.e[j], __ffma2_rn(fb, make_float2(-s2.x, -s2.y), __fmul2_rn(fa, c2)));
        rope_set(&b.e[j], __ffma2_rn(fa, s2, __fmul2_rn(fb, c2)));
      }
    }
  };
  const long long ldxh = p.ldxh, ldyh = p.ldyh;
  int n = h1 - h0;
  for (; n >= ROPE_BATCH; n -= ROPE_BATCH) {      // a batch's loads are in flight together
    VT a[ROPE_BATCH], b[ROPE_BATCH];
#pragma unroll
    for (int k = 0; k < ROPE_BATCH; ++k, x += ldxh) {
      a[k] = *reinterpret_cast<const VT*>(x);
      if (HALVES) b[k] = *reinterpret_cast<const VT*>(x + pairs);
    }
#pragma unroll
    for (int k = 0; k < ROPE_BATCH; ++k, y += ldyh) {
      turn_head(a[k], b[k]);
      *reinterpret_cast<VT*>(y) = a[k];
      if (HALVES) *reinterpret_cast<VT*>(y + pairs) = b[k];
    }
  }
  for (; n > 0; --n, x += ldxh, y += ldyh) {
    VT a = *reinterpret_cast<const VT*>(x), b;
    if (HALVES) b = *reinterpret_cast<const VT*>(x + pairs);
    turn_head(a, b);
    *reinterpret_cast<VT*>(y) = a;
    if (HALVES) *reinterpret_cast<VT*>(y + pairs) = b;
  }
}

template <typename T, int V, bool HALVES, int ALIGN = V * (int)sizeof(T)>
cudaError_t launch_v(const RopeTurns& t, RopeArgs a, int tokens, int head_dim, cudaStream_t st) {
  if (HALVES) {
    a.rot_units = a.pairs / V;
    a.units = a.rot_units + (head_dim - 2 * a.pairs) / V;
  } else {
    a.rot_units = 0;
    a.units = head_dim / V;
  }
  a.work = (long long)tokens * a.units;
  // Heads per thread: 8 while that leaves 64 threads per SM; smaller batches
  // spread the heads instead, down to one a thread.  The trigonometry of a
  // vector costs as much as several heads: 1024 tokens x 32 x 72 take 5.0 us
  // with 8 heads a thread and 7.6 with 2; 16 tokens 2.7 with 8 and 2.1 with 1;
  // 4608 x 64 x 128 27.5 with 8, 42.8 with 4 and 26.1 with 16, with which
  // 2048 x 32 x 128 takes 11.8 instead of 9.7.
  int hpt = 8;
  while (hpt > 1 && a.work * ((a.heads + hpt - 1) / hpt) < 148 * 64) hpt >>= 1;
  a.heads_per_thread = hpt;
  const long long blocks = (a.work + ROPE_THREADS - 1) / ROPE_THREADS;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)((a.heads + hpt - 1) / hpt));
  return launch_op(rope_kernel<T, V, HALVES, ALIGN>, grid, ROPE_THREADS, 0, 1, st, t, a);
}

// The widest vector (up to 16 bytes) that every address is a multiple of.
template <typename T>
cudaError_t launch_t(const svdq_rope_plan* plan, const RopeArgs& a, int tokens, int head_dim,
                     cudaStream_t st) {
  constexpr int E = (int)sizeof(T);
  const bool halves = plan->pairing == SVDQ_ROPE_HALVES;
  uint64_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                  (uint64_t)(a.ldxt * E) | (uint64_t)(a.ldyt * E) | (uint64_t)(a.ldxh * E) |
                  (uint64_t)(a.ldyh * E) | (uint64_t)head_dim * E;
  if (halves) bits |= (uint64_t)a.pairs * E;
  int v = 16 / E;
  while (v > 1 && (bits & (uint64_t)(v * E - 1)) != 0) v >>= 1;
  const RopeTurns& t = plan->t;
  if (halves) {
    if constexpr (E == 2)
      if (v == 8) return launch_v<T, 8, true>(t, a, tokens, head_dim, st);
    if (v == 4) return launch_v<T, 4, true>(t, a, tokens, head_dim, st);
    if (v == 2) return launch_v<T, 2, true>(t, a, tokens, head_dim, st);
    return launch_v<T, 1, true>(t, a, tokens, head_dim, st);
  }
  if constexpr (E == 2)
    if (v == 8) return launch_v<T, 8, false>(t, a, tokens, head_dim, st);
  if (v == 4) return launch_v<T, 4, false>(t, a, tokens, head_dim, st);
  if (v == 2) return launch_v<T, 2, false>(t, a, tokens, head_dim, st);
  return launch_v<T, 2, false, E>(t, a, tokens, head_dim, st);    // element by element
}

}  // namespace

// Fraction of a turn, times 2^64 and modulo that, of `freq` radians (below 2^20
// in magnitude), to the nearest: freq = m 2^e with a 53-bit m and e <= -33, and
// m / 2 pi comes from the first 128 bits of 1 / 2 pi in integers, so that the
// error before the last rounding is below 2^53 2^-128 2^e, whatever the size.
uint64_t turn_of(double freq) {
  // floor(2^128 / 2 pi)
  constexpr unsigned __int128 INV_2PI = (unsigned __int128)0x28BE60DB9391054Aull << 64 | 0x7F09D5F47D4D3770ull;
  int exp = 0;
  const double frac = std::frexp(std::fabs(freq), &exp);             // freq = frac 2^exp
  const uint64_t m = (uint64_t)std::ldexp(frac, 53);
  // m INV_2PI is the turns times 2^(128 - e), e = exp - 53; `high` leaves out its
  // last 64 bits, so that the result's last bit is bit -e of it, 33 or more
  const unsigned __int128 low = (unsigned __int128)m * (uint64_t)INV_2PI;
  const unsigned __int128 high = (unsigned __int128)m * (uint64_t)(INV_2PI >> 64) + (uint64_t)(low >> 64);
  const int shift = 53 - exp;
  if (frac == 0.0 || shift > 128) return 0;                          // below half of the last bit
  const unsigned __int128 half = (high >> (shift - 1)) + 1;
  const uint64_t turn = (uint64_t)(half >> 1);
  return freq < 0.0 ? 0 - turn : turn;
}

cudaError_t launch_rope(const svdq_rope_plan* plan, int dtype, int tokens, int heads,
                        int head_dim, const int32_t* pos, int pos_rows, int ld_pos, const void* X,
                        long long ldxt, long long ldxh, void* Y, long long ldyt, long long ldyh,
                        int inverse, cudaStream_t st) {
  RopeArgs a{};
  a.pos = pos; a.x = X; a.y = Y;
  a.ldxt = ldxt; a.ldxh = ldxh; a.ldyt = ldyt; a.ldyh = ldyh;
  a.pos_rows = pos_rows; a.ld_pos = ld_pos;
  a.heads = heads; a.pairs = plan->t.pairs;
  a.inverse = inverse; a.in_place = X == Y;
  if (dtype == SVDQ_DTYPE_BF16) return launch_t<__nv_bfloat16>(plan, a, tokens, head_dim, st);
  if (dtype == SVDQ_DTYPE_F16) return launch_t<__half>(plan, a, tokens, head_dim, st);
  return launch_t<float>(plan, a, tokens, head_dim, st);
}

}  // namespace svdq

extern "C" {

svdq_status svdq_rope_create(int n_axes, const int* pairs_per_axis, const double* freq,
                             int pairing, svdq_rope_plan** out) {
  if (!out) return SVDQ_ERR_INVALID_ARG;
  *out = nullptr;
  if (!pairs_per_axis || !freq || n_axes < 1 || n_axes > SVDQ_ROPE_MAX_AXES ||
      (pairing != SVDQ_ROPE_INTERLEAVED && pairing != SVDQ_ROPE_HALVES))
    return SVDQ_ERR_INVALID_ARG;
  int pairs = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (pairs_per_axis[a] < 0 || pairs_per_axis[a] > SVDQ_ROPE_MAX_PAIRS) return SVDQ_ERR_SHAPE;
    pairs += pairs_per_axis[a];
  }
  if (pairs < 1 || pairs > SVDQ_ROPE_MAX_PAIRS) return SVDQ_ERR_SHAPE;
  for (int p = 0; p < pairs; ++p)
    if (!(std::fabs(freq[p]) < 1048576.0)) return SVDQ_ERR_NUMERIC;
  svdq_rope_plan* plan = new (std::nothrow) svdq_rope_plan();
  if (!plan) return SVDQ_ERR_OOM;
  plan->pairing = pairing;
  plan->t.pairs = pairs;
  plan->t.axes = n_axes;
  int p = 0;
  for (int a = 0; a < n_axes; ++a)
    for (int j = 0; j < pairs_per_axis[a]; ++j, ++p) {
      plan->t.axis[p] = (uint8_t)a;
      plan->t.turn[p] = svdq::turn_of(freq[p]);
    }
  *out = plan;
  return SVDQ_OK;
}

void svdq_rope_free(svdq_rope_plan* plan) { delete plan; }

svdq_status svdq_rope(const svdq_rope_plan* plan, int dtype, int tokens, int heads, int head_dim,
                      const int32_t* positions, int pos_rows, int ld_pos, const void* X,
                      long long ldx_token, long long ldx_head, void* Y, long long ldy_token,
                      long long ldy_head, int inverse, cudaStream_t stream) {
  if (!plan || dtype < SVDQ_DTYPE_BF16 || dtype > SVDQ_DTYPE_F32) return SVDQ_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 0 || pos_rows < (tokens ? 1 : 0) || ld_pos < plan->t.axes || head_dim < 2 ||
      head_dim % 2 != 0 || head_dim < 2 * plan->t.pairs || ldx_token < 0 || ldx_head < 0 ||
      ldy_token < 0 || ldy_head < 0)
    return SVDQ_ERR_SHAPE;
  if (head_dim > SVDQ_ROPE_MAX_HEAD_DIM || heads > SVDQ_ROPE_MAX_HEADS) return SVDQ_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0) return SVDQ_OK;
  if (!positions || !X || !Y) return SVDQ_ERR_INVALID_ARG;
  // two heads or tokens never share an element of Y: all heads lie within a
  // token's stride, or all tokens within a head's
  const __int128 hd = head_dim;
  const bool in_token = (heads == 1 || ldy_head >= hd) &&
                        (tokens == 1 || ldy_token >= (__int128)(heads - 1) * ldy_head + hd);
  const bool in_head = (tokens == 1 || ldy_token >= hd) &&
                       (heads == 1 || ldy_head >= (__int128)(tokens - 1) * ldy_token + hd);
  if (!in_token && !in_head) return SVDQ_ERR_SHAPE;
  if (X == Y && ((tokens > 1 && ldx_token != ldy_token) || (heads > 1 && ldx_head != ldy_head)))
    return SVDQ_ERR_INVALID_ARG;
  const uintptr_t e = dtype == SVDQ_DTYPE_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(X) & e) || (reinterpret_cast<uintptr_t>(Y) & e) ||
      (reinterpret_cast<uintptr_t>(positions) & 3))
    return SVDQ_ERR_ALIGNMENT;
  {
    const int es = svdq::dtype_size(dtype);
    auto extent = [&](const void* p, long long token, long long head) {
      return svdq::extent(p, (long long)head_dim * es, tokens, heads, token * es, head * es);
    };
    const svdq::Extent y = extent(Y, ldy_token, ldy_head);
    const svdq::Extent pos = svdq::extent_rows(positions, pos_rows < tokens ? pos_rows : tokens, plan->t.axes,
                                               ld_pos, 4);
    if ((X != Y && svdq::overlap(y, extent(X, ldx_token, ldx_head))) || svdq::overlap(y, pos))
      return SVDQ_ERR_INVALID_ARG;
  }
  return svdq::status_of(svdq::launch_rope(plan, dtype, tokens, heads, head_dim, positions, pos_rows, ld_pos, X,
                                           ldx_token, ldx_head, Y, ldy_token, ldy_head, inverse, stream));
}

}  // extern "C"
