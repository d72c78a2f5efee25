// Beam search: of each group's K beams x V tokens the n candidates of highest score, and the beams' states moved to where
// their parents' successors are.
//   score(b, t) = scores[b] + logits[b, t] - log sum_t' exp(logits[b, t'])
//
// One pass over the logits leaves, for every row, its sum of exponentials and the largest logit of every run of G consecutive
// tokens.  The n best candidates (score first, then the lowest beam and token) lie in the n runs whose largest logits are the
// best in that same order: a run that n others precede cannot hold a candidate that fewer than n precede.  So what is left
// is to select n of K V / G runs, then n of their n G tokens.
//
// Which of two beams' candidates is the better one depends on the difference of two such logarithms, and among thousands of
// candidates some lie closer than fp32's rounding.  So each exponential is formed to 2^-28.8 (2^-31.4 on the mean; 2^(j/32) from
// a table in two words, P. T. P. Tang's reduction, and a polynomial of degree 3), added into two words (the sum is off by 2^-27
// at most, by 2^-31 on the mean), and scores are compared in two fp32 words.  Equal logits of one row stay equal, and so do equal
// rows: which values are added to which goes by their tokens, wherever a row begins in memory.  A token with all of its row's sum has
// the logarithm 0.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace gbla {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr float kInf = __builtin_huge_valf();
constexpr double kLn2 = 0.6931471805599453;

// 2^(j / 32) / (1 + j / 32) = hi + lo, hi of 18 bits: times (1 + j / 32) 2^q, which the rounded exponent's own bits make, it is exact
__device__ const float kExpHi[32] = {
    0x1p+0f, 0x1.fb5b8p-1f, 0x1.f7378p-1f, 0x1.f38bp-1f, 0x1.f04d8p-1f, 0x1.ed768p-1f, 0x1.eaff8p-1f, 0x1.e8e28p-1f,
    0x1.e7198p-1f, 0x1.e5ap-1f, 0x1.e4718p-1f, 0x1.e3898p-1f, 0x1.e2e58p-1f, 0x1.e281p-1f, 0x1.e2598p-1f, 0x1.e26dp-1f,
    0x1.e2b8p-1f, 0x1.e3388p-1f, 0x1.e3edp-1f, 0x1.e4d38p-1f, 0x1.e5ea8p-1f, 0x1.e72f8p-1f, 0x1.e8a28p-1f, 0x1.ea418p-1f,
    0x1.ec0b8p-1f, 0x1.edff8p-1f, 0x1.f01c8p-1f, 0x1.f2618p-1f, 0x1.f4ce8p-1f, 0x1.f762p-1f, 0x1.fa1cp-1f, 0x1.fcfb8p-1f,
};
__device__ const float kExpLo[32] = {
    0x0p+0f, -0x1.fd0268p-20f, 0x1.45997ap-21f, 0x1.6dc7a4p-20f, -0x1.1f909cp-20f, -0x1.9cb2a4p-21f, -0x1.60e976p-21f, -0x1.fbcb98p-20f,
    -0x1.894a0ep-21f, -0x1.3965fep-21f, -0x1.1b5fd8p-20f, 0x1.acef48p-20f, -0x1.36643ep-20f, 0x1.014d7ep-24f, 0x1.d1967ep-20f, -0x1.67559p-20f,
    -0x1.110082p-20f, 0x1.2a661ep-20f, 0x1.3ff29p-20f, 0x1.38d8dap-21f, -0x1.feaabp-20f, 0x1.65eb56p-20f, -0x1.22e3d8p-23f, -0x1.14a9b8p-21f,
    -0x1.99e158p-21f, -0x1.14c836p-20f, -0x1.872644p-21f, 0x1.7c2b28p-20f, -0x1.5bc508p-22f, 0x1.789ea6p-22f, -0x1.387142p-20f, -0x1.67e88p-20f,
};
constexpr float kL = 0x1.715476p+5f, kLlo = 0x1.4ae0cp-21f;  // 32 / ln 2 in two words
// 2^(f / 32) - 1 = f (c1 + f (c2 + f c3)): c_k = (ln 2 / 32)^k / k!, and in c2 the next term too: for f^4 the multiple of f^2 that is
// nearest on |f| <= 1/2, (sqrt 2 - 1) / 2, which leaves 2^-33
constexpr float kC1 = 0x1.62e43p-6f, kC2 = 0x1.ebfce6p-13f, kC3 = 0x1.c6b08ep-20f;

// Logarithms: c_j of 8 bits next to 1 / (1 + (j + 1/2) / 64), and -ln c_j in two words
__device__ const float kLogC[64] = {
    0x1.fcp-1f, 0x1.f4p-1f, 0x1.ecp-1f, 0x1.e6p-1f, 0x1.dep-1f, 0x1.d8p-1f, 0x1.dp-1f, 0x1.cap-1f,
    0x1.c4p-1f, 0x1.bep-1f, 0x1.b8p-1f, 0x1.b2p-1f, 0x1.acp-1f, 0x1.a6p-1f, 0x1.a2p-1f, 0x1.9cp-1f,
    0x1.98p-1f, 0x1.92p-1f, 0x1.8ep-1f, 0x1.88p-1f, 0x1.84p-1f, 0x1.8p-1f, 0x1.7ap-1f, 0x1.76p-1f,
    0x1.72p-1f, 0x1.6ep-1f, 0x1.6ap-1f, 0x1.66p-1f, 0x1.62p-1f, 0x1.5ep-1f, 0x1.5ap-1f, 0x1.58p-1f,
    0x1.54p-1f, 0x1.5p-1f, 0x1.4cp-1f, 0x1.4ap-1f, 0x1.46p-1f, 0x1.42p-1f, 0x1.4p-1f, 0x1.3cp-1f,
    0x1.3ap-1f, 0x1.36p-1f, 0x1.34p-1f, 0x1.3p-1f, 0x1.2ep-1f, 0x1.2cp-1f, 0x1.28p-1f, 0x1.26p-1f,
    0x1.24p-1f, 0x1.2p-1f, 0x1.1ep-1f, 0x1.1cp-1f, 0x1.1ap-1f, 0x1.16p-1f, 0x1.14p-1f, 0x1.12p-1f,
    0x1.1p-1f, 0x1.0ep-1f, 0x1.0cp-1f, 0x1.0ap-1f, 0x1.08p-1f, 0x1.06p-1f, 0x1.04p-1f, 0x1.02p-1f,
};
__device__ const float kLogHi[64] = {
    0x1.010158p-7f, 0x1.849252p-6f, 0x1.466aeep-5f, 0x1.aaef2ep-5f, 0x1.1973bep-4f, 0x1.4d3116p-4f, 0x1.9335e6p-4f, 0x1.c8858p-4f,
    0x1.fe8914p-4f, 0x1.1aa2b8p-3f, 0x1.365fccp-3f, 0x1.527e5ep-3f, 0x1.6f0128p-3f, 0x1.8beafep-3f, 0x1.9f6c4p-3f, 0x1.bd0874p-3f,
    0x1.d1038p-3f, 0x1.ef5adep-3f, 0x1.01eae6p-2f, 0x1.1178e8p-2f, 0x1.1bf996p-2f, 0x1.269622p-2f, 0x1.36b678p-2f, 0x1.419b42p-2f,
    0x1.4c9e0ap-2f, 0x1.57bf76p-2f, 0x1.63003p-2f, 0x1.6e60eep-2f, 0x1.79e266p-2f, 0x1.858558p-2f, 0x1.914a86p-2f, 0x1.973a34p-2f,
    0x1.a3344p-2f, 0x1.af5296p-2f, 0x1.bb9612p-2f, 0x1.c1c606p-2f, 0x1.ce42f2p-2f, 0x1.dae754p-2f, 0x1.e148a2p-2f, 0x1.ee2a16p-2f,
    0x1.f4aa7ep-2f, 0x1.00e5aep-1f, 0x1.04360cp-1f, 0x1.0ae76ep-1f, 0x1.0e4898p-1f, 0x1.11af82p-1f, 0x1.188ee4p-1f, 0x1.1c0784p-1f,
    0x1.1f8636p-1f, 0x1.269622p-1f, 0x1.2a2786p-1f, 0x1.2dbf56p-1f, 0x1.315da4p-1f, 0x1.38ae22p-1f, 0x1.3c608p-1f, 0x1.4019c2p-1f,
    0x1.43dap-1f, 0x1.47a152p-1f, 0x1.4b6fd6p-1f, 0x1.4f45a8p-1f, 0x1.5322e2p-1f, 0x1.5707a2p-1f, 0x1.5af406p-1f, 0x1.5ee82ap-1f,
};
__device__ const float kLogLo[64] = {
    -0x1.4ee432p-32f, 0x1.191958p-31f, -0x1.7a4382p-30f, -0x1.e09dep-30f, -0x1.d73554p-29f, -0x1.6fc0aap-31f, -0x1.535b3cp-31f, 0x1.bc4b24p-32f,
    -0x1.890aa6p-30f, -0x1.dc08d6p-31f, -0x1.fd4dfep-28f, 0x1.286d64p-29f, 0x1.6ead58p-28f, 0x1.671fd2p-28f, 0x1.c2259ap-29f, -0x1.f109d4p-29f,
    -0x1.b3543p-28f, 0x1.373ffap-29f, -0x1.3b272ep-27f, 0x1.13f23ep-29f, 0x1.ad35cap-29f, -0x1.d9648ep-27f, -0x1.283ddep-27f, 0x1.eaf464p-29f,
    -0x1.e8d3c4p-30f, -0x1.86e5cp-27f, 0x1.67558ap-27f, 0x1.abc65cp-28f, 0x1.0f9f68p-27f, -0x1.12468p-27f, 0x1.adfb44p-29f, 0x1.89ab56p-29f,
    0x1.127d3cp-29f, -0x1.b6e646p-27f, -0x1.1fc742p-28f, 0x1.27f474p-27f, -0x1.fe6e3p-28f, 0x1.0992c2p-27f, -0x1.76364cp-28f, -0x1.297d84p-27f,
    0x1.c06326p-27f, 0x1.6c81eap-27f, -0x1.89fc54p-29f, 0x1.682a7ep-28f, 0x1.847338p-27f, 0x1.e3ad54p-28f, 0x1.e4794cp-30f, 0x1.35ccp-26f,
    -0x1.cf4d3ap-32f, -0x1.d9648ep-26f, 0x1.a1d82p-26f, -0x1.09e418p-26f, 0x1.0d01a2p-27f, -0x1.1cd124p-26f, 0x1.86d7f6p-26f, 0x1.25ca94p-29f,
    -0x1.a0db88p-26f, 0x1.fa28b4p-27f, 0x1.f2e184p-26f, 0x1.ad270cp-28f, 0x1.a19e16p-27f, 0x1.aee31ap-27f, -0x1.e4db1p-28f, 0x1.448324p-26f,
};
constexpr float kLn2A = 0x1.63p-1f, kLn2B = -0x1.bdp-13f, kLn2C = -0x1.05c61p-29f;  // ln 2; A and B times 13 bits are exact

// A logit's E values of a 16-byte piece.
template <typename T>
__device__ __forceinline__ float piece(const uint4& w, int j) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
  if (sizeof(T) == 2) return j & 1 ? bf_hi(q[j / 2]) : bf_lo(q[j / 2]);
  return __uint_as_float(q[j & 3]);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float o;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
  return o;
}

// The row's tokens begin so many values behind a 16-byte boundary.
template <typename T>
__device__ __forceinline__ int row_offset(const BeamArgs& a, int64_t row) {
  return (int)((reinterpret_cast<uintptr_t>(a.logits) + row * a.ld * sizeof(T)) % 16 / sizeof(T));
}
// E mask bits from token t, a multiple of E, of a row.
template <int E>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* m, int words, int t) {
  const int w = t >> 5;
  return (w < words ? m[w] : 0u) >> (t & 31) & ((1u << E) - 1);
}
// Of the values of two pieces those from the off-th on, a piece of them.
template <typename T>
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int off) {
  uint32_t q[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int words = off * (int)sizeof(T) / 4;
  if (words & 2) {
#pragma unroll
    for (int i = 0; i < 6; ++i) q[i] = q[i + 2];
  }
  if (words & 1) {
#pragma unroll
    for (int i = 0; i < 5; ++i) q[i] = q[i + 1];
  }
  if (sizeof(T) == 2 && off & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __funnelshift_r(q[i], q[i + 1], 16);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
// The power of two that exponentials of logits up to `top` are summed relative to: e^top is at most it, and above a quarter of it.
__device__ __forceinline__ int octave(float top) { return (int)floorf(top * 1.44269504f) + 1; }
__device__ __forceinline__ double sum_of(const BeamPart& p) {
  return p.far ? __hiloint2double(p.hi, __float_as_int(p.lo)) : (double)p.hi * (1. / 65536.) + (double)p.lo;
}

constexpr int kU = kBeamPieces;
template <int V> struct Int { static constexpr int value = V; };

// i / d for i d < 2^32 as a multiplication: `by` is ceil(2^32 / d), or 0 for d = 1.
__device__ __forceinline__ uint32_t recip(uint32_t d) { return d == 1 ? 0 : 0xffffffffu / d + 1; }
__device__ __forceinline__ uint32_t quot(uint32_t i, uint32_t by) { return by ? __umulhi(i, by) : i; }

// The larger of two packed bf16 values each; of NaN and a number the number (of two NaN that), or NaN.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t o;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
  return o;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t o;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
  return o;
}
// The largest of a piece's values (no NaN).
template <typename T>
__device__ __forceinline__ float piece_max(const uint4& w) {
  if (sizeof(T) == 2) {
    const uint32_t m = max2(max2(w.x, w.y), max2(w.z, w.w));
    return fmaxf(bf_lo(m), bf_hi(m));
  }
  return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
// A piece with -infinity in place of the values without a mask bit.
template <typename T>
__device__ __forceinline__ uint4 masked(uint4 w, uint32_t ok) {
  auto pick = [&](uint32_t v, int j) {
    if (sizeof(T) == 4) return ok >> j & 1 ? v : 0xff800000u;
    const uint32_t keep = (ok >> 2 * j & 1 ? 0xffffu : 0u) | (ok >> (2 * j + 1) & 1 ? 0xffff0000u : 0u);
    return (v & keep) | (0xff80ff80u & ~keep);
  };
  return make_uint4(pick(w.x, 0), pick(w.y, 1), pick(w.z, 2), pick(w.w, 3));
}

// The largest of each run of 2^lg pieces: v[u] is the lane's of the u-th 32 of the warp's pieces; run g is stored at out[g] where it is
// below `end`.  From 8 lanes on the pieces are dealt out to the lanes while they are compared: 7 exchanges and those of what is left of
// lg, in place of 8 lg.
__device__ __forceinline__ void store_runs(float (&v)[kU], int lg, float* out, int end) {
  static_assert(kU == 8, "three halvings");
  const int lane = threadIdx.x & 31, per = 32 >> lg;  // runs of 32 pieces
  if (lg > 5) {  // of 64, 128 or all 256 pieces
    int n = kU;
#pragma unroll
    for (int h = 0; h < 3; ++h) {
      if (h >= lg - 5) break;
      n >>= 1;
#pragma unroll
      for (int u = 0; u < kU >> (h + 1); ++u) v[u] = fmaxf(v[2 * u], v[2 * u + 1]);
    }
#pragma unroll
    for (int u = 0; u < kU / 2; ++u) {
      if (u >= n) break;
      for (int o = 16; o; o >>= 1) v[u] = fmaxf(v[u], __shfl_xor_sync(FULL, v[u], o));
      if (lane == 0 && u < end) out[u] = v[u];
    }
    return;
  }
  if (lg < 3) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      for (int o = 1; o < 1 << lg; o <<= 1) v[u] = fmaxf(v[u], __shfl_xor_sync(FULL, v[u], o));
      const int g = u * per + (lane >> lg);
      if ((lane & ((1 << lg) - 1)) == 0 && g < end) out[g] = v[u];
    }
    return;
  }
  int o = 1 << (lg - 1), u = 0;
#pragma unroll
  for (int h = kU / 2; h; h >>= 1, o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float other = __shfl_xor_sync(FULL, upper ? v[i] : v[i + h], o);
      v[i] = fmaxf(upper ? v[i + h] : v[i], other);
    }
    u += upper ? h : 0;
  }
  const int mine = o ? 2 * o : 1;  // lanes that now hold the same
  for (; o; o >>= 1) v[0] = fmaxf(v[0], __shfl_xor_sync(FULL, v[0], o));
  const int g = u * per + (lane >> lg);
  if ((lane & (mine - 1)) == 0 && g < end) out[g] = v[0];
}

enum BeamMask { MASK_NONE, MASK_CANDIDATES, MASK_SUM };  // no mask; of the candidates alone; of the sum, too
// A warp takes kU pieces a lane of one row.  Bound by instructions, 19 a value, 16 of them in the fp32 pipe (a plain exponential takes
// 6): 33.5 M bf16 logits in 29 us, 0.34 of a copy's rate, 16.8 M fp32 ones under a mask in 23, 0.43.  (Rows by way of shared memory
// in persistent CTAs: 10 us more.)  SHIFT: rows do not all begin at 16-byte boundaries, and are moved to them in registers, as
// which values are added to which must not depend on it (64 x 16 beams, the whole selection: 43.2 us for rows of 32767 tokens, 45.1 for rows
// of 32768 at a stride of 32769, 39.4 for whole pieces, 40.4 with the shifts compiled in; words picked by selects: 44.3, 46.1).
template <typename T, BeamMask MASK, bool SHIFT>
__global__ void __launch_bounds__(256, 4) k_beam_rows(const BeamArgs a) {
  pdl_enter();
  constexpr int E = 16 / sizeof(T);
  __shared__ float hi_tab[32], lo_tab[32];
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    hi_tab[lane] = kExpHi[lane];
    lo_tab[lane] = kExpLo[lane];
  }
  __syncthreads();
  const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t row = task / a.tasks;
  const int tile = (int)(task - row * a.tasks);
  if (row >= (int64_t)a.B * a.K || (a.done && a.done[row])) return;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const int first = tile * (kU * 32 * E), t0 = first + lane * E, off = SHIFT ? row_offset<T>(a, row) : 0;  // the tokens of the warp's, the lane's first value
  const uint32_t* mask = MASK == MASK_NONE ? nullptr : a.allowed + row * a.words;
  constexpr uint32_t LOWEST = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -infinity
  uint4 w[kU], tail;  // tail: of a row that does not begin at a boundary, the piece after the warp's
  if (first >= off && first - off + (kU * 32 + (off ? 1 : 0)) * E <= a.V) {
#pragma unroll
    for (int u = 0; u < kU; ++u) w[u] = __ldcs(reinterpret_cast<const uint4*>(x + t0 - off) + u * 32);
    if (off) tail = __ldcs(reinterpret_cast<const uint4*>(x + first - off) + kU * 32);
  } else {
    auto piece_at = [&](int t) {  // of tokens t ..
      uint32_t q[4] = {LOWEST, LOWEST, LOWEST, LOWEST};
      if (t >= 0 && t + E <= a.V) return __ldcs(reinterpret_cast<const uint4*>(x + t));
      if (t > -E && t < a.V) {  // the row's edges, value by value
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (t + j >= 0 && t + j < a.V) {
            if (sizeof(T) == 2) {
              const uint32_t v = reinterpret_cast<const uint16_t*>(x)[t + j];
              q[j / 2] = j & 1 ? (q[j / 2] & 0xffffu) | v << 16 : (q[j / 2] & 0xffff0000u) | v;
            } else {
              q[j & 3] = reinterpret_cast<const uint32_t*>(x)[t + j];
            }
          }
      }
      return make_uint4(q[0], q[1], q[2], q[3]);
    };
#pragma unroll
    for (int u = 0; u < kU; ++u) w[u] = piece_at(t0 - off + u * 32 * E);
    if (off) tail = piece_at(first - off + kU * 32 * E);
  }
  if (SHIFT && off) {  // pieces of memory to pieces of tokens: what a lane's token piece lacks is in the piece that follows, the next lane's
    auto following = [&](int u) {  // of lane 31, the first lane's next piece
      return __shfl_sync(FULL, lane ? w[u].x : u + 1 < kU ? w[u + 1 < kU ? u + 1 : 0].x : tail.x, (lane + 1) & 31);
    };
    for (int k = off * (int)sizeof(T) / 4; k; --k) {  // a word at a time, the first of the piece that follows after the last
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t got = following(u);
        w[u] = make_uint4(w[u].y, w[u].z, w[u].w, got);
      }
      tail = make_uint4(tail.y, tail.z, tail.w, tail.x);
    }
    if (sizeof(T) == 2 && off & 1) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t got = following(u);
        w[u] = make_uint4(__funnelshift_r(w[u].x, w[u].y, 16), __funnelshift_r(w[u].y, w[u].z, 16), __funnelshift_r(w[u].z, w[u].w, 16), __funnelshift_r(w[u].w, got, 16));
      }
    }
  }
  // the largest value of each run, and of all that are summed; w: what is summed
  float top = -kInf, run[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    if (MASK == MASK_SUM) w[u] = masked<T>(w[u], mask_bits<E>(mask, a.words, t0 + u * 32 * E));
    run[u] = piece_max<T>(w[u]);
    top = fmaxf(top, run[u]);
    if (MASK == MASK_CANDIDATES) run[u] = piece_max<T>(masked<T>(w[u], mask_bits<E>(mask, a.words, t0 + u * 32 * E)));
  }
  const int mine = kU * 32 >> a.lg;  // the warp's runs
  store_runs(run, a.lg, a.top + row * a.runs + (int64_t)tile * mine, a.runs - tile * mine);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
  BeamPart part;
  if (fabsf(top) <= 4096.f) {
    const float floor_ = top - 80.f;  // what is below counts as e^-80 (bf16: e^-64 to e^-80) of the largest: nothing
    // rounded up: further down (96 below -4064 to nearest) the exponent of 2^(n / 32 - e) leaves its field
    const uint32_t floor1 = (__float_as_uint(floor_) + (floor_ > 0.f ? 0xffffu : 0u)) >> 16, floor2 = floor1 | floor1 << 16;
    const int e = octave(top);
    const uint32_t bias = (uint32_t)(127 - e) << 23;
    // two values at a time.  sum: on the grid of 2^-16 that its start fixes; lo: what the grid cuts off, and the rest
    float2 sum = two(192.f), lo = two(0.f);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float2 rest = two(0.f);  // of one piece first: 8 additions a value goes through, not 32
      const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int j = 0; j < E; j += 2) {
        float2 v;
        if (sizeof(T) == 2) {
          const uint32_t c = max2_nan(q[j / 2], floor2);
          v = make_float2(bf_lo(c), bf_hi(c));
        } else {
          v = make_float2(max_nan(__uint_as_float(q[j & 3]), floor_), max_nan(__uint_as_float(q[(j + 1) & 3]), floor_));
        }
        const float2 k = __ffma2_rn(v, two(kL), two(12582912.f));  // rounded to 32nds of an octave: n + 1.5 2^23
        const float2 n = __ffma2_rn(k, two(-1.f), two(12582912.f));  // -n
        const float2 f = __ffma2_rn(v, two(kLlo), __ffma2_rn(v, two(kL), n));
        const float2 p = __fmul2_rn(f, __ffma2_rn(f, __ffma2_rn(f, two(kC3), two(kC2)), two(kC1)));
        const uint32_t bx = __float_as_uint(k.x), by = __float_as_uint(k.y);
        // n's lower 5 bits are j, the others the octave: (1 + j / 32) 2^(n / 32 - e)
        const float2 scale = make_float2(__uint_as_float((bx << 18) + bias), __uint_as_float((by << 18) + bias));
        const float2 h = make_float2(hi_tab[bx & 31], hi_tab[by & 31]), l = make_float2(lo_tab[bx & 31], lo_tab[by & 31]);
        const float2 h2 = __fmul2_rn(h, scale), next = __fadd2_rn(sum, h2);
        const float2 cut = __ffma2_rn(__ffma2_rn(sum, two(-1.f), next), two(-1.f), h2);  // h2 - (next - sum): exact
        rest = __fadd2_rn(rest, __ffma2_rn(__ffma2_rn(h, p, __ffma2_rn(l, p, l)), scale, cut));  // (h + l) (1 + p) - h: l p counts
        sum = next;
      }
      lo = __fadd2_rn(lo, rest);
    }
    // the grid's parts are whole numbers of 2^-16, at most 2^22 a lane: exact as integers.  What of lo is on the grid joins them, so the
    // exchanges round values below 2^-12 (a value's rest, 0.011 of it at most, has gone through 7 additions on the mean by then)
    float r = lo.x + lo.y;
    const int more = __float2int_rn(r * 65536.f);
    r = __fmaf_rn((float)more, -0x1p-16f, r);
    part.hi = __reduce_add_sync(FULL, (int)((sum.x - 192.f) * 65536.f) + (int)((sum.y - 192.f) * 65536.f) + more);
    for (int o = 16; o; o >>= 1) r += __shfl_xor_sync(FULL, r, o);
    part.lo = r;
    part.top = top;
    part.far = 0;
  } else if (top > -kInf) {  // far from 0 (or infinite): in 64 bits
    double s = 0.;
    for (int u = 0; u < kU; ++u)
      for (int j = 0; j < E; ++j) {
        float v = -kInf;
        const int t = t0 + u * 32 * E + j;
        if (t >= 0 && t < a.V) v = to_f(x[t]);
        if (MASK == MASK_SUM && !(t >= 0 && t < a.V && mask[t >> 5] >> (t & 31) & 1)) v = -kInf;
        s += exp((double)v - (double)top);
      }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    part = BeamPart{__double2hiint(s), __int_as_float(__double2loint(s)), top, 1};
  } else {  // nothing above -infinity; a NaN among them shows
    float q = 0.f;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float v = piece<T>(w[u], j);
        if (v != v) q = v;
      }
    for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(FULL, q, o);
    part = BeamPart{0, q, -kInf, 0};
  }
  if (lane == 0) a.part[task] = part;
}

// ---------------------------------------------------------------- selection
// Candidates are compared by (key, lowest place): key the order of the score's two fp32 words, 0 for no candidate.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// a + b = s + the returned
__device__ __forceinline__ float two_sum(float a, float b, float& s) {
  s = __fadd_rn(a, b);
  const float v = __fadd_rn(s, -a);
  return __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -v)), __fadd_rn(b, -v));
}
// base (two words) + (x - ref)
__device__ __forceinline__ uint64_t key_of(float2 base, float x, float ref) {
  if (!(x > -kInf) || !(base.x > -kInf)) return 0;  // NaN too
  float s, e = base.y;
  if (ref != 0.f) {
    float d;
    const float l = two_sum(x, -ref, d);
    x = d;
    if (fabsf(l) < kInf) e = __fadd_rn(e, l);
  }
  e = __fadd_rn(two_sum(base.x, x, s), e);
  float hi = __fadd_rn(s, e), lo = __fadd_rn(e, -__fadd_rn(hi, -s));
  if (!(fabsf(lo) < kInf)) lo = 0.f, hi = s;  // an infinite score, or one at the end of the range
  if (hi != hi) return 0;
  return (uint64_t)ordered(hi) << 32 | ordered(lo);
}
__device__ __forceinline__ float score_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

constexpr int kPick = 1024;   // threads
constexpr int kBins = 2 * kPick;
constexpr int kBeamCount = 256; // items whose ranks are counted (256: 2.5 us, sorted by warps 4; the counts grow with their square)
struct PickSmem {
  uint64_t key[kBeamItems];       // the items at hand; the kept ones first
  uint64_t kept[kBeamMost];
  uint32_t at[kBeamItems];
  uint32_t kept_at[kBeamMost];
  uint32_t run[kBeamMost];        // the kept runs: row,
  int token[kBeamMost];           // first token
  float2 base[kBeamMost];         // rows: the score of a logit at ref
  float ref[kBeamMost];           // rows: what logits are taken relative to; kInf: ended
  int hist[kBins];
  uint32_t red[64];
  int n, digit, need, whole;
};
__device__ __forceinline__ PickSmem& pick_smem() {
  extern __shared__ __align__(16) unsigned char raw[];
  return *reinterpret_cast<PickSmem*>(raw);
}
// An item is kept if its key is above `key`, or equal and its place at most `at`.
struct Cut { uint64_t key; uint32_t at; };
// Of the keys > 0 that a thread has seen: the largest and the smallest upper word, and how many.
struct Seen {
  uint32_t top = 0, bottom = 0xffffffffu;
  int live = 0;
  __device__ __forceinline__ void add(uint64_t k) {
    if (!k) return;
    top = max(top, (uint32_t)(k >> 32));
    bottom = min(bottom, (uint32_t)(k >> 32));
    ++live;
  }
};

// The term of a row's largest logit as the pass over the logits formed it, relative to 2^e, in two words.
__device__ __forceinline__ float2 own_term(float v, int e) {
  const float k = __fmaf_rn(v, kL, 12582912.f), n = __fadd_rn(12582912.f, -k), f = __fmaf_rn(v, kLlo, __fmaf_rn(v, kL, n));
  const float p = __fmul_rn(f, __fmaf_rn(f, __fmaf_rn(f, kC3, kC2), kC1));
  const uint32_t b = __float_as_uint(k);
  const float scale = __uint_as_float((b << 18) + ((uint32_t)(127 - e) << 23)), h = kExpHi[b & 31], l = kExpLo[b & 31];
  const float h2 = __fmul_rn(h, scale), grid = __fadd_rn(__fadd_rn(192.f, h2), -192.f);
  const float rest = __fmaf_rn(__fmaf_rn(h, p, __fmaf_rn(l, p, l)), scale, __fadd_rn(h2, -grid));
  float hi;
  const float lo = two_sum(grid, rest, hi);
  return make_float2(hi, lo);
}
// ln((s + t) 2^q0), s > 0 and normal, t its rest, in two words: table-driven (P. T. P. Tang), r = m c - 1 below 0.01.  q0 and the exponent
// of s together below 2^13 (logits up to 4096 give 5941 at most): n times kLn2A and kLn2B is exact; to 2^-33, as the lower word is rounded
// at 2^-36 three times there (below 2^10 to 2^-36).
__device__ __forceinline__ float2 log2w(float s, float t, float q0) {
  const uint32_t b = __float_as_uint(s);
  const int q = (int)(b >> 23) - 127, j = b >> 17 & 63;
  const float inv = __uint_as_float((uint32_t)(127 - q) << 23), mh = __fmul_rn(s, inv), ml = __fmul_rn(t, inv);
  const float c = kLogC[j], ph = __fmul_rn(mh, c), r1 = __fadd_rn(ph, -1.f);
  const float r0 = __fadd_rn(__fmaf_rn(mh, c, -ph), __fmul_rn(ml, c)), r = __fadd_rn(r1, r0), rl = __fadd_rn(r0, -__fadd_rn(r, -r1));
  const float poly = r * r * __fmaf_rn(r, __fmaf_rn(r, __fmaf_rn(r, 0.2f, -0.25f), 1.f / 3.f), -0.5f);
  const float n = (float)q + q0;
  float hi, lo = two_sum(__fmul_rn(n, kLn2A), __fmul_rn(n, kLn2B), hi);
  lo = __fadd_rn(lo, two_sum(hi, kLogHi[j], hi));
  lo = __fadd_rn(lo, two_sum(hi, r, hi));
  return make_float2(hi, __fadd_rn(lo, __fadd_rn(__fmaf_rn(n, kLn2C, kLogLo[j]), __fadd_rn(poly, rl))));
}

// The number of the CTA's counts before this thread's.
__device__ __forceinline__ int count_before(PickSmem& s, int v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s.red[warp] = (uint32_t)inc;
  __syncthreads();
  const unsigned sum = __reduce_add_sync(FULL, lane < warp ? s.red[lane] : 0u);
  return (int)sum + inc - v;
}

// Among items [0, cnt), more than `want` of them live (key > 0), the cut that keeps `want`: digits of 11 bits from the highest in
// which the keys differ, then, where more keys are equal than are kept, of the place.  same(i): item i agrees in all digits so far.
template <bool PLACE>
__device__ __forceinline__ bool digits(PickSmem& s, int cnt, uint64_t eq, uint64_t& pre, int& shift, int& need) {
  const int tid = threadIdx.x;
  bool whole = false;
  while (shift > 0 && !whole) {
    const int bits = min(11, shift), to = shift - bits;
    s.hist[tid] = 0;
    s.hist[tid + kPick] = 0;
    __syncthreads();
    for (int i = tid; i < cnt; i += kPick) {
      const uint64_t k = s.key[i];
      if (PLACE ? k == eq : k != 0) {
        const uint64_t v = PLACE ? (uint64_t)~s.at[i] & 0xffffffffu : k;  // the lowest place first
        if (shift == 64 || v >> shift == pre) atomicAdd(&s.hist[(int)(v >> to) & ((1 << bits) - 1)], 1);
      }
    }
    __syncthreads();
    const int b1 = kBins - 1 - 2 * tid, c1 = s.hist[b1], c0 = s.hist[b1 - 1];  // from the top bin down, two a thread
    const int above = count_before(s, c0 + c1);
    if (above < need && need <= above + c0 + c1) {
      const bool first = need <= above + c1;
      const int left = first ? need - above : need - above - c1;
      s.digit = first ? b1 : b1 - 1;
      s.need = left;
      s.whole = left == (first ? c1 : c0);
    }
    __syncthreads();
    pre = (shift == 64 ? 0 : pre << bits) | (uint64_t)s.digit;
    need = s.need;
    whole = s.whole;
    shift = to;
  }
  return whole;
}

// Of items [0, cnt) the `want` best to the front, in any order; returns how many there are (fewer: no more candidates).  seen: of the
// threads' shares of the items.  low: a key that none of the kept is below; 1 if they are fewer than `want`.
__device__ __forceinline__ int select_best(int cnt, int want, Seen seen, uint64_t& low) {
  PickSmem& s = pick_smem();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t top = __reduce_max_sync(FULL, seen.top), bottom = __reduce_min_sync(FULL, seen.bottom);
  int live = __reduce_add_sync(FULL, seen.live);
  if (lane == 0) s.red[warp] = top, s.red[32 + warp] = bottom, s.hist[warp] = live;
  __syncthreads();  // (the items are written, too)
  top = __reduce_max_sync(FULL, s.red[lane]);
  bottom = __reduce_min_sync(FULL, s.red[32 + lane]);
  live = __reduce_add_sync(FULL, s.hist[lane]);
  if (tid == 0) s.n = 0;
  __syncthreads();
  Cut cut{0, 0};
  low = live < want ? 1 : (uint64_t)bottom << 32;
  if (live > want) {
    int need = want, shift = 32 + (top == bottom ? 0 : 32 - __clz((int)(top ^ bottom)));
    uint64_t pre = shift < 64 ? ((uint64_t)top << 32) >> shift : 0;
    if (digits<false>(s, cnt, 0, pre, shift, need)) {
      low = pre << shift;
      cut.key = low - 1;  // everything from `low` up
    } else {
      low = cut.key = pre;
      uint64_t at = 0;
      int bits = 32;
      digits<true>(s, cnt, cut.key, at, bits, need);
      cut.at = ~(uint32_t)(at << bits);  // (places differ: the last digit's items are all kept)
    }
  }
  // the kept ones aside, then to the front
  for (int i0 = 0; i0 < cnt; i0 += kPick) {
    const int i = i0 + tid;
    const uint64_t k = i < cnt ? s.key[i] : 0;
    const bool keep = k && (k > cut.key || (k == cut.key && s.at[i] <= cut.at));
    const unsigned m = __ballot_sync(FULL, keep);
    if (!m) continue;
    int first = 0;
    if (lane == 0) first = atomicAdd(&s.n, __popc(m));
    first = __shfl_sync(FULL, first, 0);
    if (keep) {
      const int to = first + __popc(m & ((1u << lane) - 1));
      s.kept[to] = k;
      s.kept_at[to] = s.at[i];
    }
  }
  __syncthreads();
  const int n = s.n;
  if (tid < n) {
    s.key[tid] = s.kept[tid];
    s.at[tid] = s.kept_at[tid];
  }
  __syncthreads();
  return n;
}
// The same of items that are there already.  Seldom called: not inlined, so that what is in the way of every call stays short.
__device__ __noinline__ int select_again(int cnt, int want, uint64_t& low) {
  PickSmem& s = pick_smem();
  Seen seen;
  for (int i = threadIdx.x; i < cnt; i += kPick) seen.add(s.key[i]);
  __syncthreads();
  return select_best(cnt, want, seen, low);
}

// A CTA a group: the rows' logarithms, the n best runs, the n best tokens of those, in order.  Bound by the latency of some
// twenty steps that the CTA takes together: K = 16 of V = 32768 in 11 us beside the rows' 29, K = n = 256 of V = 2048 in 16 beside 23.
template <typename T, bool SHIFT>
__global__ void __launch_bounds__(kPick) k_beam_pick(const BeamArgs a) {
  pdl_enter();
  PickSmem& s = pick_smem();
  constexpr int E = 16 / sizeof(T);
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * a.K;
  if (blockIdx.x == 0 && tid == 0) *a.err = 0;
  // the rows' sums from their parts, 1 to 32 threads a row
  int team = 1;
  while (team < a.tasks && team < 32) team <<= 1;
  for (int b0 = 0; b0 < a.K; b0 += kPick / team) {
    const int b = b0 + tid / team, t = tid % team;
    const bool is = b < a.K, ended = is && a.done && a.done[row0 + b], mine = is && !ended;
    const float c = is ? a.scores[row0 + b] : 0.f;
    const BeamPart* p = a.part + (row0 + b) * a.tasks;
    float best = -kInf, most = -kInf;  // the largest logit of the parts near 0; of those far from it
    for (int i = t; mine && i < a.tasks; i += team) {
      const BeamPart q = p[i];
      if (q.far) most = fmaxf(most, q.top);
      else best = fmaxf(best, q.top);
    }
    for (int o = team / 2; o; o >>= 1) {
      best = fmaxf(best, __shfl_xor_sync(FULL, best, o));
      most = fmaxf(most, __shfl_xor_sync(FULL, most, o));
    }
    float2 at0 = make_float2(-kInf, 0.f);  // no value above -infinity, or a NaN among them: no candidates
    float ref = 0.f;
    // (known to the row's threads) the row has logits far from 0, and not so far below the others that they count for nothing: in 64 bits,
    // below
    const bool far = most > -kInf && !(most < best - 200.f);
    {
      const int e = best > -kInf ? octave(best) : 0;
      const float2 own = own_term(best > -kInf ? best : 0.f, e);
      float hi = 0.f, lo = 0.f;
      for (int i = t; mine && !far && i < a.tasks; i += team) {
        const BeamPart q = p[i];
        if (q.far) {  // 0, or NaN
          if (sum_of(q) != sum_of(q)) hi = __int_as_float(0x7fffffff);
          continue;
        }
        const int d = q.top > -kInf ? e - octave(q.top) : 120;
        const float f = d < 120 ? __uint_as_float((uint32_t)(127 - d) << 23) : 0.f;  // (a part without values is 0, or NaN)
        lo += two_sum(hi, (float)(q.hi >> 12) * 0x1p-4f * f, hi);
        lo += two_sum(hi, (float)(q.hi & 4095) * 0x1p-16f * f, hi);
        lo += two_sum(hi, q.lo * f, hi);
      }
      for (int o = team / 2; o; o >>= 1) {
        const float oh = __shfl_xor_sync(FULL, hi, o), ol = __shfl_xor_sync(FULL, lo, o);
        lo = lo + ol + two_sum(hi, oh, hi);
      }
      lo = two_sum(hi, lo, hi);
      if (hi > 0.f) {
        // where the largest logit has more than half the mass: relative to it, by its own term, so that the term's error counts for the
        // other half alone, and a logit that has all of it has the logarithm 0 exactly (a beam whose next token is given keeps its score)
        const bool half = own.x > 0.5f * hi;
        float2 l = log2w(hi, lo, half ? 0.f : (float)e);
        float from = c, rest = 0.f;
        if (half) {
          const float2 m = log2w(own.x, own.y, 0.f);
          const bool all = (hi - own.x) + (lo - own.y) < 0x1p-40f * hi;
          l.y = all ? 0.f : l.y - m.y;
          l.y += two_sum(all ? 0.f : l.x, all ? 0.f : -m.x, l.x);
          rest = two_sum(c, -best, from);
        }
        const float more = two_sum(from, -l.x, at0.x);
        at0.y = fabsf(at0.x) < kInf ? two_sum(at0.x, more + (rest - l.y), at0.x) : 0.f;
      }
    }
    if (__any_sync(FULL, far)) {  // relative to the largest part's, a logit itself if it is a far one.  The warp's other rows keep theirs
      double e = best > -kInf ? (double)best : -kInf, sum = 0.;
      if (far && (double)most > e) e = (double)most, ref = most;
      for (int i = t; mine && far && i < a.tasks; i += team) {
        const BeamPart q = p[i];
        sum += sum_of(q) * (q.top > -kInf ? exp((q.far ? (double)q.top : (double)octave(q.top) * kLn2) - e) : 1.);
      }
      for (int o = team / 2; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
      if (sum > 0.) {
        const double v = (double)c - ((ref != 0.f ? 0. : e) + log(sum));
        at0.x = (float)v;
        if (fabsf(at0.x) < kInf) at0.y = (float)(v - (double)at0.x);
      }
    }
    if (ended) at0 = make_float2(c, 0.f), ref = kInf;
    if (is && t == 0) {
      s.base[b] = at0.x > -kInf ? at0 : make_float2(-kInf, 0.f);  // NaN: no candidates
      s.ref[b] = ref;
    }
  }
  __syncthreads();
  // the n best runs, kBeamItems at a time
  const uint32_t runs = (uint32_t)a.runs, all = (uint32_t)a.K * runs;
  const float* tops = a.top + row0 * a.runs;
  const uint32_t by = (uint64_t)all * runs >> 32 ? 0 : recip(runs);  // i / runs as a multiplication where that is exact
  int have = 0;
  uint64_t low = 1;
  for (uint32_t i0 = 0; i0 < all;) {
    const int more = (int)min((uint32_t)(kBeamItems - have), all - i0);
    Seen seen;
    if (tid < have) seen.add(s.key[tid]);
    for (int j0 = tid; j0 < more; j0 += 4 * kPick) {
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = j0 + u * kPick < more ? tops[i0 + j0 + u * kPick] : 0.f;  // (an ended beam's: anything)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u * kPick;
        if (j >= more) continue;
        const uint32_t i = i0 + j, b = by ? __umulhi(i, by) : i / runs;
        const float ref = s.ref[b];
        const bool ended = ref == kInf;
        const uint64_t k = ended && i != b * runs ? 0 : key_of(s.base[b], ended ? 0.f : v[u], ended ? 0.f : ref);
        s.at[have + j] = i;
        s.key[have + j] = k;
        seen.add(k);
      }
    }
    have = select_best(have + more, a.n, seen, low);
    i0 += more;
  }
  if (tid < have) {
    const uint32_t i = s.at[tid], b = i / runs;
    s.run[tid] = b;
    s.token[tid] = (int)((i - b * runs) << a.lg) * E;
  }
  if (tid == 0) s.n = 0;
  __syncthreads();
  // their tokens, a piece a thread: those not below `low`, which is n runs' largest at least: few more than n, unless many are alike
  const int pieces = have << a.lg;
  const float lowest = score_of(low);
  auto tokens = [&](int i0, auto many) {  // of pieces i0, i0 + kPick ..
    constexpr int U = decltype(many)::value;
    uint4 w[U];
    uint32_t ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kPick;
      ok[u] = 0;
      if (i >= pieces) continue;
      const uint32_t b = s.run[i >> a.lg];
      const int j = i & ((1 << a.lg) - 1), t0 = s.token[i >> a.lg] + j * E;
      if (s.ref[b] == kInf) {
        ok[u] = j == 0 ? 1 : 0;
        continue;
      }
      const int64_t at = row0 + b;
      ok[u] = a.allowed ? mask_bits<E>(a.allowed + at * a.words, a.words, t0) : (1u << E) - 1;
      const int off = SHIFT ? row_offset<T>(a, at) : 0;
      const T* x = static_cast<const T*>(a.logits) + at * a.ld + t0 - off;  // where that is a 16-byte boundary
      if (t0 >= off && t0 - off + (off ? 2 : 1) * E <= a.V) {
        w[u] = *reinterpret_cast<const uint4*>(x);
        if (off) w[u] = shifted<T>(w[u], *reinterpret_cast<const uint4*>(x + E), off);
      } else {  // an end of the row: its tokens are all looked at below
        w[u] = make_uint4(0, 0, 0, 0);
        ok[u] &= t0 + E > a.V ? (t0 < a.V ? (1u << (a.V - t0)) - 1 : 0u) : ~0u;
        ok[u] |= ok[u] << 16;
      }
    }
    uint32_t found = 0;  // E bits a piece
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ok[u]) continue;
      const uint32_t b = s.run[(i0 + u * kPick) >> a.lg];
      // what is below this as one sum of fp32, off by 2^-23 of either number at most, is below `low` (NaN: nothing is)
      const float bx = s.base[b].x, ref = s.ref[b], least = lowest - 0x1p-21f * (fabsf(lowest) + fabsf(bx)) - 1e-30f;
      uint32_t bits = ok[u] >> 16;
      if (ref == kInf) bits = 1;
      if (!bits) {
#pragma unroll
        for (int j = 0; j < E; ++j) bits |= bx + (piece<T>(w[u], j) - ref) < least ? 0u : 1u << j;
        bits &= ok[u];
      }
      found |= bits << (u * E);
    }
    for (; found; found &= found - 1) {  // few
      const int q = __ffs((int)found) - 1, i = i0 + q / E * kPick;
      const uint32_t b = s.run[i >> a.lg];
      const bool ended = s.ref[b] == kInf;
      const int t = ended ? a.eos : s.token[i >> a.lg] + (i & ((1 << a.lg) - 1)) * E + q % E;
      const float x = ended ? 0.f : to_f(static_cast<const T*>(a.logits)[(row0 + b) * a.ld + t]);
      const uint64_t k = key_of(s.base[b], x, ended ? 0.f : s.ref[b]);
      if (k < low) continue;
      const int to = atomicAdd(&s.n, 1);
      if (to >= kBeamItems) continue;
      s.key[to] = k;
      s.at[to] = b * (uint32_t)a.V + (uint32_t)t;
    }
  };
  for (int i0 = 0; i0 < pieces; i0 += 4 * kPick) tokens(i0 + tid, Int<4>{});
  __syncthreads();
  int cnt = s.n;
  __syncthreads();
  if (cnt > kBeamItems) {  // many alike: again, as many at a time as there is room for
    if (tid == 0) s.n = 0;
    __syncthreads();
    for (int i0 = 0; i0 < pieces; i0 += kPick) {
      tokens(i0 + tid, Int<1>{});
      __syncthreads();
      cnt = s.n;
      __syncthreads();
      if (cnt > kBeamItems - kPick * E) {
        uint64_t l;
        select_again(cnt, a.n, l);
        low = max(low, l);
      }
    }
    cnt = s.n;
    __syncthreads();
  }
  if (cnt > kPick) {
    uint64_t l;
    cnt = select_again(cnt, a.n, l);
  }
  // in order, by (key descending, place ascending): an item's rank is how many precede it
  int rank = kBeamMost;
  uint64_t key = 0;
  uint32_t at = 0xffffffffu;
  if (cnt <= kBeamCount) {  // counted among all, by the keys' upper words, `team` threads an item
    int team = 32;
    while (team > 1 && team * cnt > kPick) team >>= 1;
    const int quads = (cnt + 3) / 4;
    for (int i = tid; i < quads * 4; i += kPick) s.kept_at[i] = i < cnt ? (uint32_t)(s.key[i] >> 32) : 0;
    __syncthreads();
    const int item = tid / team, part = tid % team;
    int above = 0, alike = 0;
    if (item < cnt) {
      key = s.key[item];
      at = s.at[item];
      const uint32_t hi = (uint32_t)(key >> 32);
      for (int q = part; q < quads; q += team) {
        const uint4 o = *reinterpret_cast<const uint4*>(s.kept_at + 4 * q);
        above += (o.x > hi) + (o.y > hi) + (o.z > hi) + (o.w > hi);
        alike += (o.x == hi) + (o.y == hi) + (o.z == hi) + (o.w == hi);
      }
    }
    for (int o = team / 2; o; o >>= 1) {
      above += __shfl_xor_sync(FULL, above, o);
      alike += __shfl_xor_sync(FULL, alike, o);
    }
    if (item < cnt && part == 0) {
      if (alike > 1)  // (itself among them)
        for (int q = 0; q < cnt; ++q) {
          const uint64_t k = s.key[q];
          above += k >> 32 == key >> 32 && (k > key || (k == key && s.at[q] < at));
        }
      rank = above;
    }
  } else {  // an item a thread: each warp sorts its 32, then how many of each warp's precede an item is found by halving
    if (tid < cnt) key = s.key[tid], at = s.at[tid];
    const int warps = (cnt + 31) / 32, lane = tid & 31;
    __syncthreads();
    if (tid < warps * 32) {
#pragma unroll
      for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) {
          const uint64_t ok = __shfl_xor_sync(FULL, key, j);
          const uint32_t oa = __shfl_xor_sync(FULL, at, j);
          const bool better = key > ok || (key == ok && at < oa);
          if (better != (((lane & j) == 0) == ((lane & k) == 0))) key = ok, at = oa;
        }
      s.key[tid] = key;
      s.at[tid] = at;
      s.kept_at[tid] = (uint32_t)(key >> 32);
    }
    __syncthreads();
    if (tid < warps * 32 && key) {
      const uint32_t hi = (uint32_t)(key >> 32);
      const uint32_t* upper = s.kept_at;
      rank = lane;
      for (int w0 = 0; w0 < warps; w0 += 4) {  // four warps' at a time, by the keys' upper words
        int pos[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) pos[u] = min(w0 + u, warps - 1) * 32;
#pragma unroll
        for (int st = 16; st; st >>= 1)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (upper[pos[u] + st - 1] > hi) pos[u] += st;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int w = w0 + u, end = w * 32 + 32;
          if (w >= warps || w == tid >> 5) continue;
          if (upper[pos[u]] > hi) ++pos[u];
          while (pos[u] < end && upper[pos[u]] == hi) {  // alike so far
            const uint64_t k = s.key[pos[u]];
            if (k < key || (k == key && s.at[pos[u]] > at)) break;
            ++pos[u];
          }
          rank += pos[u] - w * 32;
        }
      }
    }
  }
  const int have_n = min(cnt, a.n);
  const int64_t o = (int64_t)blockIdx.x * a.n;
  if (rank < have_n) {
    const uint32_t b = at / (uint32_t)a.V, t = at - b * (uint32_t)a.V;
    a.out_scores[o + rank] = score_of(key);
    a.out_tokens[o + rank] = (int)t;
    a.out_parents[o + rank] = (int)b;
    if (a.out_done) a.out_done[o + rank] = (a.done && a.done[row0 + b]) || (int)t == a.eos;
  }
  if (tid >= have_n && tid < a.n) {
    a.out_scores[o + tid] = -kInf;
    a.out_tokens[o + tid] = -1;
    a.out_parents[o + tid] = 0;
    if (a.out_done) a.out_done[o + tid] = 0;
  }
}

// ------------------------------------------------------------------ reorder
constexpr int kMove = kBeamMoveUnits / 256;  // accesses of a thread, all on their way before the first is stored

// Within one tensor a CTA takes all K rows of one group over a few columns: it reads every row that goes on before it writes one.
// U: the access's type.  (50 MB in and out of 16 beams each: 6.8 us, as a copy.)
template <typename U>
__device__ __forceinline__ void move_within(const BeamState& t, const BeamMove& m, int task) {
  const int units = (int)(t.row_bytes / sizeof(U)), cols = m.cols, chunks = t.ctas / m.B, b = task / chunks, chunk = task - b * chunks;
  const int c0 = chunk * cols, nc = min(cols, units - c0), total = nc * m.n;
  const uint32_t by = recip(nc);
  U* rows = static_cast<U*>(t.dst) + (int64_t)b * m.n * units + c0;
  U v[kMove];
  int to[kMove];
#pragma unroll
  for (int u = 0; u < kMove; ++u) {
    const int i = threadIdx.x + u * 256;
    to[u] = -1;
    if (i >= total) continue;
    const int k = (int)quot(i, by), c = i - k * nc, p = m.parents[(int64_t)b * m.n + k];
    if ((unsigned)p >= (unsigned)m.K || p == k) continue;
    v[u] = rows[(int64_t)p * units + c];
    to[u] = k;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kMove; ++u)
    if (to[u] >= 0) rows[(int64_t)to[u] * units + (threadIdx.x + u * 256 - to[u] * nc)] = v[u];
}
// Between two, kBeamMoveUnits consecutive accesses of the destination, whatever rows they are in: 100 MB to 100 MB in 27 us, as a copy
// (by columns of a group as above 38: the pieces of a row that a CTA takes are 128 bytes).
template <typename U>
__device__ __forceinline__ void move_between(const BeamState& t, const BeamMove& m, int task) {
  const int64_t units = t.row_bytes / (int64_t)sizeof(U), all = units * m.B * m.n, i0 = (int64_t)task * kBeamMoveUnits;
  const int64_t row0 = i0 / units;
  const int off = (int)(i0 - row0 * units), b0 = (int)(row0 / m.n), k0 = (int)(row0 - (int64_t)b0 * m.n);
  const bool wide = units >= kBeamMoveUnits;  // one row, or two
  const uint32_t by = wide ? 0 : recip((uint32_t)units), by_n = recip(m.n);  // i < 2 kBeamMoveUnits
  const U* src = static_cast<const U*>(t.src);
  U* dst = static_cast<U*>(t.dst) + i0;
  U v[kMove];
  bool is[kMove];
#pragma unroll
  for (int u = 0; u < kMove; ++u) {
    const int j = threadIdx.x + u * 256;
    is[u] = false;
    if (i0 + j >= all) continue;
    const int64_t i = off + (int64_t)j;
    const uint32_t r = wide ? i >= units : quot((uint32_t)i, by), g = quot(k0 + r, by_n);
    const int p = m.parents[row0 + r];
    if ((unsigned)p >= (unsigned)m.K) continue;
    v[u] = src[((int64_t)(b0 + g) * m.K + p) * units + (i - (int64_t)r * units)];
    is[u] = true;
  }
#pragma unroll
  for (int u = 0; u < kMove; ++u)
    if (is[u]) dst[threadIdx.x + u * 256] = v[u];
}
template <typename U>
__device__ __forceinline__ void move_rows(const BeamState& t, const BeamMove& m, int task) {
  if (t.dst == t.src) move_within<U>(t, m, task);
  else move_between<U>(t, m, task);
}
__global__ void __launch_bounds__(256) k_beam_move(const __grid_constant__ BeamTable tab, const BeamMove m) {
  pdl_enter();
  if (blockIdx.x == 0) {  // one CTA looks at every parent and alone reports
    int bad = 0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < (int64_t)m.B * m.n; i += 256) bad |= (unsigned)m.parents[i] >= (unsigned)m.K;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *m.err = bad ? 1 : 0;
    return;
  }
  const int cta = (int)blockIdx.x - 1;
  int k = 0;
  while (k + 1 < tab.n && tab.t[k + 1].first <= cta) ++k;
  const BeamState& t = tab.t[k];
  const int task = cta - t.first;
  if (t.unit == 16) move_rows<uint4>(t, m, task);
  else if (t.unit == 4) move_rows<uint32_t>(t, m, task);
  else move_rows<uint8_t>(t, m, task);
}

}  // namespace

// Whether some row does not begin at a 16-byte boundary.
static bool shifts(const BeamArgs& a, bool f32) {
  return (reinterpret_cast<uintptr_t>(a.logits) | (uintptr_t)a.ld * (f32 ? 4 : 2)) % 16 != 0;
}
template <typename T, bool SHIFT>
static cudaError_t rows(const BeamArgs& a, cudaStream_t st) {
  const int64_t tasks = (int64_t)a.B * a.K * a.tasks;
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3((unsigned)((tasks + 7) / 8)), dim3(256), 0, st, a); };
  return !a.allowed ? go(k_beam_rows<T, MASK_NONE, SHIFT>) : a.over_allowed ? go(k_beam_rows<T, MASK_SUM, SHIFT>) : go(k_beam_rows<T, MASK_CANDIDATES, SHIFT>);
}
cudaError_t launch_beam_rows(const BeamArgs& a, bool f32, cudaStream_t st) {
  if (shifts(a, f32)) return f32 ? rows<float, true>(a, st) : rows<bf16, true>(a, st);
  return f32 ? rows<float, false>(a, st) : rows<bf16, false>(a, st);
}
cudaError_t launch_beam_pick(const BeamArgs& a, bool f32, cudaStream_t st) {
  auto go = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PickSmem));
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3((unsigned)a.B), dim3(kPick), sizeof(PickSmem), st, a);
  };
  if (shifts(a, f32)) return f32 ? go(k_beam_pick<float, true>) : go(k_beam_pick<bf16, true>);
  return f32 ? go(k_beam_pick<float, false>) : go(k_beam_pick<bf16, false>);
}
cudaError_t launch_beam_move(const BeamTable& t, const BeamMove& m, int ctas, cudaStream_t st) {
  return launch_pdl(k_beam_move, dim3((unsigned)ctas + 1), dim3(256), 0, st, t, m);
}

}  // namespace gbla
