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
// candidates some lie closer than fp32's rounding.  So each exponential is formed to 2^-30 (2^(j/32) from a table in two
// words, P. T. P. Tang's reduction, and a polynomial of degree 4), added into two words (the sum is off by 2^-27 at most, by
// 2^-31 on the mean), and scores are compared in two fp32 words.  Equal logits of one row stay equal.
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
// 2^(f / 32) - 1 = f (c1 + f (c2 + f (c3 + f c4))): c_k = (ln 2 / 32)^k / k!, the next term below 2^-39 at |f| = 1/2
constexpr float kC1 = 0x1.62e43p-6f, kC2 = 0x1.ebfbep-13f, kC3 = 0x1.c6b08ep-20f, kC4 = 0x1.3b2ab6p-27f;

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

// The row's tokens begin `off` values behind a 16-byte boundary; places are counted from that boundary.
template <typename T>
__device__ __forceinline__ int row_offset(const BeamArgs& a, int64_t row) {
  return (int)((reinterpret_cast<uintptr_t>(a.logits) + row * a.ld * sizeof(T)) % 16 / sizeof(T));
}
// E mask bits from token t (below 0: bits of no token) of a row.
template <int E>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* m, int words, int t) {
  const int w = t >> 5;  // -1 for t < 0
  const uint32_t lo = w >= 0 && w < words ? m[w] : 0u, hi = w + 1 < words && (t & 31) + E > 32 ? m[w + 1] : 0u;
  return __funnelshift_r(lo, hi, t & 31) & ((1u << E) - 1);
}

__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ double sum_of(const BeamPart& p) {
  return p.far ? __hiloint2double(p.hi, __float_as_int(p.lo)) : (double)p.hi * (1. / 65536.) + (double)p.lo;
}

constexpr int kU = kBeamPieces;

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

// A warp takes kU pieces a lane of one row.  Bound by instructions, some 16 a value (a plain exponential takes 6).
template <typename T>
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
  const int t0 = tile * (kU * 32 * E) + lane * E - row_offset<T>(a, row);  // the token of the lane's first value
  const uint32_t* mask = a.allowed ? a.allowed + row * a.words : nullptr;
  constexpr uint32_t LOWEST = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -infinity
  uint4 w[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int t = t0 + u * 32 * E;
    w[u] = make_uint4(LOWEST, LOWEST, LOWEST, LOWEST);
    if (t >= 0 && t + E <= a.V) {
      w[u] = __ldcs(reinterpret_cast<const uint4*>(x + t));
    } else if (t > -E && t < a.V) {  // the row's edges, value by value
      uint32_t q[4] = {LOWEST, LOWEST, LOWEST, LOWEST};
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
      w[u] = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
  // the largest value of each run, and of all that are summed; w: what is summed
  float top = -kInf;
  const int per = 32 >> a.lg;  // runs of the warp's 32 pieces
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    float run = piece_max<T>(w[u]);
    if (mask) {
      const uint4 m = masked<T>(w[u], mask_bits<E>(mask, a.words, t0 + u * 32 * E));
      top = fmaxf(top, run);
      run = piece_max<T>(m);
      if (a.over_allowed) w[u] = m;
    }
    top = fmaxf(top, run);
    for (int o = 1; o < 1 << a.lg; o <<= 1) run = fmaxf(run, __shfl_xor_sync(FULL, run, o));
    const int g = (tile * kU + u) * per + (lane >> a.lg);
    if ((lane & ((1 << a.lg) - 1)) == 0 && g < a.runs) a.top[row * a.runs + g] = run;
  }
  if (mask && a.over_allowed) {
    top = -kInf;
#pragma unroll
    for (int u = 0; u < kU; ++u) top = fmaxf(top, piece_max<T>(w[u]));
  }
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
  BeamPart part;
  if (fabsf(top) <= 4096.f) {
    const float floor_ = top - 80.f;  // what is below counts as e^-80 of the largest: nothing
    const uint32_t floor2 = pack_bf16(floor_, floor_);
    const int e = (int)floorf(top * 1.44269504f) + 1;
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
        const float2 p = __fmul2_rn(f, __ffma2_rn(f, __ffma2_rn(f, __ffma2_rn(f, two(kC4), two(kC3)), two(kC2)), two(kC1)));
        const uint32_t bx = __float_as_uint(k.x), by = __float_as_uint(k.y);
        // n's lower 5 bits are j, the others the octave: (1 + j / 32) 2^(n / 32 - e)
        const float2 scale = make_float2(__uint_as_float((bx << 18) + bias), __uint_as_float((by << 18) + bias));
        const float2 h = make_float2(hi_tab[bx & 31], hi_tab[by & 31]), l = make_float2(lo_tab[bx & 31], lo_tab[by & 31]);
        const float2 h2 = __fmul2_rn(h, scale), next = __fadd2_rn(sum, h2);
        const float2 cut = __ffma2_rn(__ffma2_rn(sum, two(-1.f), next), two(-1.f), h2);  // h2 - (next - sum): exact
        rest = __fadd2_rn(rest, __ffma2_rn(__ffma2_rn(h, p, l), scale, cut));
        sum = next;
      }
      lo = __fadd2_rn(lo, rest);
    }
    // the grid's parts are whole numbers of 2^-16, at most 2^22 a lane: exact as integers
    part.hi = __reduce_add_sync(FULL, (int)((sum.x - 192.f) * 65536.f) + (int)((sum.y - 192.f) * 65536.f));
    float r = lo.x + lo.y;
    for (int o = 16; o; o >>= 1) r += __shfl_xor_sync(FULL, r, o);
    part.lo = r;
    part.ref = (float)e;
    part.far = 0;
  } else if (top > -kInf) {  // far from 0 (or infinite): in 64 bits
    double s = 0.;
    for (int u = 0; u < kU; ++u)
      for (int j = 0; j < E; ++j) {
        float v = -kInf;
        const int t = t0 + u * 32 * E + j;
        if (t >= 0 && t < a.V) v = to_f(x[t]);
        if (a.over_allowed && mask && !(t >= 0 && t < a.V && mask[t >> 5] >> (t & 31) & 1)) v = -kInf;
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
struct PickSmem {
  uint64_t key[kBeamItems];       // the items at hand; the kept ones first
  uint64_t kept[kBeamMost];
  double expo[kBeamMost];         // rows' references; then the kept runs
  uint32_t at[kBeamItems];
  uint32_t kept_at[kBeamMost];
  double total[kBeamMost];        // rows' sums of exponentials; then their base scores
  float ref[kBeamMost];           // what a row's logits are taken relative to
  int hist[kBins];
  uint32_t red[64];
  int n, digit, need, whole;
};
// An item is kept if its key is above `key`, or equal and its place at most `at`.
struct Cut { uint64_t key; uint32_t at; };

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

// Of items [0, cnt) the `want` best to the front, in any order; returns how many there are (fewer: no more candidates).  low: a key
// that none of the kept is below; 1 if they are fewer than `want`.
__device__ int select_best(PickSmem& s, int cnt, int want, uint64_t& low) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t top = 0, bottom = 0xffffffffu;  // of the keys' upper words
  int live = 0;
  for (int i = tid; i < cnt; i += kPick) {
    const uint64_t k = s.key[i];
    if (k) {
      top = max(top, (uint32_t)(k >> 32));
      bottom = min(bottom, (uint32_t)(k >> 32));
      ++live;
    }
  }
  top = __reduce_max_sync(FULL, top);
  bottom = __reduce_min_sync(FULL, bottom);
  live = __reduce_add_sync(FULL, live);
  __syncthreads();
  if (lane == 0) s.red[warp] = top, s.red[32 + warp] = bottom, s.hist[warp] = live;
  __syncthreads();
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

// A CTA a group: the rows' logarithms, the n best runs, the n best tokens of those, in order.
template <typename T>
__global__ void __launch_bounds__(kPick) k_beam_pick(const BeamArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) unsigned char raw[];
  PickSmem& s = *reinterpret_cast<PickSmem*>(raw);
  constexpr int E = 16 / sizeof(T);
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * a.K;
  if (blockIdx.x == 0 && tid == 0) *a.err = 0;
  float2* base = reinterpret_cast<float2*>(s.total);  // [K], over the sums once they are used
  // the rows' sums from their parts, 1 to 32 threads a row
  int team = 1;
  while (team < a.tasks && team < 32) team <<= 1;
  for (int b0 = 0; b0 < a.K; b0 += kPick / team) {
    const int b = b0 + tid / team, t = tid % team;
    const BeamPart* p = a.part + (row0 + b) * a.tasks;
    const bool mine = b < a.K && !(a.done && a.done[row0 + b]);
    float best = -kInf, most = -kInf;  // of the parts near 0: as powers of two, exactly; of those far from it
    for (int i = t; mine && i < a.tasks; i += team) {
      if (p[i].far) most = fmaxf(most, p[i].ref);
      else best = fmaxf(best, p[i].ref);
    }
    for (int o = team / 2; o; o >>= 1) {
      best = fmaxf(best, __shfl_xor_sync(FULL, best, o));
      most = fmaxf(most, __shfl_xor_sync(FULL, most, o));
    }
    const bool far = most > -kInf;
    double e = best > -kInf ? (double)best * kLn2 : -kInf, sum = 0.;  // the sum is sum exp(e)
    float ref = 0.f;
    if (far && (double)most > e) e = (double)most, ref = most;  // relative to a logit itself where it is far from 0
    for (int i = t; mine && i < a.tasks; i += team) {
      const BeamPart q = p[i];
      double f = 1.;  // (a part without values has a sum of 0, or NaN)
      if (q.ref > -kInf && far) f = exp((q.far ? (double)q.ref : (double)q.ref * kLn2) - e);
      else if (q.ref > -kInf) f = q.ref > best - 1000.f ? __hiloint2double((1023 + (int)(q.ref - best)) << 20, 0) : 0.;
      sum += sum_of(q) * f;
    }
    for (int o = team / 2; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    if (b < a.K && t == 0) s.total[b] = sum, s.expo[b] = ref != 0.f ? 0. : e, s.ref[b] = ref;
  }
  __syncthreads();
  float2 mine = make_float2(-kInf, 0.f);
  if (tid < a.K) {
    const float c = a.scores[row0 + tid];
    if (a.done && a.done[row0 + tid]) {
      mine = make_float2(c, 0.f);
    } else {
      const double sum = s.total[tid];
      if (sum > 0.) {  // else no value above -infinity, or a NaN among them
        const double v = (double)c - (s.expo[tid] + log(sum));
        mine.x = (float)v;
        if (fabsf(mine.x) < kInf) mine.y = (float)(v - (double)mine.x);
      }
    }
    if (!(mine.x > -kInf)) mine = make_float2(-kInf, 0.f);  // NaN: no candidates
  }
  __syncthreads();
  if (tid < a.K) base[tid] = mine;
  __syncthreads();
  // the n best runs, kBeamItems at a time
  const uint32_t runs = (uint32_t)a.runs, all = (uint32_t)a.K * runs;
  const float* tops = a.top + row0 * a.runs;
  int have = 0;
  uint64_t low = 1;
  for (uint32_t i0 = 0; i0 < all;) {
    const int more = (int)min((uint32_t)(kBeamItems - have), all - i0);
    for (int j = tid; j < more; j += kPick) {
      const uint32_t i = i0 + j, b = i / runs;
      s.at[have + j] = i;
      s.key[have + j] = a.done && a.done[row0 + b] ? (i == b * runs ? key_of(base[b], 0.f, 0.f) : 0) : key_of(base[b], tops[i], s.ref[b]);
    }
    __syncthreads();
    have = select_best(s, have + more, a.n, low);
    i0 += more;
  }
  uint32_t* run = reinterpret_cast<uint32_t*>(s.expo);  // out of the way of the tokens
  if (tid < have) run[tid] = s.at[tid];
  if (tid == 0) s.n = 0;
  __syncthreads();
  // their tokens, a piece a thread: those not below `low`, which is n runs' largest at least
  const int pieces = have << a.lg;
  for (int i0 = 0; i0 < pieces; i0 += kPick) {
    const int i = i0 + tid;
    if (i < pieces) {
      const uint32_t r = run[i >> a.lg], b = r / runs;
      const int64_t row = row0 + b;
      const float2 bs = base[b];
      const float ref = s.ref[b];
      auto put = [&](float x, float rf, uint32_t t) {
        const uint64_t k = key_of(bs, x, rf);
        if (k < low) return;
        const int to = atomicAdd(&s.n, 1);
        s.key[to] = k;
        s.at[to] = b * (uint32_t)a.V + t;
      };
      if (a.done && a.done[row]) {
        if ((i & ((1 << a.lg) - 1)) == 0) put(0.f, 0.f, (uint32_t)a.eos);
      } else {
        const int t0 = (int)(((r - b * runs) << a.lg) + (i & ((1 << a.lg) - 1))) * E - row_offset<T>(a, row);
        const T* x = static_cast<const T*>(a.logits) + row * a.ld;
        // what is below this as one sum of fp32, off by 2^-23 of either number at most, is below `low` (NaN: nothing is)
        const float lowest = score_of(low), least = lowest - 0x1p-21f * (fabsf(lowest) + fabsf(bs.x)) - 1e-30f;
        const bool inside = t0 >= 0 && t0 + E <= a.V;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (inside) w = *reinterpret_cast<const uint4*>(x + t0);
        uint32_t ok = (1u << E) - 1;
        if (a.allowed) ok = mask_bits<E>(a.allowed + row * a.words, a.words, t0);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const int t = t0 + j;
          if (!inside && (t < 0 || t >= a.V)) continue;
          const float v = inside ? piece<T>(w, j) : to_f(x[t]);
          if ((ok >> j & 1) && !(bs.x + (v - ref) < least)) put(v, ref, (uint32_t)t);
        }
      }
    }
    __syncthreads();
    const int cnt = s.n;
    __syncthreads();
    if (cnt > kBeamItems - kPick * E) {  // room for as many again
      uint64_t l;
      select_best(s, cnt, a.n, l);
      low = max(low, l);
    }
  }
  int cnt = s.n;
  __syncthreads();
  if (cnt > kPick) {
    uint64_t l;
    cnt = select_best(s, cnt, a.n, l);
  }
  // in order, an item a thread: bitonic, by (key descending, place ascending)
  int size = 1;
  while (size < cnt) size <<= 1;
  uint64_t key = tid < cnt ? s.key[tid] : 0;
  uint32_t at = tid < cnt ? s.at[tid] : 0xffffffffu;
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      uint64_t ok;
      uint32_t oa;
      if (j < 32) {
        ok = __shfl_xor_sync(FULL, key, j);
        oa = __shfl_xor_sync(FULL, at, j);
      } else {
        __syncthreads();
        s.key[tid] = key;
        s.at[tid] = at;
        __syncthreads();
        ok = s.key[tid ^ j];
        oa = s.at[tid ^ j];
      }
      const bool better = key > ok || (key == ok && at < oa);
      if (better != (((tid & j) == 0) == ((tid & k) == 0))) key = ok, at = oa;
    }
  const int have_n = min(cnt, a.n);
  if (tid < a.n) {
    const int64_t o = (int64_t)blockIdx.x * a.n + tid;
    const bool is = tid < have_n;
    const uint32_t b = is ? at / (uint32_t)a.V : 0, t = at - b * (uint32_t)a.V;
    a.out_scores[o] = is ? score_of(key) : -kInf;
    a.out_tokens[o] = is ? (int)t : -1;
    a.out_parents[o] = (int)b;
    if (a.out_done) a.out_done[o] = is && ((a.done && a.done[row0 + b]) || (int)t == a.eos);
  }
}

// ------------------------------------------------------------------ reorder
// A CTA takes all K rows of one group over a few columns of one tensor: it reads every row that goes on before it writes one,
// so the rows may be moved within their tensor.  U: the access's type.
template <typename U>
__device__ __forceinline__ void move_rows(const BeamState& t, const BeamMove& m, int task) {
  const int chunks = t.chunks, b = task / chunks, chunk = task - b * chunks;
  const int units = (int)(t.row_bytes / sizeof(U)), cols = m.cols;
  const int c0 = chunk * cols, nc = min(cols, units - c0), total = nc * m.n;
  const U* src = static_cast<const U*>(t.src) + (int64_t)b * m.K * units + c0;
  U* dst = static_cast<U*>(t.dst) + (int64_t)b * m.n * units + c0;
  U v[8];
  bool is[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int i = threadIdx.x + u * 256;
    is[u] = false;
    if (i >= total) continue;
    const int k = i / nc, c = i - k * nc, p = m.parents[(int64_t)b * m.n + k];
    if ((unsigned)p >= (unsigned)m.K || (t.dst == t.src && p == k)) continue;
    v[u] = src[(int64_t)p * units + c];
    is[u] = true;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int i = threadIdx.x + u * 256;
    if (!is[u]) continue;
    const int k = i / nc, c = i - k * nc;
    dst[(int64_t)k * units + c] = v[u];
  }
}
__global__ void __launch_bounds__(256) k_beam_move(const __grid_constant__ BeamTable tab, const BeamMove m) {
  pdl_enter();
  if (blockIdx.x == gridDim.x - 1) {  // the last CTA looks at every parent and alone reports
    int bad = 0;
    for (int64_t i = threadIdx.x; i < (int64_t)m.B * m.n; i += 256) bad |= (unsigned)m.parents[i] >= (unsigned)m.K;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *m.err = bad ? 1 : 0;
    return;
  }
  int k = 0;
  while (k + 1 < tab.n && tab.t[k + 1].first <= (int)blockIdx.x) ++k;
  const BeamState& t = tab.t[k];
  const int task = (int)blockIdx.x - t.first;
  if (t.unit == 16) move_rows<uint4>(t, m, task);
  else if (t.unit == 4) move_rows<uint32_t>(t, m, task);
  else move_rows<uint8_t>(t, m, task);
}

}  // namespace

cudaError_t launch_beam_rows(const BeamArgs& a, bool f32, cudaStream_t st) {
  const int64_t tasks = (int64_t)a.B * a.K * a.tasks;
  const dim3 grid((unsigned)((tasks + 7) / 8));
  return f32 ? launch_pdl(k_beam_rows<float>, grid, dim3(256), 0, st, a) : launch_pdl(k_beam_rows<bf16>, grid, dim3(256), 0, st, a);
}
cudaError_t launch_beam_pick(const BeamArgs& a, bool f32, cudaStream_t st) {
  auto go = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PickSmem));
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3((unsigned)a.B), dim3(kPick), sizeof(PickSmem), st, a);
  };
  return f32 ? go(k_beam_pick<float>) : go(k_beam_pick<bf16>);
}
cudaError_t launch_beam_move(const BeamTable& t, const BeamMove& m, int ctas, cudaStream_t st) {
  return launch_pdl(k_beam_move, dim3((unsigned)ctas + 1), dim3(256), 0, st, t, m);
}

}  // namespace gbla
