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

// 2^(j / 32) = hi + lo
__device__ const float kExpHi[32] = {
    0x1.0p+0f, 0x1.059b0ep+0f, 0x1.0b5586p+0f, 0x1.11301ep+0f, 0x1.172b84p+0f, 0x1.1d4874p+0f, 0x1.2387a6p+0f, 0x1.29e9ep+0f,
    0x1.306fep+0f, 0x1.371a74p+0f, 0x1.3dea64p+0f, 0x1.44e086p+0f, 0x1.4bfdaep+0f, 0x1.5342b6p+0f, 0x1.5ab07ep+0f, 0x1.6247ecp+0f,
    0x1.6a09e6p+0f, 0x1.71f75ep+0f, 0x1.7a1148p+0f, 0x1.82589ap+0f, 0x1.8ace54p+0f, 0x1.93737cp+0f, 0x1.9c4918p+0f, 0x1.a5503cp+0f,
    0x1.ae89fap+0f, 0x1.b7f77p+0f, 0x1.c199bep+0f, 0x1.cb720ep+0f, 0x1.d5818ep+0f, 0x1.dfc974p+0f, 0x1.ea4afap+0f, 0x1.f50766p+0f,
};
__device__ const float kExpLo[32] = {
    0x0.0p+0f, -0x1.9d4f52p-25f, 0x1.9f3122p-25f, -0x1.fdb496p-25f, -0x1.c15742p-27f, -0x1.d2e8cap-25f, 0x1.ceac48p-25f, -0x1.5c0424p-25f,
    0x1.4636e2p-25f, -0x1.18aac6p-25f, 0x1.824684p-25f, 0x1.8624b4p-30f, -0x1.593abcp-25f, -0x1.2c561p-25f, -0x1.5bd5ecp-27f, -0x1.f8b55p-25f,
    0x1.9fcef4p-26f, 0x1.1d8beep-25f, -0x1.829fdp-25f, -0x1.accc7cp-26f, 0x1.15506ep-27f, -0x1.e64744p-25f, 0x1.51f848p-27f, -0x1.b83b54p-25f,
    -0x1.a94b14p-26f, -0x1.a09438p-25f, -0x1.3d56b2p-27f, -0x1.8837ccp-27f, -0x1.822dbcp-27f, -0x1.908c94p-25f, 0x1.52486cp-27f, -0x1.246ebp-26f,
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

constexpr int kU = kBeamPieces;

// A warp takes kU pieces a lane of one row.
template <typename T>
__global__ void __launch_bounds__(256) k_beam_rows(const BeamArgs a) {
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
  uint32_t ok[kU];
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
    ok[u] = mask ? mask_bits<E>(mask, a.words, t) : (1u << E) - 1;
  }
  // the largest value of each run, and of all that are summed
  float top = -kInf;
  const int per = 32 >> a.lg;  // runs of the warp's 32 pieces
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    float all = -kInf, run = -kInf;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float v = piece<T>(w[u], j);
      all = fmaxf(all, v);
      if (ok[u] >> j & 1) run = fmaxf(run, v);
    }
    top = fmaxf(top, a.over_allowed ? run : all);
    for (int o = 1; o < 1 << a.lg; o <<= 1) run = fmaxf(run, __shfl_xor_sync(FULL, run, o));
    const int g = (tile * kU + u) * per + (lane >> a.lg);
    if ((lane & ((1 << a.lg) - 1)) == 0 && g < a.runs) a.top[row * a.runs + g] = run;
  }
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
  BeamPart part;
  if (fabsf(top) <= 4096.f) {
    const float floor_ = top - 80.f;  // what is below counts as e^-80 of the largest: nothing
    const int e = (int)floorf(top * 1.44269504f) + 1;
    const uint32_t bias = (uint32_t)(127 - e) << 23;
    float sum = 192.f, lo = 0.f;  // sum: on the grid of 2^-16 that its start fixes; lo: what the grid cuts off, and the rest
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float rest = 0.f;  // of one piece first: 16 additions a value goes through, not 64
#pragma unroll
      for (int j = 0; j < E; ++j) {
        float v = piece<T>(w[u], j);
        if (a.over_allowed && !(ok[u] >> j & 1)) v = -kInf;
        v = max_nan(v, floor_);
        const float k = __fmaf_rn(v, kL, 12582912.f);  // rounded to 32nds of an octave
        const float n = __fadd_rn(k, -12582912.f);
        const float f = __fmaf_rn(v, kLlo, __fmaf_rn(v, kL, -n));
        const float p = f * __fmaf_rn(f, __fmaf_rn(f, __fmaf_rn(f, kC4, kC3), kC2), kC1);
        const uint32_t b = __float_as_uint(k);
        const float scale = __uint_as_float(((b & ~31u) << 18) + bias);  // 2^(floor(n / 32) - e)
        const float h = hi_tab[b & 31], h2 = __fmul_rn(h, scale);
        const float next = __fadd_rn(sum, h2);
        rest += __fmaf_rn(__fmaf_rn(h, p, lo_tab[b & 31]), scale, __fadd_rn(h2, -__fadd_rn(next, -sum)));
        sum = next;
      }
      lo += rest;
    }
    double s = (double)__fadd_rn(sum, -192.f) + (double)lo;
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    part = BeamPart{s, (float)e, 0};
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
    part = BeamPart{s, top, 1};
  } else {  // nothing above -infinity; a NaN among them shows
    float q = 0.f;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float v = piece<T>(w[u], j);
        if (v != v && (!a.over_allowed || (ok[u] >> j & 1))) q = v;
      }
    for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(FULL, q, o);
    part = BeamPart{(double)q, -kInf, 0};
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
constexpr int kBins = 2048;
struct PickSmem {
  uint64_t key[kBeamItems];      // the items at hand; the kept ones first
  uint64_t kept[kBeamMost];
  double total[kBeamMost];       // rows' sums of exponentials; then their base scores
  double expo[kBeamMost];
  uint32_t at[kBeamItems];
  uint32_t kept_at[kBeamMost];
  float ref[kBeamMost];          // what a row's logits are taken relative to
  int hist[kBins];
  uint64_t red[32];
  uint64_t red2[32];
  int n, digit, need, whole;
};

// Of items [0, cnt) the `want` best to the front, in any order; returns how many there are (fewer: no more candidates).
__device__ int select_best(PickSmem& s, int cnt, int want) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the live ones, and the range of their keys
  uint64_t top = 0, low = ~0ull;
  int live = 0;
  for (int i = tid; i < cnt; i += kPick) {
    const uint64_t k = s.key[i];
    if (k) {
      top = max(top, k);
      low = min(low, k);
      ++live;
    }
  }
  for (int o = 16; o; o >>= 1) {
    top = max(top, __shfl_xor_sync(FULL, top, o));
    low = min(low, __shfl_xor_sync(FULL, low, o));
  }
  live = __reduce_add_sync(FULL, live);
  __syncthreads();
  if (tid == 0) s.n = 0;
  if (lane == 0) s.red[warp] = top, s.red2[warp] = low;
  __syncthreads();
  if (lane == 0 && live) atomicAdd(&s.n, live);
  for (int w = 0; w < 32; ++w) {
    top = max(top, s.red[w]);
    low = min(low, s.red2[w]);
  }
  __syncthreads();
  live = s.n;
  // the threshold: keys above `pre` in the bits above `shift` are kept, those equal there go on; at last by the place, whose
  // lowest value is the best
  uint64_t key_min = 1, key_eq = 0;  // kept: key >= key_min, or key == key_eq and place <= at_max
  uint32_t at_max = 0;
  if (live > want) {
    int need = want;
    const uint64_t diff = top ^ low;
    int shift = diff ? 64 - __clzll((long long)diff) : 0;  // bits [shift, 64) are common
    uint64_t pre = shift < 64 ? top >> shift : 0;
    bool whole = false;
    while (shift > 0 && !whole) {
      const int bits = min(11, shift), to = shift - bits;
      for (int i = tid; i < kBins; i += kPick) s.hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < cnt; i += kPick) {
        const uint64_t k = s.key[i];
        if (k && (shift == 64 || k >> shift == pre)) atomicAdd(&s.hist[(int)(k >> to) & ((1 << bits) - 1)], 1);
      }
      __syncthreads();
      // thread t: bins from the top, two each
      const int b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
      const int c1 = s.hist[b1], c0 = s.hist[b0];
      int inc = c1 + c0;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) s.red[warp] = (uint64_t)inc;
      __syncthreads();
      int above = inc - c1 - c0;
      for (int w = 0; w < warp; ++w) above += (int)s.red[w];
      if (above < need && need <= above + c1) s.digit = b1, s.need = need - above, s.whole = need == above + c1;
      if (above + c1 < need && need <= above + c1 + c0) s.digit = b0, s.need = need - above - c1, s.whole = need == above + c1 + c0;
      __syncthreads();
      pre = (shift == 64 ? 0 : pre << bits) | (uint64_t)s.digit;
      need = s.need;
      whole = s.whole;
      shift = to;
      __syncthreads();
    }
    key_min = pre << shift;  // everything from here up, if the last digit's items are all kept
    if (!whole) {            // more equal keys than are kept: by place
      key_eq = key_min;
      key_min = key_eq + 1;
      uint32_t apre = 0;
      int ashift = 32;
      bool all = false;
      while (ashift > 0 && !all) {
        const int bits = min(11, ashift), to = ashift - bits;
        for (int i = tid; i < kBins; i += kPick) s.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < cnt; i += kPick)
          if (s.key[i] == key_eq && (ashift == 32 || s.at[i] >> ashift == apre)) atomicAdd(&s.hist[(s.at[i] >> to) & ((1u << bits) - 1)], 1);
        __syncthreads();
        const int b0 = 2 * tid, b1 = b0 + 1;  // from the lowest place
        const int c0 = s.hist[b0], c1 = s.hist[b1];
        int inc = c0 + c1;
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(FULL, inc, o);
          if (lane >= o) inc += v;
        }
        if (lane == 31) s.red[warp] = (uint64_t)inc;
        __syncthreads();
        int before = inc - c0 - c1;
        for (int w = 0; w < warp; ++w) before += (int)s.red[w];
        if (before < need && need <= before + c0) s.digit = b0, s.need = need - before, s.whole = need == before + c0;
        if (before + c0 < need && need <= before + c0 + c1) s.digit = b1, s.need = need - before - c0, s.whole = need == before + c0 + c1;
        __syncthreads();
        apre = (ashift == 32 ? 0 : apre << bits) | (uint32_t)s.digit;
        need = s.need;
        all = s.whole;
        ashift = to;
        __syncthreads();
      }
      at_max = ashift ? (apre << ashift) | ((1u << ashift) - 1) : apre;
    }
  }
  // the kept ones aside, then to the front
  if (tid == 0) s.n = 0;
  __syncthreads();
  for (int i0 = 0; i0 < cnt; i0 += kPick) {
    const int i = i0 + tid;
    const uint64_t k = i < cnt ? s.key[i] : 0;
    const bool keep = k && (k >= key_min || (k == key_eq && s.at[i] <= at_max));
    const unsigned m = __ballot_sync(FULL, keep);
    int first = 0;
    if (lane == 0 && m) first = atomicAdd(&s.n, __popc(m));
    first = __shfl_sync(FULL, first, 0);
    if (keep) {
      const int to = first + __popc(m & ((1u << lane) - 1));
      s.kept[to] = k;
      s.kept_at[to] = s.at[i];
    }
  }
  __syncthreads();
  const int n = s.n;
  for (int i = tid; i < n; i += kPick) {
    s.key[i] = s.kept[i];
    s.at[i] = s.kept_at[i];
  }
  __syncthreads();
  return n;
}

// The `want` best of `total` items, item(i) -> (key, place), kBeamItems at a time.
template <typename F>
__device__ int select_all(PickSmem& s, int64_t total, int want, F&& item) {
  int have = 0;
  for (int64_t i0 = 0; i0 < total;) {
    const int more = (int)min((int64_t)(kBeamItems - have), total - i0);
    for (int i = threadIdx.x; i < more; i += kPick) item(i0 + i, s.key[have + i], s.at[have + i]);
    __syncthreads();
    have = select_best(s, have + more, want);
    i0 += more;
  }
  return have;
}

// A CTA a group: the rows' logarithms, the n best runs, the n best tokens of those, in order.
template <typename T>
__global__ void __launch_bounds__(kPick) k_beam_pick(const BeamArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) unsigned char raw[];
  PickSmem& s = *reinterpret_cast<PickSmem*>(raw);
  constexpr int E = 16 / sizeof(T);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * a.K;
  if (blockIdx.x == 0 && tid == 0) *a.err = 0;
  float2* base = reinterpret_cast<float2*>(s.total);  // [K], over the sums once they are used
  for (int b = warp; b < a.K; b += kPick / 32) {
    const BeamPart* p = a.part + (row0 + b) * a.tasks;
    const bool done = a.done && a.done[row0 + b];
    double e = 0., sum = 0.;  // the sum is sum exp(e)
    float ref = 0.f;
    if (!done) {
      float best = -kInf;  // of the parts near 0: as powers of two, exactly
      bool far = false;
      for (int i = lane; i < a.tasks; i += 32) {
        if (p[i].far) far = true;
        else best = fmaxf(best, p[i].ref);
      }
      for (int o = 16; o; o >>= 1) best = fmaxf(best, __shfl_xor_sync(FULL, best, o));
      far = __any_sync(FULL, far);
      e = best > -kInf ? (double)best * kLn2 : -kInf;
      if (far) {  // relative to the largest of all, a logit itself where it is far from 0
        float most = -kInf;
        for (int i = lane; i < a.tasks; i += 32)
          if (p[i].far) most = fmaxf(most, p[i].ref);
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(FULL, most, o));
        if ((double)most > e) e = (double)most, ref = most;
      }
      for (int i = lane; i < a.tasks; i += 32) {
        const BeamPart q = p[i];
        double f = 1.;  // (a part without values has a sum of 0, or NaN)
        if (q.ref > -kInf && far) f = exp((q.far ? (double)q.ref : (double)q.ref * kLn2) - e);
        else if (q.ref > -kInf) f = q.ref > best - 1000.f ? __longlong_as_double((long long)(1023 + (int)(q.ref - best)) << 52) : 0.;
        sum += q.s * f;
      }
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    }
    if (lane == 0) s.total[b] = sum, s.expo[b] = ref != 0.f ? 0. : e, s.ref[b] = ref;
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
  const int G = E << a.lg;
  int have = select_all(s, (int64_t)a.K * a.runs, a.n, [&](int64_t i, uint64_t& key, uint32_t& at) {
    const int b = (int)(i / a.runs), g = (int)(i - (int64_t)b * a.runs);
    at = (uint32_t)i;
    if (a.done && a.done[row0 + b]) key = g == 0 ? key_of(base[b], 0.f, 0.f) : 0;
    else key = key_of(base[b], a.top[(row0 + b) * a.runs + g], s.ref[b]);
  });
  // the runs' places, out of the way of the tokens
  uint32_t* run = reinterpret_cast<uint32_t*>(s.expo);
  for (int i = tid; i < have; i += kPick) run[i] = s.at[i];
  __syncthreads();
  have = select_all(s, (int64_t)have * G, a.n, [&](int64_t i, uint64_t& key, uint32_t& at) {
    const uint32_t r = run[i / G];
    const int b = (int)(r / (uint32_t)a.runs), g = (int)(r - (uint32_t)b * a.runs), j = (int)(i % G);
    const int64_t row = row0 + b;
    key = 0;
    at = 0;
    if (a.done && a.done[row]) {
      if (j == 0) key = key_of(base[b], 0.f, 0.f), at = (uint32_t)b * (uint32_t)a.V + (uint32_t)a.eos;
      return;
    }
    const int t = g * G + j - row_offset<T>(a, row);
    if (t < 0 || t >= a.V) return;
    if (a.allowed && !(a.allowed[row * a.words + (t >> 5)] >> (t & 31) & 1)) return;
    key = key_of(base[b], to_f(static_cast<const T*>(a.logits)[row * a.ld + t]), s.ref[b]);
    at = (uint32_t)b * (uint32_t)a.V + (uint32_t)t;
  });
  // in order: bitonic, by (key descending, place ascending)
  int size = 1;
  while (size < have) size <<= 1;
  for (int i = have + tid; i < size; i += kPick) s.key[i] = 0, s.at[i] = 0xffffffffu;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      for (int i = tid; i < size; i += kPick) {
        const int o = i ^ j;
        if (o > i) {
          const uint64_t x = s.key[i], y = s.key[o];
          const uint32_t p = s.at[i], q = s.at[o];
          const bool later = x < y || (x == y && p > q);  // i comes after o
          if (later == ((i & k) == 0)) s.key[i] = y, s.key[o] = x, s.at[i] = q, s.at[o] = p;
        }
      }
      __syncthreads();
    }
  const int64_t o0 = (int64_t)blockIdx.x * a.n;
  for (int i = tid; i < a.n; i += kPick) {
    const bool is = i < have;
    const uint32_t at = is ? s.at[i] : 0;
    const int b = (int)(at / (uint32_t)a.V), t = (int)(at - (uint32_t)b * (uint32_t)a.V);
    a.out_scores[o0 + i] = is ? score_of(s.key[i]) : -kInf;
    a.out_tokens[o0 + i] = is ? t : -1;
    a.out_parents[o0 + i] = is ? b : 0;
    if (a.out_done) a.out_done[o0 + i] = is && ((a.done && a.done[row0 + b]) || t == a.eos);
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
