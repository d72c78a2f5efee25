// Gated linear recurrence with a decay per token and channel:
//   s_t = c softplus(lam) sigmoid(r_t),  a_t = exp(-s_t),  q_t = 1 - a_t,
//   m_t = sqrt(1 - a_t^2) = sqrt(q_t (2 - q_t)),
//   h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t,  y_t = h_t,
// per sequence and channel in either direction, and its backward
//   w_t = dy_t + a_{t+1} w_{t+1}          (w = dL/dh, + dhT at the last token)
//   dx = w m sig(i),  di = w m x sig(i) (1 - sig(i)),
//   e_t = s_t dL/ds_t = -w (a s h_{t-1} - sig(i) x a^2 (s / m)),
//   dr = e (1 - sig(r)),  dlam = sum_t e_t sig(lam) / softplus(lam),  dh0 = a w at the first token.
// q is formed without cancellation (a polynomial for small s), so m keeps its
// relative accuracy for decays near 1; s / m tends to 0 with s, so dr and dlam
// stay finite where a = 1.
//
// A thread walks one channel of one sequence.  The state on entry to every
// kGlrChunk-row chunk is saved for the backward, which recomputes the states
// of a chunk from it.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace gbla {
namespace {

constexpr unsigned FULLM = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqf(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// softplus(lam), and sigmoid(lam) / softplus(lam) (1 - e^lam / 2 + .. for small e^lam).
__device__ __forceinline__ float softplus_f(float l) { return fmaxf(l, 0.f) + log1pf(expf(-fabsf(l))); }
__device__ __forceinline__ float dsoftplus_ratio(float l) {
  return l < -15.f ? 1.f : 1.f / ((1.f + expf(-l)) * softplus_f(l));
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 e = mul2(x, two(-kLog2e));
  const float2 d = add2(make_float2(ex2f(e.x), ex2f(e.y)), two(1.f));
  return make_float2(rcpf(d.x), rcpf(d.y));
}

// The gates of two values with k = c softplus(lam): a, s and m = sqrt(1 - a^2).
struct Gate2 { float2 a, s, m, sr; };
// k < 1/4 for both channels, so s < 1/4: with g = sqrt(sigmoid(r)) = rsqrt(1 + e^-r), two special functions a value, and
// polynomials (Chebyshev interpolation on [0, 1/4]) for (1 - e^-s) / s and sqrt((1 - e^-2s) / 2s), both within 1e-8.
__device__ __forceinline__ Gate2 gate2_small(float2 r, float2 k, float2 root2k) {
  Gate2 v;
  const float2 e = mul2(r, two(-kLog2e));
  const float2 d = add2(make_float2(ex2f(e.x), ex2f(e.y)), two(1.f));
  const float2 g = make_float2(rsqf(d.x), rsqf(d.y));
  v.sr = mul2(g, g);
  v.s = mul2(k, v.sr);
  const float2 s = v.s;
  float2 p = fma2(s, two(0.0075136060f), two(-0.0414906554f));
  p = fma2(s, p, two(0.1666510850f));
  p = fma2(s, p, two(-0.4999995232f));
  p = fma2(s, p, two(1.f));
  v.a = fma2(make_float2(-s.x, -s.y), p, two(1.f));
  float2 w = fma2(s, two(0.0123387622f), two(-0.0622048900f));
  w = fma2(s, w, two(0.2083072215f));
  w = fma2(s, w, two(-0.4999991953f));
  w = fma2(s, w, two(1.f));
  v.m = mul2(mul2(g, root2k), w);
  return v;
}
// Any k: q = 1 - e^-s from the polynomial below 1/4, m = sqrt(q (2 - q)).
__device__ __forceinline__ float sqf(float x);
__device__ __forceinline__ Gate2 gate2_any(float2 r, float2 k) {
  Gate2 v;
  v.sr = sigmoid2(r);
  v.s = mul2(k, v.sr);
  const float2 s = v.s, t = mul2(s, two(-kLog2e));
  float2 p = fma2(s, two(0.0075136060f), two(-0.0414906554f));
  p = fma2(s, p, two(0.1666510850f));
  p = fma2(s, p, two(-0.4999995232f));
  p = fma2(s, p, two(1.f));
  float2 q = mul2(s, p);
  v.a = add2(two(1.f), make_float2(-q.x, -q.y));
  const float2 e = make_float2(ex2f(t.x), ex2f(t.y));
  if (s.x >= 0.25f) { q.x = 1.f - e.x; v.a.x = e.x; }
  if (s.y >= 0.25f) { q.y = 1.f - e.y; v.a.y = e.y; }
  const float2 z = mul2(q, add2(two(2.f), make_float2(-q.x, -q.y)));
  v.m = make_float2(sqf(z.x), sqf(z.y));
  return v;
}
__device__ __forceinline__ float sqf(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------ chunks
// The rows are cut into chunks (slots of at least kGlrSlot rows each into their own, everything else as one stream); a
// chunk and 64 channels are a tile, a tile is one CTA's, and a warp has PER neighbouring rows of it.  A chunk's rows
// are numbered in the direction of the recurrence.
struct Span {
  int64_t r0;       // physical first row of the chunk
  int nr;           // its rows
  int b;            // its slot (slots of their own)
  int k;            // its first row in the slot
};
template <int CH>
__device__ __forceinline__ int64_t row_at(const GlrArgs& a, const Span& c, int j) {
  return a.reverse ? c.r0 + CH - 1 - j : c.r0 + j;
}
// Bits of the N <= 32 rows from j0 on: in the chunk, in a sequence, a sequence's first, its last (in the direction of the
// recurrence).  Whole warps call it.
struct Flags { uint32_t in, V, F, E; };
template <int CH, int N>
__device__ __forceinline__ Flags flags_of(const GlrArgs& a, const Span& c, int per_seq, int j0, int lane) {
  const int j = j0 + min(lane, N - 1), p = a.reverse ? CH - 1 - j : j;  // place in the chunk
  const bool in = p < c.nr;
  bool v = in, s, z;
  const int64_t row = c.r0 + p;
  if (a.seq.mode == SEQ_VARLEN) {
    s = in && (a.marks[row >> 6] >> (row & 63) & 1);
    z = in && (row + 1 == a.seq.T || (a.marks[(row + 1) >> 6] >> ((row + 1) & 63) & 1));
  } else {
    int b = c.b, pos = c.k + p;
    if (!per_seq) {
      b = (int)row / a.seq.L;
      pos = (int)row - b * a.seq.L;
    }
    const int len = a.seq.mode == SEQ_PADDED ? (in ? a.seq.lens[b] : 0) : a.seq.L;
    v = in && pos < len;
    s = v && pos == 0;
    z = v && pos == len - 1;
  }
  const uint32_t m = N == 32 ? ~0u : (1u << N) - 1;
  Flags f;
  f.in = __ballot_sync(FULLM, in) & m;
  f.V = __ballot_sync(FULLM, v) & m;
  f.F = __ballot_sync(FULLM, a.reverse ? z : s) & m;
  f.E = __ballot_sync(FULLM, a.reverse ? s : z) & m;
  return f;
}
// The sequence of a row that is in one.
__device__ __forceinline__ int seq_of(const GlrArgs& a, int64_t row) {
  if (a.seq.mode != SEQ_VARLEN) return (int)(row / a.seq.L);
  int lo = 0, hi = a.seq.n_seq - 1;  // the last b with cu[b] <= row: it is not empty
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.seq.cu[mid] <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------ the scan between chunks
// A tile publishes, per channel, what its rows do to a state that enters: h -> A h + H, as one 64-bit word {H, A}
// (present when the top bit, A's sign, is set; A = infinity stands for "a sequence starts here: h -> H").  Chunks
// form groups of 16 and groups of groups; a chunk that needs the state before it composes the words of the chunks
// before it in its group, of the groups before its own in the larger group, and the state after the last larger
// group: at most 31 words, read together.  The order of composition is fixed, so results do not depend on timing.
// Tiles are handed out by a counter in an order in which everything a tile waits for has been handed out before:
// the earliest unfinished tile waits for nothing unfinished, so every wait ends (and is bounded all the same).
constexpr uint64_t kReset = 0xFF80000000000000ull;
__device__ __forceinline__ uint64_t word(float A, float H) {
  return (uint64_t)(__float_as_uint(A) | 0x80000000u) << 32 | __float_as_uint(H);
}
__device__ __forceinline__ uint64_t reset_word(float H) { return kReset | __float_as_uint(H); }
struct Map { float A, H; bool reset; };  // reset: h -> H
__device__ __forceinline__ Map map_of(uint64_t w) {
  Map m;
  m.H = __uint_as_float((uint32_t)w);
  m.A = __uint_as_float((uint32_t)(w >> 32) & 0x7fffffffu);
  m.reset = (w >> 32) == (kReset >> 32);
  return m;
}
// first m, then n
__device__ __forceinline__ Map then(const Map& m, const Map& n) {
  Map o;
  o.reset = m.reset || n.reset;
  o.H = n.reset ? n.H : fmaf(n.A, m.H, n.H);
  o.A = m.A * n.A;  // of no use where reset
  return o;
}
__device__ __forceinline__ uint64_t word_of(const Map& m) { return m.reset ? reset_word(m.H) : word(m.A, m.H); }

__device__ __forceinline__ void publish(uint64_t* p, const Map& x) {
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(word_of(x)) : "memory");
}
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
  uint64_t x;
  asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(x) : "l"(p) : "memory");
  return x;
}
// The words of a call: of chunks, groups and larger groups, each [..][dp] with dp the channels rounded up to 64.
struct Chain {
  uint64_t* chunk; uint64_t* group; uint64_t* large;
  int k, last;      // this chunk's place in its chain, and the last one
};
__device__ __forceinline__ Chain chain_of(const GlrArgs& a, const GlrTiles& t, int s, int k, int ch) {
  // s: the sequence slot (0 for a stream); the arrays hold each slot's words in the order of its chain
  const int64_t n = t.per_seq ? t.per_seq : t.n_chunks, ng = (n + 15) >> 4, nl = (n + 255) >> 8;
  Chain c;
  c.chunk = a.words + s * n * a.dp + ch;
  c.group = a.words + ((int64_t)t.n_chunks + s * ng) * a.dp + ch;
  c.large = a.words + ((int64_t)t.n_chunks + (int64_t)(t.per_seq ? a.seq.n_seq : 1) * ng + s * nl) * a.dp + ch;
  c.k = k;
  c.last = (int)n - 1;
  return c;
}
// The 31 words that chunk c.k reads, from the oldest on: the state after the last larger group, what the groups before its
// own in the larger group do, what the chunks before it in its group do.  Four parts of 8 (the last of 7), a thread of
// each for every channel: ask() asks for a thread's at once, before they are needed; answer() waits for those that were
// not there yet, again together, and composes them.
constexpr uint64_t kIdentity = 0xBF80000000000000ull;  // h -> 1 h + 0
struct Words { uint64_t w[8]; };
__device__ __forceinline__ const uint64_t* words_at(const Chain& c, int64_t dp, int part) {
  const int l = c.k >> 8;
  return part >= 2 ? c.chunk + (int64_t)((c.k & ~15) + (part - 2) * 8) * dp : c.group + (int64_t)((l << 4) + part * 8 - 1) * dp;
}
// The word j of a part exists (the rest count as identities).
__device__ __forceinline__ bool word_is(const Chain& c, int part, int j) {
  if (part >= 2) return (part - 2) * 8 + j < (c.k & 15);
  if (part == 0 && j == 0) return c.k >= 256;
  return part * 8 + j - 1 < (c.k >> 4 & 15);
}
__device__ __forceinline__ uint64_t peek_word(const Chain& c, const uint64_t* p, int64_t dp, int part, int j) {
  return peek(part == 0 && j == 0 ? c.large + (int64_t)((c.k >> 8) - 1) * dp : p + j * dp);
}
__device__ __forceinline__ void ask(const Chain& c, int64_t dp, int part, Words& v) {
  const uint64_t* p = words_at(c, dp, part);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v.w[j] = kIdentity;
    if (word_is(c, part, j)) v.w[j] = peek_word(c, p, dp, part, j);
  }
}
// Whether to go on asking after n vain tries: bounded, and given up at once where another wait has been.
__device__ __forceinline__ bool patient(int n, int* err) {
  if ((n & 255) != 255) return true;
  if (*(volatile int*)err & kErrTimeout) return false;
  if (n < (1 << 22)) return true;
  atomicOr(err, kErrTimeout);
  return false;
}
__device__ __forceinline__ Map answer(const Chain& c, int64_t dp, int part, Words& v, int* err) {
  for (int n = 0;; ++n) {
    uint64_t there = v.w[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) there &= v.w[j];
    if (there >> 63 || !patient(n, err)) break;
    const uint64_t* p = words_at(c, dp, part);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(v.w[j] >> 63)) v.w[j] = peek_word(c, p, dp, part, j);
  }
  Map m{1.f, 0.f, false};
#pragma unroll
  for (int j = 0; j < 8; ++j) m = then(m, map_of(v.w[j]));
  return m;
}

// ------------------------------------------------------------ tiles
// A pair of neighbouring channels of a row.  VEC: pairs are aligned and whole.
template <typename T, bool VEC>
__device__ __forceinline__ float2 load2(const void* base, int64_t o, int n) {
  const T* p = (const T*)base + o;
  if (VEC) {
    if (n <= 0) return make_float2(0.f, 0.f);
    if (sizeof(T) == 2) {
      const uint32_t w = __ldg((const uint32_t*)p);
      return make_float2(bf_lo(w), bf_hi(w));
    }
    return __ldg((const float2*)p);
  }
  return make_float2(n > 0 ? to_f(p[0]) : 0.f, n > 1 ? to_f(p[1]) : 0.f);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store2(void* base, int64_t o, int n, float2 v) {
  T* p = (T*)base + o;
  if (VEC) {
    if (n <= 0) return;
    if (sizeof(T) == 2) *(uint32_t*)p = pack_bf16(v.x, v.y);
    else *(float2*)p = v;
    return;
  }
  if (n > 0) p[0] = from_f<T>(v.x);
  if (n > 1) p[1] = from_f<T>(v.y);
}

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kCtasFwd = 2;                  // an SM's
constexpr int kPerF = kGlrRowsFwd / kWarps;  // a warp's rows; a lane has two channels of each

// How a tile's rows are read: copied ahead into shared memory (rows of 16-byte pieces), or straight into registers by
// pairs of channels or single ones.
enum GlrLoad { GLR_TMA = 0, GLR_PAIRS = 1, GLR_SINGLE = 2 };

// A tile: channels from ch0, the chunk's rows, and its place k in its slot's chain (-1: no tile).
struct Tile {
  int ch0, k;
  Span c;
  int inner;        // every row is inside one sequence and neither its first nor its last
};
template <int CH>
__device__ __forceinline__ Tile tile_of(const GlrArgs& a, const GlrTiles& g, unsigned t, bool back) {
  const unsigned ncg = (unsigned)(a.dp >> 6);
  Tile o;
  o.ch0 = (int)(t % ncg) * 64;
  const unsigned w = t / ncg;
  if (g.per_seq) {
    const unsigned q = w / (unsigned)a.seq.n_seq;
    o.c.b = (int)(w - q * (unsigned)a.seq.n_seq);
    o.k = (int)q;
    o.c.k = (back ? g.per_seq - 1 - o.k : o.k) * CH;
    o.c.r0 = (int64_t)o.c.b * a.seq.L + o.c.k;
    o.c.nr = min(CH, a.seq.L - o.c.k);
    const int len = a.seq.mode == SEQ_PADDED ? a.seq.lens[o.c.b] : a.seq.L;
    o.inner = o.c.k > 0 && o.c.k + CH < len;
  } else {
    o.c.b = o.c.k = 0;
    o.k = (int)w;
    o.c.r0 = (int64_t)(back ? g.n_chunks - 1 - o.k : o.k) * CH;
    o.c.nr = (int)min((int64_t)CH, a.seq.T - o.c.r0);
    o.inner = 0;
    if (a.seq.mode == SEQ_VARLEN && o.c.r0 + CH < a.seq.T) {
      uint64_t m = a.marks[(o.c.r0 + CH) >> 6] & 1;
#pragma unroll
      for (int j = 0; j < CH / 64; ++j) m |= a.marks[(o.c.r0 >> 6) + j];
      o.inner = m == 0;
    }
  }
  return o;
}

// A pair of channels in shared memory.
template <typename T>
__device__ __forceinline__ float2 lds2(const T* p) {
  if (sizeof(T) == 2) {
    const uint32_t w = *(const uint32_t*)p;
    return make_float2(bf_lo(w), bf_hi(w));
  }
  return *(const float2*)p;
}

// The lane's rows of a tile: decays and what they add, and what they do together (A, H; a start in them: H alone).
// PLAIN: every row is inside one sequence.  sm: the lane's first row of x in shared memory, r and i one and two tiles on.
template <typename T, int LOAD, bool SMALL, bool PLAIN, int PER, int CH>
__device__ __forceinline__ void local_rows(const GlrArgs& a, const T* sm, const Span& c, const Flags& f, int j0, int ch,
                                           int nch, float2 ka, float2 root2k, float2 (&da)[PER], float2 (&u)[PER], float2& A, float2& H) {
  const int64_t step = a.reverse ? -a.ld : a.ld;
  int64_t o = LOAD == GLR_TMA ? 0 : row_at<CH>(a, c, j0) * a.ld + ch;
  A = two(1.f);
  H = two(0.f);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    float2 x, r, i;
    if (LOAD == GLR_TMA) {
      r = lds2(sm + CH * 64);
      i = lds2(sm + 2 * CH * 64);
      x = lds2(sm);
      sm += a.reverse ? -64 : 64;
    } else {
      const int n = f.V >> q & 1 ? nch : 0;
      r = load2<T, LOAD == GLR_PAIRS>(a.r, o, n);
      i = load2<T, LOAD == GLR_PAIRS>(a.i, o, n);
      x = load2<T, LOAD == GLR_PAIRS>(a.x, o, n);
      o += step;
    }
    const Gate2 g = SMALL ? gate2_small(r, ka, root2k) : gate2_any(r, ka);
    da[q] = g.a;
    u[q] = mul2(g.m, mul2(sigmoid2(i), x));
    if (!PLAIN) {
      if (!(f.V >> q & 1)) {
        da[q] = two(1.f);
        u[q] = two(0.f);
      }
      if (f.F >> q & 1) {
        if (a.h0) {
          const int64_t oh = (int64_t)seq_of(a, row_at<CH>(a, c, j0 + q)) * a.d + ch;
          if (nch > 0) u[q].x = fmaf(da[q].x, a.h0[oh], u[q].x);
          if (nch > 1) u[q].y = fmaf(da[q].y, a.h0[oh + 1], u[q].y);
        }
        H = u[q];
        continue;
      }
    }
    H = fma2(da[q], H, u[q]);
    A = mul2(A, da[q]);
  }
}

struct GlrMaps { CUtensorMap m[3]; };  // x, r, i

// Tiles in shared memory at once.
template <typename T> constexpr int stages_fwd() { return sizeof(T) == 2 ? 2 : 1; }

// Shared memory of a CTA of the forward, after its tiles of x, r and i.  A lane's two channels are {A, A, H, H}, and A = -1
// where a sequence starts.
struct GlrShared {
  float4 agg[2][kWarps][32];  // of each warp's rows; tiles take turns
  float4 before[4][32];       // of each part of the words before
  Tile tile[2];
  uint64_t full[2];
};
__device__ __forceinline__ void put_map(float4* row, int cc, const Map& m) {
  float* p = (float*)(row + (cc >> 1)) + (cc & 1);
  p[0] = m.reset ? -1.f : m.A;
  p[2] = m.H;
}
__device__ __forceinline__ Map get_map(const float4* row, int cc) {
  const float* p = (const float*)(row + (cc >> 1)) + (cc & 1);
  return Map{p[0], p[2], p[0] == -1.f};
}
// The state after what g does to h.
__device__ __forceinline__ float2 after(float4 g, float2 h) {
  const float2 o = fma2(make_float2(g.x, g.y), h, make_float2(g.z, g.w));
  return g.x == -1.f ? make_float2(g.z, g.w) : o;
}

// Forward: one pass, x, r and i read once and y written once.  Bound by the instructions of the gates (four special
// functions a value) and by memory.  Two CTAs an SM keep taking tiles, so that one's wait for the state between tiles
// is another's arithmetic; a tile's rows are copied to shared memory while an earlier one is worked on.
template <typename T, int LOAD>
__global__ void __launch_bounds__(kThreads, kCtasFwd) k_glr_fwd(const GlrArgs a, const GlrTiles tl, const __grid_constant__ GlrMaps maps) {
  constexpr int PER = kPerF, CH = kGlrRowsFwd, ST = stages_fwd<T>();
  constexpr uint32_t BYTES = 3 * CH * 64 * sizeof(T), ALL = (1u << PER) - 1;
  extern __shared__ __align__(128) uint8_t raw[];
  pdl_enter();
  if (a.err && *a.err) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cc = tid & 63, part = tid >> 6;
  uint8_t* tiles = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
  GlrShared& sh = *reinterpret_cast<GlrShared*>(tiles + (LOAD == GLR_TMA ? ST * BYTES : 0));
  const uint32_t full = smem_u32(sh.full);
  const unsigned total = (unsigned)tl.n_chunks * (unsigned)(a.dp >> 6);

  // thread 0: tile o into stage st
  auto fetch = [&](const Tile& o, int st) {
    sh.tile[st] = o;
    if (LOAD == GLR_TMA && o.k >= 0) {
      mbar_expect_tx(full + 8 * st, BYTES);
#pragma unroll
      for (int m = 0; m < 3; ++m)
        tma_load_2d(smem_u32(tiles) + st * BYTES + m * (BYTES / 3), &maps.m[m], full + 8 * st, o.ch0, (int)o.c.r0);
    }
  };
  auto take = [&]() {
    const unsigned t = (unsigned)atomicAdd(a.ticket, 1ull);
    Tile o;
    o.k = -1;
    if (t < total) o = tile_of<CH>(a, tl, t, a.reverse);
    return o;
  };
  Tile next;  // thread 0: the tile after those fetched
  if (tid == 0) {
    if (LOAD == GLR_TMA) {
      for (int st = 0; st < ST; ++st) mbar_init(full + 8 * st, 1);
      mbar_init_fence();
    }
    for (int st = 0; st < ST; ++st) fetch(take(), st);
    next = take();
  }
  __syncthreads();

  for (int it = 0;; ++it) {
    const int st = it % ST;
    const Tile t = sh.tile[st];
    const int k = t.k;
    if (k < 0) break;
    const Chain chain = chain_of(a, tl, t.c.b, k, t.ch0 + cc);
    Words words;
    ask(chain, a.dp, part, words);
    // the lane's rows
    const int ch = t.ch0 + 2 * lane, nch = a.d - ch;  // channels of this lane: 2 (or more), 1 or none
    const int j0 = warp * PER;
    const float2 ka = *(const float2*)(a.kd + ch);
    Flags f{ALL, ALL, 0, 0};
    if (!t.inner) f = flags_of<CH, PER>(a, t.c, tl.per_seq, j0, lane);
    const bool inner = LOAD == GLR_TMA && f.V == ALL && f.F == 0;
    const T* sm = (const T*)(tiles + st * BYTES) + (a.reverse ? CH - 1 - j0 : j0) * 64 + 2 * lane;
    if (LOAD == GLR_TMA && !mbar_wait_bounded(full + 8 * st, (it / ST) & 1)) atomicOr(a.err_out, kErrTimeout);
    float2 da[PER], u[PER], A, H;
    if (inner && __all_sync(FULLM, ka.x < 0.25f && ka.y < 0.25f)) {
      const float2 root2k = make_float2(sqf(2.f * ka.x), sqf(2.f * ka.y));
      local_rows<T, LOAD, true, true, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, root2k, da, u, A, H);
    } else if (inner) {
      local_rows<T, LOAD, false, true, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, ka, da, u, A, H);
    } else {
      local_rows<T, LOAD, false, false, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, ka, da, u, A, H);
    }
    float4(*agg)[32] = sh.agg[it & 1];
    agg[warp][lane] = f.F ? make_float4(-1.f, -1.f, H.x, H.y) : make_float4(A.x, A.y, H.x, H.y);
    // whether the chunk's first row begins a sequence: then nothing enters
    const bool need = !__syncthreads_or(warp == 0 && (f.F & 1)) && k > 0;
    if (tid == 0) fetch(next, st);
    Map tot{1.f, 0.f, false};
    if (part == 3 && k < chain.last) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) tot = then(tot, get_map(agg[w], cc));
      publish(chain.chunk + (int64_t)k * a.dp, tot);
    }
    if (need && (part >= 2 || k >= 16)) put_map(sh.before[part], cc, answer(chain, a.dp, part, words, a.err_out));
    if ((k & 15) == 15 && k < chain.last && part >= 2) {  // what the group does takes no other group: it does not wait for parts 0 and 1
      named_bar(1, 128);
      if (part == 3)
        publish(chain.group + (int64_t)(k >> 4) * a.dp, need ? then(then(get_map(sh.before[2], cc), get_map(sh.before[3], cc)), tot) : tot);
    }
    // the state that enters the warp's rows
    float2 h = two(0.f);
    if (need) {
      __syncthreads();
      if (k >= 16) h = after(sh.before[1][lane], after(sh.before[0][lane], h));
      h = after(sh.before[3][lane], after(sh.before[2][lane], h));
    }
    if ((k & 255) == 255 && k < chain.last && part == 3) {
      const float2 c2 = make_float2(__shfl_sync(FULLM, h.x, cc >> 1), __shfl_sync(FULLM, h.y, cc >> 1));
      const float in = cc & 1 ? c2.y : c2.x;
      publish(chain.large + (int64_t)(k >> 8) * a.dp, Map{0.f, tot.reset ? tot.H : fmaf(tot.A, in, tot.H), true});
    }
    for (int w = 0; w < warp; ++w) h = after(agg[w][lane], h);
    if (j0 % kGlrChunk == 0 && a.saved) {  // the backward's chunks are of kGlrChunk rows
      const int p = a.reverse ? CH - kGlrChunk - j0 : j0;  // physical place of the piece in the chunk
      if (p < t.c.nr) {
        const int64_t piece = tl.per_seq ? (int64_t)t.c.b * a.per_seq + (t.c.k + p) / kGlrChunk : (t.c.r0 + p) / kGlrChunk;
        store2<float, false>(a.saved, piece * a.d + ch, nch, h);
      }
    }
    // the rows again, from the state that enters them
    const int64_t step = a.reverse ? -a.d : a.d;
    int64_t o = row_at<CH>(a, t.c, j0) * a.d + ch;
    if (inner && (!a.hT || f.E == 0)) {
      if (nch > 0) {
        T* y = (T*)a.y + o;
#pragma unroll
        for (int p = 0; p < PER; ++p, y += step) {
          h = fma2(da[p], h, u[p]);
          store2<T, true>(y, 0, 2, h);
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < PER; ++p, o += step) {
        if (f.F >> p & 1) h = u[p];
        else h = fma2(da[p], h, u[p]);
        store2<T, LOAD != GLR_SINGLE>(a.y, o, f.in >> p & 1 ? nch : 0, f.V >> p & 1 ? h : two(0.f));
        if (a.hT && (f.E >> p & 1)) store2<float, false>(a.hT, (int64_t)seq_of(a, row_at<CH>(a, t.c, j0 + p)) * a.d + ch, nch, h);
      }
    }
    if (tid == 0 && next.k >= 0) next = take();
  }
}

// s / (2 sinh s) = a s / (1 - a^2), the even factor of the decay's gradient: a polynomial in s^2 below s = 1/4 (Chebyshev
// interpolation, within 4e-8).
template <bool SMALL>
__device__ __forceinline__ float2 half_s_over_sinh(const Gate2& g) {
  const float2 w = mul2(g.s, g.s);
  float2 p = fma2(w, two(0.5f * 0.0192536078f), two(0.5f * -0.1666622013f));
  p = fma2(w, p, two(0.5f));
  if (!SMALL) {
    if (g.s.x >= 0.25f) p.x = g.a.x * g.s.x * rcpf(g.m.x * g.m.x);
    if (g.s.y >= 0.25f) p.y = g.a.y * g.s.y * rcpf(g.m.y * g.m.y);
  }
  return p;
}

// What the backward holds of a row: a; p = m sig(i) (dx = w p); sig(i); s; then G = -a (s h_{t-1} - u s / (2 sinh s)) in the
// place of s (e = w G) and x (1 - sig(i)) in that of sig(i) (di = dx times it); x and dy as they came.
template <typename T> struct RowPair;
template <> struct RowPair<bf16> {
  uint32_t w;
  __device__ __forceinline__ float2 get() const { return make_float2(bf_lo(w), bf_hi(w)); }
  __device__ __forceinline__ void set(float2 v) { w = pack_bf16(v.x, v.y); }  // exact: it was bf16
};
template <> struct RowPair<float> {
  float2 v;
  __device__ __forceinline__ float2 get() const { return v; }
  __device__ __forceinline__ void set(float2 o) { v = o; }
};

constexpr int kPerB = kGlrChunk / kWarps;
constexpr int kCtasBwd = 2;  // an SM's
template <typename T> constexpr int stages_bwd() { return sizeof(T) == 2 ? 2 : 1; }

template <typename T, int LOAD, bool SMALL, bool PLAIN, int PER, int CH>
__device__ __forceinline__ void local_rows_bwd(const GlrArgs& a, const T* sm, const Span& c, const Flags& f, int j0, int ch, int nch,
                                               float2 ka, float2 root2k, float2 (&da)[PER], float2 (&pp)[PER], float2 (&gi)[PER],
                                               float2 (&s)[PER], RowPair<T> (&x)[PER], RowPair<T> (&dy)[PER], float2& A, float2& H, float2& D) {
  const int64_t step = a.reverse ? -a.ld : a.ld, stepy = a.reverse ? -a.d : a.d;
  int64_t o = LOAD == GLR_TMA ? 0 : row_at<CH>(a, c, j0) * a.ld + ch, oy = LOAD == GLR_TMA ? 0 : row_at<CH>(a, c, j0) * a.d + ch;
  A = two(1.f);
  H = D = two(0.f);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    float2 r, i;
    if (LOAD == GLR_TMA) {
      r = lds2(sm + CH * 64);
      i = lds2(sm + 2 * CH * 64);
      x[q] = *(const RowPair<T>*)sm;
      dy[q] = *(const RowPair<T>*)(sm + 3 * CH * 64);
      sm += a.reverse ? -64 : 64;
    } else {
      const int n = f.V >> q & 1 ? nch : 0;
      r = load2<T, LOAD == GLR_PAIRS>(a.r, o, n);
      i = load2<T, LOAD == GLR_PAIRS>(a.i, o, n);
      x[q].set(load2<T, LOAD == GLR_PAIRS>(a.x, o, n));
      dy[q].set(load2<T, LOAD == GLR_PAIRS>(a.dy, oy, n));
      o += step;
      oy += stepy;
    }
    const Gate2 g = SMALL ? gate2_small(r, ka, root2k) : gate2_any(r, ka);
    da[q] = g.a;
    s[q] = g.s;
    gi[q] = sigmoid2(i);
    pp[q] = mul2(g.m, gi[q]);
    if (!PLAIN) {
      if (!(f.V >> q & 1)) {
        da[q] = two(1.f);
        pp[q] = s[q] = gi[q] = two(0.f);
        x[q].set(two(0.f));
        dy[q].set(two(0.f));
      }
      if (f.F >> q & 1) {
        float2 h = two(0.f);
        if (a.h0) h = load2<float, false>(a.h0, (int64_t)seq_of(a, row_at<CH>(a, c, j0 + q)) * a.d + ch, nch);
        H = fma2(da[q], h, mul2(pp[q], x[q].get()));
        continue;
      }
    }
    H = fma2(da[q], H, mul2(pp[q], x[q].get()));
    A = mul2(A, da[q]);
  }
  if (!PLAIN && (f.F | f.E)) {  // A is the product of all decays where it counts: rows behind a start or before an end
    A = two(1.f);
#pragma unroll
    for (int q = 0; q < PER; ++q) A = mul2(A, da[q]);
  }
#pragma unroll
  for (int q = PER - 1; q >= 0; --q) {
    if (!PLAIN && (f.E >> q & 1)) D = a.dhT ? load2<float, false>(a.dhT, (int64_t)seq_of(a, row_at<CH>(a, c, j0 + q)) * a.d + ch, nch) : two(0.f);
    D = mul2(da[q], add2(D, dy[q].get()));
  }
}

struct GlrMaps4 { CUtensorMap m[4]; };  // x, r, i, dy

struct GlrSharedBwd {
  float4 agg[2][kWarps][32];   // forward: what each warp's rows do to the state; tiles take turns
  float4 gga[2][kWarps][32];   // backward: what they do to a w
  float4 before[4][32];        // of each part of the words of the chunks behind
  float2 sum[2][kWarps][32];   // dlam of each warp's rows
  Tile tile[2];
  uint64_t full[2];
};

// Backward: one pass from each sequence's end, x, r, i and dy read once, dx, dr and di written once; the states before the
// rows come from the chunk's saved one, the w behind them as the forward's states do.  As the forward, with tiles of
// kGlrChunk rows: a row's held values take eleven registers a pair of channels.
template <typename T, int LOAD>
__global__ void __launch_bounds__(kThreads, kCtasBwd) k_glr_bwd(const GlrArgs a, const GlrTiles tl, const __grid_constant__ GlrMaps4 maps) {
  constexpr int PER = kPerB, CH = kGlrChunk, ST = stages_bwd<T>();
  constexpr uint32_t BYTES = 4 * CH * 64 * sizeof(T), ALL = (1u << PER) - 1;
  extern __shared__ __align__(128) uint8_t raw[];
  pdl_enter();
  if (a.err && *a.err) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cc = tid & 63, part = tid >> 6;
  uint8_t* tiles = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
  GlrSharedBwd& sh = *reinterpret_cast<GlrSharedBwd*>(tiles + (LOAD == GLR_TMA ? ST * BYTES : 0));
  const uint32_t full = smem_u32(sh.full);
  const unsigned total = (unsigned)tl.n_chunks * (unsigned)(a.dp >> 6);

  auto fetch = [&](const Tile& o, int st) {  // thread 0: tile o into stage st
    sh.tile[st] = o;
    if (LOAD == GLR_TMA && o.k >= 0) {
      mbar_expect_tx(full + 8 * st, BYTES);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        tma_load_2d(smem_u32(tiles) + st * BYTES + m * (BYTES / 4), &maps.m[m], full + 8 * st, o.ch0, (int)o.c.r0);
    }
  };
  auto take = [&]() {
    const unsigned t = (unsigned)atomicAdd(a.ticket, 1ull);
    Tile o;
    o.k = -1;
    if (t < total) o = tile_of<CH>(a, tl, t, !a.reverse);  // the chains run against the recurrence
    return o;
  };
  // dlam of a tile: its warps' sums in order
  auto put_sum = [&](int q, int64_t piece, int ch0) {
    if (warp != 0 || !a.dlam_part) return;
    float2 v = two(0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = add2(v, sh.sum[q][w][lane]);
    store2<float, false>(a.dlam_part, piece * a.d + ch0 + 2 * lane, a.d - ch0 - 2 * lane, v);
  };
  Tile next;  // thread 0: the tile after those fetched
  if (tid == 0) {
    if (LOAD == GLR_TMA) {
      for (int st = 0; st < ST; ++st) mbar_init(full + 8 * st, 1);
      mbar_init_fence();
    }
    for (int st = 0; st < ST; ++st) fetch(take(), st);
    next = take();
  }
  __syncthreads();

  int64_t last_piece = 0;
  int last_ch0 = 0;
  int it = 0;
  for (;; ++it) {
    const int st = it % ST;
    const Tile t = sh.tile[st];
    const int k = t.k;
    if (k < 0) break;
    const Chain chain = chain_of(a, tl, t.c.b, k, t.ch0 + cc);
    Words words;
    ask(chain, a.dp, part, words);
    const int ch = t.ch0 + 2 * lane, nch = a.d - ch;
    const int64_t piece = tl.per_seq ? (int64_t)t.c.b * tl.per_seq + t.c.k / CH : t.c.r0 / CH;
    float2 h = load2<float, false>(a.saved, piece * a.d + ch, nch);  // the state before the chunk's rows
    const int j0 = warp * PER;
    const float2 ka = *(const float2*)(a.kd + ch);
    Flags f{ALL, ALL, 0, 0};
    if (!t.inner) f = flags_of<CH, PER>(a, t.c, tl.per_seq, j0, lane);
    const bool inner = LOAD == GLR_TMA && f.V == ALL && (f.F | f.E) == 0;
    const T* sm = (const T*)(tiles + st * BYTES) + (a.reverse ? CH - 1 - j0 : j0) * 64 + 2 * lane;
    if (LOAD == GLR_TMA && !mbar_wait_bounded(full + 8 * st, (it / ST) & 1)) atomicOr(a.err_out, kErrTimeout);
    float2 da[PER], pp[PER], gi[PER], s[PER], A, H, D;
    RowPair<T> x[PER], dy[PER];
    const bool small = __all_sync(FULLM, ka.x < 0.25f && ka.y < 0.25f);
    if (inner && small) {
      const float2 root2k = make_float2(sqf(2.f * ka.x), sqf(2.f * ka.y));
      local_rows_bwd<T, LOAD, true, true, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, root2k, da, pp, gi, s, x, dy, A, H, D);
    } else if (inner) {
      local_rows_bwd<T, LOAD, false, true, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, ka, da, pp, gi, s, x, dy, A, H, D);
    } else {
      local_rows_bwd<T, LOAD, false, false, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, ka, da, pp, gi, s, x, dy, A, H, D);
    }
    const int tq = it & 1;
    sh.agg[tq][warp][lane] = f.F ? make_float4(-1.f, -1.f, H.x, H.y) : make_float4(A.x, A.y, H.x, H.y);
    sh.gga[tq][warp][lane] = f.E ? make_float4(-1.f, -1.f, D.x, D.y) : make_float4(A.x, A.y, D.x, D.y);
    // whether a sequence ends with the chunk's last row: then nothing comes from behind
    const bool need = !__syncthreads_or(warp == kWarps - 1 && (f.E >> (PER - 1) & 1)) && k > 0;
    if (tid == 0) fetch(next, st);
    if (it > 0) put_sum(tq ^ 1, last_piece, last_ch0);
    last_piece = piece;
    last_ch0 = t.ch0;
    Map tot{1.f, 0.f, false};
    if (part == 3 && k < chain.last) {
#pragma unroll
      for (int w = kWarps - 1; w >= 0; --w) tot = then(tot, get_map(sh.gga[tq][w], cc));
      publish(chain.chunk + (int64_t)k * a.dp, tot);
    }
    // the states before the warp's rows, and with them what e is of w
    for (int w = 0; w < warp; ++w) h = after(sh.agg[tq][w][lane], h);
    const float2 rk = make_float2(ka.x > 0.f ? 1.f / ka.x : 0.f, ka.y > 0.f ? 1.f / ka.y : 0.f);
    float2 osr[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const float2 xv = x[q].get(), u = mul2(pp[q], xv);
      if (!inner && (f.F >> q & 1)) h = a.h0 ? load2<float, false>(a.h0, (int64_t)seq_of(a, row_at<CH>(a, t.c, j0 + q)) * a.d + ch, nch) : two(0.f);
      Gate2 g;
      g.a = da[q];
      g.s = s[q];
      float2 sg;
      if (small) {
        sg = half_s_over_sinh<true>(g);
      } else {
        const float2 z = fma2(make_float2(-da[q].x, -da[q].y), da[q], two(1.f));  // 1 - a^2, read where s >= 1/4
        g.m = make_float2(sqf(z.x), sqf(z.y));
        sg = half_s_over_sinh<false>(g);
      }
      const float2 su = mul2(sg, u), sh_ = mul2(s[q], h);
      osr[q] = fma2(make_float2(-s[q].x, -s[q].y), rk, two(1.f));
      s[q] = mul2(da[q], add2(su, make_float2(-sh_.x, -sh_.y)));  // G
      gi[q] = fma2(make_float2(-xv.x, -xv.y), gi[q], xv);         // x (1 - sig(i))
      h = fma2(da[q], h, u);
    }
    if (need && (part >= 2 || k >= 16)) put_map(sh.before[part], cc, answer(chain, a.dp, part, words, a.err_out));
    if ((k & 15) == 15 && k < chain.last && part >= 2) {
      named_bar(1, 128);
      if (part == 3)
        publish(chain.group + (int64_t)(k >> 4) * a.dp, need ? then(then(get_map(sh.before[2], cc), get_map(sh.before[3], cc)), tot) : tot);
    }
    // a w from behind the warp's rows
    float2 v = two(0.f);
    if (need) {
      __syncthreads();
      if (k >= 16) v = after(sh.before[1][lane], after(sh.before[0][lane], v));
      v = after(sh.before[3][lane], after(sh.before[2][lane], v));
    }
    if ((k & 255) == 255 && k < chain.last && part == 3) {
      const float2 c2 = make_float2(__shfl_sync(FULLM, v.x, cc >> 1), __shfl_sync(FULLM, v.y, cc >> 1));
      const float in = cc & 1 ? c2.y : c2.x;
      publish(chain.large + (int64_t)(k >> 8) * a.dp, Map{0.f, tot.reset ? tot.H : fmaf(tot.A, in, tot.H), true});
    }
    for (int w = kWarps - 1; w > warp; --w) v = after(sh.gga[tq][w][lane], v);
    // the gradients, from the last row on
    float2 dl = two(0.f);
    const int64_t step = a.reverse ? a.ldd : -a.ldd;
    int64_t o = row_at<CH>(a, t.c, j0 + PER - 1) * a.ldd + ch;
#pragma unroll
    for (int q = PER - 1; q >= 0; --q, o += step) {
      if (!inner && (f.E >> q & 1)) v = a.dhT ? load2<float, false>(a.dhT, (int64_t)seq_of(a, row_at<CH>(a, t.c, j0 + q)) * a.d + ch, nch) : two(0.f);
      const float2 w = add2(dy[q].get(), v);
      v = mul2(da[q], w);
      float2 dx = mul2(w, pp[q]), di = mul2(dx, gi[q]), e = mul2(w, s[q]), dr = mul2(e, osr[q]);
      if (inner) {
        dl = add2(dl, e);
        if (nch > 0) {
          store2<T, true>(a.dx, o, 2, dx);
          store2<T, true>(a.dr, o, 2, dr);
          store2<T, true>(a.di, o, 2, di);
        }
      } else {
        const bool ok = f.V >> q & 1;
        const int n = f.in >> q & 1 ? nch : 0;
        if (ok) dl = add2(dl, e);
        store2<T, LOAD != GLR_SINGLE>(a.dx, o, n, ok ? dx : two(0.f));
        store2<T, LOAD != GLR_SINGLE>(a.dr, o, n, ok ? dr : two(0.f));
        store2<T, LOAD != GLR_SINGLE>(a.di, o, n, ok ? di : two(0.f));
        if (a.dh0 && (f.F >> q & 1)) store2<float, false>(a.dh0, (int64_t)seq_of(a, row_at<CH>(a, t.c, j0 + q)) * a.d + ch, nch, v);
        if (!ok) v = dy[q].get();  // (0: a row of no sequence hands nothing on, whatever entered)
      }
    }
    sh.sum[tq][warp][lane] = dl;
    if (tid == 0 && next.k >= 0) next = take();
  }
  __syncthreads();
  if (it > 0) put_sum((it - 1) & 1, last_piece, last_ch0);
}

// dlam's partial rows n0 = blockIdx.y, n0 + gridDim.y, .. of 64 channels, summed in order, times the derivative of softplus over it.
__global__ void __launch_bounds__(256) k_glr_dlam(const float* part, int64_t n, int d, const float* lam, float* out) {
  pdl_enter();
  __shared__ float red[4][64];
  const int ch = blockIdx.x * 64 + (threadIdx.x & 63), p = threadIdx.x >> 6;
  float v = 0.f;
  if (ch < d) {
    const int64_t step = (int64_t)gridDim.y * 4;
#pragma unroll 8
    for (int64_t i = blockIdx.y * 4 + p; i < n; i += step) v += part[i * d + ch];
  }
  red[p][threadIdx.x & 63] = v;
  __syncthreads();
  if (p == 0 && ch < d)
    out[(int64_t)blockIdx.y * d + ch] = (((red[0][threadIdx.x] + red[1][threadIdx.x]) + red[2][threadIdx.x]) + red[3][threadIdx.x]) * dsoftplus_ratio(lam[ch]);
}

// c softplus(lam), the scan's words and the tile counter cleared; checks the sequence data and, for packed sequences,
// marks the rows that begin one (the error word and the marks are 0 on entry).
__global__ void __launch_bounds__(256) k_glr_prep(const GlrArgs a, int64_t words, int* err) {
  pdl_enter();
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)gridDim.x * 256;
  if (id == 0) {
    *a.ticket = 0;
    if (a.seq.mode == SEQ_DENSE) *err = 0;
  }
  for (int64_t i = id; i < a.dp; i += n) a.kd[i] = i < a.d ? a.c * softplus_f(a.lam[i]) : 0.f;
  for (int64_t i = id; i < words / 2; i += n) ((ulonglong2*)a.words)[i] = make_ulonglong2(0, 0);
  if (a.seq.mode == SEQ_DENSE) return;
  for (int64_t b = id; b < a.seq.n_seq; b += n) {
    if (a.seq.mode == SEQ_PADDED) {
      if (a.seq.lens[b] < 0 || a.seq.lens[b] > a.seq.L) atomicOr(err, 1);
      continue;
    }
    const int lo = a.seq.cu[b], hi = a.seq.cu[b + 1];
    if (lo < 0 || hi < lo || hi > a.seq.T || (b == 0 && lo != 0) || (b == a.seq.n_seq - 1 && hi != a.seq.T)) {
      atomicOr(err, 1);
      continue;
    }
    if (lo < hi) atomicOr((unsigned long long*)a.marks + (lo >> 6), 1ull << (lo & 63));
  }
}

// A sequence without tokens hands its state on.
__global__ void __launch_bounds__(256) k_glr_empty(const GlrArgs a, const float* from, float* to) {
  if (a.err && *a.err) return;
  for (int b = blockIdx.x; b < a.seq.n_seq; b += gridDim.x) {
    const int n = a.seq.mode == SEQ_VARLEN ? a.seq.cu[b + 1] - a.seq.cu[b] : a.seq.lens[b];
    if (n == 0)
      for (int ch = threadIdx.x; ch < a.d; ch += 256) to[(int64_t)b * a.d + ch] = from ? from[(int64_t)b * a.d + ch] : 0.f;
  }
}

}  // namespace

namespace {
// Pairs of channels are whole and aligned.
bool pairs_ok(const GlrArgs& a, size_t es) {
  uintptr_t bad = (uintptr_t)(a.d & 1) | (uintptr_t)(a.ld & 1) | (uintptr_t)(a.ldd & 1);
  for (const void* p : {a.x, a.r, a.i, (const void*)a.y, a.dy, (const void*)a.dx, (const void*)a.dr, (const void*)a.di})
    bad |= reinterpret_cast<uintptr_t>(p) & (2 * es - 1);
  return bad == 0;
}
}  // namespace

cudaError_t launch_glr_prep(const GlrArgs& a, int64_t words, int* err, cudaStream_t st) {
  const int64_t n = std::max<int64_t>(std::max<int64_t>(words / 2, a.dp), a.seq.mode == SEQ_DENSE ? 1 : a.seq.n_seq);
  const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)sm_count() * 8);
  return launch_pdl(k_glr_prep, dim3(grid), dim3(256), 0, st, a, words, err);
}
cudaError_t launch_glr_empty(const GlrArgs& a, const float* from, float* to, cudaStream_t st) {
  k_glr_empty<<<(unsigned)std::min(a.seq.n_seq, 4096), 256, 0, st>>>(a, from, to);
  return cudaGetLastError();
}

namespace {
// A map of [rows][d] with row stride ld, its box 64 channels of `box` rows; false where TMA does not take it.
bool rows_map(CUtensorMap* m, const void* p, bool f32, int d, int64_t T, int64_t ld, int box) {
  const size_t es = f32 ? 4 : 2;
  auto enc = encoder();
  if (!enc || reinterpret_cast<uintptr_t>(p) % 16 || ld * es % 16 || (size_t)d * es % 16 || ld * es >= (1ull << 40)) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)T}, strides[1] = {(cuuint64_t)(ld * es)};
  cuuint32_t boxes[2] = {64, (cuuint32_t)box}, es1[2] = {1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides,
             boxes, es1, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
cudaError_t run_glr_fwd(const GlrArgs& a, const GlrTiles& t, cudaStream_t st) {
  constexpr bool f32 = sizeof(T) == 4;
  GlrMaps maps{};
  const bool tma = reinterpret_cast<uintptr_t>(a.y) % (2 * sizeof(T)) == 0 &&
                   rows_map(&maps.m[0], a.x, f32, a.d, a.seq.T, a.ld, kGlrRowsFwd) &&
                   rows_map(&maps.m[1], a.r, f32, a.d, a.seq.T, a.ld, kGlrRowsFwd) &&
                   rows_map(&maps.m[2], a.i, f32, a.d, a.seq.T, a.ld, kGlrRowsFwd);
  const size_t smem = 128 + sizeof(GlrShared) + (tma ? stages_fwd<T>() * (size_t)3 * kGlrRowsFwd * 64 * sizeof(T) : 0);
  const dim3 grid((unsigned)std::min<int64_t>((int64_t)t.n_chunks * (a.dp >> 6), (int64_t)sm_count() * kCtasFwd));
  auto kernel = tma ? k_glr_fwd<T, GLR_TMA> : pairs_ok(a, sizeof(T)) ? k_glr_fwd<T, GLR_PAIRS> : k_glr_fwd<T, GLR_SINGLE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(kThreads), smem, st, a, t, maps);
}
}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, const GlrTiles& t, bool f32, cudaStream_t st) {
  return f32 ? run_glr_fwd<float>(a, t, st) : run_glr_fwd<bf16>(a, t, st);
}

namespace {
template <typename T>
cudaError_t run_glr_bwd(const GlrArgs& a, const GlrTiles& t, cudaStream_t st) {
  constexpr bool f32 = sizeof(T) == 4;
  GlrMaps4 maps{};
  const bool tma = pairs_ok(a, sizeof(T)) && rows_map(&maps.m[0], a.x, f32, a.d, a.seq.T, a.ld, kGlrChunk) &&
                   rows_map(&maps.m[1], a.r, f32, a.d, a.seq.T, a.ld, kGlrChunk) &&
                   rows_map(&maps.m[2], a.i, f32, a.d, a.seq.T, a.ld, kGlrChunk) &&
                   rows_map(&maps.m[3], a.dy, f32, a.d, a.seq.T, a.d, kGlrChunk);
  const size_t smem = 128 + sizeof(GlrSharedBwd) + (tma ? stages_bwd<T>() * (size_t)4 * kGlrChunk * 64 * sizeof(T) : 0);
  const dim3 grid((unsigned)std::min<int64_t>((int64_t)t.n_chunks * (a.dp >> 6), (int64_t)sm_count() * kCtasBwd));
  auto kernel = tma ? k_glr_bwd<T, GLR_TMA> : pairs_ok(a, sizeof(T)) ? k_glr_bwd<T, GLR_PAIRS> : k_glr_bwd<T, GLR_SINGLE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(kThreads), smem, st, a, t, maps);
}
}  // namespace

cudaError_t launch_glr_bwd(const GlrArgs& a, const GlrTiles& t, bool f32, cudaStream_t st) {
  return f32 ? run_glr_bwd<float>(a, t, st) : run_glr_bwd<bf16>(a, t, st);
}

cudaError_t launch_glr_dlam(const GlrArgs& a, int64_t n, int rows, float* out, cudaStream_t st) {
  return launch_pdl(k_glr_dlam, dim3((unsigned)(a.dp >> 6), (unsigned)rows), dim3(256), 0, st, (const float*)a.dlam_part, n, a.d, a.lam, out);
}

}  // namespace gbla
