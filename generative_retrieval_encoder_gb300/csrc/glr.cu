// Gated linear recurrence with a decay per token and channel:
//   s_t = c softplus(lam) sigmoid(r_t),  a_t = exp(-s_t),  q_t = 1 - a_t,
//   m_t = sqrt(1 - a_t^2) = sqrt(q_t (2 - q_t)),
//   h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t,  y_t = h_t,
// per sequence and channel in either direction, and its backward
//   w_t = dy_t + a_{t+1} w_{t+1}          (w = dL/dh, + dhT at the last token)
//   dx = w m sig(i),  di = w m x sig(i) (1 - sig(i)),
//   e_t = s_t dL/ds_t = -w a (s h_{t-1} - u s / (2 sinh s)),  u = m sig(i) x,
//   dr = e (1 - sig(r)),  dlam = sum_t e_t sig(lam) / softplus(lam),  dh0 = a w at the first token.
// (dL/ds = -a w (h_{t-1} - (a / m) sig(i) x), and a^2 s / m^2 = a s / (2 sinh s).)  q is formed without cancellation (a
// polynomial for small s), so m keeps its relative accuracy for decays near 1; s / (2 sinh s) is 1/2 at s = 0, so dr
// and dlam stay finite where a = 1.  States, decays and sums are fp32; y and the gradients are rounded once.
//
// What a call cannot do without (bf16): forward 8 bytes a value, backward 14; and four special functions a value and
// direction, which at 6.8 TB/s take half the special function units' time.  The scan runs along the rows, so the rows are
// cut: tiles of 128 (forward) or 64 rows x 64 channels, whose effects on a state are composed across tiles while the rows'
// values stay on the chip (scan_* below): every input is read once.  Measured (whole calls back to back, launches included):
//   forward  B = 32, L = 2048, d = 512 (268 MB)   65 us, 4.1 TB/s (72 with L2 flushed before each);
//            B = 8, L = 32768 (1.07 GB)  257 us, 4.2 TB/s
//            one sequence of 65536 rows (268 MB)  98 us, 2.7 TB/s; packed, d = 1024 (1.35 GB)  350 us, 3.9 TB/s
//   forward and backward  B = 16, L = 8192 (1.48 GB)  424 us, 3.5 TB/s; packed, d = 1024 (2.67 GB)  741 us, 3.6 TB/s
// Without the waits between tiles (a copy that left them out) the forward takes 61, 200, 59 and 284 us, and without the
// gates too 47, 162, 46 and 218: what is left above the copy is first the gates' instructions, then the tiles of one chain
// that are worked on at the same time and so wait for one another, most where one sequence has few channels.
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
// The rows are cut into chunks (GlrCut); a chunk and 64 channels are a tile, a tile is one CTA's, and a warp has PER neighbouring rows of it.  A chunk's rows
// are numbered in the direction of the recurrence.
struct Span {
  int64_t r0;       // physical first row of the chunk
  int nr;           // its rows
  int b;            // its slot or sequence (where those are cut by themselves)
  int k;            // its first row in that
  int len;          // that one's valid rows
};
template <int CH>
__device__ __forceinline__ int64_t row_at(const GlrArgs& a, const Span& c, int j) {
  return a.reverse ? c.r0 + CH - 1 - j : c.r0 + j;
}
// Bits of the N <= 32 rows from j0 on: in the chunk, in a sequence, a sequence's first, its last (in the direction of the
// recurrence).  Whole warps call it.
struct Flags { uint32_t in, V, F, E; };
template <int CH, int N>
__device__ __forceinline__ Flags flags_of(const GlrArgs& a, const Span& c, int cut, int j0, int lane) {
  const int j = j0 + min(lane, N - 1), p = a.reverse ? CH - 1 - j : j;  // place in the chunk
  const bool in = p < c.nr;
  bool v = in, s, z;
  const int64_t row = c.r0 + p;
  if (cut == GLR_STREAM && a.seq.mode == SEQ_VARLEN) {
    s = in && (a.marks[row >> 6] >> (row & 63) & 1);
    z = in && (row + 1 == a.seq.T || (a.marks[(row + 1) >> 6] >> ((row + 1) & 63) & 1));
  } else {
    int pos = c.k + p, len = c.len;
    if (cut == GLR_STREAM) {
      const int b = (int)row / a.seq.L;
      pos = (int)row - b * a.seq.L;
      len = a.seq.mode == SEQ_PADDED ? (in ? a.seq.lens[b] : 0) : a.seq.L;
    }
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
__device__ __forceinline__ int seq_of(const GlrArgs& a, int64_t row) {  // (rows that begin or end one only: few)
  if (a.seq.mode != SEQ_VARLEN) return (int)(row / a.seq.L);
  int lo = 0, hi = a.seq.n_seq - 1;  // the last b with cu[b] <= row: it is not empty
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.seq.cu[mid] <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------ tiles
constexpr int kWarpsF = 8, kWarpsB = 8;                                       // of a CTA, forward and backward
constexpr int kPerF = kGlrRowsFwd / kWarpsF, kPerB = kGlrRowsBwd / kWarpsB;     // a warp's rows; a lane has two channels of each
constexpr int kCtasFwd = 2, kCtasBwd = 3;                                     // an SM's

// How a tile's rows are read: copied ahead into shared memory (rows of 16-byte pieces), or straight into registers by
// pairs of channels or single ones.
enum GlrLoad { GLR_TMA = 0, GLR_PAIRS = 1, GLR_SINGLE = 2 };

// A tile: channels from ch0, the chunk's rows, its place k in its chain (-1: no tile) of last + 1, and where the chain's words
// for it, its saved states and its partial row of dlam are.
struct Tile {
  int ch0, k, last;
  int inner;        // every row is inside one sequence and neither its first nor its last
  Span c;
  int64_t own, near, far, large;  // the chunk's word; its group's first; the one before its larger group's first; the larger group before
  int64_t piece, row;
};
__device__ __forceinline__ unsigned quotient(unsigned n, GlrDiv d) {  // n / divisor (Granlund and Montgomery's method)
  const unsigned t = __umulhi(n, d.m);
  return d.s < 0 ? n : (t + ((n - t) >> 1)) >> d.s;
}
// What of tile t has to be asked of memory.
template <int CH>
__device__ __forceinline__ int4 asked_of(const GlrArgs& a, const GlrTiles& g, unsigned t, bool back) {
  const unsigned w = quotient(t, g.by_cg);
  int4 e = make_int4(0, a.seq.L, 0, 0);
  if (g.cut == GLR_SEQS) e = g.order[w];
  if (g.cut == GLR_SLOTS && a.seq.mode == SEQ_PADDED) e.y = a.seq.lens[w - quotient(w, g.by_seq) * (unsigned)a.seq.n_seq];
  if (g.cut == GLR_STREAM && a.seq.mode == SEQ_VARLEN) {  // whether rows of the chunk, or the one behind, begin a sequence
    const int64_t r0 = (int64_t)(back ? g.n_chunks - 1 - (int)w : (int)w) * CH;
    uint64_t m = 1;
    if (r0 + CH < a.seq.T) {
      m = a.marks[(r0 + CH) >> 6] & 1;
#pragma unroll
      for (int j = 0; j < CH / 64; ++j) m |= a.marks[(r0 >> 6) + j];
    }
    e.x = (int)(uint32_t)m;
    e.y = (int)(uint32_t)(m >> 32);
  }
  return e;
}
// Tile t of the call's with that; back: the chain runs from the last chunk.
template <int CH>
__device__ __forceinline__ void tile_of(const GlrArgs& a, const GlrTiles& g, unsigned t, bool back, const int4& e, Tile& o) {
  const unsigned w = quotient(t, g.by_cg);
  o.ch0 = (int)(t - w * (unsigned)(a.dp >> 6)) * 64;
  int row0 = 0, s = 0, n = g.n_chunks, k = (int)w, rows = a.seq.T;
  if (g.cut == GLR_SLOTS) {
    const unsigned q = quotient(w, g.by_seq);
    s = (int)(w - q * (unsigned)a.seq.n_seq);
    k = (int)q;
    n = g.per_seq;
    row0 = s * a.seq.L;
    rows = a.seq.L;
  } else if (g.cut == GLR_SEQS) {
    row0 = e.x;
    s = e.z;
    k = e.w;
    rows = e.y;
    n = (rows + CH - 1) / CH;
  }
  const int c = back ? n - 1 - k : k;
  o.k = k;
  o.last = n - 1;
  o.c.b = s;
  o.c.k = c * CH;
  o.c.r0 = (int64_t)row0 + o.c.k;
  o.c.nr = min(CH, rows - o.c.k);
  o.c.len = e.y;
  o.inner = g.cut == GLR_STREAM ? a.seq.mode == SEQ_VARLEN && (e.x | e.y) == 0 : o.c.k > 0 && o.c.k + CH < e.y;
  // words of chunks, of groups of 16, of 16 groups: those of a chain in a row, in its order
  const int64_t chunk = row0 / CH + s, group = (int64_t)g.n_words + row0 / (16 * CH) + s, large = (int64_t)g.n_words + g.n_groups + row0 / (256 * CH) + s;
  o.own = (chunk + k) * a.dp + o.ch0;
  o.near = (chunk + (k & ~15)) * a.dp + o.ch0;
  o.far = (group + (k >> 8 << 4) - 1) * a.dp + o.ch0;
  o.large = (large + (k >> 8) - 1) * a.dp + o.ch0;
  o.piece = (g.cut == GLR_SLOTS ? (int64_t)s * a.pieces : row0 / kGlrPiece + s) + o.c.k / kGlrPiece;
  o.row = g.cut == GLR_SLOTS ? (int64_t)s * n + c : row0 / CH + s + c;
}

// ------------------------------------------------------------ the scan between chunks
// A tile publishes, per channel, what its rows do to a state that enters: h -> A h + H, as one 64-bit word {H, A}
// (present when the top bit, A's sign, is set: one word, so nothing else has to be ordered).  A = 0: a sequence starts here, h -> H
// whatever h was.  A product of decays is never 0: one below the fp32 range counts as its smallest value, 2^-149, so that a state
// that is NaN or infinite stays so to its sequence's end (and a finite one adds 2^-149 of itself at most).  Chunks form
// groups of 16 and groups of groups; a chunk that needs the state before it composes the words of the chunks before it in
// its group, of the groups before its own in the larger group, and the state after the last larger group: at most 31
// words, read together.  The order of composition is fixed, so results do not depend on timing.
// Tiles are handed out by a counter in an order in which everything a tile waits for has been handed out before:
// the earliest unfinished tile waits for nothing unfinished, so every wait ends (and is bounded all the same).
struct Map { float A, H; };
struct Map2 { float2 A, H; };  // of a lane's two channels
constexpr uint64_t kIdentity = 0xBF80000000000000ull;  // h -> 1 h + 0
__device__ __forceinline__ uint64_t word_of(float A, float H) {
  uint32_t a;  // (written as C++ this comes out as the float -|A|, which loses a NaN's sign: the word would never be there)
  asm("or.b32 %0, %1, 0x80000000;" : "=r"(a) : "r"(__float_as_uint(A)));
  return (uint64_t)a << 32 | __float_as_uint(H);
}
constexpr float kTiny = 0x1p-149f;
// The product p of decays, the least of them low: 0 where one of them is, and only there.
__device__ __forceinline__ float product(float p, float low) { return fmaxf(p, fminf(low, kTiny)); }
__device__ __forceinline__ float2 product(float2 p, float2 low) { return make_float2(product(p.x, low.x), product(p.y, low.y)); }
__device__ __forceinline__ float2 least(float2 a, float2 b) { return make_float2(fminf(a.x, b.x), fminf(a.y, b.y)); }
__device__ __forceinline__ float2 after(const Map2& n, float2 h) {
  const float2 o = fma2(n.A, h, n.H);
  return make_float2(n.A.x == 0.f ? n.H.x : o.x, n.A.y == 0.f ? n.H.y : o.y);
}
// First m, then n.
__device__ __forceinline__ Map2 then(const Map2& m, const Map2& n) { return Map2{product(mul2(m.A, n.A), least(m.A, n.A)), after(n, m.H)}; }
// What a warp's rows do, A the product of their decays; start: nothing from before them gets through.  A NaN decay (it has made H
// NaN) counts as 2^-149 too: no A is NaN then, so a start ends what is before it.  (fmaxf takes the number of a NaN and a number.)
__device__ __forceinline__ Map2 map_of(float2 A, float2 H, bool start) {
  return Map2{start ? two(0.f) : make_float2(fmaxf(A.x, kTiny), fmaxf(A.y, kTiny)), H};
}
// In shared memory: {A, A, H, H} of a lane's two channels.
__device__ __forceinline__ Map2 map_at(const float4& g) { return Map2{make_float2(g.x, g.y), make_float2(g.z, g.w)}; }
__device__ __forceinline__ float4 packed(const Map2& m) { return make_float4(m.A.x, m.A.y, m.H.x, m.H.y); }
__device__ __forceinline__ void publish(uint64_t* p, const Map2& m) {
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(word_of(m.A.x, m.H.x)), "l"(word_of(m.A.y, m.H.y)) : "memory");
}
// x, or where `is` the word at p (a predicated load: no branch).
__device__ __forceinline__ uint64_t peek(const uint64_t* p, bool is, uint64_t x) {
  asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %2, 0;\n @q ld.relaxed.gpu.global.b64 %0, [%1];\n}" : "+l"(x) : "l"(p), "r"((uint32_t)is) : "memory");
  return x;
}

// The 31 words that a chunk reads, from the oldest on (the larger group's, 15 groups', 15 chunks'), in W / 2 parts for the W
// warps of a CTA, a thread of each part for every channel: ask() asks for a thread's at once, before they are needed;
// answer() waits for those that were not there yet, again together, and composes them.  Words that do not exist are
// identities.
template <int W> struct Words { uint64_t w[64 / W]; };
// Whether chunk k has words of this part at all.
template <int W>
__device__ __forceinline__ bool part_is(int k, int part) {
  constexpr int N = 64 / W, FAR = W / 4;
  return part >= FAR ? (k & 15) > (part - FAR) * N : k >= 16 && (part == 0 || (k >> 4 & 15) >= part * N);
}
template <int W>
__device__ __forceinline__ uint64_t peek_word(const GlrArgs& a, const Tile& t, int part, int cc, int j, bool want, uint64_t x) {
  constexpr int N = 64 / W, FAR = W / 4;  // words of a part; the parts of groups
  const int lim = part >= FAR ? (t.k & 15) - (part - FAR) * N : (t.k >> 4 & 15) + 1 - part * N;
  int64_t at = (part >= FAR ? t.near + (part - FAR) * N * a.dp : t.far + part * N * a.dp) + j * a.dp;
  bool is = j < lim;
  if (j == 0 && part == 0) {
    at = t.large;
    is = t.k >= 256;
  }
  return peek(a.words + at + cc, is && want, x);
}
template <int W>
__device__ __forceinline__ void ask(const GlrArgs& a, const Tile& t, int part, int cc, Words<W>& v) {
  if (!part_is<W>(t.k, part)) return;
#pragma unroll
  for (int j = 0; j < 64 / W; ++j) v.w[j] = peek_word<W>(a, t, part, cc, j, true, kIdentity);
}
// Whether to go on asking after n vain tries: bounded, and given up at once where another wait has been.
__device__ __forceinline__ bool patient(int n, int* err) {
  if ((n & 255) != 255) return true;
  if (*(volatile int*)err & kErrTimeout) return false;
  if (n < (1 << 22)) return true;
  atomicOr(err, kErrTimeout);
  return false;
}
template <int W>
__device__ __forceinline__ Map answer(const GlrArgs& a, const Tile& t, int part, int cc, Words<W>& v) {
  for (int n = 0;; ++n) {
    uint64_t there = v.w[0];
#pragma unroll
    for (int j = 1; j < 64 / W; ++j) there &= v.w[j];
    if (there >> 63 || !patient(n, a.err_out)) break;
#pragma unroll
    for (int j = 0; j < 64 / W; ++j) v.w[j] = peek_word<W>(a, t, part, cc, j, !(v.w[j] >> 63), v.w[j]);
  }
  Map m{1.f, 0.f};
  float low = 1.f;
#pragma unroll
  for (int j = 0; j < 64 / W; ++j) {  // one after the other
    const float A = __uint_as_float((uint32_t)(v.w[j] >> 32) & 0x7fffffffu), H = __uint_as_float((uint32_t)v.w[j]);
    m = Map{m.A * A, A == 0.f ? H : fmaf(A, m.H, H)};
    low = fminf(low, A);
  }
  return Map{product(m.A, low), m.H};
}

// Shared memory of the scan: what the rows of each warp (in the chain's order) do; the parts of the words.
template <int W> struct ScanShared {
  float4 agg[W][32];
  float4 before[W / 2][32];
};
// After the warps' maps are in sc.agg: what those before warp vw do, composed; the last warp publishes the tile's word.
template <int W>
__device__ __forceinline__ Map2 scan_local(const GlrArgs& a, const Tile& t, const ScanShared<W>& sc, int vw, int lane, Map2& total) {
  Map2 m{two(1.f), two(0.f)};
  float2 low = two(1.f);
  if (t.inner) {  // no start among the rows
    for (int w = 0; w < vw; ++w) {
      const Map2 n = map_at(sc.agg[w][lane]);
      m = Map2{mul2(m.A, n.A), fma2(n.A, m.H, n.H)};
    }
  } else {
    for (int w = 0; w < vw; ++w) {
      const Map2 n = map_at(sc.agg[w][lane]);
      m = Map2{mul2(m.A, n.A), after(n, m.H)};
      low = least(low, n.A);
    }
  }
  m.A = product(m.A, low);
  if (vw == W - 1) {
    total = then(m, map_at(sc.agg[vw][lane]));
    if (t.k < t.last) publish(a.words + t.own + 2 * lane, total);
  }
  return m;
}
// This thread's part of the words into sc.before; a full group's word published (it takes no other group's: it does not wait
// for the parts of those).
template <int W>
__device__ __forceinline__ void scan_words(const GlrArgs& a, const Tile& t, ScanShared<W>& sc, int vw, int lane, bool need, Words<W>& words, const Map2& total) {
  constexpr int P = W / 2, FAR = W / 4;
  const int part = vw >> 1, cc = (vw & 1) * 32 + lane;
  if (need && part_is<W>(t.k, part)) {
    const Map m = answer<W>(a, t, part, cc, words);
    float* p = (float*)&sc.before[part][cc >> 1] + (cc & 1);
    p[0] = m.A;
    p[2] = m.H;
  }
  if ((t.k & 15) == 15 && t.k < t.last && part >= FAR) {
    named_bar(1, W * 16);
    if (vw == W - 1) {
      Map2 m = total;
      if (need) {
#pragma unroll
        for (int q = P - 1; q >= FAR; --q)
          if (part_is<W>(t.k, q)) m = then(map_at(sc.before[q][lane]), m);
      }
      publish(a.words + t.far + (int64_t)((t.k >> 4 & 15) + 1) * a.dp + 2 * lane, m);
    }
  }
}
// The state that enters the tile.  Whole CTAs call it (need is the same for all).
template <int W>
__device__ __forceinline__ float2 scan_state(const GlrArgs& a, const Tile& t, const ScanShared<W>& sc, int vw, int lane, bool need, const Map2& total) {
  float2 h = two(0.f);
  __syncthreads();
  if (need) {
#pragma unroll
    for (int q = 0; q < W / 2; ++q)
      if (part_is<W>(t.k, q)) h = after(map_at(sc.before[q][lane]), h);
  }
  if ((t.k & 255) == 255 && t.k < t.last && vw == W - 1)
    publish(a.words + t.large + a.dp + 2 * lane, Map2{two(0.f), after(total, h)});
  return h;
}

// Thread 0's side of a CTA's tiles: the ticket of a tile is drawn as soon as the one before is fetched, what it needs from
// memory asked for a good while later, and looked at later still, so that no step waits.
struct Drawn { unsigned t; int4 e; };

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

// Shared memory of a CTA of the forward, after its tiles of x, r and i.
struct GlrShared {
  ScanShared<kWarpsF> sc;
  Tile tile[4];                // the CTA's n-th at n & 3
  uint64_t full[2];
};

// Forward: one pass, x, r and i read once and y written once.  Bound by the instructions of the gates (four special
// functions and 36 instructions a value in all; 42 % of the issue slots), by the waits between tiles and by memory.  Two CTAs
// an SM keep taking tiles, so that one's wait for the state between tiles is another's arithmetic; a tile's rows are copied
// to shared memory while an earlier one is worked on.  A lane holds a and u of its 16 rows between the two halves of a tile: 64
// registers, hence two CTAs.  Other shapes (B = 8, L = 32768): 64-row tiles 365 us with three CTAs of 8 x 8 rows, 466 with four
// of 4 x 16 (the composition costs the same for half the rows); one CTA of 16 x 16 rows 250, but 71 against 65 us at L = 2048;
// forming the decays twice to hold u alone, three CTAs, 324.
template <typename T, int LOAD>
__global__ void __launch_bounds__(kWarpsF * 32, kCtasFwd) k_glr_fwd(const GlrArgs a, const GlrTiles tl, const __grid_constant__ GlrMaps maps) {
  constexpr int PER = kPerF, CH = kGlrRowsFwd, ST = stages_fwd<T>();
  constexpr uint32_t BYTES = 3 * CH * 64 * sizeof(T), ALL = (1u << PER) - 1;
  extern __shared__ __align__(128) uint8_t raw[];
  pdl_enter();
  if (a.err && *a.err) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* tiles = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
  GlrShared& sh = *reinterpret_cast<GlrShared*>(tiles + (LOAD == GLR_TMA ? ST * BYTES : 0));
  const uint32_t full = smem_u32(sh.full);
  const unsigned total = (unsigned)(tl.cut == GLR_SEQS ? *tl.n_order : tl.n_chunks) * (unsigned)(a.dp >> 6);

  // thread 0: the CTA's n-th tile
  auto fetch = [&](const Drawn& d, int n) {
    Tile& o = sh.tile[n & 3];
    o.k = -1;
    if (d.t >= total) return;
    tile_of<CH>(a, tl, d.t, a.reverse, d.e, o);
    if (LOAD == GLR_TMA) {
      const int st = n % ST;
      mbar_expect_tx(full + 8 * st, BYTES);
#pragma unroll
      for (int m = 0; m < 3; ++m)
        tma_load_2d(smem_u32(tiles) + st * BYTES + m * (BYTES / 3), &maps.m[m], full + 8 * st, o.ch0, (int)o.c.r0);
    }
  };
  Drawn next;
  if (tid == 0) {
    if (LOAD == GLR_TMA) {
      for (int st = 0; st < ST; ++st) mbar_init(full + 8 * st, 1);
      mbar_init_fence();
    }
    for (int n = 0; n <= ST; ++n) {
      next.t = (unsigned)atomicAdd(a.ticket, 1ull);
      if (next.t < total) next.e = asked_of<CH>(a, tl, next.t, a.reverse);
      if (n < ST) fetch(next, n);
    }
  }
  __syncthreads();

  for (int it = 0;; ++it) {
    const int st = it % ST;
    const Tile& me = sh.tile[it & 3];
    if (me.k < 0) break;
    Words<kWarpsF> words;
    ask(a, me, warp >> 1, (warp & 1) * 32 + lane, words);
    // the lane's rows
    const int ch = me.ch0 + 2 * lane, nch = a.d - ch;  // channels of this lane: 2 (or more), 1 or none
    const int j0 = warp * PER;
    const float2 ka = *(const float2*)(a.kd + ch);
    Flags f{ALL, ALL, 0, 0};
    if (!me.inner) f = flags_of<CH, PER>(a, me.c, tl.cut, j0, lane);
    const bool inner = LOAD == GLR_TMA && f.V == ALL && f.F == 0;
    const T* sm = (const T*)(tiles + st * BYTES) + (a.reverse ? CH - 1 - j0 : j0) * 64 + 2 * lane;
    if (LOAD == GLR_TMA && !mbar_wait_bounded(full + 8 * st, (it / ST) & 1)) atomicOr(a.err_out, kErrTimeout);
    float2 da[PER], u[PER], A, H;
    if (inner && __all_sync(FULLM, ka.x < 0.25f && ka.y < 0.25f)) {
      const float2 root2k = make_float2(sqf(2.f * ka.x), sqf(2.f * ka.y));
      local_rows<T, LOAD, true, true, PER, CH>(a, sm, me.c, f, j0, ch, nch, ka, root2k, da, u, A, H);
    } else if (inner) {
      local_rows<T, LOAD, false, true, PER, CH>(a, sm, me.c, f, j0, ch, nch, ka, ka, da, u, A, H);
    } else {
      local_rows<T, LOAD, false, false, PER, CH>(a, sm, me.c, f, j0, ch, nch, ka, ka, da, u, A, H);
    }
    sh.sc.agg[warp][lane] = packed(map_of(A, H, f.F != 0));
    // whether the chunk's first row begins a sequence: then nothing enters
    const bool need = !__syncthreads_or(warp == 0 && (f.F & 1)) && me.k > 0;
    if (tid == 0) {
      fetch(next, it + ST);
      if (next.t < total) next.t = (unsigned)atomicAdd(a.ticket, 1ull);
    }
    Map2 tot;
    const Map2 pre = scan_local(a, me, sh.sc, warp, lane, tot);
    scan_words(a, me, sh.sc, warp, lane, need, words, tot);
    float2 h = after(pre, scan_state(a, me, sh.sc, warp, lane, need, tot));
    // the rows again, from the state that enters them; every kGlrPiece rows it is saved
    static_assert(PER % kGlrPiece == 0, "a warp's rows are whole pieces");
    auto save = [&](int p) {  // before the warp's row p
      const int at = a.reverse ? CH - kGlrPiece - j0 - p : j0 + p;  // physical place of the piece in the chunk
      if (at < me.c.nr) store2<float, false>(a.saved, (me.piece + at / kGlrPiece) * a.d + ch, nch, h);
    };
    const int64_t step = a.reverse ? -a.d : a.d;
    int64_t o = row_at<CH>(a, me.c, j0) * a.d + ch;
    if (inner && (!a.hT || f.E == 0)) {
      if (nch > 0) {
        T* y = (T*)a.y + o;
#pragma unroll
        for (int p = 0; p < PER; ++p, y += step) {
          if (p % kGlrPiece == 0 && a.saved) save(p);
          h = fma2(da[p], h, u[p]);
          store2<T, true>(y, 0, 2, h);
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < PER; ++p, o += step) {
        if (p % kGlrPiece == 0 && a.saved) save(p);
        if (f.F >> p & 1) h = u[p];
        else h = fma2(da[p], h, u[p]);
        store2<T, LOAD != GLR_SINGLE>(a.y, o, f.in >> p & 1 ? nch : 0, f.V >> p & 1 ? h : two(0.f));
        if (a.hT && (f.E >> p & 1)) store2<float, false>(a.hT, (int64_t)seq_of(a, row_at<CH>(a, me.c, j0 + p)) * a.d + ch, nch, h);
      }
    }
    if (tid == 0 && next.t < total) next.e = asked_of<CH>(a, tl, next.t, a.reverse);
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

constexpr int kStagesBwd = 2;

// The backward goes over a tile's rows twice (they stay in shared memory): first for the decays, which with dy are all that
// the scan of w takes, then, with w known, for everything else.  Held in between: a, and dy, whose place w takes.

// The lane's rows, what they do together to a w from behind: w -> A w + D (an end in them: D alone).  sm: the lane's first row of
// x in shared memory, r, i and dy one, two and three tiles on.
template <typename T, int LOAD, bool SMALL, bool PLAIN, int PER, int CH>
__device__ __forceinline__ void decays_bwd(const GlrArgs& a, const T* sm, const Span& c, const Flags& f, int j0, int ch, int nch, float2 ka,
                                           float2 (&da)[PER], RowPair<T> (&dy)[PER], float2& A, float2& D) {
  const int64_t step = a.reverse ? -a.ld : a.ld, stepy = a.reverse ? -a.d : a.d;
  int64_t o = LOAD == GLR_TMA ? 0 : row_at<CH>(a, c, j0) * a.ld + ch, oy = LOAD == GLR_TMA ? 0 : row_at<CH>(a, c, j0) * a.d + ch;
  A = two(1.f);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    float2 r;
    if (LOAD == GLR_TMA) {
      r = lds2(sm + CH * 64);
      dy[q] = *(const RowPair<T>*)(sm + 3 * CH * 64);
      sm += a.reverse ? -64 : 64;
    } else {
      const int n = f.V >> q & 1 ? nch : 0;
      r = load2<T, LOAD == GLR_PAIRS>(a.r, o, n);
      dy[q].set(load2<T, LOAD == GLR_PAIRS>(a.dy, oy, n));
      o += step;
      oy += stepy;
    }
    da[q] = SMALL ? gate2_small(r, ka, ka).a : gate2_any(r, ka).a;
    if (!PLAIN && !(f.V >> q & 1)) {
      da[q] = two(1.f);
      dy[q].set(two(0.f));
    }
    A = mul2(A, da[q]);
  }
  D = two(0.f);
#pragma unroll
  for (int q = PER - 1; q >= 0; --q) {
    if (!PLAIN && (f.E >> q & 1))
      D = a.dhT ? load2<float, false>(a.dhT, (int64_t)seq_of(a, row_at<CH>(a, c, j0 + q)) * a.d + ch, nch) : two(0.f);
    D = mul2(da[q], add2(D, dy[q].get()));
  }
}

// The gradients: w of every row from the last on, v what comes from behind it; then from the first row on, from the state h
// before it.  dl: the rows' share of dlam.
template <typename T, int LOAD, bool SMALL, bool PLAIN, int PER, int CH>
__device__ __forceinline__ void gradients(const GlrArgs& a, const T* sm, const Span& c, const Flags& f, int j0, int ch, int nch, float2 ka,
                                          float2 root2k, const float2 (&da)[PER], const RowPair<T> (&dy)[PER], float2 v, float2 h, float2& dl) {
  float2 w[PER];
#pragma unroll
  for (int q = PER - 1; q >= 0; --q) {
    if (!PLAIN && (f.E >> q & 1)) v = a.dhT ? load2<float, false>(a.dhT, (int64_t)seq_of(a, row_at<CH>(a, c, j0 + q)) * a.d + ch, nch) : two(0.f);
    w[q] = add2(dy[q].get(), v);
    v = mul2(da[q], w[q]);
    if (!PLAIN && a.dh0 && (f.F >> q & 1)) store2<float, false>(a.dh0, (int64_t)seq_of(a, row_at<CH>(a, c, j0 + q)) * a.d + ch, nch, v);
  }
  dl = two(0.f);
  const int64_t step = a.reverse ? -a.ld : a.ld, stepd = a.reverse ? -a.ldd : a.ldd;
  int64_t o = LOAD == GLR_TMA ? 0 : row_at<CH>(a, c, j0) * a.ld + ch;
  const int64_t od = row_at<CH>(a, c, j0) * a.ldd + ch;
  T *px = (T*)a.dx + od, *pr = (T*)a.dr + od, *pi = (T*)a.di + od;
#pragma unroll
  for (int q = 0; q < PER; ++q, px += stepd, pr += stepd, pi += stepd) {
    float2 r, i, x;
    const bool ok = PLAIN || (f.V >> q & 1);
    if (LOAD == GLR_TMA) {
      r = lds2(sm + CH * 64);
      i = lds2(sm + 2 * CH * 64);
      x = lds2(sm);
      sm += a.reverse ? -64 : 64;
    } else {
      const int n = ok ? nch : 0;
      r = load2<T, LOAD == GLR_PAIRS>(a.r, o, n);
      i = load2<T, LOAD == GLR_PAIRS>(a.i, o, n);
      x = load2<T, LOAD == GLR_PAIRS>(a.x, o, n);
      o += step;
    }
    if (!PLAIN && (f.F >> q & 1))
      h = a.h0 ? load2<float, false>(a.h0, (int64_t)seq_of(a, row_at<CH>(a, c, j0 + q)) * a.d + ch, nch) : two(0.f);
    Gate2 g = SMALL ? gate2_small(r, ka, root2k) : gate2_any(r, ka);
    const float2 gi = sigmoid2(i), p = mul2(g.m, gi), u = mul2(p, x), sh = mul2(g.s, h);
    g.a = ok ? da[q] : g.a;
    const float2 G = mul2(g.a, fma2(half_s_over_sinh<SMALL>(g), u, make_float2(-sh.x, -sh.y)));  // e = w G
    h = fma2(g.a, h, u);
    const float2 dx = mul2(w[q], p), di = mul2(dx, fma2(make_float2(-x.x, -x.y), gi, x)), e = mul2(w[q], G);
    const float2 dr = mul2(e, add2(two(1.f), make_float2(-g.sr.x, -g.sr.y)));
    if (PLAIN) {
      dl = add2(dl, e);
      if (nch > 0) {
        store2<T, true>(px, 0, 2, dx);
        store2<T, true>(pr, 0, 2, dr);
        store2<T, true>(pi, 0, 2, di);
      }
    } else {
      const int n = f.in >> q & 1 ? nch : 0;
      if (ok) dl = add2(dl, e);
      else h = two(0.f);
      store2<T, LOAD != GLR_SINGLE>(px, 0, n, ok ? dx : two(0.f));
      store2<T, LOAD != GLR_SINGLE>(pr, 0, n, ok ? dr : two(0.f));
      store2<T, LOAD != GLR_SINGLE>(pi, 0, n, ok ? di : two(0.f));
    }
  }
}

struct GlrMaps4 { CUtensorMap m[4]; };  // x, r, i, dy

struct GlrSharedBwd {
  ScanShared<kWarpsB> sc;      // what the rows do to a w
  float2 sum[kWarpsB][32];      // dlam of each warp's rows
  Tile tile[4];                // the CTA's n-th at n & 3
  uint64_t full[2];
};

// Backward: one pass from each sequence's end, x, r, i and dy read once, dx, dr and di written once; the states before a
// warp's rows come from the saved one, the w behind them as the forward's states do.  As the forward, with half the rows in a
// tile and three CTAs an SM: 80 registers, for which a thread spills 56 bytes (bf16 rows copied by TMA) to 148; holding everything
// from the first pass took 128, two CTAs and spilled too: 541 against 426 us for both directions at B = 16, L = 8192.  In fp32 the
// two stages of one CTA take an SM's shared memory.  Bound by instructions (81 a value, 50 % of the issue slots) and the waits
// between tiles.  Every tile has two barriers between the first and the second pass, so what one tile leaves in
// shared memory for them is read before the next one's is written.
template <typename T, int LOAD>
__global__ void __launch_bounds__(kWarpsB * 32, kCtasBwd) k_glr_bwd(const GlrArgs a, const GlrTiles tl, const __grid_constant__ GlrMaps4 maps) {
  constexpr int PER = kPerB, CH = kGlrRowsBwd, ST = kStagesBwd;
  constexpr uint32_t BYTES = 4 * CH * 64 * sizeof(T), ALL = (1u << PER) - 1;
  extern __shared__ __align__(128) uint8_t raw[];
  pdl_enter();
  if (a.err && *a.err) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, vw = kWarpsB - 1 - warp;  // vw: in the order of the chain
  uint8_t* tiles = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
  GlrSharedBwd& sh = *reinterpret_cast<GlrSharedBwd*>(tiles + (LOAD == GLR_TMA ? ST * BYTES : 0));
  const uint32_t full = smem_u32(sh.full);
  const unsigned total = (unsigned)(tl.cut == GLR_SEQS ? *tl.n_order : tl.n_chunks) * (unsigned)(a.dp >> 6);

  auto fetch = [&](const Drawn& d, int n) {  // thread 0: the CTA's n-th tile (the chains run against the recurrence)
    Tile& o = sh.tile[n & 3];
    o.k = -1;
    if (d.t >= total) return;
    tile_of<CH>(a, tl, d.t, !a.reverse, d.e, o);
    if (LOAD == GLR_TMA) {
      const int st = n % ST;
      mbar_expect_tx(full + 8 * st, BYTES);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        tma_load_2d(smem_u32(tiles) + st * BYTES + m * (BYTES / 4), &maps.m[m], full + 8 * st, o.ch0, (int)o.c.r0);
    }
  };
  // dlam of a tile: its warps' sums in order
  auto put_sum = [&](int64_t row, int ch0) {
    if (warp != 0 || !a.dlam_part) return;
    float2 v = two(0.f);
#pragma unroll
    for (int w = 0; w < kWarpsB; ++w) v = add2(v, sh.sum[w][lane]);
    store2<float, false>(a.dlam_part, row * a.d + ch0 + 2 * lane, a.d - ch0 - 2 * lane, v);
  };
  Drawn next;
  if (tid == 0) {
    if (LOAD == GLR_TMA) {
      for (int st = 0; st < ST; ++st) mbar_init(full + 8 * st, 1);
      mbar_init_fence();
    }
    for (int n = 0; n <= ST; ++n) {
      next.t = (unsigned)atomicAdd(a.ticket, 1ull);
      if (next.t < total) next.e = asked_of<CH>(a, tl, next.t, !a.reverse);
      if (n < ST) fetch(next, n);
    }
  }
  __syncthreads();

  int64_t last_row = 0;
  int last_ch0 = 0;
  int it = 0;
  for (;; ++it) {
    const int st = it % ST;
    const Tile& t = sh.tile[it & 3];
    if (t.k < 0) break;
    const int ch = t.ch0 + 2 * lane, nch = a.d - ch;
    Words<kWarpsB> words;
    ask(a, t, vw >> 1, (vw & 1) * 32 + lane, words);
    const int64_t row = t.row;
    const int j0 = warp * PER;
    static_assert(PER == kGlrPiece, "a warp's rows are a piece");
    const int at = a.reverse ? CH - PER - j0 : j0;  // physical place of the warp's piece in the chunk
    const int64_t piece = t.piece + at / PER;
    const float2 h = load2<float, false>(a.saved, piece * a.d + ch, at < t.c.nr ? nch : 0);
    const float2 ka = *(const float2*)(a.kd + ch);
    Flags f{ALL, ALL, 0, 0};
    if (!t.inner) f = flags_of<CH, PER>(a, t.c, tl.cut, j0, lane);
    const bool plain = LOAD == GLR_TMA && f.V == ALL && (f.F | f.E) == 0 && __all_sync(FULLM, ka.x < 0.25f && ka.y < 0.25f);
    const T* sm = (const T*)(tiles + st * BYTES) + (a.reverse ? CH - 1 - j0 : j0) * 64 + 2 * lane;
    if (LOAD == GLR_TMA && !mbar_wait_bounded(full + 8 * st, (it / ST) & 1)) atomicOr(a.err_out, kErrTimeout);
    float2 da[PER], A, D;
    RowPair<T> dy[PER];
    if (plain) decays_bwd<T, LOAD, true, true, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, da, dy, A, D);
    else decays_bwd<T, LOAD, false, false, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, da, dy, A, D);
    sh.sc.agg[vw][lane] = packed(map_of(A, D, f.E != 0));
    // whether a sequence ends with the chunk's last row: then nothing comes from behind
    const bool need = !__syncthreads_or(warp == kWarpsB - 1 && (f.E >> (PER - 1) & 1)) && t.k > 0;
    if (tid == 0 && it > 0) {  // the tile before has been gone over: its place is free
      fetch(next, it + 1);
      if (next.t < total) next.t = (unsigned)atomicAdd(a.ticket, 1ull);
    }
    if (it > 0) put_sum(last_row, last_ch0);
    last_row = row;
    last_ch0 = t.ch0;
    Map2 tot;
    const Map2 pre = scan_local(a, t, sh.sc, vw, lane, tot);
    scan_words(a, t, sh.sc, vw, lane, need, words, tot);
    const float2 v = after(pre, scan_state(a, t, sh.sc, vw, lane, need, tot));
    float2 dl;
    if (plain) gradients<T, LOAD, true, true, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, make_float2(sqf(2.f * ka.x), sqf(2.f * ka.y)), da, dy, v, h, dl);
    else gradients<T, LOAD, false, false, PER, CH>(a, sm, t.c, f, j0, ch, nch, ka, ka, da, dy, v, h, dl);
    sh.sum[warp][lane] = dl;
    if (tid == 0 && next.t < total) next.e = asked_of<CH>(a, tl, next.t, !a.reverse);
  }
  __syncthreads();
  if (it > 0) put_sum(last_row, last_ch0);
}

// Rows n0 = blockIdx.y, n0 + gridDim.y, .. of [n][d] for 64 channels, summed in order; lam: times the derivative of softplus over it.
__global__ void __launch_bounds__(256) k_glr_dlam(const float* part, int64_t n, int d, const float* lam, const int* err, float* out) {
  pdl_enter();
  if (err && *err) return;
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
  if (p == 0 && ch < d) {
    const float s = ((red[0][threadIdx.x] + red[1][threadIdx.x]) + red[2][threadIdx.x]) + red[3][threadIdx.x];
    out[(int64_t)blockIdx.y * d + ch] = lam ? s * dsoftplus_ratio(lam[ch]) : s;
  }
}

// c softplus(lam), the scan's words and the tile counter cleared; checks the sequence data; marks the rows that begin a packed
// sequence (STREAM), or counts the chunks of every level (SEQS: chunk k of n at level k levels / n, rounded down, so a
// sequence's chunks are at different ones, in order).  The error word, marks and counts are 0 on entry.
__global__ void __launch_bounds__(256) k_glr_prep(const GlrArgs a, const GlrTiles tl, int64_t words, int64_t parts, int* level, int* err) {
  pdl_enter();
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)gridDim.x * 256;
  if (id == 0) {
    *a.ticket = 0;
    if (a.seq.mode == SEQ_DENSE) *err = 0;
  }
  for (int64_t i = id; i < a.dp; i += n) a.kd[i] = i < a.d ? a.c * softplus_f(a.lam[i]) : 0.f;
  for (int64_t i = id; i < words / 2; i += n) ((ulonglong2*)a.words)[i] = make_ulonglong2(0, 0);
  if (a.seq.mode == SEQ_DENSE) return;
  if (tl.cut == GLR_SEQS)  // rows of dlam's partial sums that no chunk has
    for (int64_t i = id; i < parts; i += n) a.dlam_part[i] = 0.f;
  const int lane = threadIdx.x & 31;
  for (int64_t b = id >> 5; b < a.seq.n_seq; b += n >> 5) {  // a warp each
    if (a.seq.mode == SEQ_PADDED) {
      if (lane == 0 && (a.seq.lens[b] < 0 || a.seq.lens[b] > a.seq.L)) atomicOr(err, 1);
      continue;
    }
    const int lo = a.seq.cu[b], hi = a.seq.cu[b + 1];
    if (lo < 0 || hi < lo || hi > a.seq.T || (b == 0 && lo != 0) || (b == a.seq.n_seq - 1 && hi != a.seq.T)) {
      if (lane == 0) atomicOr(err, 1);
      continue;
    }
    if (tl.cut == GLR_SEQS) {
      const int c = (hi - lo + tl.rows - 1) / tl.rows;
      for (int k = lane; k < c; k += 32) atomicAdd(level + (int64_t)k * tl.levels / c, 1);
    } else if (lane == 0 && lo < hi) {
      atomicOr((unsigned long long*)a.marks + (lo >> 6), 1ull << (lo & 63));
    }
  }
}

// Counts to first places: their sums before, in place; the sum of all to *total.  One CTA.
__global__ void __launch_bounds__(1024) k_glr_levels(int* level, int n, int* total, const int* err) {
  pdl_enter();
  __shared__ int wsum[32];
  __shared__ int carry;
  if (threadIdx.x == 0) carry = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int base = 0; base < n; base += 4096) {
    const int i = base + threadIdx.x * 4;
    int v[4], s = 0;
    for (int j = 0; j < 4; ++j) s += v[j] = i + j < n ? level[i + j] : 0;
    int x = s;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULLM, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    int at = before + x - s;
    for (int j = 0; j < 4; ++j) {
      if (i + j < n) level[i + j] = at;
      at += v[j];
    }
    __syncthreads();
    if (threadIdx.x == 1023) carry = before + x;
    __syncthreads();
  }
  if (threadIdx.x == 0) *total = *err ? 0 : carry;
}

// The chunks in the order of their levels (within one in any order: results do not depend on it).  In this order the next chunk
// of a sequence comes many tiles later, when its predecessor's words are long there: 64 packed sequences of d = 1024 take 341
// us forward (64 .. 16384 rows) against 505 in one stream, where all tiles at work are neighbours, and 471 backward (64 .. 8192)
// against 923.
__global__ void __launch_bounds__(256) k_glr_place(const GlrArgs a, const GlrTiles tl, int* level) {
  pdl_enter();
  if (*a.err) return;
  const int lane = threadIdx.x & 31;
  for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5; b < a.seq.n_seq; b += (int64_t)gridDim.x * 8) {
    const int lo = a.seq.cu[b], hi = a.seq.cu[b + 1], c = (hi - lo + tl.rows - 1) / tl.rows;
    for (int k = lane; k < c; k += 32)
      const_cast<int4*>(tl.order)[atomicAdd(level + (int64_t)k * tl.levels / c, 1)] = make_int4(lo, hi - lo, (int)b, k);
  }
}

// A few tokens of many sequences (one of each: serving): a thread for two channels of a sequence, no scan and no other launch.
// Bound by the latency of a load a row where there are few threads (B = 16, L = 1, d = 512: 1.8 us on the device, against 16 of
// the tiles with their preparation), by memory where there are many (B = 4096, L = 64: 4.7 TB/s).
template <typename T, bool VEC>
__global__ void __launch_bounds__(128) k_glr_step(const GlrArgs a, int* err) {
  pdl_enter();
  const int pairs = (a.d + 1) / 2;
  const int64_t id = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (id == 0) *err = 0;
  if (id >= (int64_t)a.seq.n_seq * pairs) return;
  const int64_t b = id / pairs;
  const int ch = 2 * (int)(id - b * pairs), nch = a.d - ch;
  const int64_t row0 = b * a.seq.L + (a.reverse ? a.seq.L - 1 : 0), step = a.reverse ? -1 : 1;
  float2 r = load2<T, VEC>(a.r, row0 * a.ld + ch, nch), i = load2<T, VEC>(a.i, row0 * a.ld + ch, nch), x = load2<T, VEC>(a.x, row0 * a.ld + ch, nch);
  float2 h = a.h0 ? load2<float, false>(a.h0, b * a.d + ch, nch) : two(0.f), ka = two(0.f);
  ka.x = a.c * softplus_f(a.lam[ch]);
  if (nch > 1) ka.y = a.c * softplus_f(a.lam[ch + 1]);
  for (int t = 0; t < a.seq.L; ++t) {
    const Gate2 g = gate2_any(r, ka);
    h = fma2(g.a, h, mul2(g.m, mul2(sigmoid2(i), x)));
    store2<T, VEC>(a.y, (row0 + t * step) * a.d + ch, nch, h);
    if (t + 1 == a.seq.L) break;
    const int64_t o = (row0 + (t + 1) * step) * a.ld + ch;
    r = load2<T, VEC>(a.r, o, nch);
    i = load2<T, VEC>(a.i, o, nch);
    x = load2<T, VEC>(a.x, o, nch);
  }
  if (a.hT) store2<float, false>(a.hT, b * a.d + ch, nch, h);
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

cudaError_t launch_glr_prep(const GlrArgs& a, const GlrTiles& t, int64_t words, int64_t parts, int* level, int* err, cudaStream_t st) {
  const int64_t n = std::max<int64_t>(std::max<int64_t>(words / 2, a.dp), a.seq.mode == SEQ_DENSE ? 1 : (int64_t)a.seq.n_seq * 32);
  const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)sm_count() * 8);
  return launch_pdl(k_glr_prep, dim3(grid), dim3(256), 0, st, a, t, words, parts, level, err);
}
cudaError_t launch_glr_order(const GlrArgs& a, const GlrTiles& t, int* level, cudaStream_t st) {
  const cudaError_t e = launch_pdl(k_glr_levels, dim3(1), dim3(1024), 0, st, level, t.levels, const_cast<int*>(t.n_order), a.err);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.seq.n_seq + 7) / 8, (int64_t)sm_count() * 4);
  return launch_pdl(k_glr_place, dim3(grid), dim3(256), 0, st, a, t, level);
}
cudaError_t launch_glr_step(const GlrArgs& a, bool f32, int* err, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)a.seq.n_seq * ((a.d + 1) / 2) + 127) / 128));
  if (f32) return launch_pdl(pairs_ok(a, 4) ? k_glr_step<float, true> : k_glr_step<float, false>, grid, dim3(128), 0, st, a, err);
  return launch_pdl(pairs_ok(a, 2) ? k_glr_step<bf16, true> : k_glr_step<bf16, false>, grid, dim3(128), 0, st, a, err);
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
  return launch_pdl(kernel, grid, dim3(kWarpsF * 32), smem, st, a, t, maps);
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
  const bool tma = pairs_ok(a, sizeof(T)) && rows_map(&maps.m[0], a.x, f32, a.d, a.seq.T, a.ld, kGlrRowsBwd) &&
                   rows_map(&maps.m[1], a.r, f32, a.d, a.seq.T, a.ld, kGlrRowsBwd) &&
                   rows_map(&maps.m[2], a.i, f32, a.d, a.seq.T, a.ld, kGlrRowsBwd) &&
                   rows_map(&maps.m[3], a.dy, f32, a.d, a.seq.T, a.d, kGlrRowsBwd);
  const size_t smem = 128 + sizeof(GlrSharedBwd) + (tma ? kStagesBwd * (size_t)4 * kGlrRowsBwd * 64 * sizeof(T) : 0);
  const dim3 grid((unsigned)std::min<int64_t>((int64_t)t.n_chunks * (a.dp >> 6), (int64_t)sm_count() * kCtasBwd));
  auto kernel = tma ? k_glr_bwd<T, GLR_TMA> : pairs_ok(a, sizeof(T)) ? k_glr_bwd<T, GLR_PAIRS> : k_glr_bwd<T, GLR_SINGLE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(kWarpsB * 32), smem, st, a, t, maps);
}
}  // namespace

cudaError_t launch_glr_bwd(const GlrArgs& a, const GlrTiles& t, bool f32, cudaStream_t st) {
  return f32 ? run_glr_bwd<float>(a, t, st) : run_glr_bwd<bf16>(a, t, st);
}

cudaError_t launch_glr_dlam(const GlrArgs& a, int64_t n, float* sums, float* out, cudaStream_t st) {
  const dim3 cols((unsigned)(a.dp >> 6));
  const float* part = a.dlam_part;
  if (n > kDlamRows) {
    const cudaError_t e = launch_pdl(k_glr_dlam, dim3(cols.x, kDlamRows), dim3(256), 0, st, part, n, a.d, (const float*)nullptr, (const int*)a.err, sums);
    if (e != cudaSuccess) return e;
    part = sums;
    n = kDlamRows;
  }
  return launch_pdl(k_glr_dlam, cols, dim3(256), 0, st, part, n, a.d, a.lam, (const int*)a.err, out);
}

}  // namespace gbla
