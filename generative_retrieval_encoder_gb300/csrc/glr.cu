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
#include "mbarrier.cuh"
#include "pdl.cuh"

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
__device__ __forceinline__ float sigmoid_f(float x) { return rcpf(1.f + ex2f(-kLog2e * x)); }

// softplus(lam), and sigmoid(lam) / softplus(lam) (1 - e^lam / 2 + .. for small e^lam).
__device__ __forceinline__ float softplus_f(float l) { return fmaxf(l, 0.f) + log1pf(expf(-fabsf(l))); }
__device__ __forceinline__ float dsoftplus_ratio(float l) {
  return l < -15.f ? 1.f : 1.f / ((1.f + expf(-l)) * softplus_f(l));
}

// The gates of one value: decay a, s, m = sqrt(1 - a^2) and s / m.
struct Gate { float a, s, m, sm, sr; };
__device__ __forceinline__ Gate gate_of(float r, float k) {
  Gate g;
  g.sr = sigmoid_f(r);
  g.s = k * g.sr;
  const float s = g.s;
  // q = 1 - e^-s: the series up to s^6 below 1/4 (the next term is below 5e-8 of it)
  float p = fmaf(s, -1.f / 720.f, 1.f / 120.f);
  p = fmaf(s, p, -1.f / 24.f);
  p = fmaf(s, p, 1.f / 6.f);
  p = fmaf(s, p, -0.5f);
  p = fmaf(s, p, 1.f);
  const float e = ex2f(-kLog2e * s);
  const float q = s < 0.25f ? s * p : 1.f - e;
  g.a = s < 0.25f ? 1.f - q : e;
  const float z = q * (2.f - q);
  const float rs = z >= 1.2e-38f ? rsqf(z) : 0.f;
  g.m = z * rs;
  g.sm = s * rs;
  return g;
}

// ------------------------------------------------------------ chunks
// The rows are cut into chunks of 64 (slots of at least kGlrSlot rows each into their own, everything else as one
// stream), a chunk and 64 channels are a tile, a tile is one CTA's.  A chunk's rows are numbered in the direction of
// the recurrence; F, E, V: the rows that are a sequence's first, its last, and in a sequence at all.
struct Rows {
  int64_t r0;       // physical first row
  int nr;           // rows of the chunk
  uint64_t F, E, V;
};
__device__ __forceinline__ Rows rows_of(const GlrArgs& a, int64_t chunk, int lane) {
  Rows c;
  uint64_t S, Z;
  if (a.seq.mode == SEQ_VARLEN) {
    c.r0 = chunk * kGlrChunk;
    c.nr = (int)min((int64_t)kGlrChunk, a.seq.T - c.r0);
    S = a.marks[chunk];
    const uint64_t nxt = c.r0 + kGlrChunk < a.seq.T ? a.marks[chunk + 1] : 1;
    c.V = c.nr == 64 ? ~0ull : (1ull << c.nr) - 1;
    Z = (S >> 1) | (nxt << 63);
    if (c.nr < 64) Z |= 1ull << (c.nr - 1);
  } else {
    uint32_t v[2], s[2], z[2];
    if (a.per_seq) {
      const int64_t b = chunk / a.per_seq;
      const int k = (int)(chunk - b * a.per_seq) * kGlrChunk;
      c.r0 = b * a.seq.L + k;
      c.nr = min(kGlrChunk, a.seq.L - k);
      const int len = a.seq.mode == SEQ_PADDED ? a.seq.lens[b] : a.seq.L;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int pos = k + lane + 32 * q;
        const bool in = pos < len;
        v[q] = __ballot_sync(FULLM, in);
        s[q] = __ballot_sync(FULLM, in && pos == 0);
        z[q] = __ballot_sync(FULLM, in && pos == len - 1);
      }
    } else {
      c.r0 = chunk * kGlrChunk;
      c.nr = (int)min((int64_t)kGlrChunk, a.seq.T - c.r0);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t row = c.r0 + lane + 32 * q;
        const int b = (int)(row / a.seq.L), pos = (int)(row - (int64_t)b * a.seq.L);
        const bool there = row < a.seq.T;
        const int len = a.seq.mode == SEQ_PADDED ? (there ? a.seq.lens[b] : 0) : a.seq.L;
        const bool in = there && pos < len;
        v[q] = __ballot_sync(FULLM, in);
        s[q] = __ballot_sync(FULLM, in && pos == 0);
        z[q] = __ballot_sync(FULLM, in && pos == len - 1);
      }
    }
    c.V = v[0] | (uint64_t)v[1] << 32;
    S = s[0] | (uint64_t)s[1] << 32;
    Z = z[0] | (uint64_t)z[1] << 32;
  }
  if (a.reverse) {
    c.V = __brevll(c.V);
    c.F = __brevll(Z);
    c.E = __brevll(S);
  } else {
    c.F = S;
    c.E = Z;
  }
  return c;
}
__device__ __forceinline__ int64_t row_at(const GlrArgs& a, const Rows& c, int j) {
  return a.reverse ? c.r0 + 63 - j : c.r0 + j;
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

__device__ __forceinline__ void publish(uint64_t* p, const Map& x, const Map& y) {
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(word_of(x)), "l"(word_of(y)) : "memory");
}
__device__ __forceinline__ void peek(const uint64_t* p, uint64_t& x, uint64_t& y) {
  asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "l"(p) : "memory");
}
// Waits for a pair of words: bounded, and given up at once where another wait has been.
__device__ __forceinline__ void await(const uint64_t* p, uint64_t& x, uint64_t& y, int* err) {
  for (int n = 0; !(x >> 63 & y >> 63); ++n) {
    if (n > 64) __nanosleep(100);
    if ((n & 1023) == 1023 && (*(volatile int*)err & kErrTimeout)) break;
    if (n > (1 << 22)) {
      atomicOr(err, kErrTimeout);
      break;
    }
    peek(p, x, y);
  }
}

// The words of a call: of chunks, groups and larger groups, each [..][dp] with dp the channels rounded up to 64.
struct Chain {
  const uint64_t* chunk; const uint64_t* group; const uint64_t* large;
  int k;            // this chunk's place in its chain
};
__device__ __forceinline__ Chain chain_of(const GlrArgs& a, int64_t s, int k, int ch) {
  // s: the sequence slot (0 for a stream); the arrays hold each slot's words in the order of its chain
  const int64_t n = a.per_seq ? a.per_seq : a.n_chunks, ng = (n + 15) >> 4, nl = (n + 255) >> 8;
  Chain c;
  c.chunk = a.words + (s * n) * a.dp + ch;
  c.group = a.words + ((int64_t)a.n_chunks + s * ng) * a.dp + ch;
  c.large = a.words + ((int64_t)a.n_chunks + (int64_t)(a.per_seq ? a.seq.n_seq : 1) * ng + s * nl) * a.dp + ch;
  c.k = k;
  return c;
}
// Warp w's share, composed, of the words that chunk k reads: warps 0-3 the larger group's state and the groups before,
// warps 4-7 the chunks before.
__device__ __forceinline__ void look_back(const Chain& c, int64_t dp, int warp, int* err, Map& x, Map& y) {
  x.A = y.A = 1.f;
  x.H = y.H = 0.f;
  x.reset = y.reset = false;
  const int g = c.k >> 4, l = c.k >> 8, q = warp & 3;
  const int n = warp < 4 ? (g & 15) + (l > 0) : c.k & 15;
  const int lo = q * n >> 2, m = ((q + 1) * n >> 2) - lo;
  const uint64_t* p[4];
  uint64_t wx[4], wy[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= m) break;
    const int i = lo + j;
    p[j] = warp >= 4 ? c.chunk + (int64_t)((g << 4) + i) * dp
           : l > 0   ? (i == 0 ? c.large + (int64_t)(l - 1) * dp : c.group + (int64_t)((l << 4) + i - 1) * dp)
                     : c.group + (int64_t)i * dp;
    peek(p[j], wx[j], wy[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= m) break;
    await(p[j], wx[j], wy[j], err);
    x = then(x, map_of(wx[j]));
    y = then(y, map_of(wy[j]));
  }
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

constexpr int kWarps = 8, kPer = kGlrChunk / kWarps;  // a warp's rows; a lane has two channels of each

// The tile of this CTA: channels from *ch0, chunk (physical) *chunk, slot *s and place *k in its chain.
__device__ __forceinline__ void tile_of(const GlrArgs& a, unsigned long long t, bool back, int& ch0, int64_t& chunk, int64_t& s, int& k) {
  const unsigned ncg = (unsigned)(a.dp >> 6);
  ch0 = (int)(t % ncg) * 64;
  t /= ncg;
  if (a.per_seq) {
    s = (int64_t)(t % (unsigned)a.seq.n_seq);
    k = (int)(t / (unsigned)a.seq.n_seq);
    chunk = s * a.per_seq + (back ? a.per_seq - 1 - k : k);
  } else {
    s = 0;
    k = (int)t;
    chunk = back ? a.n_chunks - 1 - k : k;
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_glr_fwd(const GlrArgs a) {
  __shared__ float4 agg[kWarps][32];       // {A, H} of each warp's rows, two channels
  __shared__ float4 back[kWarps][32];      // of each warp's share of the words before
  __shared__ int back_reset[kWarps];
  __shared__ unsigned long long tile_s;
  if (a.err && *a.err) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) tile_s = atomicAdd(a.ticket, 1ull);
  __syncthreads();
  int ch, k;
  int64_t chunk, slot;
  tile_of(a, tile_s, a.reverse, ch, chunk, slot, k);
  ch += 2 * lane;
  const int nch = a.d - ch;  // channels of this lane: 2, 1 or none
  const Rows c = rows_of(a, chunk, lane);

  // the lane's rows: a and u
  float2 ka = make_float2(0.f, 0.f);
  if (nch > 0) ka.x = a.c * softplus_f(a.lam[ch]);
  if (nch > 1) ka.y = a.c * softplus_f(a.lam[ch + 1]);
  const int j0 = warp * kPer;
  const uint32_t V = (uint32_t)(c.V >> j0) & 0xffu, F = (uint32_t)(c.F >> j0) & 0xffu, E = (uint32_t)(c.E >> j0) & 0xffu;
  float2 x[kPer], r[kPer], i[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int64_t o = row_at(a, c, j0 + q) * a.ld + ch;
    const int n = V >> q & 1 ? nch : 0;
    r[q] = load2<T, VEC>(a.r, o, n);
    i[q] = load2<T, VEC>(a.i, o, n);
    x[q] = load2<T, VEC>(a.x, o, n);
  }
  float2 da[kPer], u[kPer];
  Map mx{1.f, 0.f, false}, my{1.f, 0.f, false};
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const Gate gx = gate_of(r[q].x, ka.x), gy = gate_of(r[q].y, ka.y);
    da[q] = make_float2(gx.a, gy.a);
    u[q] = make_float2(gx.m * sigmoid_f(i[q].x) * x[q].x, gy.m * sigmoid_f(i[q].y) * x[q].y);
    if (!(V >> q & 1)) {
      da[q] = make_float2(1.f, 1.f);
      u[q] = make_float2(0.f, 0.f);
    }
    if (F >> q & 1) {
      if (a.h0) {
        const int64_t o = (int64_t)seq_of(a, row_at(a, c, j0 + q)) * a.d + ch;
        if (nch > 0) u[q].x = fmaf(da[q].x, a.h0[o], u[q].x);
        if (nch > 1) u[q].y = fmaf(da[q].y, a.h0[o + 1], u[q].y);
      }
      mx.H = u[q].x;
      my.H = u[q].y;
      mx.reset = my.reset = true;
    } else {
      mx.H = fmaf(da[q].x, mx.H, u[q].x);
      my.H = fmaf(da[q].y, my.H, u[q].y);
      mx.A *= da[q].x;
      my.A *= da[q].y;
    }
  }
  agg[warp][lane] = make_float4(mx.A, mx.H, my.A, my.H);
  __syncthreads();

  // what the warps before do together
  Map px{1.f, 0.f, false}, py{1.f, 0.f, false};
  for (int w = 0; w < warp; ++w) {
    const float4 g = agg[w][lane];
    const bool rs = (c.F >> (w * kPer) & 0xff) != 0;
    px = then(px, Map{g.x, g.y, rs});
    py = then(py, Map{g.z, g.w, rs});
  }
  const Chain chain = chain_of(a, slot, k, ch);
  const int64_t last = a.per_seq ? a.per_seq : a.n_chunks;
  Map tx, ty;
  if (warp == kWarps - 1) {
    tx = then(px, mx);
    ty = then(py, my);
    if (k + 1 < last) publish(const_cast<uint64_t*>(chain.chunk) + (int64_t)k * a.dp, tx, ty);
  }
  // the state that enters, where the chunk does not begin with a sequence
  const int first = __ffsll(c.V) - 1;
  const bool need = first >= 0 && !(c.F >> first & 1);
  float2 in = make_float2(0.f, 0.f);
  if (need) {
    Map bx, by;
    look_back(chain, a.dp, warp, a.err_out, bx, by);
    back[warp][lane] = make_float4(bx.A, bx.H, by.A, by.H);
    if (lane == 0) back_reset[warp] = bx.reset;
    __syncthreads();
    Map sx{1.f, 0.f, false}, sy{1.f, 0.f, false};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 g = back[w][lane];
      const bool rs = back_reset[w];
      sx = then(sx, Map{g.x, g.y, rs});
      sy = then(sy, Map{g.z, g.w, rs});
    }
    in = make_float2(sx.H, sy.H);
    if (a.saved && warp == 0) store2<float, false>(a.saved, chunk * a.d + ch, nch, in);
  }
  if (warp == kWarps - 1 && (k & 15) == 15 && k + 1 < last) {
    Map gx{1.f, 0.f, false}, gy{1.f, 0.f, false};
    if (need)
      for (int w = 4; w < 8; ++w) {
        const float4 g = back[w][lane];
        gx = then(gx, Map{g.x, g.y, back_reset[w] != 0});
        gy = then(gy, Map{g.z, g.w, back_reset[w] != 0});
      }
    publish(const_cast<uint64_t*>(chain.group) + (int64_t)(k >> 4) * a.dp, then(gx, tx), then(gy, ty));
    if ((k & 255) == 255)
      publish(const_cast<uint64_t*>(chain.large) + (int64_t)(k >> 8) * a.dp, Map{0.f, tx.reset ? tx.H : fmaf(tx.A, in.x, tx.H), true},
              Map{0.f, ty.reset ? ty.H : fmaf(ty.A, in.y, ty.H), true});
  }
  // the rows again, from the state that enters them
  float2 h = make_float2(px.reset ? px.H : fmaf(px.A, in.x, px.H), py.reset ? py.H : fmaf(py.A, in.y, py.H));
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int j = j0 + q;
    const int64_t row = row_at(a, c, j);
    if (F >> q & 1) {
      h = u[q];
    } else {
      h.x = fmaf(da[q].x, h.x, u[q].x);
      h.y = fmaf(da[q].y, h.y, u[q].y);
    }
    const bool in_chunk = (a.reverse ? 63 - j : j) < c.nr;
    store2<T, VEC>(a.y, row * a.d + ch, in_chunk ? nch : 0, V >> q & 1 ? h : make_float2(0.f, 0.f));
    if (a.hT && (E >> q & 1)) store2<float, false>(a.hT, (int64_t)seq_of(a, row) * a.d + ch, nch, h);
  }
}

// Sequence b's first row and valid rows.
__device__ __forceinline__ void seq_rows(const SeqDesc& s, int b, int64_t& row0, int& n) {
  if (s.mode == SEQ_VARLEN) {
    row0 = s.cu[b];
    n = s.cu[b + 1] - s.cu[b];
  } else {
    row0 = (int64_t)b * s.L;
    n = s.mode == SEQ_PADDED ? s.lens[b] : s.L;
  }
}
// The chunk of a row (the tiles of GlrArgs), and whether the row is its first in the direction of the recurrence.
__device__ __forceinline__ int64_t chunk_of(const GlrArgs& a, int b, int64_t row, int64_t row0, bool& first, bool& last) {
  const int64_t p = a.per_seq ? row - row0 : row;
  const int64_t c = p / kGlrChunk + (a.per_seq ? (int64_t)b * a.per_seq : 0);
  const bool lo = p % kGlrChunk == 0, hi = p % kGlrChunk == kGlrChunk - 1;
  first = a.reverse ? hi : lo;
  last = a.reverse ? lo : hi;
  return c;
}

template <typename T>
__global__ void __launch_bounds__(256) k_glr_bwd(const GlrArgs a) {
  if (a.err && *a.err) return;
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= (int64_t)a.seq.n_seq * a.d) return;
  const int b = (int)(id / a.d), ch = (int)(id % a.d);
  int64_t row0;
  int n;
  seq_rows(a.seq, b, row0, n);
  const float k = a.c * softplus_f(a.lam[ch]);
  float w = a.dhT ? a.dhT[id] : 0.f, dl = 0.f;  // w: a_{t+1} w_{t+1}
  int hi = n;                                   // rows [lo, hi) of the recurrence: one chunk's
  while (hi > 0) {
    int lo = hi - 1;
    float before[kGlrChunk];
    float h = 0.f;
    for (;; --lo) {  // back to the first row of the chunk, or of the sequence
      const int64_t row = a.reverse ? row0 + n - 1 - lo : row0 + lo;
      bool first, last;
      const int64_t c = chunk_of(a, b, row, row0, first, last);
      if (lo == 0) { h = a.h0 ? a.h0[id] : 0.f; break; }
      if (first) { h = a.saved[c * a.d + ch]; break; }
    }
    for (int t = lo; t < hi; ++t) {
      const int64_t row = a.reverse ? row0 + n - 1 - t : row0 + t;
      const int64_t o = row * a.ld + ch;
      before[t - lo] = h;
      const Gate g = gate_of(to_f(((const T*)a.r)[o]), k);
      h = fmaf(g.a, h, g.m * sigmoid_f(to_f(((const T*)a.i)[o])) * to_f(((const T*)a.x)[o]));
    }
    for (int t = hi - 1; t >= lo; --t) {
      const int64_t row = a.reverse ? row0 + n - 1 - t : row0 + t;
      const int64_t o = row * a.ld + ch, od = row * a.ldd + ch;
      const Gate g = gate_of(to_f(((const T*)a.r)[o]), k);
      const float gi = sigmoid_f(to_f(((const T*)a.i)[o])), x = to_f(((const T*)a.x)[o]);
      w += to_f(((const T*)a.dy)[row * a.d + ch]);
      const float e = -w * (g.a * g.s * before[t - lo] - gi * x * g.a * g.a * g.sm);
      ((T*)a.dx)[od] = from_f<T>(w * g.m * gi);
      ((T*)a.di)[od] = from_f<T>(w * g.m * x * gi * (1.f - gi));
      ((T*)a.dr)[od] = from_f<T>(e * (1.f - g.sr));
      dl += e;
      w *= g.a;
    }
    hi = lo;
  }
  if (a.dh0) a.dh0[id] = w;
  if (a.dlam_part) a.dlam_part[id] = dl * dsoftplus_ratio(a.lam[ch]);
  if (a.seq.mode == SEQ_PADDED)
    for (int t = n; t < a.seq.L; ++t) {
      const int64_t od = (row0 + t) * a.ldd + ch;
      ((T*)a.dx)[od] = ((T*)a.dr)[od] = ((T*)a.di)[od] = from_f<T>(0.f);
    }
}

// Checks the sequence data and, for packed sequences, marks the rows that begin one.
__global__ void __launch_bounds__(256) k_glr_prep(const GlrArgs a, int* err) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= a.seq.n_seq) return;
  if (a.seq.mode == SEQ_PADDED) {
    if (a.seq.lens[b] < 0 || a.seq.lens[b] > a.seq.L) atomicOr(err, 1);
    return;
  }
  const int lo = a.seq.cu[b], hi = a.seq.cu[b + 1];
  if (lo < 0 || hi < lo || hi > a.seq.T || (b == 0 && lo != 0) || (b == a.seq.n_seq - 1 && hi != a.seq.T)) {
    atomicOr(err, 1);
    return;
  }
  if (lo < hi) atomicOr((unsigned long long*)a.marks + lo / kGlrChunk, 1ull << (lo % kGlrChunk));
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

cudaError_t launch_glr_prep(const GlrArgs& a, int* err, cudaStream_t st) {
  k_glr_prep<<<(unsigned)((a.seq.n_seq + 255) / 256), 256, 0, st>>>(a, err);
  return cudaGetLastError();
}
cudaError_t launch_glr_empty(const GlrArgs& a, const float* from, float* to, cudaStream_t st) {
  k_glr_empty<<<(unsigned)std::min(a.seq.n_seq, 4096), 256, 0, st>>>(a, from, to);
  return cudaGetLastError();
}

cudaError_t launch_glr_fwd(const GlrArgs& a, bool f32, cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.n_chunks * (a.dp >> 6));
  if (f32) {
    if (pairs_ok(a, 4)) k_glr_fwd<float, true><<<grid, 256, 0, st>>>(a);
    else k_glr_fwd<float, false><<<grid, 256, 0, st>>>(a);
  } else {
    if (pairs_ok(a, 2)) k_glr_fwd<bf16, true><<<grid, 256, 0, st>>>(a);
    else k_glr_fwd<bf16, false><<<grid, 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_glr_bwd(const GlrArgs& a, bool f32, cudaStream_t st) {
  const int64_t n = (int64_t)a.seq.n_seq * a.d;
  const unsigned grid = (unsigned)((n + 255) / 256);
  if (f32) k_glr_bwd<float><<<grid, 256, 0, st>>>(a);
  else k_glr_bwd<bf16><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace gbla
