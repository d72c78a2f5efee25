// Token embedding: rows of a table by ids, k of them a token side by side, and the table's gradient.
//   y[slot] = scale table[ids[slot]],   dtable[v] = scale * sum of dy[slot] over the slots with ids[slot] = v
// (slot = token k + which of its ids; an id below 0, or of a row that is in no sequence, has a row of zeros and no gradient).
//
// The gradient goes by sorted slots, so that each row of the table is written once, in one fixed order of its slots: a stable
// counting sort by the id's digits (no CTA waits for another: a tile's place among its digit's keys comes from the counts of
// the tiles before it), then the sums, kEmbedCap sorted places a group of threads.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace gbla {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kMaxBins = 1 << kEmbedDigit;  // a thread's each, at most
static_assert(kMaxBins <= kThreads && kEmbedCap % 4 == 0 && kEmbedCap <= 32, "");

// The id of a slot, -1 for none.  An id past the table or a length outside [0, L] counts as none and is `bad`.
__device__ __forceinline__ int id_of(const EmbedArgs& a, int64_t slot, bool& bad) {
  const int64_t id = a.wide_ids ? static_cast<const int64_t*>(a.ids)[slot] : (int64_t)static_cast<const int32_t*>(a.ids)[slot];
  if (a.lens) {
    const int row = (int)slot / a.k, b = row / a.L, len = a.lens[b];
    if (len < 0 || len > a.L) {
      bad = true;
      return -1;
    }
    if (row - b * a.L >= len) return -1;
  }
  if (id >= a.V) {
    bad = true;
    return -1;
  }
  return id < 0 ? -1 : (int)id;
}
__device__ __forceinline__ int id_of(const EmbedArgs& a, int64_t slot) {  // and says so in the error word
  bool bad = false;
  const int id = id_of(a, slot, bad);
  if (bad) atomicOr(a.err, 1);
  return id;
}

template <typename T>
__device__ __forceinline__ uint4 scaled(uint4 w, float s) {
  if (sizeof(T) == 2)
    return make_uint4(pack_bf16(bf_lo(w.x) * s, bf_hi(w.x) * s), pack_bf16(bf_lo(w.y) * s, bf_hi(w.y) * s),
                      pack_bf16(bf_lo(w.z) * s, bf_hi(w.z) * s), pack_bf16(bf_lo(w.w) * s, bf_hi(w.w) * s));
  return make_uint4(__float_as_uint(__uint_as_float(w.x) * s), __float_as_uint(__uint_as_float(w.y) * s),
                    __float_as_uint(__uint_as_float(w.z) * s), __float_as_uint(__uint_as_float(w.w) * s));
}

// A CTA takes `per` slots: their ids once, then the rows as one run of y.  ROWS: rows of `cols` accesses of 16 bytes each, four in flight a
// thread.  Bound by memory: 131072 rows of 512 bf16 from a table of 32768 in 27 us, 0.9 of a copy's rate with the table read once (L2
// holds it).  PAIRS, VALUES: y in pieces of 16 bytes of whatever rows, read from the table by two bf16 or by single values (`per` is a
// multiple of a piece's values): 65536 rows of 510 in 19 us, of 511 in 29, of 512 by ROWS in 14; value by value 62.  SINGLE: of a y that
// is not aligned, value by value, `cols` of them a row; of a scale that is not finite, too, as the others multiply the zeros of no token.
enum EmbedRows { SINGLE, ROWS, PAIRS, VALUES };
template <typename T, EmbedRows M>
__global__ void __launch_bounds__(kThreads) k_embed_fwd(const EmbedArgs a, int per, int cols, uint32_t by_cols, bool check) {
  pdl_enter();
  __shared__ int id[1024];
  if (check && blockIdx.x == gridDim.x - 1) {  // one CTA looks at every id and alone reports: no launch to clear the error word first
    bool bad = false;
    for (int64_t i = threadIdx.x; i < a.n; i += kThreads) id_of(a, i, bad);
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.err = any ? 1 : 0;
    return;
  }
  const int64_t s0 = (int64_t)blockIdx.x * per;
  const int ns = (int)min((int64_t)per, a.n - s0);
  for (int i = threadIdx.x; i < ns; i += kThreads) {
    bool bad = false;
    id[i] = id_of(a, s0 + i, bad);
    if (bad && !check) atomicOr(a.err, 1);
  }
  __syncthreads();
  const T* tab = static_cast<const T*>(a.table);
  T* y = static_cast<T*>(a.y) + s0 * a.d;
  if constexpr (M == PAIRS || M == VALUES) {
    constexpr int E = 16 / sizeof(T), V = M == PAIRS ? 2 : 1;
    const int total = ns * a.d;  // (below 2^24: `per` is a piece's values, or total some 1024 pieces)
    for (int e = threadIdx.x * E; e < total; e += kThreads * E) {
      int k = by_cols ? (int)__umulhi((uint32_t)e, by_cols) : e / a.d, c = e - k * a.d;
      uint32_t q[E / V];
      int row = id[k];
#pragma unroll
      for (int j = 0; j < E; j += V) {
        if (c == a.d && e + j < total) c = 0, row = id[++k];
        q[j / V] = 0;
        if (row >= 0 && e + j < total) {
          const T* at = tab + (int64_t)row * a.d + c;
          if constexpr (M == VALUES && sizeof(T) == 2) q[j / V] = *reinterpret_cast<const uint16_t*>(at);
          else q[j / V] = *reinterpret_cast<const uint32_t*>(at);
        }
        c += V;
      }
      uint4 w;
      if constexpr (M == VALUES && sizeof(T) == 2) w = make_uint4(q[0] | q[1] << 16, q[2] | q[3] << 16, q[4] | q[5] << 16, q[6] | q[7] << 16);
      else w = make_uint4(q[0], q[1], q[2], q[3]);
      w = scaled<T>(w, a.scale);
      if (e + E <= total) {
        *reinterpret_cast<uint4*>(y + e) = w;
      } else {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (e + j < total) y[e + j] = from_f<T>(sizeof(T) == 2 ? (j & 1 ? bf_hi(u[j / 2 & 3]) : bf_lo(u[j / 2 & 3])) : __uint_as_float(u[j & 3]));
      }
    }
  } else {
    const int64_t total = (int64_t)ns * cols;  // more than 2^16 for one slot alone
    for (int64_t i0 = threadIdx.x; i0 < total; i0 += 4 * kThreads) {
      uint4 v[4];
      float f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * kThreads;
        v[u] = make_uint4(0, 0, 0, 0);
        f[u] = 0.f;
        if (i >= total) continue;
        const int s = per == 1 ? 0 : cols == 1 ? (int)i : (int)__umulhi((uint32_t)i, by_cols), c = (int)(i - (int64_t)s * cols);
        const int k = id[s];
        if (k < 0) continue;
        if (M == ROWS) v[u] = __ldg(reinterpret_cast<const uint4*>(tab + (int64_t)k * a.d) + c);
        else f[u] = to_f(tab[(int64_t)k * a.d + c]) * a.scale;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * kThreads;
        if (i >= total) continue;
        if (M == ROWS) reinterpret_cast<uint4*>(y)[i] = scaled<T>(v[u], a.scale);
        else y[i] = from_f<T>(f[u]);
      }
    }
  }
}

// ------------------------------------------------------------------ the sort
// Two launches a digit, bound by latency: 131072 slots in 26 us by two digits of 8 bits with tiles of 512 keys (1024 keys, whose CTAs are
// fewer: 75 us for the whole gradient against 71; 2048: 80).
// A tile's keys: a warp takes an eighth of them, consecutive, 32 a round.
constexpr int kRounds = kEmbedTile / kThreads;
template <int R>
__device__ __forceinline__ int64_t place_of(int tile, int round) {
  return (int64_t)tile * (R * kThreads) + (threadIdx.x >> 5) * (R * 32) + round * 32 + (threadIdx.x & 31);
}
// The key at a place of the pass's input: an id, V for none (last of all), V too past the end.
__device__ __forceinline__ int key_at(const EmbedArgs& a, const EmbedSort& s, int64_t i, bool first) {
  if (i >= a.n) return a.V;
  if (!first) return s.key_in[i];
  const int id = id_of(a, i);
  return id < 0 ? a.V : id;
}

// Of a table of more rows than there are slots the whole gradient is cleared meanwhile: the sort's CTAs are few and wait for latencies, so
// each of its launches has more CTAs that clear a share, kFill values each.  Of a smaller one the rows that no id has are cleared beside
// the sums, which write the others.  (4 hashes into a million rows of 128, 512 MB: 109 us against 122; 32768 rows of 512 and 131072 slots,
// 67 MB: 79 against 71.)
constexpr int kFill = 16384;
bool embed_fills(const EmbedArgs& a) { return a.V > a.n; }
__device__ __forceinline__ bool fill(const EmbedFill& f, int tiles) {
  if ((int)blockIdx.x < tiles) return false;
  const int64_t lo = f.lo + ((int64_t)blockIdx.x - tiles) * kFill, hi = min(f.hi, lo + kFill);
  if (f.wide) {
    for (int64_t i = lo + threadIdx.x * 4; i < hi; i += kThreads * 4) {
      if (i + 4 <= hi) *reinterpret_cast<float4*>(f.p + i) = make_float4(0.f, 0.f, 0.f, 0.f);
      else
        for (int64_t j = i; j < hi; ++j) f.p[j] = 0.f;
    }
  } else {
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) f.p[i] = 0.f;
  }
  return true;
}

// Each tile's keys by digit, and the sums of kEmbedTiles tiles.
__global__ void __launch_bounds__(kThreads) k_embed_count(const EmbedArgs a, const EmbedSort s, const EmbedFill f, int bins, int shift, bool first) {
  pdl_enter();
  if (fill(f, s.tiles)) return;
  __shared__ int count[kMaxBins];
  for (int i = threadIdx.x; i < bins; i += kThreads) count[i] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = place_of<kRounds>(blockIdx.x, r);
    if (i < a.n) atomicAdd(&count[(key_at(a, s, i, first) >> shift) & (bins - 1)], 1);
  }
  __syncthreads();
  int* tile = s.count + (int64_t)blockIdx.x * kMaxBins;
  int* sum = s.sums + (int64_t)(blockIdx.x / kEmbedTiles) * kMaxBins;
  for (int i = threadIdx.x; i < bins; i += kThreads) {
    const int c = count[i];
    tile[i] = c;
    if (c) atomicAdd(&sum[i], c);
  }
}

// Of more than kEmbedGroups groups of tiles: their sums become the sums of the groups before each, the digits' totals behind them, so that
// a tile reads two rows of them, not all, which would take the square of the slots.  (8 columns, 32768 rows; with this launch and
// without: 524288 slots 68 us and 67, 786432 83 and 87, 4194304 302 and 492, 16777216 1102 and 4284.)  A thread a digit and 32nd of the
// groups.
__global__ void __launch_bounds__(1024) k_embed_scan(int* sums, int groups) {
  pdl_enter();
  __shared__ int red[32][32];
  constexpr int U = 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* col = sums + blockIdx.x * 32 + lane;
  const int per = (groups + 31) / 32, lo = min(groups, warp * per), hi = min(groups, lo + per);
  int sum = 0;
#pragma unroll 8
  for (int g = lo; g < hi; ++g) sum += col[(int64_t)g * kMaxBins];
  red[warp][lane] = sum;
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    const int c = red[w][lane];
    at += w < warp ? c : 0;
    all += c;
  }
  if (warp == 0) col[(int64_t)groups * kMaxBins] = all;
  for (int g = lo; g < hi; g += U) {
    int c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) c[u] = g + u < hi ? col[(int64_t)(g + u) * kMaxBins] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g + u < hi) col[(int64_t)(g + u) * kMaxBins] = at;
      at += c[u];
    }
  }
}

// The sum of the values of the CTA's threads before this one.
__device__ __forceinline__ int sum_before(int v, int* red) {
  int inc = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, inc, o);
    if ((threadIdx.x & 31) >= o) inc += x;
  }
  if ((threadIdx.x & 31) == 31) red[threadIdx.x >> 5] = inc;
  __syncthreads();
  int at = inc - v;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) at += w < (int)(threadIdx.x >> 5) ? red[w] : 0;
  return at;
}

// A tile's keys and slots to their places by the digit at `shift`.  ALL: a single tile, every pass in this one CTA, which also
// counts.
template <bool ALL, int R>
__global__ void __launch_bounds__(kThreads) k_embed_place(const EmbedArgs a, EmbedSort s, const EmbedFill f, int bits, int shift, bool first) {
  pdl_enter();
  if (fill(f, s.tiles)) return;
  __shared__ uint16_t warp_count[kThreads / 32][kMaxBins];
  __shared__ int base[kMaxBins];
  __shared__ int red[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tile = blockIdx.x, bins = 1 << bits;
  if (ALL) {  // no launch before this one cleared the words that it and the next ones count in
    if (threadIdx.x == 0) *a.err = *s.n_long = 0;
    __syncthreads();
  }
  for (;;) {
    for (int i = lane; i < bins; i += 32) warp_count[warp][i] = 0;
    __syncwarp();
    int key[R], rank[R], own[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t i = place_of<R>(tile, r);
      key[r] = key_at(a, s, i, first);
      own[r] = first || i >= a.n ? (int)i : s.slot_in[i];
    }
    // keys of the thread's digit (bins <= kThreads): of all tiles, and of the tiles before this one; on their way meanwhile
    int all = 0, before = 0;
    if (!ALL && threadIdx.x < bins) {
      const int g0 = tile / kEmbedTiles, groups = (s.tiles + kEmbedTiles - 1) / kEmbedTiles;
      if (groups > kEmbedGroups) {
        all = s.sums[(int64_t)groups * kMaxBins + threadIdx.x];
        before = s.sums[(int64_t)g0 * kMaxBins + threadIdx.x];
      } else {
#pragma unroll 8
        for (int g = 0; g < groups; ++g) {
          const int c = s.sums[(int64_t)g * kMaxBins + threadIdx.x];
          all += c;
          before += g < g0 ? c : 0;
        }
      }
#pragma unroll 16
      for (int t = g0 * kEmbedTiles; t < tile; ++t) before += s.count[(int64_t)t * kMaxBins + threadIdx.x];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = place_of<R>(tile, r) < a.n;
      const int digit = (key[r] >> shift) & (bins - 1);
      const unsigned same = __match_any_sync(FULL, in ? digit : -1);
      const int ahead = warp_count[warp][digit];
      __syncwarp();
      rank[r] = ahead + __popc(same & ((1u << lane) - 1));
      if (in && lane == __ffs(same) - 1) warp_count[warp][digit] = (uint16_t)(ahead + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    // where each digit's keys of this tile begin: all smaller digits, then the tiles before this one
    if (threadIdx.x < bins) {
      int sum = 0;  // the warps' counts become each warp's start within the tile
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        const int c = warp_count[w][threadIdx.x];
        warp_count[w][threadIdx.x] = (uint16_t)sum;
        sum += c;
      }
      if (ALL) all = sum;
    }
    const int at = sum_before(all, red) + before;
    if (threadIdx.x < bins) base[threadIdx.x] = at;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t i = place_of<R>(tile, r);
      if (i >= a.n) continue;
      const int digit = (key[r] >> shift) & (bins - 1);
      const int to = base[digit] + warp_count[warp][digit] + rank[r];
      s.key_out[to] = key[r];
      s.slot_out[to] = own[r];
    }
    if (!ALL) return;
    __syncthreads();
    shift += bits;
    if (shift >= s.key_bits) break;
    first = false;
    s.key_in = s.key_out;
    s.slot_in = s.slot_out;
    s.key_out = s.key_in == s.keys[0] ? s.keys[1] : s.keys[0];
    s.slot_out = s.slot_in == s.slots[0] ? s.slots[1] : s.slots[0];
  }
}

// ------------------------------------------------------------------ the sums
// A chunk is kEmbedCap places of the sorted order.  Runs (the places of one id) of up to kEmbedCap places are summed by the chunk
// in which they begin, also past its end; each chunk sums its part of a longer run into a partial row: 2 c for the run that its
// first place is in, 2 c + 1 for one that begins later.  So a group of threads goes through a chunk's rows of dy at a stretch,
// eight of them in flight whatever ids they are of, and stores a sum where the id changes.  (131072 rows of 512 bf16, read from where the
// sort sends it: 35 us with 67 MB of the table's gradient cleared beside, 0.85 of a copy's rate; chunks of 16 or 64 places 4 to 8 us more,
// rows by way of shared memory 4 more.)
// A thread takes P pieces of E columns each, G E columns apart: 16 bytes where rows are whole pieces of that, else pairs of bf16, or two
// fp32, or a single bf16 where rows are odd.  (65536 slots of 511 columns, V = 32768: fp32 67 us, by one value 80; bf16 92, by two 98,
// and 193 by eight, whose stores alone fill the instruction cache; 8192 of 201: 32, 39 and 79.  1000 of 100 bf16: 14 in pairs.)
template <int BYTES> struct Bits;
template <> struct Bits<16> { using type = uint4; };
template <> struct Bits<4> { using type = uint32_t; };
template <> struct Bits<2> { using type = uint16_t; };
template <typename T, int E>
using Piece = typename Bits<E * sizeof(T)>::type;
template <typename T, int E>
__device__ __forceinline__ float value(const Piece<T, E>& w, int j) {
  uint32_t q;
  if constexpr (sizeof(w) == 16) q = (&w.x)[sizeof(T) == 2 ? j / 2 : j];
  else q = w;
  if (sizeof(T) == 4) return __uint_as_float(q);
  return j & 1 ? bf_hi(q) : bf_lo(q);
}

// The rows of the ids without a slot, kThreads of them a CTA: which of them occur is read from the sorted keys between the first
// and the last of them, up to kScan places; among more each is looked for (500000 places of 1000
// ids, a few of them most: the whole gradient 74 us, 203 by reading all).
constexpr int kScan = 16384;
__device__ void clear_rows(const EmbedArgs& a, const int* key, int64_t v0) {
  __shared__ int64_t bound[2];
  __shared__ unsigned there[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kThreads / 32) there[threadIdx.x] = 0;
  if (warp < 2) {  // the first place of a key >= v, 32 places looked at at a time
    const int64_t v = min(v0 + warp * kThreads, (int64_t)a.V);
    int64_t lo = 0, hi = a.n;  // it is in [lo, hi]
    while (lo < hi) {
      const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
      const unsigned m = __ballot_sync(FULL, i < hi && key[i] < v);  // a prefix of the lanes
      const int k = __popc(m);
      const int64_t l = lo;
      lo = k ? l + (k - 1) * step + 1 : l;
      hi = min(hi, l + k * step);
    }
    if (lane == 0) bound[warp] = lo;
  }
  __syncthreads();
  if (bound[1] - bound[0] > kScan) {  // (frequent ids) a thread looks for its own, three places at a time
    const int64_t v = v0 + threadIdx.x;
    int64_t lo = bound[0], hi = bound[1];  // the first place of a key >= v is in [lo, hi]
    while (lo < hi) {
      const int64_t q = (hi - lo + 3) / 4, p0 = lo + q - 1, p1 = min(p0 + q, hi - 1), p2 = min(p0 + 2 * q, hi - 1);
      const int k0 = key[p0], k1 = key[p1], k2 = key[p2];
      if (k0 >= v) hi = p0;
      else if (k1 >= v) lo = p0 + 1, hi = p1;
      else if (k2 >= v) lo = p1 + 1, hi = p2;
      else lo = p2 + 1;
    }
    const unsigned m = __ballot_sync(FULL, lo < bound[1] && key[lo] == v);
    if (lane == 0) there[warp] = m;
  } else {  // four keys a load, four loads on their way
    for (int64_t i0 = (bound[0] & ~(int64_t)3) + threadIdx.x * 4; i0 < bound[1]; i0 += kThreads * 16) {
      int4 k[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * kThreads * 4;
        k[u] = i < bound[1] ? *reinterpret_cast<const int4*>(key + i) : make_int4(-1, -1, -1, -1);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * kThreads * 4;
        const int q[4] = {k[u].x, k[u].y, k[u].z, k[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (i + j < bound[0] || i + j >= bound[1]) continue;
          const int r = q[j] - (int)v0;
          if (!(reinterpret_cast<volatile unsigned*>(there)[r >> 5] >> (r & 31) & 1)) atomicOr(&there[r >> 5], 1u << (r & 31));
        }
      }
    }
  }
  __syncthreads();
  const bool wide = a.d % 4 == 0 && reinterpret_cast<uintptr_t>(a.dtable) % 16 == 0;
  for (unsigned m = ~there[warp]; m; m &= m - 1) {
    const int64_t v = v0 + warp * 32 + __ffs(m) - 1;
    if (v >= a.V) break;
    float* out = a.dtable + v * a.d;
    if (wide)
      for (int c = lane * 4; c < a.d; c += 128) *reinterpret_cast<float4*>(out + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    else
      for (int c = lane; c < a.d; c += 32) out[c] = 0.f;
  }
}

// Groups of G threads, G E P columns of a chunk each: the first `chunk_ctas` CTAs; the others, if any, clear the rows of the ids without
// a slot.
template <typename T, int G, int E, int P>
__global__ void __launch_bounds__(kThreads, 4) k_embed_rows(const EmbedArgs a, const EmbedSort s, int blocks, int chunk_ctas) {
  pdl_enter();
  if ((int)blockIdx.x >= chunk_ctas) {
    clear_rows(a, s.key_out, ((int64_t)blockIdx.x - chunk_ctas) * kThreads);
    return;
  }
  using W = Piece<T, E>;
  constexpr int C = kEmbedCap;
  constexpr int U = 8;  // rows in flight (16 of short rows, in half as many CTAs: 168 us against 152 for 1000000 slots of 32 columns)
  // the keys from C places before the chunk to C behind it, and the slots from its first place on
  __shared__ __align__(16) int keys[kThreads / G][3 * C];
  __shared__ __align__(16) int slots[kThreads / G][2 * C];
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const unsigned team = G == 32 ? FULL : ((1u << (G & 31)) - 1) << (threadIdx.x & 31 & ~(G - 1));
  const int64_t task = (int64_t)blockIdx.x * (kThreads / G) + grp;
  const int64_t chunk = task / blocks;
  const int block = (int)(task - chunk * blocks), c = block * (G * E * P) + t * E;
  const int64_t lo = chunk * C;
  if (lo >= a.n) return;
  int *key = keys[grp] + C, *slot = slots[grp];  // by place - lo
  const int len = (int)min((int64_t)C, a.n - lo);
  // four at a time (chunks begin at multiples of 4, the arrays' ends are padded); before the first place -1, behind the last one the most
#pragma unroll
  for (int q = t; q < 3 * C / 4; q += G) {
    const int64_t i = lo - C + 4 * q;
    int4 k = make_int4(-1, -1, -1, -1);
    if (i >= 0) {
      const int4 none = make_int4(0x7fffffff, 0x7fffffff, 0x7fffffff, 0x7fffffff);
      k = i < a.n ? *reinterpret_cast<const int4*>(s.key_out + i) : none;
      if (i + 1 >= a.n) k.y = none.y;
      if (i + 2 >= a.n) k.z = none.z;
      if (i + 3 >= a.n) k.w = none.w;
    }
    *reinterpret_cast<int4*>(keys[grp] + 4 * q) = k;
    if (4 * q >= C && i < a.n) *reinterpret_cast<int4*>(slot + 4 * q - C) = *reinterpret_cast<const int4*>(s.slot_out + i);
  }
  __syncwarp(team);
  const int k0 = key[0], k1 = key[len - 1];
  if (k0 >= a.V) return;  // sorted last: slots without an id, nothing else
  // the places nearest to the chunk's first and last one that have another key than it, before and behind
  int b0 = -C - 1, f0 = 2 * C, b1 = -1, f1 = 2 * C;
  if (G >= 16) {
#pragma unroll
    for (int j = t - C; j < 2 * C; j += G) {
      const int k = key[j];
      if (j < 0 && k != k0) b0 = max(b0, j);
      if (j > 0 && k != k0) f0 = min(f0, j);
      if (j >= 0 && j < len && k != k1) b1 = max(b1, j);
      if (j >= len && k != k1) f1 = min(f1, j);
    }
#pragma unroll
    for (int o = G / 2; o; o >>= 1) {
      b0 = max(b0, __shfl_xor_sync(team, b0, o));
      f0 = min(f0, __shfl_xor_sync(team, f0, o));
      b1 = max(b1, __shfl_xor_sync(team, b1, o));
      f1 = min(f1, __shfl_xor_sync(team, f1, o));
    }
  } else {  // by halving, every thread the same: each is in [lower, upper] (1000000 slots of 32 columns:
           // 116 us, 123 by reading all keys)
    int l0 = -C, u0 = 0, l1 = 1, u1 = 2 * C, l2 = 0, u2 = len - 1, l3 = len, u3 = 2 * C;
    auto halve = [&](int& l, int& u, int k) {  // the first place of a key >= k
      if (l >= u) return;
      const int m = (l + u) >> 1;
      if (key[m] >= k) u = m;
      else l = m + 1;
    };
#pragma unroll
    for (int step = 0; step < 7; ++step) {  // (2 C <= 2^6)
      halve(l0, u0, k0);
      halve(l1, u1, k0 + 1);
      halve(l2, u2, k1);
      halve(l3, u3, k1 + 1);
    }
    b0 = l0 - 1, f0 = l1, b1 = l2 - 1, f1 = l3;
  }
  // the first run is the places (b0, f0), the last one (b1, f1), as far as they are looked at: C before and behind
  const bool long0 = f0 - b0 - 1 > C, same = b1 < 0, long1 = k1 < a.V && (same ? long0 : f1 - b1 - 1 > C);
  int from = 0, to = len;
  if (!long0 && b0 != -1) from = f0;  // another chunk's
  if (!long1) {
    if (k1 < a.V) {
      to = f1;
    } else {  // the ids end in this chunk
      to = 0;
      while (key[to] < a.V) ++to;
    }
  }
  const int l1 = long0 ? min(f0, len) : 0, m0 = long1 && !same ? b1 + 1 : 0x7fffffff;  // of long runs: places below l1 and from m0 on
  if (block == 0 && t == 0) {  // a long run's first chunk lists it, its last one says so
    if (long0 && b0 == -1) s.longs[atomicAdd(s.n_long, 1)] = make_int2(k0, (int)(2 * chunk));
    if (m0 < len) s.longs[atomicAdd(s.n_long, 1)] = make_int2(k1, (int)(2 * chunk + 1));
    if (long0 && f0 <= len) s.last[k0] = (int)(2 * chunk);
  }
  // where the sum that ends at a place goes: -1 on to the next place, -2, -3 the chunk's partial rows, else the id's row.  In place of the
  // keys, from the first of them on
  int* dest = key - C;
  int d[2 * C / G];
#pragma unroll
  for (int q = 0; q < 2 * C / G; ++q) {
    const int j = t + q * G, k = key[j];
    const bool ends = j >= from && j < to && (j == to - 1 || key[j + 1] != k);
    d[q] = !ends ? -1 : j < l1 ? -2 : j >= m0 ? -3 : k;
  }
  __syncwarp(team);  // (all have read the keys)
#pragma unroll
  for (int q = 0; q < 2 * C / G; ++q) dest[t + q * G] = d[q];
  __syncwarp(team);
  const T* dy = static_cast<const T*>(a.dy);
  float acc[P][E];
  auto clear = [&] {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < E; ++j) acc[p][j] = 0.f;
  };
  clear();
  for (int i = from; i < to; i += U) {
    W w[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* at = dy + (i + u < to ? (int64_t)slot[i + u] * a.d : 0) + c;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        w[u][p] = W{};
        if (i + u < to && c + p * G * E < a.d) w[u][p] = __ldcs(reinterpret_cast<const W*>(at + p * G * E));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= to) continue;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < E; ++j) acc[p][j] += value<T, E>(w[u][p], j);
      const int k = dest[i + u];
      if (k == -1) continue;
      const float scale = k < 0 ? 1.f : a.scale;
      float* out = (k < 0 ? s.part + (2 * chunk - 2 - k) * a.d : a.dtable + (int64_t)k * a.d) + c;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (c + p * G * E >= a.d) continue;
        float* o = out + p * G * E;
        if constexpr (E % 4 == 0) {
#pragma unroll
          for (int j = 0; j < E; j += 4)
            *reinterpret_cast<float4*>(o + j) = make_float4(acc[p][j] * scale, acc[p][j + 1] * scale, acc[p][j + 2] * scale, acc[p][j + 3] * scale);
        } else if constexpr (E == 2) {
          *reinterpret_cast<float2*>(o) = make_float2(acc[p][0] * scale, acc[p][1] * scale);
        } else {
          *o = acc[p][0] * scale;
        }
      }
      clear();
    }
  }
}

// hi + lo + v, in two words again (64-bit additions have a hundredth of fp32's rate: 35 us for what takes 6)
__device__ __forceinline__ void add2(float& hi, float& lo, float v) {
  const float s = __fadd_rn(hi, v), b = __fadd_rn(s, -hi);
  lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -b)), __fadd_rn(v, -b)));
  hi = s;
}
// The value of two words: of an infinite (or no) number the upper one, as lo is NaN then.
__device__ __forceinline__ float sum2(float hi, float lo) { return fabsf(hi) <= 3.402823466e38f ? hi + lo : hi; }

// The ids of long runs, 32 columns of one (128 where rows are whole pieces of 16 bytes) a task: their partial rows are added in two
// words, by a warp in order, or, of more than kWarpRows, by the CTA's warps each every eighth row.  Bound by
// latency: 6 us for the ids of 131072 slots that have more than 32 each.
constexpr int kWarpRows = 24;
template <int C>
struct Join {
  float hi[C], lo[C];
  // rows p, p + step .. of up to last, of those below `first` that one
  __device__ __forceinline__ void add(const float* part, int d, int p, int step, int first, int last) {
    constexpr int U = 8;  // in flight
#pragma unroll
    for (int j = 0; j < C; ++j) hi[j] = lo[j] = 0.f;
    for (; p <= last; p += U * step) {
      float v[U][C];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = max(p + u * step, first);
        const float* at = part + (int64_t)r * d;
        if (C == 4) {
          const float4 q = r <= last ? *reinterpret_cast<const float4*>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[u][C > 3 ? 3 : 0] = q.w; v[u][C > 2 ? 2 : 0] = q.z; v[u][C > 1 ? 1 : 0] = q.y; v[u][0] = q.x;
        } else {
          v[u][0] = r <= last ? *at : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p + u * step > last) break;
#pragma unroll
        for (int j = 0; j < C; ++j) add2(hi[j], lo[j], v[u][j]);
      }
    }
  }
};
template <int C>
__global__ void __launch_bounds__(kThreads) k_embed_join(const EmbedArgs a, const EmbedSort s) {
  pdl_enter();
  constexpr int W = kThreads / 32;
  __shared__ float2 red[W][32 * C];
  __shared__ int2 big[W];  // the warps' tasks that are the CTA's: the run, its first column
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, blocks = (a.d + 32 * C - 1) / (32 * C);
  const int n_long = *s.n_long;
  const int64_t tasks = (int64_t)n_long * blocks;
  for (int64_t t0 = (int64_t)blockIdx.x * W; t0 < tasks; t0 += (int64_t)gridDim.x * W) {
    const int64_t task = t0 + warp;
    Join<C> sum;
    int n_rows = 0;
    if (task < tasks) {
      // (one id's columns go to different CTAs: a frequent one's are long tasks)
      const int b = (int)(task / n_long), which = (int)(task - (int64_t)b * n_long), c0 = b * 32 * C, c = c0 + lane * C;
      const int2 run = s.longs[which];  // the id, and its first partial row: maybe the odd one of its chunk, then each chunk's even one
      const int last = s.last[run.x], first = (run.y | 1) - 1;
      n_rows = (last - first) / 2 + 1;
      if (n_rows > kWarpRows) {
        if (lane == 0) big[warp] = make_int2(which, c0);
      } else if (c < a.d) {
        sum.add(s.part + c, a.d, first, 2, run.y, last);
        float* out = a.dtable + (int64_t)run.x * a.d + c;
#pragma unroll
        for (int j = 0; j < C; ++j) out[j] = sum2(sum.hi[j], sum.lo[j]) * a.scale;
      }
    }
    if (!__syncthreads_or(n_rows > kWarpRows)) continue;
    // (each warp's own answer, known to all)
    if (lane == 0 && n_rows <= kWarpRows) big[warp] = make_int2(-1, 0);
    __syncthreads();
    for (int k = 0; k < W; ++k) {
      const int2 it = big[k];
      if (it.x < 0) continue;
      const int2 run = s.longs[it.x];
      const int c = it.y + lane * C;
      if (c < a.d) {
        sum.add(s.part + c, a.d, (run.y | 1) - 1 + 2 * warp, 2 * W, run.y, s.last[run.x]);
#pragma unroll
        for (int j = 0; j < C; ++j) red[warp][lane * C + j] = make_float2(sum.hi[j], sum.lo[j]);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 32 * C; i += kThreads) {
        if (it.y + i >= a.d) continue;
        float h = red[0][i].x, l = red[0][i].y;
#pragma unroll
        for (int w = 1; w < W; ++w) {
          add2(h, l, red[w][i].x);
          l += red[w][i].y;
        }
        a.dtable[(int64_t)run.x * a.d + it.y + i] = sum2(h, l) * a.scale;
      }
      __syncthreads();
    }
    __syncthreads();  // all have read `big` to its end (entries of -1 pass no barrier) before the next turn writes it
  }
}

template <typename T, int E, int P>
cudaError_t rows(const EmbedArgs& a, const EmbedSort& s, cudaStream_t st) {
  const int64_t chunks = (a.n + kEmbedCap - 1) / kEmbedCap, clear = embed_fills(a) ? 0 : ((int64_t)a.V + kThreads - 1) / kThreads;
  auto go = [&](auto kernel, int G) {
    const int blocks = (a.d + G * E * P - 1) / (G * E * P), per = kThreads / G;
    const int64_t ctas = (chunks * blocks + per - 1) / per;
    return launch_pdl(kernel, dim3((unsigned)(ctas + clear)), dim3(kThreads), 0, st, a, s, blocks, (int)ctas);
  };
  const int v = (a.d + E * P - 1) / (E * P);
  return v <= 4 ? go(k_embed_rows<T, 4, E, P>, 4) : v <= 8 ? go(k_embed_rows<T, 8, E, P>, 8)
         : v <= 16 ? go(k_embed_rows<T, 16, E, P>, 16) : go(k_embed_rows<T, 32, E, P>, 32);
}

__global__ void __launch_bounds__(kThreads) k_zero(uint4* p, int64_t n) {
  pdl_enter();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) p[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace

// Up to so many ids one more CTA of the forward checks them, 32 a thread, while the others copy (a launch that clears the error word
// is 1 us on the device and 2 on the host); of more, each reports what it finds.
constexpr int64_t kCheckIds = 8192;
bool embed_fwd_clears(const EmbedArgs& a) { return a.n <= kCheckIds; }

cudaError_t launch_embed_fwd(const EmbedArgs& a, bool f32, cudaStream_t st) {
  const int es = f32 ? 4 : 2, E = 16 / es;
  const uintptr_t tab = reinterpret_cast<uintptr_t>(a.table), y = reinterpret_cast<uintptr_t>(a.y);
  const bool finite = std::fabs(a.scale) <= 3.402823466e38f;
  const EmbedRows m = !finite ? SINGLE : ((uintptr_t)a.d * es | tab | y) % 16 == 0 ? ROWS : y % 16 ? SINGLE : !f32 && a.d % 2 == 0 && tab % 4 == 0 ? PAIRS : VALUES;
  const int cols = m == ROWS ? a.d / E : a.d;
  // about four accesses a thread; of pieces also 16 slots' at least
  const int per = m == ROWS || m == SINGLE ? std::max(1, 1024 / cols) : std::min(1024, std::max(1, 1024 / a.d) * E);
  // i / cols = the high word of i ceil(2^32 / cols) for i cols < 2^32: here i < per cols
  const uint32_t by = cols == 1 || (int64_t)per * cols * cols >> 32 ? 0 : (uint32_t)((0x100000000ull + cols - 1) / cols);
  const bool check = embed_fwd_clears(a);
  const dim3 grid((unsigned)((a.n + per - 1) / per + (check ? 1 : 0)));
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kThreads), 0, st, a, per, cols, by, check); };
  if (f32) return go(m == ROWS ? k_embed_fwd<float, ROWS> : m == VALUES ? k_embed_fwd<float, VALUES> : k_embed_fwd<float, SINGLE>);
  return go(m == ROWS ? k_embed_fwd<bf16, ROWS> : m == PAIRS ? k_embed_fwd<bf16, PAIRS> : m == VALUES ? k_embed_fwd<bf16, VALUES> : k_embed_fwd<bf16, SINGLE>);
}

// Share `i` of `n` of the gradient's values, from a multiple of 4 on.
EmbedFill embed_fill(const EmbedArgs& a, int i, int n) {
  const int64_t all = embed_fills(a) ? (int64_t)a.V * a.d : 0;
  auto cut = [&](int k) { return k == n ? all : all / n * k / 4 * 4; };
  return EmbedFill{a.dtable, cut(i), cut(i + 1), reinterpret_cast<uintptr_t>(a.dtable) % 16 == 0};
}
unsigned fill_ctas(const EmbedFill& f) { return (unsigned)((f.hi - f.lo + kFill - 1) / kFill); }

cudaError_t launch_embed_count(const EmbedArgs& a, const EmbedSort& s, const EmbedFill& f, int bits, int shift, cudaStream_t st) {
  return launch_pdl(k_embed_count, dim3((unsigned)s.tiles + fill_ctas(f)), dim3(kThreads), 0, st, a, s, f, 1 << bits, shift, shift == 0);
}
cudaError_t launch_embed_scan(const EmbedSort& s, cudaStream_t st) {
  const int groups = (s.tiles + kEmbedTiles - 1) / kEmbedTiles;
  return launch_pdl(k_embed_scan, dim3(kMaxBins / 32), dim3(1024), 0, st, s.sums, groups);
}
cudaError_t launch_embed_place(const EmbedArgs& a, const EmbedSort& s, const EmbedFill& f, int bits, int shift, cudaStream_t st) {
  const dim3 grid((unsigned)s.tiles + fill_ctas(f));
  if (s.tiles == 1)  // (rounds without keys cost time, too: 1023 keys 14.0 us in 4 rounds a pass, 16.6 in 8)
    return launch_pdl(a.n <= kEmbedOne / 2 ? k_embed_place<true, kEmbedOne / 2 / kThreads> : k_embed_place<true, kEmbedOne / kThreads>, grid,
                      dim3(kThreads), 0, st, a, s, f, bits, 0, true);
  return launch_pdl(k_embed_place<false, kRounds>, grid, dim3(kThreads), 0, st, a, s, f, bits, shift, shift == 0);
}
cudaError_t launch_embed_rows(const EmbedArgs& a, const EmbedSort& s, bool f32, cudaStream_t st) {
  const size_t es = f32 ? 4 : 2;
  const uintptr_t dy = reinterpret_cast<uintptr_t>(a.dy), out = reinterpret_cast<uintptr_t>(a.dtable);
  const bool wide = ((uintptr_t)(a.d * es) | (uintptr_t)a.d * 4 | dy | out) % 16 == 0;
  if (f32) return wide ? rows<float, 4, 1>(a, s, st) : rows<float, 1, 2>(a, s, st);
  if (wide) return rows<bf16, 8, 1>(a, s, st);
  return a.d % 2 == 0 && dy % 4 == 0 && out % 8 == 0 ? rows<bf16, 2, 1>(a, s, st) : rows<bf16, 1, 1>(a, s, st);
}
cudaError_t launch_embed_join(const EmbedArgs& a, const EmbedSort& s, cudaStream_t st) {
  const int C = a.d % 4 == 0 ? 4 : 1;  // (the partial rows are in the workspace: aligned)
  // at most one long run in more than kEmbedCap places
  const int64_t most = (a.n / (kEmbedCap + 1) * ((a.d + 32 * C - 1) / (32 * C)) + 7) / 8;
  return launch_pdl(C == 4 ? k_embed_join<4> : k_embed_join<1>, dim3((unsigned)std::min<int64_t>(most, sm_count() * 4)), dim3(kThreads), 0,
                    st, a, s);
}
cudaError_t launch_zero(void* p, size_t bytes, cudaStream_t st) {
  const int64_t n = (int64_t)(bytes / 16);
  return launch_pdl(k_zero, dim3((unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, sm_count() * 8)), dim3(kThreads), 0, st,
                    static_cast<uint4*>(p), n);
}

}  // namespace gbla
