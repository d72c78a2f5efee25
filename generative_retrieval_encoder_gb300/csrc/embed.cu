// Token embedding: rows of a table by ids, k of them a token side by side, and the table's gradient.
//   y[slot] = scale table[ids[slot]],   dtable[v] = scale * sum of dy[slot] over the slots with ids[slot] = v
// (slot = token k + which of its ids; an id below 0, or of a row that is in no sequence, has a row of zeros and no gradient).
//
// The gradient goes by sorted slots, so that each row of the table is written once, in one fixed order of its slots: a stable
// counting sort by the id's digits (no CTA waits for another: a tile's place among its digit's keys comes from the counts of
// the tiles before it), each id's range in the sorted order, then the sums, kEmbedCap sorted places a group of threads.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace gbla {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kMaxBins = 1 << kEmbedDigit;

// The id of a slot, -1 for none.  An id past the table or a length outside [0, L] sets the error word and counts as none.
__device__ __forceinline__ int id_of(const EmbedArgs& a, int64_t slot) {
  const int64_t id = a.wide_ids ? static_cast<const int64_t*>(a.ids)[slot] : (int64_t)static_cast<const int32_t*>(a.ids)[slot];
  if (a.lens) {
    const int row = (int)slot / a.k, b = row / a.L, len = a.lens[b];
    if (len < 0 || len > a.L) {
      atomicOr(a.err, 1);
      return -1;
    }
    if (row - b * a.L >= len) return -1;
  }
  if (id >= a.V) {
    atomicOr(a.err, 1);
    return -1;
  }
  return id < 0 ? -1 : (int)id;
}

template <typename T>
__device__ __forceinline__ uint4 scaled(uint4 w, float s) {
  if (sizeof(T) == 2)
    return make_uint4(pack_bf16(bf_lo(w.x) * s, bf_hi(w.x) * s), pack_bf16(bf_lo(w.y) * s, bf_hi(w.y) * s),
                      pack_bf16(bf_lo(w.z) * s, bf_hi(w.z) * s), pack_bf16(bf_lo(w.w) * s, bf_hi(w.w) * s));
  return make_uint4(__float_as_uint(__uint_as_float(w.x) * s), __float_as_uint(__uint_as_float(w.y) * s),
                    __float_as_uint(__uint_as_float(w.z) * s), __float_as_uint(__uint_as_float(w.w) * s));
}

// A CTA takes `per` slots: their ids once, then the rows as one run of `cols` accesses each (16 bytes where WIDE, one value
// else), four in flight a thread.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_embed_fwd(const EmbedArgs a, int per, int cols, uint32_t by_cols) {
  pdl_enter();
  __shared__ int id[1024];
  if (gridDim.x == 1) {  // nobody else has an error to report
    if (threadIdx.x == 0) *a.err = 0;
    __syncthreads();
  }
  const int64_t s0 = (int64_t)blockIdx.x * per;
  const int ns = (int)min((int64_t)per, a.n - s0);
  for (int i = threadIdx.x; i < ns; i += kThreads) id[i] = id_of(a, s0 + i);
  __syncthreads();
  const T* tab = static_cast<const T*>(a.table);
  T* y = static_cast<T*>(a.y) + s0 * a.d;
  constexpr int E = WIDE ? 16 / sizeof(T) : 1;
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
      if (WIDE) v[u] = __ldg(reinterpret_cast<const uint4*>(tab + (int64_t)k * a.d) + c);
      else f[u] = to_f(tab[(int64_t)k * a.d + c]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + u * kThreads;
      if (i >= total) continue;
      if (WIDE) reinterpret_cast<uint4*>(y)[i] = scaled<T>(v[u], a.scale);
      else y[i] = from_f<T>(f[u] * a.scale);
    }
  }
}

// ------------------------------------------------------------------ the sort
// A tile's keys: a warp takes kEmbedTile / 8 consecutive ones, 32 a round.
constexpr int kRounds = kEmbedTile / kThreads;
__device__ __forceinline__ int64_t place_of(int tile, int round) {
  return (int64_t)tile * kEmbedTile + (threadIdx.x >> 5) * (kRounds * 32) + round * 32 + (threadIdx.x & 31);
}
// The key at a place of the pass's input: an id, V for none (last of all), V too past the end.
__device__ __forceinline__ int key_at(const EmbedArgs& a, const EmbedSort& s, int64_t i, bool first) {
  if (i >= a.n) return a.V;
  if (!first) return s.key_in[i];
  const int id = id_of(a, i);
  return id < 0 ? a.V : id;
}

// Each tile's keys by digit, and the sums of kEmbedTiles tiles.
__global__ void __launch_bounds__(kThreads) k_embed_count(const EmbedArgs a, const EmbedSort s, int bins, int shift, bool first) {
  pdl_enter();
  __shared__ int count[kMaxBins];
  for (int i = threadIdx.x; i < bins; i += kThreads) count[i] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = place_of(blockIdx.x, r);
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

// Exclusive sums over `bins` values of smem by the CTA, `v` in place.
__device__ __forceinline__ void scan_bins(int* v, int bins, int* red) {
  constexpr int P = (kMaxBins + kThreads - 1) / kThreads;
  int own[P], sum = 0;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int i = threadIdx.x * P + j;
    own[j] = i < bins ? v[i] : 0;
    sum += own[j];
  }
  int inc = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, inc, o);
    if ((threadIdx.x & 31) >= o) inc += x;
  }
  if ((threadIdx.x & 31) == 31) red[threadIdx.x >> 5] = inc;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < (int)(threadIdx.x >> 5); ++w) at += red[w];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int i = threadIdx.x * P + j;
    if (i < bins) v[i] = at;
    at += own[j];
  }
  __syncthreads();
}

// The sorted places' boundaries: range[v] = (first place of v, the one behind its last).
__device__ __forceinline__ void mark(const EmbedArgs& a, const int* key, int2* range, int64_t i) {
  const int k = key[i], before = i > 0 ? key[i - 1] : -1;
  if (k == before) return;
  if (k < a.V) range[k].x = (int)i;
  if (before >= 0) range[before].y = (int)i;
}

// A tile's keys and slots to their places by the digit at `shift`.  ALL: a single tile, every pass in this one CTA, which also
// counts, and marks the ranges.
template <bool ALL>
__global__ void __launch_bounds__(kThreads) k_embed_place(const EmbedArgs a, EmbedSort s, int bits, int shift, bool first) {
  pdl_enter();
  __shared__ uint16_t warp_count[kThreads / 32][kMaxBins];
  __shared__ int base[kMaxBins];
  __shared__ int red[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tile = blockIdx.x, bins = 1 << bits;
  for (;;) {
    for (int i = lane; i < bins; i += 32) warp_count[warp][i] = 0;
    __syncwarp();
    int key[kRounds], rank[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int64_t i = place_of(tile, r);
      key[r] = key_at(a, s, i, first);
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const bool in = place_of(tile, r) < a.n;
      const int digit = (key[r] >> shift) & (bins - 1);
      const unsigned same = __match_any_sync(FULL, in ? digit : -1);
      const int before = warp_count[warp][digit];
      __syncwarp();
      rank[r] = before + __popc(same & ((1u << lane) - 1));
      if (in && lane == __ffs(same) - 1) warp_count[warp][digit] = (uint16_t)(before + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    // where each digit's keys of this tile begin: all smaller digits, then the tiles before this one
    for (int i = threadIdx.x; i < bins; i += kThreads) {
      int sum = 0;  // the warps' counts become each warp's start within the tile
      for (int w = 0; w < kThreads / 32; ++w) {
        const int c = warp_count[w][i];
        warp_count[w][i] = (uint16_t)sum;
        sum += c;
      }
      if (!ALL) {
        const int groups = (s.tiles + kEmbedTiles - 1) / kEmbedTiles;
        sum = 0;
#pragma unroll 8
        for (int g = 0; g < groups; ++g) sum += s.sums[(int64_t)g * kMaxBins + i];
      }
      base[i] = sum;
    }
    __syncthreads();
    scan_bins(base, bins, red);
    if (!ALL) {
      for (int i = threadIdx.x; i < bins; i += kThreads) {
        const int g0 = tile / kEmbedTiles;
        int sum = base[i];
#pragma unroll 4
        for (int g = 0; g < g0; ++g) sum += s.sums[(int64_t)g * kMaxBins + i];
#pragma unroll 16
        for (int t = g0 * kEmbedTiles; t < tile; ++t) sum += s.count[(int64_t)t * kMaxBins + i];
        base[i] = sum;
      }
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int64_t i = place_of(tile, r);
      if (i >= a.n) continue;
      const int digit = (key[r] >> shift) & (bins - 1);
      const int to = base[digit] + warp_count[warp][digit] + rank[r];
      s.key_out[to] = key[r];
      s.slot_out[to] = first ? (int)i : s.slot_in[i];
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
  for (int64_t i = threadIdx.x; i <= a.n; i += kThreads) {
    if (i < a.n) mark(a, s.key_out, s.range, i);
    else if (s.key_out[i - 1] < a.V) s.range[s.key_out[i - 1]].y = (int)i;
  }
}

__global__ void __launch_bounds__(kThreads) k_embed_mark(const EmbedArgs a, const int* key, int2* range) {
  pdl_enter();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < a.n) mark(a, key, range, i);
  if (i == a.n - 1 && key[i] < a.V) range[key[i]].y = (int)a.n;
}

// ------------------------------------------------------------------ the sums
// A chunk is kEmbedCap places of the sorted order.  Runs (the places of one id) of up to kEmbedCap places are summed by the chunk
// in which they begin, also past its end; each chunk sums its part of a longer run into a partial row: 2 c for the run that its
// first place is in, 2 c + 1 for one that begins later.  So a group of threads goes through a chunk's rows of dy at a stretch,
// eight of them in flight whatever ids they are of, and stores a sum where the id changes.
template <typename T, bool WIDE>
struct Sum {
  static constexpr int E = 16 / sizeof(T);
  float v[E];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = 0.f;
  }
  __device__ __forceinline__ void store(float scale, float* out, int c, int d, int step) const {
    if (WIDE) {
      if (c >= d) return;
#pragma unroll
      for (int j = 0; j < E; j += 4)
        *reinterpret_cast<float4*>(out + c + j) = make_float4(v[j] * scale, v[j + 1] * scale, v[j + 2] * scale, v[j + 3] * scale);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (c + j * step < d) out[c + j * step] = v[j] * scale;
    }
  }
};

// Groups of G threads, G E columns each.  The first `chunk_ctas` CTAs take chunks, the others the rows of ids without a slot: a
// warp 32 table rows.
template <typename T, int G, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_embed_rows(const EmbedArgs a, const EmbedSort s, int blocks, int chunk_ctas) {
  pdl_enter();
  constexpr int E = 16 / sizeof(T), U = WIDE ? 8 : 2;
  if ((int)blockIdx.x >= chunk_ctas) {
    const int64_t v0 = (((int64_t)blockIdx.x - chunk_ctas) * (kThreads / 32) + (threadIdx.x >> 5)) * 32;
    const int lane = threadIdx.x & 31;
    bool none = false;
    if (v0 + lane < a.V) {
      const int2 r = s.range[v0 + lane];
      none = r.x == r.y;
    }
    for (unsigned m = __ballot_sync(FULL, none); m; m &= m - 1) {
      float* out = a.dtable + (v0 + __ffs(m) - 1) * a.d;
      if (a.d % 4 == 0 && reinterpret_cast<uintptr_t>(a.dtable) % 16 == 0)
        for (int c = lane * 4; c < a.d; c += 128) *reinterpret_cast<float4*>(out + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      else
        for (int c = lane; c < a.d; c += 32) out[c] = 0.f;
    }
    return;
  }
  const int t = threadIdx.x % G;
  const int64_t task = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
  const int64_t chunk = task / blocks;
  const int c = (int)(task - chunk * blocks) * G * E + (WIDE ? t * E : t);
  const int64_t lo = chunk * kEmbedCap;
  if (lo >= a.n) return;
  const int64_t hi = min(a.n, lo + kEmbedCap);
  const int *key = s.key_out, *slot = s.slot_out;
  const T* dy = static_cast<const T*>(a.dy);
  // the places to go through
  const int k0 = key[lo], k1 = key[hi - 1];
  int from = (int)lo, to = (int)hi;
  int l1 = (int)lo, m0 = 0x7fffffff;  // of long runs: places below l1 and from m0 on
  const int2 none = make_int2(0, 0), r0 = k0 < a.V ? s.range[k0] : none, r1 = k1 < a.V ? s.range[k1] : none;
  if (k0 >= a.V) return;  // sorted last: nothing but slots without an id
  if (r0.y - r0.x > kEmbedCap) l1 = min(r0.y, (int)hi);
  else if (r0.x < lo) from = r0.y;  // another chunk's
  if (k1 >= a.V) {
    // the ids end in this chunk: behind the last of them
    int x = (int)lo, y = (int)hi - 1;  // key[x] < V <= key[y]
    while (y - x > 1) {
      const int mid = (x + y) >> 1;
      if (key[mid] < a.V) x = mid; else y = mid;
    }
    to = y;
  } else if (r1.y - r1.x <= kEmbedCap) {
    to = r1.y;
  } else if (k1 != k0) {
    m0 = r1.x;
    if (t == 0 && c < G * E) {  // a long run's first chunk lists it
      const int at = atomicAdd(s.n_long, 1);
      s.longs[at] = make_int2(k1, (int)(2 * chunk + 1));
    }
  }
  if (l1 > lo && r0.x == lo && t == 0 && c < G * E) {
    const int at = atomicAdd(s.n_long, 1);
    s.longs[at] = make_int2(k0, (int)(2 * chunk));
  }
  Sum<T, WIDE> acc;
  acc.clear();
  int now = -1;
  auto flush = [&](int i) {  // the sum of the run whose last place is i - 1
    if (now < 0) return;
    if (i - 1 < l1) acc.store(1.f, s.part + 2 * chunk * a.d, c, a.d, G);
    else if (i - 1 >= m0) acc.store(1.f, s.part + (2 * chunk + 1) * a.d, c, a.d, G);
    else acc.store(a.scale, a.dtable + (int64_t)now * a.d, c, a.d, G);
  };
  for (int i = from; i < to; i += U) {
    int k[U], at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = i + u < to ? key[i + u] : -1;
      at[u] = i + u < to ? slot[i + u] : -1;
    }
    uint4 w[U];
    float f[U][WIDE ? 1 : E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (WIDE) {
        w[u] = make_uint4(0, 0, 0, 0);
        if (at[u] >= 0 && c < a.d) w[u] = __ldcs(reinterpret_cast<const uint4*>(dy + (int64_t)at[u] * a.d + c));
      } else {
#pragma unroll
        for (int j = 0; j < (WIDE ? 1 : E); ++j) f[u][j] = at[u] >= 0 && c + j * G < a.d ? to_f(dy[(int64_t)at[u] * a.d + c + j * G]) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k[u] < 0) continue;
      if (k[u] != now) {
        flush(i + u);
        now = k[u];
        acc.clear();
      }
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        acc.v[j] += !WIDE ? f[u][WIDE ? 0 : j] : sizeof(T) == 2 ? (j & 1 ? bf_hi(q[(j / 2) & 3]) : bf_lo(q[(j / 2) & 3])) : __uint_as_float(q[j & 3]);
      }
    }
  }
  flush(to);
}

// The ids of long runs: a CTA adds the partial rows of one, 32 columns, a warp every eighth of them, in 64 bits.
__global__ void __launch_bounds__(kThreads) k_embed_join(const EmbedArgs a, const EmbedSort s) {
  pdl_enter();
  __shared__ double red[kThreads / 32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, blocks = (a.d + 31) / 32;
  const int64_t tasks = (int64_t)*s.n_long * blocks;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int which = (int)(task / blocks), c = (int)(task - (int64_t)which * blocks) * 32 + lane;
    const int2 run = s.longs[which];
    const int64_t first = run.y, last = 2 * (int64_t)((s.range[run.x].y - 1) / kEmbedCap);
    double sum = 0.;
    if (c < a.d) {
      if (warp == 0) sum = s.part[first * a.d + c];
#pragma unroll 8
      for (int64_t p = (first | 1) + 1 + 2 * warp; p <= last; p += 2 * (kThreads / 32)) sum += s.part[p * a.d + c];
    }
    __syncthreads();
    red[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < a.d) {
      for (int w = 1; w < kThreads / 32; ++w) sum += red[w][lane];
      a.dtable[(int64_t)run.x * a.d + c] = (float)(sum * (double)a.scale);
    }
  }
}

template <typename T, bool WIDE>
cudaError_t rows(const EmbedArgs& a, const EmbedSort& s, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  const int64_t chunks = (a.n + kEmbedCap - 1) / kEmbedCap, empty = ((int64_t)a.V + kThreads - 1) / kThreads;
  auto go = [&](auto kernel, int G) {
    const int blocks = (a.d + G * E - 1) / (G * E), per = kThreads / G;
    const int64_t ctas = (chunks * blocks + per - 1) / per;
    return launch_pdl(kernel, dim3((unsigned)(ctas + empty)), dim3(kThreads), 0, st, a, s, blocks, (int)ctas);
  };
  const int v = (a.d + E - 1) / E;
  return v <= 4 ? go(k_embed_rows<T, 4, WIDE>, 4) : v <= 8 ? go(k_embed_rows<T, 8, WIDE>, 8)
         : v <= 16 ? go(k_embed_rows<T, 16, WIDE>, 16) : go(k_embed_rows<T, 32, WIDE>, 32);
}

__global__ void __launch_bounds__(kThreads) k_zero(uint4* p, int64_t n) {
  pdl_enter();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) p[i] = make_uint4(0, 0, 0, 0);
}

// Accesses a row of the forward takes: of 16 bytes where rows and tensors allow it, of one value else.
int row_cols(const EmbedArgs& a, bool f32, bool& wide) {
  const size_t es = f32 ? 4 : 2;
  wide = ((uintptr_t)(a.d * es) | reinterpret_cast<uintptr_t>(a.table) | reinterpret_cast<uintptr_t>(a.y)) % 16 == 0;
  return wide ? (int)(a.d * es / 16) : a.d;
}

}  // namespace

// Slots of a CTA of the forward, about four accesses a thread.
int embed_fwd_ctas(const EmbedArgs& a, bool f32) {
  bool wide;
  const int per = std::max(1, 1024 / row_cols(a, f32, wide));
  return (int)((a.n + per - 1) / per);
}

cudaError_t launch_embed_fwd(const EmbedArgs& a, bool f32, cudaStream_t st) {
  bool wide;
  const int cols = row_cols(a, f32, wide), per = std::max(1, 1024 / cols);
  // i / cols = the high word of i ceil(2^32 / cols) for i cols < 2^32: here i < 1024 and cols <= 1024
  const uint32_t by = cols == 1 ? 0 : (uint32_t)((0x100000000ull + cols - 1) / cols);
  const dim3 grid((unsigned)embed_fwd_ctas(a, f32));
  if (f32) return wide ? launch_pdl(k_embed_fwd<float, true>, grid, dim3(kThreads), 0, st, a, per, cols, by)
                       : launch_pdl(k_embed_fwd<float, false>, grid, dim3(kThreads), 0, st, a, per, cols, by);
  return wide ? launch_pdl(k_embed_fwd<bf16, true>, grid, dim3(kThreads), 0, st, a, per, cols, by)
              : launch_pdl(k_embed_fwd<bf16, false>, grid, dim3(kThreads), 0, st, a, per, cols, by);
}

cudaError_t launch_embed_count(const EmbedArgs& a, const EmbedSort& s, int bits, int shift, cudaStream_t st) {
  return launch_pdl(k_embed_count, dim3((unsigned)s.tiles), dim3(kThreads), 0, st, a, s, 1 << bits, shift, shift == 0);
}
cudaError_t launch_embed_place(const EmbedArgs& a, const EmbedSort& s, int bits, int shift, cudaStream_t st) {
  if (s.tiles == 1) return launch_pdl(k_embed_place<true>, dim3(1), dim3(kThreads), 0, st, a, s, bits, 0, true);
  return launch_pdl(k_embed_place<false>, dim3((unsigned)s.tiles), dim3(kThreads), 0, st, a, s, bits, shift, shift == 0);
}
cudaError_t launch_embed_mark(const EmbedArgs& a, const EmbedSort& s, cudaStream_t st) {
  return launch_pdl(k_embed_mark, dim3((unsigned)((a.n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, a, (const int*)s.key_out,
                    s.range);
}
cudaError_t launch_embed_rows(const EmbedArgs& a, const EmbedSort& s, bool f32, cudaStream_t st) {
  const size_t es = f32 ? 4 : 2;
  const bool wide = ((uintptr_t)(a.d * es) | (uintptr_t)a.d * 4 | reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.dtable)) % 16 == 0;
  if (f32) return wide ? rows<float, true>(a, s, st) : rows<float, false>(a, s, st);
  return wide ? rows<bf16, true>(a, s, st) : rows<bf16, false>(a, s, st);
}
cudaError_t launch_embed_join(const EmbedArgs& a, const EmbedSort& s, cudaStream_t st) {
  return launch_pdl(k_embed_join, dim3((unsigned)std::min<int64_t>((a.n + kEmbedCap - 1) / kEmbedCap * ((a.d + 31) / 32), sm_count() * 8)),
                    dim3(kThreads), 0, st, a, s);
}
cudaError_t launch_zero(void* p, size_t bytes, cudaStream_t st) {
  const int64_t n = (int64_t)(bytes / 16);
  return launch_pdl(k_zero, dim3((unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, sm_count() * 8)), dim3(kThreads), 0, st,
                    static_cast<uint4*>(p), n);
}

}  // namespace gbla
