// Layer norm between the blocks, with the residual stream's addition.
//   s = x + res (rounded to the io type, which is what is normed and kept),
//   m = mean s, r = 1 / sqrt(mean (s - m)^2 + eps), z = (s - m) r, y = z w + b
// and its backward, g = dy w:
//   dx = r (g - mean g - z mean(g z)) + ds,  dw = sum_rows dy z,  db = sum_rows dy.
//
// A group of G threads holds a row, N values each, so mean and squares are taken
// from registers (the squares about the mean itself: no cancellation) and every
// tensor is read once.  Rows longer than 8192 values go by CTA in passes over L2.
// Additions and products are of two values at a time: bf16 rows are otherwise bound
// by instructions (backward 91 us against 80 at 16 x 8192 rows of 512).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace gbla {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 256;

// Up to so many slots one CTA checks their lengths while the others work (a launch that clears the error word is 1 us on the device and
// 2 on the host); of more, the first row of each reports what it finds.
constexpr int kCheckSlots = 8192;

// Whether row `row` belongs to its sequence; a length outside [0, L] sets the error word and counts as 0.
__device__ __forceinline__ bool row_valid(const LnArgs& a, int64_t row) {
  if (!a.lens) return true;
  const int b = (int)row / a.L, len = a.lens[b];
  if (len < 0 || len > a.L) {
    if (a.slots > kCheckSlots && row == (int64_t)b * a.L) atomicOr(a.err, 1);
    return false;
  }
  return row - (int64_t)b * a.L < len;
}
// The error word.  With lengths to check that is the first CTA's only work (a.first = 1): it alone reports, and returns true.
__device__ __forceinline__ bool check_slots(const LnArgs& a) {
  if (blockIdx.x > 0 || a.slots > kCheckSlots) return false;
  int bad = 0;
  if (a.first) {
    for (int b = threadIdx.x; b < a.slots; b += kThreads) bad |= a.lens[b] < 0 || a.lens[b] > a.L;
    bad = __syncthreads_or(bad);
  }
  if (threadIdx.x == 0) *a.err = bad ? 1 : 0;
  return a.first;
}

// How a row's values lie with its threads.  SINGLE: one value an access.  PIECES: 16 bytes an access, rows begin at 16-byte boundaries.
// SHIFTED: the same of rows (bf16, of any number of values in 16-byte aligned tensors) that begin `off` values behind a boundary: the
// pieces are those of memory, what they hold of other rows is masked, and the ends of a row are stored value by value.
enum LnRows { SINGLE, PIECES, SHIFTED };
// The values that row `row` begins behind a 16-byte boundary.
template <typename T, LnRows M>
__device__ __forceinline__ int row_off(int64_t row, int d) {
  constexpr int E = 16 / sizeof(T);
  return M == SHIFTED ? ((int)row & (E - 1)) * (d & (E - 1)) & (E - 1) : 0;
}
// The column of value i of thread t in a row of G threads: pieces dealt out in turn, or single values.  Outside [0, d): none.
template <typename T, int G, LnRows M>
__device__ __forceinline__ int col_of(int i, int t, int off) {
  constexpr int E = 16 / sizeof(T);
  return M != SINGLE ? ((i / E) * G + t) * E + i % E - off : i * G + t;
}

// The thread's N values of a row as they lie in memory (0 outside the row): bf16 values stay two to a register until they are used.
template <typename T, int G, int N, LnRows M>
struct Row {
  static constexpr int E = 16 / sizeof(T);
  static constexpr bool WIDE = M != SINGLE;
  uint4 w[WIDE ? N / E : 1];
  float v[WIDE ? 1 : N];
  // The piece's values one by one, or by pairs.
  __device__ static __forceinline__ uint4 singles(const T* p, int c, int d) {
    uint32_t u[4] = {0, 0, 0, 0};
    if (d % 2 == 0 && reinterpret_cast<uintptr_t>(p) % 4 == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((unsigned)(c + 2 * j) < (unsigned)d) u[j] = *reinterpret_cast<const uint32_t*>(p + c + 2 * j);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((unsigned)(c + j) < (unsigned)d) u[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[c + j] << (j & 1 ? 16 : 0);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void load(const T* p, int t, int d) {  // (SHIFTED rows come by way of shared memory)
    if (WIDE) {
#pragma unroll
      for (int i = 0; i < N / E; ++i) {
        const int c = (i * G + t) * E;
        w[i] = c < d ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[WIDE ? 0 : i] = i * G + t < d ? to_f(p[i * G + t]) : 0.f;
    }
  }
  // Of a vector of d values that itself begins anywhere (w, b).
  __device__ __forceinline__ void load_vec(const T* p, int t, int d, int off) {
    if (M != SHIFTED) {
      load(p, t, d);
    } else {
#pragma unroll
      for (int i = 0; i < N / E; ++i) w[WIDE ? i : 0] = singles(p, (i * G + t) * E - off, d);
    }
  }
  // The same by way of the thread's own places in shared memory, kThreads apart: asked for now, read when it has come.  What is behind
  // the row's end is not read (zeros).
  __device__ static __forceinline__ void ask(uint4* mine, const T* p, int t, int d, int off) {
#pragma unroll
    for (int i = 0; i < N / E; ++i) {
      const int c = (i * G + t) * E - off;
      const bool some = c < d;
      cp_async16(smem_u32(mine + i * kThreads), p + (some ? c : -off), !some ? 0 : M == SHIFTED ? min(E, d - c) * (int)sizeof(T) : 16);
    }
  }
  __device__ __forceinline__ void take(const uint4* mine, int t, int off) {
#pragma unroll
    for (int i = 0; i < N / E; ++i) w[WIDE ? i : 0] = mine[i * kThreads];
    if (M == SHIFTED && t == 0 && off) {  // the row before's
      auto keep = [&](uint32_t v, int k) { return v & ((2 * k >= off ? 0xffffu : 0u) | (2 * k + 1 >= off ? 0xffff0000u : 0u)); };
      w[0] = make_uint4(keep(w[0].x, 0), keep(w[0].y, 1), keep(w[0].z, 2), keep(w[0].w, 3));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (WIDE ? N / E : 1); ++i) w[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < (WIDE ? 1 : N); ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ void ones() {
    const uint32_t o = sizeof(T) == 2 ? 0x3f803f80u : 0x3f800000u;
#pragma unroll
    for (int i = 0; i < (WIDE ? N / E : 1); ++i) w[i] = make_uint4(o, o, o, o);
#pragma unroll
    for (int i = 0; i < (WIDE ? 1 : N); ++i) v[i] = 1.f;
  }
  // Values 2 k and 2 k + 1.
  __device__ __forceinline__ float2 get(int k) const {
    if (!WIDE) return make_float2(v[WIDE ? 0 : 2 * k], v[WIDE ? 0 : 2 * k + 1]);
    const uint4& q = w[WIDE ? 2 * k / E : 0];
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
    if (sizeof(T) == 2) return make_float2(bf_lo(u[k & 3]), bf_hi(u[k & 3]));
    return make_float2(__uint_as_float(u[2 * k & 3]), __uint_as_float(u[(2 * k + 1) & 3]));
  }
};
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
// Stores the values of the thread, f(k) the pair 2 k, 2 k + 1.
template <typename T, int G, int N, LnRows M, typename F>
__device__ __forceinline__ void store_row(T* p, int t, int d, int off, F&& f) {
  constexpr int E = 16 / sizeof(T);
  if (M != SINGLE) {
#pragma unroll
    for (int i = 0; i < N; i += E) {
      const int c = col_of<T, G, M>(i, t, off);
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        const float2 q = f(i / 2 + k);
        if (sizeof(T) == 2) u[k & 3] = pack_bf16(q.x, q.y);
        else u[2 * k & 3] = __float_as_uint(q.x), u[(2 * k + 1) & 3] = __float_as_uint(q.y);
      }
      if (M == SHIFTED && (c < 0 || c + E > d)) {  // an end of the row, or outside
        if (d % 2 == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((unsigned)(c + 2 * j) < (unsigned)d) *reinterpret_cast<uint32_t*>(p + c + 2 * j) = u[j];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if ((unsigned)(c + j) < (unsigned)d) reinterpret_cast<uint16_t*>(p)[c + j] = (uint16_t)(u[j / 2] >> (j & 1 ? 16 : 0));
        }
      } else if (c < d) {
        *reinterpret_cast<uint4*>(p + c) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 q = f(i / 2);
      if (i * G + t < d) p[i * G + t] = from_f<T>(q.x);
      if ((i + 1) * G + t < d) p[(i + 1) * G + t] = from_f<T>(q.y);
    }
  }
}

// The sums of M values over the G threads of a row, in a fixed order, in every thread.  Rows of more than a warp meet at a barrier of
// their own; `red` [kThreads / 32][M], another one than the last time.
template <int G, int M>
__device__ __forceinline__ void group_sum(float (&v)[M], float (*red)[M]) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o; o >>= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(FULL, v[m], o);
  if (G > 32) {
    constexpr int W = G > 32 ? G / 32 : 1;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int m = 0; m < M; ++m) red[warp][m] = v[m];
    // (its number written out: a register's counts as all 16, of which an SM has few)
    const int own = threadIdx.x / G;
    if (G == kThreads) __syncthreads();
    else if (own == 0) asm volatile("bar.sync 1, %0;" ::"n"(G) : "memory");
    else if (own == 1) asm volatile("bar.sync 2, %0;" ::"n"(G) : "memory");
    else if (own == 2) asm volatile("bar.sync 3, %0;" ::"n"(G) : "memory");
    else asm volatile("bar.sync 4, %0;" ::"n"(G) : "memory");
    const int w0 = warp / W * W;
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = red[w0][m];
#pragma unroll
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] += red[w0 + w][m];
  }
}

// The forward's CTAs an SM, and the rows that those of SHIFTED rows ask for ahead.
template <typename T, int N, LnRows M>
constexpr int kLnFwdCtas = N == 32 || (N == 24 && M == SHIFTED) ? 2 : M != PIECES ? 3 : N * sizeof(T) <= 32 ? 5 : 4;
constexpr int kLnFwdAhead = 2;

// A row a group and no loop: bound by memory (two rows in, two out, 16 x 8192 rows of 512 bf16 in 78 us, the rate of a copy; 5 CTAs an SM
// ask for enough at a time, which rows unpacked to fp32 as they are loaded, in three CTAs, did not: 122 us).  One token of 16 sequences
// takes 2 us, a launch.  SHIFTED rows in a loop, with w and b read once for a group: 65536 of 500 bf16 in 46 us, 0.84 of a copy's rate,
// of 511 in 61 (value by value 135).
template <typename T, int G, int N, LnRows M>
__global__ void __launch_bounds__(kThreads, kLnFwdCtas<T, N, M>) k_ln_fwd(const LnArgs a) {
  pdl_enter();
  __shared__ float red[2][kThreads / 32][1];
  using R = Row<T, G, N, M>;
  const int t = threadIdx.x % G;
  const float inv = 1.f / (float)a.d;
  if (check_slots(a)) return;
  const int64_t r00 = (int64_t)(blockIdx.x - a.first) * (kThreads / G), step = (int64_t)(gridDim.x - a.first) * (kThreads / G);
  const int off = row_off<T, M>(r00 + threadIdx.x / G, a.d);
  R w, b;
  auto affine = [&] {
    if (a.w) w.load_vec(static_cast<const T*>(a.w), t, a.d, off);
    else w.ones();
    if (a.b) b.load_vec(static_cast<const T*>(a.b), t, a.d, off);
    else b.clear();
  };
  constexpr int A = kLnFwdAhead, P = N * (int)sizeof(T) / 16;
  extern __shared__ __align__(16) unsigned char dyn[];
  uint4* ring = reinterpret_cast<uint4*>(dyn) + threadIdx.x;  // SHIFTED: [A][2 P][kThreads]
  auto ask = [&](int64_t row, int slot) {
    if (row < a.rows && row_valid(a, row)) {
      uint4* to = ring + slot * 2 * P * kThreads;
      R::ask(to, static_cast<const T*>(a.x) + row * a.ldx, t, a.d, off);
      if (a.res) R::ask(to + P * kThreads, static_cast<const T*>(a.res) + row * a.d, t, a.d, off);
    }
    cp_async_commit();
  };
  if (M == SHIFTED) {
#pragma unroll
    for (int k = 0; k < A; ++k) ask(r00 + threadIdx.x / G + k * step, k);
    affine();
  }
  int slot = 0;
  for (int64_t r0 = r00; r0 < a.rows; r0 += step) {  // (as often in every thread of the CTA)
    const int64_t row = r0 + threadIdx.x / G;
    const bool in = row < a.rows, live = in && row_valid(a, row);
    float2 s[N / 2];  // two values at a time
    {
      R x, q;
      x.clear();
      q.clear();
      if (M == SHIFTED) {
        cp_async_wait<A - 1>();
        if (live) {
          x.take(ring + slot * 2 * P * kThreads, t, off);
          if (a.res) q.take(ring + (slot * 2 + 1) * P * kThreads, t, off);
        }
        ask(row + A * step, slot);
        slot = slot + 1 == A ? 0 : slot + 1;
      } else if (live) {
        x.load(static_cast<const T*>(a.x) + row * a.ldx, t, a.d);
        if (a.res) q.load(static_cast<const T*>(a.res) + row * a.d, t, a.d);
      }
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        s[k] = x.get(k);
        if (!a.res) continue;
        s[k] = __fadd2_rn(s[k], q.get(k));
        if (sizeof(T) == 2) {
          const uint32_t u = pack_bf16(s[k].x, s[k].y);
          s[k] = make_float2(bf_lo(u), bf_hi(u));
        }
      }
    }
    if (in && a.sum) store_row<T, G, N, M>(static_cast<T*>(a.sum) + row * a.d, t, a.d, off, [&](int k) { return s[k]; });
    float2 q = two(0.f);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) q = __fadd2_rn(q, s[k]);
    float m[1] = {q.x + q.y}, v[1];
    group_sum<G, 1>(m, red[0]);
    const float mean = m[0] * inv;
    q = two(0.f);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      s[k] = __fadd2_rn(s[k], two(-mean));
      // (pieces are of one row or of none)
      const int c0 = col_of<T, G, M>(M == PIECES ? 2 * k / R::E * R::E : 2 * k, t, off), c1 = M == PIECES ? c0 : col_of<T, G, M>(2 * k + 1, t, off);
      if ((unsigned)c0 >= (unsigned)a.d) s[k].x = 0.f;
      if ((unsigned)c1 >= (unsigned)a.d) s[k].y = 0.f;
      q = __ffma2_rn(s[k], s[k], q);
    }
    v[0] = q.x + q.y;
    group_sum<G, 1>(v, red[1]);
    if (in) {
      const float r = live ? 1.f / sqrtf(v[0] * inv + a.eps) : 0.f;
      if (M != SHIFTED) affine();
      store_row<T, G, N, M>(static_cast<T*>(a.y) + row * a.d, t, a.d, off, [&](int k) {
        const float2 y = __ffma2_rn(__fmul2_rn(s[k], two(r)), w.get(k), b.get(k));
        return live ? y : two(0.f);
      });
      if (a.stats && t == 0) reinterpret_cast<float2*>(a.stats)[row] = make_float2(live ? mean : 0.f, r);
    }
    if (M != SHIFTED) break;
  }
  if (M == SHIFTED) cp_async_wait<0>();
}

// Rows that the backward asks for ahead: what is in flight covers the memory's latency with the two CTAs an SM that the column
// sums' registers allow.  Bound by memory: three rows in, one out, 16 x 8192 rows of 512 bf16 in 78 us, the rate of a copy (91 with the
// statistics read when they are needed and one value at a time; before that, 107 by registers alone, 90 with three rows ahead).  Rows
// of more than 2048 by the few that are at work at once, which wait for one another's sums: 4096 at 0.65, 5120 to 8192, in one CTA, at 0.57
// (without rows ahead 0.45).
template <typename T, int N, LnRows M>
constexpr int kAhead = M == SINGLE ? 0 : 2;

template <typename T, int G, int N, LnRows M>
__global__ void __launch_bounds__(kThreads, N == 32 ? 1 : N == 8 ? 3 : 2) k_ln_bwd(const LnArgs a) {
  pdl_enter();
  __shared__ float red[2][kThreads / 32][2];
  extern __shared__ __align__(16) unsigned char dyn[];
  float* acc = reinterpret_cast<float*>(dyn);  // at the end: [R][G N], the groups' column sums, where the CTA has several
  uint4* ring = reinterpret_cast<uint4*>(dyn) + threadIdx.x;  // [kAhead][3 (N / E)][kThreads]
  constexpr int R = kThreads / G, A = kAhead<T, N, M>, P = N * (int)sizeof(T) / 16;
  using Mine = Row<T, G, N, M>;
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const float inv = 1.f / (float)a.d;
  if (check_slots(a)) return;
  const int64_t cta = blockIdx.x - a.first, ctas = gridDim.x - a.first;
  Mine w, x, y, s;
  float2 dw[N / 2], db[N / 2];  // two values at a time
#pragma unroll
  for (int k = 0; k < N / 2; ++k) dw[k] = db[k] = two(0.f);
  const int64_t step = ctas * R;  // a multiple of the values of a piece (ln_ctas): a group's rows all begin alike
  const int off = row_off<T, M>(cta * R + grp, a.d);
  if (a.w) w.load_vec(static_cast<const T*>(a.w), t, a.d, off);
  else w.ones();
  s.clear();
  auto stats = [&](int64_t row) {
    return row < a.rows ? reinterpret_cast<const float2*>(a.stats)[row] : make_float2(0.f, 0.f);
  };
  float2 next = stats(cta * R + grp);
  auto ask = [&](int64_t row, int slot) {
    if (row < a.rows && row_valid(a, row)) {
      uint4* to = ring + slot * 3 * P * kThreads;
      Mine::ask(to, static_cast<const T*>(a.x) + row * a.ldx, t, a.d, off);
      Mine::ask(to + P * kThreads, static_cast<const T*>(a.dy) + row * a.d, t, a.d, off);
      if (a.ds) Mine::ask(to + 2 * P * kThreads, static_cast<const T*>(a.ds) + row * a.d, t, a.d, off);
    }
    cp_async_commit();
  };
  if (A > 0) {
#pragma unroll
    for (int k = 0; k < A; ++k) ask(cta * R + grp + k * step, k);
  }
  int slot = 0, turn = 0;
  for (int64_t r0 = cta * R; r0 < a.rows; r0 += step) {  // (as often in every thread of the CTA)
    const int64_t row = r0 + grp;
    const bool in = row < a.rows, live = in && row_valid(a, row);
    const float2 st = live ? next : make_float2(0.f, 0.f);
    next = stats(row + step);
    if (A > 0) cp_async_wait<(A > 0 ? A - 1 : 0)>();
    if (live) {
      if (A > 0) {
        const uint4* from = ring + slot * 3 * P * kThreads;
        x.take(from, t, off);
        y.take(from + P * kThreads, t, off);
        if (a.ds) s.take(from + 2 * P * kThreads, t, off);
      } else {
        x.load(static_cast<const T*>(a.x) + row * a.ldx, t, a.d);
        y.load(static_cast<const T*>(a.dy) + row * a.d, t, a.d);
        if (a.ds) s.load(static_cast<const T*>(a.ds) + row * a.d, t, a.d);
      }
    } else {
      x.clear();
      y.clear();
      s.clear();
    }
    const float2 mean = two(-st.x), r = two(st.y);
    float2 c0 = two(0.f), c1 = two(0.f);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {  // outside the row: dy is 0 there
      const float2 z = __fmul2_rn(__fadd2_rn(x.get(k), mean), r), q = y.get(k), g = __fmul2_rn(q, w.get(k));
      dw[k] = __ffma2_rn(q, z, dw[k]);
      db[k] = __fadd2_rn(db[k], q);
      c0 = __fadd2_rn(c0, g);
      c1 = __ffma2_rn(g, z, c1);
    }
    float c[2] = {c0.x + c0.y, c1.x + c1.y};
    group_sum<G, 2>(c, red[turn]);
    turn ^= 1;
    c0 = two(-c[0] * inv);
    c1 = two(-c[1] * inv);
    if (in)
      store_row<T, G, N, M>(static_cast<T*>(a.dx) + row * a.d, t, a.d, off, [&](int k) {
        const float2 z = __fmul2_rn(__fadd2_rn(x.get(k), mean), r), g = __fmul2_rn(y.get(k), w.get(k));
        return __ffma2_rn(__ffma2_rn(z, c1, __fadd2_rn(g, c0)), r, s.get(k));
      });
    if (A > 0) {  // into the places whose values are used by now
      ask(row + A * step, slot);
      slot = slot + 1 == A ? 0 : slot + 1;
    }
  }
  if (A > 0) cp_async_wait<0>();
  if (!a.part) return;
  // [CTA][dw | db][d], the CTA's rows summed in the order of its groups
  float* out = a.part + cta * 2 * a.d;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (R == 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = col_of<T, G, M>(i, t, off);
        const float2 q = which ? db[i / 2] : dw[i / 2];
        if ((unsigned)c < (unsigned)a.d) out[which * a.d + c] = i & 1 ? q.y : q.x;
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = col_of<T, G, M>(i, t, off);
        const float2 q = which ? db[i / 2] : dw[i / 2];
        if (c >= 0) acc[grp * (G * N) + c] = i & 1 ? q.y : q.x;
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += kThreads) {
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < R; ++k) q += acc[k * (G * N) + c];
        out[which * a.d + c] = q;
      }
    }
  }
}

// Rows of any length, a CTA each: three passes over the row, from L2 after the first, six CTAs an SM (3355 rows of 10000 bf16: forward
// 69 us, 0.57 of a copy's rate, backward 85, 0.46; in two CTAs an SM 94 and 132, value by value 318 of both).
__device__ __forceinline__ float cta_sum(float v, float* red) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kThreads / 32; ++w) v += red[w];
  return v;
}
// The row's values a piece (or as many single ones) a thread at a time.
template <typename T, LnRows M>
using Part = Row<T, kThreads, 16 / (int)sizeof(T), M>;
template <typename T>
constexpr int kPart = kThreads * 16 / (int)sizeof(T);
template <typename T, LnRows M, typename F>
__device__ __forceinline__ void store_part(T* p, int d, F&& f) {
  store_row<T, kThreads, 16 / (int)sizeof(T), M>(p, threadIdx.x, d, 0, f);
}
template <typename T, LnRows M>
__global__ void __launch_bounds__(kThreads) k_ln_fwd_long(const LnArgs a) {
  pdl_enter();
  __shared__ float red[kThreads / 32];
  constexpr int E = 16 / (int)sizeof(T);
  const int t = threadIdx.x;
  const float inv = 1.f / (float)a.d;
  if (check_slots(a)) return;
  const int64_t cta = blockIdx.x - a.first, ctas = gridDim.x - a.first;
  const T *w = static_cast<const T*>(a.w), *b = static_cast<const T*>(a.b);
  for (int64_t row = cta; row < a.rows; row += ctas) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* res = a.res ? static_cast<const T*>(a.res) + row * a.d : nullptr;
    T* sum = a.sum ? static_cast<T*>(a.sum) + row * a.d : nullptr;
    T* y = static_cast<T*>(a.y) + row * a.d;
    if (!row_valid(a, row)) {
      for (int c = 0; c < a.d; c += kPart<T>) {
        if (sum) store_part<T, M>(sum + c, a.d - c, [](int) { return two(0.f); });
        store_part<T, M>(y + c, a.d - c, [](int) { return two(0.f); });
      }
      if (a.stats && t == 0) reinterpret_cast<float2*>(a.stats)[row] = make_float2(0.f, 0.f);
      continue;
    }
    // s of the thread's values from column c on; a thread's own columns in every pass, so what it stored (sum may be x or res) is what it
    // reads again
    float2 s[E / 2];
    auto load = [&](const T* p, const T* q, int c) {
      Part<T, M> v, u;
      v.load(p + c, t, a.d - c);
      if (q) u.load(q + c, t, a.d - c);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        s[k] = v.get(k);
        if (!q) continue;
        s[k] = __fadd2_rn(s[k], u.get(k));
        s[k] = make_float2(to_f(from_f<T>(s[k].x)), to_f(from_f<T>(s[k].y)));
      }
    };
    float2 q = two(0.f);
    for (int c = 0; c < a.d; c += kPart<T>) {
      load(x, res, c);
      if (sum) store_part<T, M>(sum + c, a.d - c, [&](int k) { return s[k]; });
#pragma unroll
      for (int k = 0; k < E / 2; ++k) q = __fadd2_rn(q, s[k]);
    }
    const float mean = cta_sum(q.x + q.y, red) * inv;
    const T *p1 = res && sum ? sum : x, *p2 = res && !sum ? res : nullptr;
    q = two(0.f);
    for (int c = 0; c < a.d; c += kPart<T>) {
      load(p1, p2, c);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        float2 e = __fadd2_rn(s[k], two(-mean));
        if (c + col_of<T, kThreads, M>(2 * k, t, 0) >= a.d) e.x = 0.f;
        if (c + col_of<T, kThreads, M>(2 * k + 1, t, 0) >= a.d) e.y = 0.f;
        q = __ffma2_rn(e, e, q);
      }
    }
    const float r = 1.f / sqrtf(cta_sum(q.x + q.y, red) * inv + a.eps);
    for (int c = 0; c < a.d; c += kPart<T>) {
      load(p1, p2, c);
      Part<T, M> wp, bp;
      if (w) wp.load(w + c, t, a.d - c);
      else wp.ones();
      if (b) bp.load(b + c, t, a.d - c);
      else bp.clear();
      store_part<T, M>(y + c, a.d - c, [&](int k) { return __ffma2_rn(__fmul2_rn(__fadd2_rn(s[k], two(-mean)), two(r)), wp.get(k), bp.get(k)); });
    }
    if (a.stats && t == 0) reinterpret_cast<float2*>(a.stats)[row] = make_float2(mean, r);
  }
}
template <typename T, LnRows M>
__global__ void __launch_bounds__(kThreads) k_ln_bwd_long(const LnArgs a) {
  pdl_enter();
  __shared__ float red[kThreads / 32];
  constexpr int E = 16 / (int)sizeof(T);
  const int t = threadIdx.x;
  const float inv = 1.f / (float)a.d;
  if (check_slots(a)) return;
  const int64_t cta = blockIdx.x - a.first, ctas = gridDim.x - a.first;
  const T* w = static_cast<const T*>(a.w);
  for (int64_t row = cta; row < a.rows; row += ctas) {
    const T *x = static_cast<const T*>(a.x) + row * a.ldx, *dy = static_cast<const T*>(a.dy) + row * a.d;
    const T* ds = a.ds ? static_cast<const T*>(a.ds) + row * a.d : nullptr;
    T* dx = static_cast<T*>(a.dx) + row * a.d;
    if (!row_valid(a, row)) {
      for (int c = 0; c < a.d; c += kPart<T>) store_part<T, M>(dx + c, a.d - c, [](int) { return two(0.f); });
      continue;
    }
    const float2 st = reinterpret_cast<const float2*>(a.stats)[row];
    float2 g[E / 2], z[E / 2];
    auto load = [&](int c) {  // g and z of the thread's values from column c on; past the row's end g is 0
      Part<T, M> xp, yp, wp;
      xp.load(x + c, t, a.d - c);
      yp.load(dy + c, t, a.d - c);
      if (w) wp.load(w + c, t, a.d - c);
      else wp.ones();
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        g[k] = __fmul2_rn(yp.get(k), wp.get(k));
        z[k] = __fmul2_rn(__fadd2_rn(xp.get(k), two(-st.x)), two(st.y));
      }
    };
    float2 q0 = two(0.f), q1 = two(0.f);
    for (int c = 0; c < a.d; c += kPart<T>) {
      load(c);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        q0 = __fadd2_rn(q0, g[k]);
        q1 = __ffma2_rn(g[k], z[k], q1);
      }
    }
    const float c0 = -cta_sum(q0.x + q0.y, red) * inv, c1 = -cta_sum(q1.x + q1.y, red) * inv;
    for (int c = 0; c < a.d; c += kPart<T>) {
      load(c);
      Part<T, M> sp;
      if (ds) sp.load(ds + c, t, a.d - c);
      else sp.clear();
      store_part<T, M>(dx + c, a.d - c, [&](int k) { return __ffma2_rn(__ffma2_rn(z[k], two(c1), __fadd2_rn(g[k], two(c0))), two(st.y), sp.get(k)); });
    }
  }
}
// The long rows' column sums: CTA (x, y) kPart columns of the y-th range of rows.
template <typename T, LnRows M>
__global__ void __launch_bounds__(kThreads) k_ln_cols_long(const LnArgs a) {
  pdl_enter();
  constexpr int E = 16 / (int)sizeof(T);
  const int c = blockIdx.x * kPart<T>, t = threadIdx.x;
  const int64_t lo = a.rows * blockIdx.y / gridDim.y, hi = a.rows * (blockIdx.y + 1) / gridDim.y;
  float2 dw[E / 2], db[E / 2];
#pragma unroll
  for (int k = 0; k < E / 2; ++k) dw[k] = db[k] = two(0.f);
#pragma unroll 2
  for (int64_t row = lo; row < hi; ++row) {
    if (!row_valid(a, row)) continue;
    const float2 st = reinterpret_cast<const float2*>(a.stats)[row];
    Part<T, M> x, y;
    x.load(static_cast<const T*>(a.x) + row * a.ldx + c, t, a.d - c);
    y.load(static_cast<const T*>(a.dy) + row * a.d + c, t, a.d - c);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
      dw[k] = __ffma2_rn(y.get(k), __fmul2_rn(__fadd2_rn(x.get(k), two(-st.x)), two(st.y)), dw[k]);
      db[k] = __fadd2_rn(db[k], y.get(k));
    }
  }
  float* out = a.part + (int64_t)blockIdx.y * 2 * a.d;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int at = c + col_of<T, kThreads, M>(i, t, 0);
    if (at >= a.d) continue;
    out[at] = i & 1 ? dw[i / 2].y : dw[i / 2].x;
    out[a.d + at] = i & 1 ? db[i / 2].y : db[i / 2].x;
  }
}

// dw | db from `n` partial rows of 2 d sums: 32 columns a CTA, its 32 warps take every 32nd partial, then their sums in order (304 rows
// of 1024 in 2 us, by latency).
__global__ void __launch_bounds__(1024) k_ln_cols(const float* part, int n, int d, float* dw, float* db) {
  pdl_enter();
  __shared__ float red[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < 2 * (int64_t)d)
#pragma unroll 8
    for (int k = warp; k < n; k += 32) v += part[(int64_t)k * 2 * d + c];
  red[warp][lane] = v;
  __syncthreads();
  v = red[lane][warp];  // a warp a column: its 32 sums in a fixed tree
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  const int64_t col = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && col < 2 * (int64_t)d) {
    if (col < d) {
      if (dw) dw[col] = v;
    } else if (db) {
      db[col - d] = v;
    }
  }
}

template <int V> struct Int { static constexpr int value = V; };
template <typename T, int G, int N, LnRows M>
cudaError_t run_fwd(const LnArgs& a, cudaStream_t st) {
  constexpr int per = kThreads / G, alike = per < 8 ? 8 / per : 1;
  int64_t ctas = (a.rows + per - 1) / per;
  if (M != SHIFTED) return launch_pdl(k_ln_fwd<T, G, N, M>, dim3((unsigned)(ctas + a.first)), dim3(kThreads), 0, st, a);
  // the scale and the bias are read value by value, once for all rows of a group, which begin alike: as many CTAs as there is room for
  ctas = std::min<int64_t>(ctas, (int64_t)sm_count() * kLnFwdCtas<T, N, M>);
  ctas = (ctas + alike - 1) / alike * alike;
  const size_t smem = (size_t)kLnFwdAhead * 2 * N * sizeof(T) * kThreads;
  if (smem > 32 << 10) {
    const cudaError_t e = cudaFuncSetAttribute(k_ln_fwd<T, G, N, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_ln_fwd<T, G, N, M>, dim3((unsigned)(ctas + a.first)), dim3(kThreads), smem, st, a);
}
template <typename T, int G, int N, LnRows M>
cudaError_t run_bwd(const LnArgs& a, int ctas, cudaStream_t st) {
  const size_t ring = (size_t)kAhead<T, N, M> * 3 * N * sizeof(T) * kThreads;
  const size_t smem = std::max(ring, a.part && kThreads / G > 1 ? (size_t)kThreads * N * 4 : 0);
  if (smem > 32 << 10) {
    const cudaError_t e = cudaFuncSetAttribute(k_ln_bwd<T, G, N, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_ln_bwd<T, G, N, M>, dim3((unsigned)(ctas + a.first)), dim3(kThreads), smem, st, a);
}
template <typename T, LnRows M>
cudaError_t pick(const LnArgs& a, bool bwd, int ctas, cudaStream_t st) {
  const LnGroup g = ln_group(a.d, sizeof(T) == 4, bwd);
  auto is = [&](auto G, auto N) { return g.threads == G.value && g.values == N.value; };
  cudaError_t e = cudaErrorNotSupported;
  auto go = [&](auto G, auto N) {
    if (!is(G, N)) return;
    if (!bwd) e = run_fwd<T, G.value, N.value, M>(a, st);
    else if constexpr (N.value != 24) e = run_bwd<T, G.value, N.value, M>(a, ctas, st);
  };
  auto all = [&](auto N, auto... G) { (go(G, N), ...); };
  if constexpr (sizeof(T) == 4) {
    all(Int<8>{}, Int<8>{}, Int<16>{}, Int<32>{});
    all(Int<16>{}, Int<32>{}, Int<64>{}, Int<128>{}, Int<256>{});
  } else {
    all(Int<8>{}, Int<4>{});
    all(Int<16>{}, Int<4>{}, Int<8>{}, Int<16>{}, Int<32>{}, Int<64>{}, Int<128>{}, Int<256>{});
    all(Int<24>{}, Int<4>{}, Int<8>{}, Int<16>{}, Int<32>{}, Int<64>{}, Int<128>{}, Int<256>{});
  }
  go(Int<256>{}, Int<32>{});
  if (g.threads) return e;
  constexpr LnRows L = M == PIECES ? PIECES : SINGLE;
  return launch_pdl(bwd ? k_ln_bwd_long<T, L> : k_ln_fwd_long<T, L>, dim3((unsigned)(ctas + a.first)), dim3(kThreads), 0, st, a);
}

}  // namespace

bool ln_clears(const LnArgs& a) { return a.slots <= kCheckSlots; }
// Threads of a row and values of each; 0: a CTA in passes.  Of bf16 16 values or, where they fill the threads better, 24 (64 MB a tensor,
// forward: 768 columns 41 us, in 64 threads of 16 51; 64 columns 42, in 8 threads of 8 50); the backward's column sums have no registers
// for 24 (384 columns 60 us, by 24 65; 1536 64, 79).  Of fp32, whose values take twice the registers, 8 to 16.
LnGroup ln_group(int d, bool f32, bool bwd) {
  if (f32) {
    for (int g = 8; g <= 32; g *= 2)
      if (d <= 8 * g) return {g, 8};
    for (int g = 32; g <= 256; g *= 2)
      if (d <= 16 * g) return {g, 16};
  } else {
    // rows that are not whole pieces may begin so far behind a boundary (8187, 8189, 8190 and 8191 columns are longer than any group's for that:
    // forward 116 us, backward 157, 8192 46 and 77)
    d += d % 8 == 0 ? 0 : d % 4 == 0 ? 4 : d % 2 == 0 ? 6 : 7;
    if (d <= 32) return {4, 8};
    for (int g = 4; g <= 256; g *= 2)
      for (int n = 16; n <= (bwd ? 16 : 24); n += 8)
        if (d <= n * g) return {g, n};
  }
  return d <= 8192 ? LnGroup{256, 32} : LnGroup{0, 0};
}
int ln_ctas(int64_t rows, int d, bool f32) {
  const int g = ln_group(d, f32, true).threads, per = g ? kThreads / g : 1, alike = per < 8 ? 8 / per : 1;  // CTAs whose rows are a multiple of 8
  const int64_t most = std::min<int64_t>((rows + per - 1) / per, (int64_t)sm_count() * (g ? 2 : 6));  // (as many as there is room for)
  return (int)((most + alike - 1) / alike * alike);
}
int ln_parts(int64_t rows, int d, bool f32) { return ln_group(d, f32, true).threads ? ln_ctas(rows, d, f32) : (int)std::min<int64_t>(rows, 64); }

static LnRows ln_rows(const LnArgs& a, bool f32) {
  const size_t es = f32 ? 4 : 2;
  uintptr_t rows = 0;  // where the rows' tensors begin
  for (const void* q : {a.x, a.res, (const void*)a.sum, (const void*)a.y, a.dy, a.ds, (const void*)a.dx}) rows |= reinterpret_cast<uintptr_t>(q);
  const uintptr_t all = rows | reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.b) | (uintptr_t)(a.d * es) | (uintptr_t)(a.ldx * es);
  return all % 16 == 0 ? PIECES : !f32 && rows % 16 == 0 && (a.ldx - a.d) % 8 == 0 ? SHIFTED : SINGLE;
}
cudaError_t launch_ln(LnArgs a, bool f32, bool bwd, cudaStream_t st) {
  a.first = a.slots > 0 && a.slots <= kCheckSlots;
  const int ctas = ln_ctas(a.rows, a.d, f32);
  const LnRows m = ln_rows(a, f32);
  if (f32) return m == PIECES ? pick<float, PIECES>(a, bwd, ctas, st) : pick<float, SINGLE>(a, bwd, ctas, st);
  return m == PIECES ? pick<bf16, PIECES>(a, bwd, ctas, st) : m == SHIFTED ? pick<bf16, SHIFTED>(a, bwd, ctas, st) : pick<bf16, SINGLE>(a, bwd, ctas, st);
}
cudaError_t launch_ln_cols_long(const LnArgs& a, bool f32, cudaStream_t st) {
  const int part = f32 ? kPart<float> : kPart<bf16>;
  const dim3 grid((unsigned)((a.d + part - 1) / part), (unsigned)ln_parts(a.rows, a.d, f32));
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kThreads), 0, st, a); };
  const bool pieces = ln_rows(a, f32) == PIECES;
  if (f32) return pieces ? go(k_ln_cols_long<float, PIECES>) : go(k_ln_cols_long<float, SINGLE>);
  return pieces ? go(k_ln_cols_long<bf16, PIECES>) : go(k_ln_cols_long<bf16, SINGLE>);
}
cudaError_t launch_ln_cols(const LnArgs& a, bool f32, float* dw, float* db, cudaStream_t st) {
  return launch_pdl(k_ln_cols, dim3((unsigned)((2 * (int64_t)a.d + 31) / 32)), dim3(1024), 0, st, (const float*)a.part,
                    ln_parts(a.rows, a.d, f32), a.d, dw, db);
}

}  // namespace gbla
