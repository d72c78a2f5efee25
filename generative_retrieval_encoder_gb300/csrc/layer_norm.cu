// Layer norm between the blocks, with the residual stream's addition.
//   s = x + res (rounded to the io type, which is what is normed and kept),
//   m = mean s, r = 1 / sqrt(mean (s - m)^2 + eps), z = (s - m) r, y = z w + b
// and its backward, g = dy w:
//   dx = r (g - mean g - z mean(g z)) + ds,  dw = sum_rows dy z,  db = sum_rows dy.
//
// A group of G threads holds a row, N values each, so mean and squares are taken
// from registers (the squares about the mean itself: no cancellation) and every
// tensor is read once.  Rows longer than 8192 values go by CTA in passes over L2.
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

// The column of value i of thread t in a row of G threads: 16-byte pieces dealt out in turn (WIDE), or single values.
template <typename T, int G, bool WIDE>
__device__ __forceinline__ int col_of(int i, int t) {
  constexpr int E = 16 / sizeof(T);
  return WIDE ? ((i / E) * G + t) * E + i % E : i * G + t;
}

// The thread's N values of a row as they lie in memory (0 past d): bf16 values stay two to a register until they are used.
template <typename T, int G, int N, bool WIDE>
struct Row {
  static constexpr int E = 16 / sizeof(T);
  uint4 w[WIDE ? N / E : 1];
  float v[WIDE ? 1 : N];
  __device__ __forceinline__ void load(const T* p, int t, int d) {
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
  // The same by way of the thread's own places in shared memory, kThreads apart: asked for now, read when it has come.
  __device__ static __forceinline__ void ask(uint4* mine, const T* p, int t, int d) {
#pragma unroll
    for (int i = 0; i < N / E; ++i) {
      const int c = (i * G + t) * E;
      cp_async16(smem_u32(mine + i * kThreads), p + (c < d ? c : 0), c < d ? 16 : 0);
    }
  }
  __device__ __forceinline__ void take(const uint4* mine) {
#pragma unroll
    for (int i = 0; i < N / E; ++i) w[WIDE ? i : 0] = mine[i * kThreads];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (WIDE ? N / E : 1); ++i) w[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < (WIDE ? 1 : N); ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ float get(int i) const {
    if (!WIDE) return v[WIDE ? 0 : i];
    const uint4& q = w[WIDE ? i / E : 0];
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
    if (sizeof(T) == 2) return i & 1 ? bf_hi(u[(i % E) / 2]) : bf_lo(u[(i % E) / 2]);
    return __uint_as_float(u[i & 3]);
  }
};
// Stores the values f(0) .. f(N - 1) of the thread.
template <typename T, int G, int N, bool WIDE, typename F>
__device__ __forceinline__ void store_row(T* p, int t, int d, F&& f) {
  constexpr int E = 16 / sizeof(T);
  if (WIDE) {
#pragma unroll
    for (int i = 0; i < N; i += E) {
      const int c = col_of<T, G, true>(i, t);
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = sizeof(T) == 2 ? pack_bf16(f(i + 2 * k), f(i + 2 * k + 1)) : __float_as_uint(f(i + k));
      if (c < d) *reinterpret_cast<uint4*>(p + c) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * G + t < d) p[i * G + t] = from_f<T>(f(i));
  }
}

// The sums of M values over the G threads of a row, in a fixed order, in every thread.  Rows of more than a warp meet at two CTA
// barriers; `red` [kThreads / 32][M].
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
    __syncthreads();
    const int w0 = warp / W * W;
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = red[w0][m];
#pragma unroll
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] += red[w0 + w][m];
    __syncthreads();
  }
}

// A row a group and no loop: bound by memory (two rows in, two out, 16 x 8192 rows of 512 bf16 in 80 us, 0.99 of a copy's rate; 5 CTAs
// an SM ask for enough at a time, which rows unpacked to fp32 as they are loaded, in three CTAs, did not: 122 us).  One token of 16
// sequences takes 2 us, a launch.
template <typename T, int G, int N, bool WIDE>
__global__ void __launch_bounds__(kThreads, N == 32 ? 2 : !WIDE ? 3 : N * sizeof(T) <= 32 ? 5 : 4) k_ln_fwd(const LnArgs a) {
  pdl_enter();
  __shared__ float red[kThreads / 32][1];
  using R = Row<T, G, N, WIDE>;
  const int t = threadIdx.x % G;
  const float inv = 1.f / (float)a.d;
  if (check_slots(a)) return;
  const int64_t cta = blockIdx.x - a.first, ctas = gridDim.x - a.first;
  const int64_t row = cta * (kThreads / G) + threadIdx.x / G;
  const bool in = row < a.rows, live = in && row_valid(a, row);
  float s[N];
  {
    R x, q;
    x.clear();
    q.clear();
    if (live) {
      x.load(static_cast<const T*>(a.x) + row * a.ldx, t, a.d);
      if (a.res) q.load(static_cast<const T*>(a.res) + row * a.d, t, a.d);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = a.res ? to_f(from_f<T>(x.get(i) + q.get(i))) : x.get(i);
  }
  if (in && a.sum) store_row<T, G, N, WIDE>(static_cast<T*>(a.sum) + row * a.d, t, a.d, [&](int i) { return s[i]; });
  float m[1] = {0.f}, v[1] = {0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) m[0] += s[i];
  group_sum<G, 1>(m, red);
  const float mean = m[0] * inv;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float c = s[i] - mean;
    v[0] += col_of<T, G, WIDE>(i, t) < a.d ? c * c : 0.f;
  }
  group_sum<G, 1>(v, red);
  if (!in) return;
  const float r = live ? 1.f / sqrtf(v[0] * inv + a.eps) : 0.f;
  R w, b;
  if (a.w) w.load(static_cast<const T*>(a.w), t, a.d);
  if (a.b) b.load(static_cast<const T*>(a.b), t, a.d);
  store_row<T, G, N, WIDE>(static_cast<T*>(a.y) + row * a.d, t, a.d, [&](int i) {
    float z = (s[i] - mean) * r;
    if (a.w) z *= w.get(i);
    if (a.b) z += b.get(i);
    return live ? z : 0.f;
  });
  if (a.stats && t == 0) reinterpret_cast<float2*>(a.stats)[row] = make_float2(live ? mean : 0.f, r);
}

// Rows that the backward asks for ahead: what is in flight covers the memory's latency with the two CTAs an SM that the column
// sums' registers allow.  Bound by memory, and by what is in flight at the turns of a row: three rows in, one out, 16 x 8192 rows of 512
// bf16 in 89 us, 0.89 of a copy's rate (107 by registers alone, 90 with three rows ahead; 64 threads a row, 8 values each in three CTAs,
// 115: the sums of a row then meet at CTA barriers).
template <typename T, int N, bool WIDE>
constexpr int kAhead = !WIDE || N == 32 ? 0 : 2;

template <typename T, int G, int N, bool WIDE>
__global__ void __launch_bounds__(kThreads, N == 32 ? 1 : N == 8 ? 3 : 2) k_ln_bwd(const LnArgs a) {
  pdl_enter();
  __shared__ float red[kThreads / 32][2];
  extern __shared__ __align__(16) unsigned char dyn[];
  float* acc = reinterpret_cast<float*>(dyn);  // at the end: [R][G N], the groups' column sums, where the CTA has several
  uint4* ring = reinterpret_cast<uint4*>(dyn) + threadIdx.x;  // [kAhead][3 (N / E)][kThreads]
  constexpr int R = kThreads / G, A = kAhead<T, N, WIDE>, P = N * (int)sizeof(T) / 16;
  using Mine = Row<T, G, N, WIDE>;
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const float inv = 1.f / (float)a.d;
  if (check_slots(a)) return;
  const int64_t cta = blockIdx.x - a.first, ctas = gridDim.x - a.first;
  Mine w, x, y, s;
  float dw[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = db[i] = 0.f;
  if (a.w) w.load(static_cast<const T*>(a.w), t, a.d);
  s.clear();
  const int64_t step = ctas * R;
  auto ask = [&](int64_t row, int slot) {
    if (row < a.rows && row_valid(a, row)) {
      uint4* to = ring + slot * 3 * P * kThreads;
      Mine::ask(to, static_cast<const T*>(a.x) + row * a.ldx, t, a.d);
      Mine::ask(to + P * kThreads, static_cast<const T*>(a.dy) + row * a.d, t, a.d);
      if (a.ds) Mine::ask(to + 2 * P * kThreads, static_cast<const T*>(a.ds) + row * a.d, t, a.d);
    }
    cp_async_commit();
  };
  if (A > 0) {
#pragma unroll
    for (int k = 0; k < A; ++k) ask(cta * R + grp + k * step, k);
  }
  int slot = 0;
  for (int64_t r0 = cta * R; r0 < a.rows; r0 += step) {  // (as often in every thread of the CTA)
    const int64_t row = r0 + grp;
    const bool in = row < a.rows, live = in && row_valid(a, row);
    float mean = 0.f, r = 0.f;
    if (A > 0) cp_async_wait<(A > 0 ? A - 1 : 0)>();
    if (live) {
      const float2 st = reinterpret_cast<const float2*>(a.stats)[row];
      if (A > 0) {
        const uint4* from = ring + slot * 3 * P * kThreads;
        x.take(from);
        y.take(from + P * kThreads);
        if (a.ds) s.take(from + 2 * P * kThreads);
      } else {
        x.load(static_cast<const T*>(a.x) + row * a.ldx, t, a.d);
        y.load(static_cast<const T*>(a.dy) + row * a.d, t, a.d);
        if (a.ds) s.load(static_cast<const T*>(a.ds) + row * a.d, t, a.d);
      }
      mean = st.x;
      r = st.y;
    } else {
      x.clear();
      y.clear();
      s.clear();
    }
    float c[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = (x.get(i) - mean) * r, q = y.get(i), g = a.w ? q * w.get(i) : q;  // past d: dy is 0 there
      dw[i] += q * z;
      db[i] += q;
      c[0] += g;
      c[1] += g * z;
    }
    group_sum<G, 2>(c, red);
    const float c0 = c[0] * inv, c1 = c[1] * inv;
    if (in)
      store_row<T, G, N, WIDE>(static_cast<T*>(a.dx) + row * a.d, t, a.d, [&](int i) {
        const float z = (x.get(i) - mean) * r, q = y.get(i);
        const float g = r * ((a.w ? q * w.get(i) : q) - c0 - z * c1);
        return a.ds ? g + s.get(i) : g;
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
        const int c = col_of<T, G, WIDE>(i, t);
        if (c < a.d) out[which * a.d + c] = which ? db[i] : dw[i];
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) acc[grp * (G * N) + col_of<T, G, WIDE>(i, t)] = which ? db[i] : dw[i];
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

// Rows of any length, a CTA each: three passes over the row, from L2 after the first.
__device__ __forceinline__ float cta_sum(float v, float* red) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kThreads / 32; ++w) v += red[w];
  return v;
}
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ln_fwd_long(const LnArgs a) {
  pdl_enter();
  __shared__ float red[kThreads / 32];
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
      for (int c = threadIdx.x; c < a.d; c += kThreads) {
        if (sum) sum[c] = from_f<T>(0.f);
        y[c] = from_f<T>(0.f);
      }
      if (a.stats && threadIdx.x == 0) reinterpret_cast<float2*>(a.stats)[row] = make_float2(0.f, 0.f);
      continue;
    }
    // a thread's own columns in every pass, so what it stored (sum may be x or res) is what it reads again
    const T *p = res && sum ? sum : x, *q = res && !sum ? res : nullptr;
    auto at = [&](int c) { return q ? to_f(from_f<T>(to_f(p[c]) + to_f(q[c]))) : to_f(p[c]); };
    float m = 0.f, v = 0.f;
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      const T s = res ? from_f<T>(to_f(x[c]) + to_f(res[c])) : x[c];
      if (sum) sum[c] = s;
      m += to_f(s);
    }
    m = cta_sum(m, red) * inv;
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      const float e = at(c) - m;
      v += e * e;
    }
    const float r = 1.f / sqrtf(cta_sum(v, red) * inv + a.eps);
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      float z = (at(c) - m) * r;
      if (w) z *= to_f(w[c]);
      if (b) z += to_f(b[c]);
      y[c] = from_f<T>(z);
    }
    if (a.stats && threadIdx.x == 0) reinterpret_cast<float2*>(a.stats)[row] = make_float2(m, r);
  }
}
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ln_bwd_long(const LnArgs a) {
  pdl_enter();
  __shared__ float red[kThreads / 32];
  const float inv = 1.f / (float)a.d;
  if (check_slots(a)) return;
  const int64_t cta = blockIdx.x - a.first, ctas = gridDim.x - a.first;
  const T* w = static_cast<const T*>(a.w);
  for (int64_t row = cta; row < a.rows; row += ctas) {
    const T *x = static_cast<const T*>(a.x) + row * a.ldx, *dy = static_cast<const T*>(a.dy) + row * a.d;
    const T* ds = a.ds ? static_cast<const T*>(a.ds) + row * a.d : nullptr;
    T* dx = static_cast<T*>(a.dx) + row * a.d;
    if (!row_valid(a, row)) {
      for (int c = threadIdx.x; c < a.d; c += kThreads) dx[c] = from_f<T>(0.f);
      continue;
    }
    const float2 st = reinterpret_cast<const float2*>(a.stats)[row];
    float c0 = 0.f, c1 = 0.f;
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      const float g = to_f(dy[c]) * (w ? to_f(w[c]) : 1.f);
      c0 += g;
      c1 += g * ((to_f(x[c]) - st.x) * st.y);
    }
    c0 = cta_sum(c0, red) * inv;
    c1 = cta_sum(c1, red) * inv;
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      const float g = to_f(dy[c]) * (w ? to_f(w[c]) : 1.f), z = (to_f(x[c]) - st.x) * st.y;
      dx[c] = from_f<T>(st.y * (g - c0 - z * c1) + (ds ? to_f(ds[c]) : 0.f));
    }
  }
}
// The long rows' column sums: CTA (x, y) 256 columns of the y-th range of rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ln_cols_long(const LnArgs a) {
  pdl_enter();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.d) return;
  const int64_t lo = a.rows * blockIdx.y / gridDim.y, hi = a.rows * (blockIdx.y + 1) / gridDim.y;
  float dw = 0.f, db = 0.f;
  for (int64_t row = lo; row < hi; ++row) {
    if (!row_valid(a, row)) continue;
    const float2 st = reinterpret_cast<const float2*>(a.stats)[row];
    const float g = to_f(static_cast<const T*>(a.dy)[row * a.d + c]);
    dw += g * ((to_f(static_cast<const T*>(a.x)[row * a.ldx + c]) - st.x) * st.y);
    db += g;
  }
  float* out = a.part + (int64_t)blockIdx.y * 2 * a.d;
  out[c] = dw;
  out[a.d + c] = db;
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

template <typename T, int G, int N, bool WIDE>
cudaError_t run(const LnArgs& a, bool bwd, int ctas, cudaStream_t st) {
  if (!bwd) return launch_pdl(k_ln_fwd<T, G, N, WIDE>, dim3((unsigned)((a.rows + kThreads / G - 1) / (kThreads / G)) + a.first), dim3(kThreads), 0, st, a);
  const size_t ring = (size_t)kAhead<T, N, WIDE> * 3 * N * sizeof(T) * kThreads;
  const size_t smem = std::max(ring, a.part && kThreads / G > 1 ? (size_t)kThreads * N * 4 : 0);
  if (smem > 32 << 10) {
    const cudaError_t e = cudaFuncSetAttribute(k_ln_bwd<T, G, N, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_ln_bwd<T, G, N, WIDE>, dim3((unsigned)(ctas + a.first)), dim3(kThreads), smem, st, a);
}
template <typename T, bool WIDE>
cudaError_t pick(const LnArgs& a, bool bwd, int ctas, cudaStream_t st) {
  switch (ln_group(a.d)) {
    case 8: return run<T, 8, 8, WIDE>(a, bwd, ctas, st);
    case 16: return run<T, 16, 8, WIDE>(a, bwd, ctas, st);
    case 32: return a.d <= 256 ? run<T, 32, 8, WIDE>(a, bwd, ctas, st) : run<T, 32, 16, WIDE>(a, bwd, ctas, st);
    case 64: return run<T, 64, 16, WIDE>(a, bwd, ctas, st);
    case 128: return run<T, 128, 16, WIDE>(a, bwd, ctas, st);
    case 256: return a.d <= 4096 ? run<T, 256, 16, WIDE>(a, bwd, ctas, st) : run<T, 256, 32, WIDE>(a, bwd, ctas, st);
  }
  if (!bwd) return launch_pdl(k_ln_fwd_long<T>, dim3((unsigned)(ctas + a.first)), dim3(kThreads), 0, st, a);
  return launch_pdl(k_ln_bwd_long<T>, dim3((unsigned)(ctas + a.first)), dim3(kThreads), 0, st, a);
}

}  // namespace

bool ln_clears(const LnArgs& a) { return a.slots <= kCheckSlots; }
// Threads of a row: 8 values each up to 256 columns, 16 up to 4096, 32 up to 8192; 0: a CTA in passes.
int ln_group(int d) {
  if (d <= 64) return 8;
  if (d <= 128) return 16;
  if (d <= 512) return 32;
  if (d <= 1024) return 64;
  if (d <= 2048) return 128;
  if (d <= 8192) return 256;
  return 0;
}
int ln_ctas(int64_t rows, int d) {
  const int g = ln_group(d), per = g ? kThreads / g : 1;
  return (int)std::min<int64_t>((rows + per - 1) / per, (int64_t)sm_count() * 2);
}
int ln_parts(int64_t rows, int d) { return ln_group(d) ? ln_ctas(rows, d) : (int)std::min<int64_t>(rows, 16); }

cudaError_t launch_ln(LnArgs a, bool f32, bool bwd, cudaStream_t st) {
  a.first = a.slots > 0 && a.slots <= kCheckSlots;
  const size_t es = f32 ? 4 : 2;
  uintptr_t bits = (uintptr_t)(a.d * es) | (uintptr_t)(a.ldx * es);
  for (const void* q : {a.x, a.res, a.w, a.b, (const void*)a.sum, (const void*)a.y, a.dy, a.ds, (const void*)a.dx})
    bits |= reinterpret_cast<uintptr_t>(q);
  const bool wide = bits % 16 == 0;
  const int ctas = ln_ctas(a.rows, a.d);
  if (f32) return wide ? pick<float, true>(a, bwd, ctas, st) : pick<float, false>(a, bwd, ctas, st);
  return wide ? pick<bf16, true>(a, bwd, ctas, st) : pick<bf16, false>(a, bwd, ctas, st);
}
cudaError_t launch_ln_cols_long(const LnArgs& a, bool f32, cudaStream_t st) {
  const dim3 grid((unsigned)((a.d + kThreads - 1) / kThreads), (unsigned)ln_parts(a.rows, a.d));
  return f32 ? launch_pdl(k_ln_cols_long<float>, grid, dim3(kThreads), 0, st, a)
             : launch_pdl(k_ln_cols_long<bf16>, grid, dim3(kThreads), 0, st, a);
}
cudaError_t launch_ln_cols(const LnArgs& a, float* dw, float* db, cudaStream_t st) {
  return launch_pdl(k_ln_cols, dim3((unsigned)((2 * (int64_t)a.d + 31) / 32)), dim3(1024), 0, st, (const float*)a.part,
                    ln_parts(a.rows, a.d), a.d, dw, db);
}

}  // namespace gbla
