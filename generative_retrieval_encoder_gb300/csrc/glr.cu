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
#include "common.cuh"
#include "kernels.h"

namespace gbla {
namespace {

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
__global__ void __launch_bounds__(256) k_glr_fwd(const GlrArgs a) {
  if (a.err && *a.err) return;
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= (int64_t)a.seq.n_seq * a.d) return;
  const int b = (int)(id / a.d), ch = (int)(id % a.d);
  int64_t row0;
  int n;
  seq_rows(a.seq, b, row0, n);
  const float k = a.c * softplus_f(a.lam[ch]);
  float h = a.h0 ? a.h0[id] : 0.f;
  for (int t = 0; t < n; ++t) {
    const int64_t row = a.reverse ? row0 + n - 1 - t : row0 + t;
    if (a.saved) {
      bool first, last;
      const int64_t c = chunk_of(a, b, row, row0, first, last);
      if (t > 0 && first) a.saved[c * a.d + ch] = h;
    }
    const int64_t o = row * a.ld + ch;
    const Gate g = gate_of(to_f(((const T*)a.r)[o]), k);
    h = fmaf(g.a, h, g.m * sigmoid_f(to_f(((const T*)a.i)[o])) * to_f(((const T*)a.x)[o]));
    ((T*)a.y)[row * a.d + ch] = from_f<T>(h);
  }
  if (a.hT) a.hT[id] = h;
  if (a.seq.mode == SEQ_PADDED)
    for (int t = n; t < a.seq.L; ++t) ((T*)a.y)[(row0 + t) * a.d + ch] = from_f<T>(0.f);
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

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, bool f32, cudaStream_t st) {
  const int64_t n = (int64_t)a.seq.n_seq * a.d;
  const unsigned grid = (unsigned)((n + 255) / 256);
  if (f32) k_glr_fwd<float><<<grid, 256, 0, st>>>(a);
  else k_glr_fwd<bf16><<<grid, 256, 0, st>>>(a);
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
