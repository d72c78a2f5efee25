// AdamW over many tensors at once, and the global gradient norm it clips by.
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g g,
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// States in fp32, or m and sqrt(v) as e4m3 values with an fp32 scale per 256
// values.  Of an 8-bit value t = |x| 448 / max |block| the bits below its step
// are rounded up with their own odds: 16 hashed bits are added below the
// last place kept, and the sum is cut off.
//
// The 8-bit states are what the fp32 operations below give, each rounded once
// (no contraction into fused multiply-adds): a value near a border between
// two codes falls on the same side wherever the same formula is computed.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace gbla {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// Two rounds of shift-xor and odd multiplications (the fraction bits of sqrt 2 and sqrt 3).
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}
// The 32 random bits of a place (the fraction bits of the golden ratio spread neighbours).
__device__ __forceinline__ uint32_t bits_of(uint64_t place, uint32_t key) {
  return mix32((uint32_t)place * 0x9E3779B9u + (uint32_t)(place >> 32) * 0xBB67AE85u + key);
}

// t in [0, 448] to an e4m3 magnitude, 16 random bits d: at the normal values (t >= 2^-6) the fraction's
// lower 20 bits, below them the fixed step 2^-9.
__device__ __forceinline__ uint32_t e4m3_up(float t, uint32_t d) {
  const uint32_t n = ((__float_as_uint(t) + (d << 4)) >> 20) - (120u << 3);
  const uint32_t s = (uint32_t)floorf(__fadd_rn(t * 512.f, (float)d * 0x1p-16f));
  return t >= 0x1p-6f ? n : s;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {  // of the low 7 bits
  const uint32_t k = code & 127u;
  return k >= 8u ? __uint_as_float((k << 20) + (120u << 23)) : (float)k * 0x1p-9f;
}

__global__ void k_adamw_begin(const AdamStep c, int64_t* step, const float* norm, AdamScalars* s) {
  pdl_enter();
  const float nm = norm ? *norm : 0.f;
  AdamScalars o;
  o.go = isfinite(nm);
  const int64_t t = *step + 1;
  if (o.go) *step = t;
  o.clip = norm && c.max_norm > 0. ? fminf(__fmul_rn(__frcp_rn(__fadd_rn(nm, 1e-6f)), (float)c.max_norm), 1.f) : 1.f;
  o.b1 = (float)c.b1; o.c1 = (float)(1. - c.b1);
  o.b2 = (float)c.b2; o.c2 = (float)(1. - c.b2);
  o.step = (float)(c.lr / (1. - pow(c.b1, (double)t)));
  o.inv = (float)(1. / sqrt(1. - pow(c.b2, (double)t)));
  o.eps = (float)c.eps;
  o.key = mix32(mix32((uint32_t)t ^ 0x9E3779B9u) + c.seed);
  *s = o;
}

// The tensor of a unit.
template <int N>
__device__ __forceinline__ int tensor_of(const AdamTable<N>& t, int unit) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.t[mid].first <= unit) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One value: m, root = sqrt(v) and p moved by g.
__device__ __forceinline__ void move(float g, float& m, float& v, float& root, float& p, const AdamScalars& s, float keep) {
  g = __fmul_rn(g, s.clip);
  m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.c1, g));
  v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(__fmul_rn(s.c2, g), g));
  root = __fsqrt_rn(v);
  p = p * keep - s.step * __fdividef(m, fmaf(root, s.inv, s.eps));
}

// A warp takes 256 values, lane l those at l, l + 32, ..
template <int N>
__global__ void __launch_bounds__(256) k_adamw(const __grid_constant__ AdamTable<N> tab, const AdamScalars* sc) {
  pdl_enter();
  const AdamScalars s = *sc;
  if (!s.go) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u0 = (int)((int64_t)tab.units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)tab.units * (blockIdx.x + 1) / gridDim.x);
  if (u0 >= u1) return;
  int k = tensor_of(tab, u0);
  for (int u = u0; u < u1; ++u) {
    while (k + 1 < tab.n && tab.t[k + 1].first <= u) ++k;
    const AdamTensor& t = tab.t[k];
    const int64_t e0 = (int64_t)(u - t.first) * kAdamUnit + warp * kAdamBlock;
    if (e0 >= t.n) continue;
    const bool q8 = t.ms != nullptr;
    const int64_t blk = e0 / kAdamBlock;
    float m[8], root[8];
    for (int j = 0; j < 8; ++j) {
      const int64_t e = e0 + lane + 32 * j;
      m[j] = root[j] = 0.f;
      if (e >= t.n) continue;
      float v;
      if (q8) {
        const uint32_t cm = ((const uint8_t*)t.m)[e], cv = ((const uint8_t*)t.v)[e];
        const float a = __fmul_rn(e4m3_value(cm), t.ms[blk]);
        m[j] = cm & 128u ? -a : a;
        v = __fmul_rn(e4m3_value(cv), t.vs[blk]);
        v = __fmul_rn(v, v);
      } else {
        m[j] = ((const float*)t.m)[e];
        v = ((const float*)t.v)[e];
      }
      const float g = t.gb ? to_f(((const bf16*)t.grad)[e]) : ((const float*)t.grad)[e];
      float p = t.master ? t.master[e] : t.pb ? to_f(((const bf16*)t.param)[e]) : ((const float*)t.param)[e];
      move(g, m[j], v, root[j], p, s, t.keep);
      if (t.master) t.master[e] = p;
      if (t.pb) ((bf16*)t.param)[e] = from_f<bf16>(p);
      else ((float*)t.param)[e] = p;
      if (!q8) {
        ((float*)t.m)[e] = m[j];
        ((float*)t.v)[e] = v;
      }
    }
    if (!q8) continue;
    // the largest magnitudes as bit patterns: a NaN or infinity is the largest of all
    uint32_t tm = 0, tv = 0;
    for (int j = 0; j < 8; ++j) {
      tm = max(tm, __float_as_uint(m[j]) & 0x7fffffffu);
      tv = max(tv, __float_as_uint(root[j]) & 0x7fffffffu);
    }
    tm = __reduce_max_sync(FULL, tm);
    tv = __reduce_max_sync(FULL, tv);
    const float fm = __uint_as_float(tm), fv = __uint_as_float(tv);
    const bool badm = !isfinite(fm), badv = !isfinite(fv);
    const float im = fm >= 0x1p-100f ? __fmul_rn(__frcp_rn(fm), 448.f) : 0.f;
    const float iv = fv >= 0x1p-100f ? __fmul_rn(__frcp_rn(fv), 448.f) : 0.f;
    __syncwarp();  // every lane has read the block's scales
    if (lane == 0) {
      t.ms[blk] = badm ? __uint_as_float(0x7fc00000u) : fm >= 0x1p-100f ? __fmul_rn(fm, 1.f / 448.f) : 0.f;
      t.vs[blk] = badv ? __uint_as_float(0x7fc00000u) : fv >= 0x1p-100f ? __fmul_rn(fv, 1.f / 448.f) : 0.f;
    }
    for (int j = 0; j < 8; ++j) {
      const int64_t e = e0 + lane + 32 * j;
      if (e >= t.n) continue;
      const uint32_t z = bits_of((uint64_t)(t.place + e), s.key);
      const float xm = fminf(__fmul_rn(fabsf(m[j]), im), 448.f), xv = fminf(__fmul_rn(root[j], iv), 448.f);
      uint32_t cm = e4m3_up(xm, z & 0xffffu) | (__float_as_uint(m[j]) >> 31 << 7);
      uint32_t cv = e4m3_up(xv, z >> 16);
      if (xv > 0.f) cv = max(cv, 1u);
      ((uint8_t*)t.m)[e] = (uint8_t)(badm ? 0x7fu : cm);
      ((uint8_t*)t.v)[e] = (uint8_t)(badv ? 0x7fu : cv);
    }
  }
}

// Sums of squares, a CTA's in one partial: a thread adds g g exactly rounded into two fp32 words (the product's own
// error and that of each addition go to the lower word), the CTA adds those in fp64 in a fixed order.
template <int N>
__global__ void __launch_bounds__(256) k_sumsq(const __grid_constant__ AdamTable<N> tab, double* part) {
  pdl_enter();
  __shared__ double red[8];
  const int u0 = (int)((int64_t)tab.units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)tab.units * (blockIdx.x + 1) / gridDim.x);
  float hi = 0.f, lo = 0.f;
  int k = u0 < u1 ? tensor_of(tab, u0) : 0;
  for (int u = u0; u < u1; ++u) {
    while (k + 1 < tab.n && tab.t[k + 1].first <= u) ++k;
    const AdamTensor& t = tab.t[k];
    for (int j = 0; j < kAdamUnit / 256; ++j) {
      const int64_t e = (int64_t)(u - t.first) * kAdamUnit + threadIdx.x + 256 * j;
      if (e >= t.n) break;
      const float g = t.gb ? to_f(((const bf16*)t.grad)[e]) : ((const float*)t.grad)[e];
      const float q = __fmul_rn(g, g), w = __fmaf_rn(g, g, -q);
      const float sum = __fadd_rn(hi, q), b = __fadd_rn(sum, -hi);
      lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fadd_rn(hi, -__fadd_rn(sum, -b)), __fadd_rn(q, -b)), w));
      hi = sum;
    }
  }
  double d = (double)hi + (double)lo;
  for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) d += red[w];
    part[blockIdx.x] = d;
  }
}

__global__ void __launch_bounds__(256) k_norm(const double* part, int n, float* norm) {
  pdl_enter();
  __shared__ double red[256];
  double d = 0.;
  for (int i = threadIdx.x; i < n; i += 256) d += part[i];
  red[threadIdx.x] = d;
  __syncthreads();
  for (int o = 128; o; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) *norm = (float)sqrt(red[0]);
}

}  // namespace

int adamw_ctas(int64_t units) { return (int)std::min<int64_t>(units, (int64_t)sm_count() * 8); }

cudaError_t launch_adamw_begin(const AdamStep& c, int64_t* step, const float* norm, AdamScalars* s, cudaStream_t st) {
  return launch_pdl(k_adamw_begin, dim3(1), dim3(1), 0, st, c, step, norm, s);
}

template <int N>
cudaError_t launch_adamw(const AdamTable<N>& t, const AdamScalars* s, cudaStream_t st) {
  return launch_pdl(k_adamw<N>, dim3((unsigned)adamw_ctas(t.units)), dim3(256), 0, st, t, s);
}
template <int N>
cudaError_t launch_sumsq(const AdamTable<N>& t, double* part, cudaStream_t st) {
  return launch_pdl(k_sumsq<N>, dim3((unsigned)adamw_ctas(t.units)), dim3(256), 0, st, t, part);
}
cudaError_t launch_norm(const double* part, int n, float* norm, cudaStream_t st) {
  return launch_pdl(k_norm, dim3(1), dim3(256), 0, st, part, n, norm);
}
template cudaError_t launch_adamw<kAdamFew>(const AdamTable<kAdamFew>&, const AdamScalars*, cudaStream_t);
template cudaError_t launch_adamw<kAdamMany>(const AdamTable<kAdamMany>&, const AdamScalars*, cudaStream_t);
template cudaError_t launch_sumsq<kAdamFew>(const AdamTable<kAdamFew>&, double*, cudaStream_t);
template cudaError_t launch_sumsq<kAdamMany>(const AdamTable<kAdamMany>&, double*, cudaStream_t);

}  // namespace gbla
