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
// The 32 random bits of a place are mix32(low word of the place * 0x9E3779B9 (the fraction bits of the golden ratio spread
// neighbours) + high word * 0xBB67AE85 + the step's key).

// |t| in [0, 448] (or two units in the last place above: the sum below does not reach the next code) to an e4m3 magnitude in the
// top byte, with 16 random bits.  From t 2^-120, where the normal values of e4m3 (t >= 2^-6) are the fp32 ones of 3 fraction
// bits, the random bits at bits 8 .. 23 of d; 0 stays 0.
__device__ __forceinline__ uint32_t e4m3_up(float t, uint32_t d) { return (__float_as_uint(t) << 4) + d; }
// Below 2^-6 the fixed step 2^-9: floor(512 t + d 2^-16) (both products exact; floor by an addition rounded down at 2^23), of
// two values; d the low or the high half of z.
__device__ __forceinline__ uint2 e4m3_low(float2 t, uint32_t z0, uint32_t z1) {
  const float2 d = make_float2((float)(uint16_t)z0, (float)(uint16_t)z1);
  const float2 s = __fadd2_rd(__ffma2_rn(d, make_float2(0x1p-16f, 0x1p-16f), __fmul2_rn(t, make_float2(512.f, 512.f))), make_float2(8388608.f, 8388608.f));
  return make_uint2(__float_as_uint(s.x) << 24, __float_as_uint(s.y) << 24);
}
// The top bytes of four words.
__device__ __forceinline__ uint32_t top4(const uint32_t (&w)[4]) {
  return __byte_perm(__byte_perm(w[0], w[1], 0x0073), __byte_perm(w[2], w[3], 0x0073), 0x5410);
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The larger of c and |a|, |b|; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float o;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(o) : "f"(a), "f"(b), "f"(c));
  return o;
}
// Two e4m3 values (exact in fp16 and fp32).
__device__ __forceinline__ float2 e4m3x2(uint32_t w) {
  uint32_t h;
  float2 o;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  asm("{\n .reg .f16 l, g;\n mov.b32 {l, g}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, g;\n}" : "=f"(o.x), "=f"(o.y) : "r"(h));
  return o;
}

__global__ void k_adamw_begin(const AdamStep c, int64_t* step, const float* norm, AdamScalars* s, int* err) {
  pdl_enter();
  *err = 0;
  const float nm = norm ? *norm : 0.f;
  AdamScalars o;
  o.go = isfinite(nm);
  const int64_t t = *step + 1;
  if (o.go) *step = t;
  o.clip = norm && c.max_norm > 0. ? fminf(__fmul_rn(__frcp_rn(__fadd_rn(nm, 1e-6f)), (float)c.max_norm), 1.f) : 1.f;
  o.b1 = (float)c.b1; o.c1 = (float)(1. - c.b1);
  o.b2 = (float)c.b2; o.c2 = (float)(1. - c.b2);
  // 1 - b^t = -expm1(t ln b): relative errors of 2^-23, in fp32 (a power in fp64 takes this one thread 9 us)
  o.step = __fdiv_rn((float)c.lr, -expm1f((float)((double)t * c.ln1)));
  o.inv = __frcp_rn(__fsqrt_rn(-expm1f((float)((double)t * c.ln2))));
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

// Two products, each rounded once.  (Scalar instructions: a packed product and a packed sum that take one another come out
// of the assembler as one fused operation, whatever rounding they ask for: an ulp off in one value of six, measured.)
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y)); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
// Two products that no sum takes.
__device__ __forceinline__ float2 times(float2 a, float2 b) { return __fmul2_rn(a, b); }
// Two values: m, v, root = sqrt(v) and p moved by g; every operation of m, v and root rounded once.
__device__ __forceinline__ void move(float2 g, float2& m, float2& v, float2& root, float2& p, const AdamScalars& s, float keep) {
  auto all = [](float x) { return make_float2(x, x); };
  g = times(g, all(s.clip));
  m = add2(mul2(all(s.b1), m), mul2(all(s.c1), g));
  v = add2(mul2(all(s.b2), v), mul2(times(all(s.c2), g), g));
  root = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 den = __ffma2_rn(root, all(s.inv), all(s.eps));
  const float2 q = times(m, make_float2(rcpf(den.x), rcpf(den.y)));  // a reciprocal of 1 ulp, and its product
  p = __ffma2_rn(all(-s.step), q, mul2(p, all(keep)));
}

// Four values at p from element e on: WIDE in one access, else the nv there are.  KEEP: they will be read again.
template <bool WIDE, bool KEEP = false>
__device__ __forceinline__ void load4(float (&o)[4], const void* p, int64_t e, bool b16, int nv) {
  if (WIDE) {
    if (b16) {
      const uint2* at = (const uint2*)((const bf16*)p + e);
      const uint2 w = KEEP ? __ldg(at) : __ldcs(at);
      o[0] = bf_lo(w.x); o[1] = bf_hi(w.x); o[2] = bf_lo(w.y); o[3] = bf_hi(w.y);
    } else {
      const float4* at = (const float4*)((const float*)p + e);
      const float4 w = KEEP ? __ldg(at) : __ldcs(at);
      o[0] = w.x; o[1] = w.y; o[2] = w.z; o[3] = w.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = j >= nv ? 0.f : b16 ? to_f(((const bf16*)p)[e + j]) : ((const float*)p)[e + j];
}
template <bool WIDE>
__device__ __forceinline__ void store4(const float (&v)[4], void* p, int64_t e, bool b16, int nv) {
  if (WIDE) {
    if (b16) __stcs((uint2*)((bf16*)p + e), make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])));
    else __stcs((float4*)((float*)p + e), make_float4(v[0], v[1], v[2], v[3]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < nv) {
      if (b16) ((bf16*)p)[e + j] = from_f<bf16>(v[j]);
      else ((float*)p)[e + j] = v[j];
    }
}
template <bool WIDE>
__device__ __forceinline__ uint32_t load4b(const void* p, int64_t e, int nv) {
  if (WIDE) return __ldcs((const uint32_t*)((const uint8_t*)p + e));
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < nv) w |= (uint32_t)((const uint8_t*)p)[e + j] << 8 * j;
  return w;
}
template <bool WIDE>
__device__ __forceinline__ void store4b(uint32_t w, void* p, int64_t e, int nv) {
  if (WIDE) {
    __stcs((uint32_t*)((uint8_t*)p + e), w);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < nv) ((uint8_t*)p)[e + j] = (uint8_t)(w >> 8 * j);
}

// A warp's block of 256 values from e0 on, lane l those at 4 l .. 4 l + 3 of either half: 16-byte accesses of fp32, and the
// block's largest magnitudes by one warp reduction each.  WIDE: the block is whole and aligned.
template <bool Q8, bool WIDE>
__device__ __forceinline__ void block_step(const AdamTensor& t, int64_t e0, const AdamScalars& s, int lane) {
  const bool pb = t.pb && !t.master;  // updated in bf16
  const int64_t blk = e0 / kAdamBlock;
  void* src = t.master ? (void*)t.master : t.param;
  float g[2][4], p[2][4], m[2][4], r[2][4];
  uint32_t wm[2], wv[2];
  int nv[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t e = e0 + 128 * h + 4 * lane;
    nv[h] = WIDE ? 4 : (int)max((int64_t)0, min((int64_t)4, t.n - e));
    load4<WIDE>(g[h], t.grad, e, t.gb, nv[h]);
    load4<WIDE>(p[h], src, e, pb, nv[h]);
    if (Q8) {
      wm[h] = load4b<WIDE>(t.m, e, nv[h]);
      wv[h] = load4b<WIDE>(t.v, e, nv[h]);
    } else {
      load4<WIDE>(m[h], t.m, e, false, nv[h]);
      load4<WIDE>(r[h], t.v, e, false, nv[h]);
    }
  }
  if (Q8) {
    const float2 sm = make_float2(t.ms[blk], t.ms[blk]), sv = make_float2(t.vs[blk], t.vs[blk]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float2 a = times(e4m3x2(wm[h] >> 8 * j), sm);
        float2 b = times(e4m3x2(wv[h] >> 8 * j), sv);
        b = times(b, b);
        m[h][j] = a.x; m[h][j + 1] = a.y;
        r[h][j] = b.x; r[h][j + 1] = b.y;
      }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      float2 a = make_float2(m[h][j], m[h][j + 1]), v = make_float2(r[h][j], r[h][j + 1]), q = make_float2(p[h][j], p[h][j + 1]), root;
      move(make_float2(g[h][j], g[h][j + 1]), a, v, root, q, s, t.keep);
      m[h][j] = a.x; m[h][j + 1] = a.y;
      if (Q8) v = root;
      r[h][j] = v.x; r[h][j + 1] = v.y;
      p[h][j] = q.x; p[h][j + 1] = q.y;
    }
    const int64_t e = e0 + 128 * h + 4 * lane;
    store4<WIDE>(p[h], src, e, pb, nv[h]);
    if (t.master) store4<WIDE>(p[h], t.param, e, true, nv[h]);
    if (!Q8) {
      store4<WIDE>(m[h], t.m, e, false, nv[h]);
      store4<WIDE>(r[h], t.v, e, false, nv[h]);
    }
  }
  if (!Q8) return;
  float fm = 0.f, fv = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!WIDE) {  // values past the end do not count
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j >= nv[h]) m[h][j] = r[h][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      fm = max_abs(m[h][j], m[h][j + 1], fm);
      fv = max_abs(r[h][j], r[h][j + 1], fv);
    }
  }
  // as bit patterns: a NaN or infinity is the largest of all
  fm = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(fm)));
  fv = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(fv)));
  const bool badm = __float_as_uint(fm) >= 0x7f800000u, badv = __float_as_uint(fv) >= 0x7f800000u;
  const float im = fm >= 0x1p-100f ? __fmul_rn(__frcp_rn(fm), 448.f) : 0.f;
  const float iv = fv >= 0x1p-100f ? __fmul_rn(__frcp_rn(fv), 448.f) : 0.f;
  __syncwarp();  // every lane has read the block's scales
  if (lane == 0) {
    t.ms[blk] = badm ? __uint_as_float(0x7fc00000u) : fm >= 0x1p-100f ? __fmul_rn(fm, 1.f / 448.f) : 0.f;
    t.vs[blk] = badv ? __uint_as_float(0x7fc00000u) : fv >= 0x1p-100f ? __fmul_rn(fv, 1.f / 448.f) : 0.f;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t cm[4], cv[4], sign[4];
    const int64_t e = e0 + 128 * h + 4 * lane;
    const uint64_t place = (uint64_t)(t.place + e);
    const uint32_t base = (uint32_t)place * 0x9E3779B9u + (uint32_t)(place >> 32) * 0xBB67AE85u + s.key;
    const float2 down = make_float2(0x1p-120f, 0x1p-120f);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {  // (four neighbours share the place's upper word: places of blocks are multiples of 256)
      const float2 xm = times(make_float2(fabsf(m[h][j]), fabsf(m[h][j + 1])), make_float2(im, im));
      const float2 xv = times(make_float2(r[h][j], r[h][j + 1]), make_float2(iv, iv));
      const float2 tm = times(xm, down), tv = times(xv, down);
      const uint32_t z0 = mix32(base + j * 0x9E3779B9u), z1 = mix32(base + (j + 1) * 0x9E3779B9u);
      const uint2 lm = e4m3_low(xm, z0, z1), lv = e4m3_low(xv, z0 >> 16, z1 >> 16);
      cm[j] = xm.x < 0x1p-6f ? lm.x : e4m3_up(tm.x, __byte_perm(z0, 0, 0x4104));
      cm[j + 1] = xm.y < 0x1p-6f ? lm.y : e4m3_up(tm.y, __byte_perm(z1, 0, 0x4104));
      cv[j] = xv.x < 0x1p-6f ? lv.x : e4m3_up(tv.x, __byte_perm(z0, 0, 0x4324));
      cv[j + 1] = xv.y < 0x1p-6f ? lv.y : e4m3_up(tv.y, __byte_perm(z1, 0, 0x4324));
      if (xv.x > 0.f) cv[j] = max(cv[j], 1u << 24);
      if (xv.y > 0.f) cv[j + 1] = max(cv[j + 1], 1u << 24);
      sign[j] = __float_as_uint(m[h][j]);
      sign[j + 1] = __float_as_uint(m[h][j + 1]);
    }
    store4b<WIDE>(badm ? 0x7f7f7f7fu : top4(cm) | (top4(sign) & 0x80808080u), t.m, e, nv[h]);
    store4b<WIDE>(badv ? 0x7f7f7f7fu : top4(cv), t.v, e, nv[h]);
  }
}

// n bytes at p will be read: 16-byte aligned, a multiple of 16.
__device__ __forceinline__ void to_l2(const void* p, int n) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n) : "memory");
}

// One pass over every tensor, tables of tensors in the launch's parameters (one launch for up to 336).  Bound by memory with
// fp32 states (12.6 M values of bf16 parameters with masters, 30 bytes each: 77 us with the norm and both small launches, 5.0
// TB/s; 57 us of it here), with 8-bit states by instructions (99 a value, 78 % of the issue slots at 5.6 TB/s; 201 M values, 18
// bytes each: 800 us with the norm, which reads 0.8 GB again).  At 64 registers and 4 CTAs an SM a warp's loads of one block do
// not cover the time it takes, so with 8-bit states its next block is brought into L2 meanwhile (860 us before; two and four
// blocks ahead are 10 and 75 us slower than one); with fp32 states 80 us with, 77 without.  5 CTAs an SM, or one wave of CTAs
// rather than two: 20 and 60 us slower.
template <int N>
__global__ void __launch_bounds__(256, 4) k_adamw(const __grid_constant__ AdamTable<N> tab, const AdamScalars* sc) {
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
    const bool wide = t.vec && e0 + kAdamBlock <= t.n;
    const int64_t e1 = e0 + kAdamUnit;
    if (t.ms && lane == 0 && t.vec && e1 + kAdamBlock <= t.n && u + 1 < u1) {
      const bool pb = t.pb && !t.master;
      to_l2((const uint8_t*)t.grad + (e1 << (t.gb ? 1 : 2)), kAdamBlock << (t.gb ? 1 : 2));
      to_l2((const uint8_t*)(t.master ? (void*)t.master : t.param) + (e1 << (pb ? 1 : 2)), kAdamBlock << (pb ? 1 : 2));
      to_l2((const uint8_t*)t.m + e1, kAdamBlock);
      to_l2((const uint8_t*)t.v + e1, kAdamBlock);
    }
    if (t.ms) {
      if (wide) block_step<true, true>(t, e0, s, lane);
      else block_step<true, false>(t, e0, s, lane);
    } else {
      if (wide) block_step<false, true>(t, e0, s, lane);
      else block_step<false, false>(t, e0, s, lane);
    }
  }
}

// Sums of squares, a CTA's in one partial: a thread adds g g into two fp32 words (the product's own error and that of each
// addition go to the lower word), the CTA adds those in fp64 in a fixed order.  A thread whose sum passes the fp32 range goes
// over its values again in fp64.  Bound by memory: 0.8 GB of fp32 gradients in two tables in 106 + 37 us, 5.7 TB/s.
template <int N>
__global__ void __launch_bounds__(256) k_sumsq(const __grid_constant__ AdamTable<N> tab, double* part) {
  pdl_enter();
  __shared__ double red[8];
  const int u0 = (int)((int64_t)tab.units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)tab.units * (blockIdx.x + 1) / gridDim.x);
  auto walk = [&](auto&& add) {  // the thread's values
    int k = u0 < u1 ? tensor_of(tab, u0) : 0;
    for (int u = u0; u < u1; ++u) {
      while (k + 1 < tab.n && tab.t[k + 1].first <= u) ++k;
      const AdamTensor& t = tab.t[k];
      float g[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t e = (int64_t)(u - t.first) * kAdamUnit + 1024 * h + 4 * threadIdx.x;
        const int nv = (int)max((int64_t)0, min((int64_t)4, t.n - e));
        if (t.vec && nv == 4) load4<true, true>(g[h], t.grad, e, t.gb, nv);
        else load4<false>(g[h], t.grad, e, t.gb, nv);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) add(g[h][j]);
    }
  };
  float hi = 0.f, lo = 0.f;
  walk([&](float v) {
    const float q = __fmul_rn(v, v), w = __fmaf_rn(v, v, -q);
    const float sum = __fadd_rn(hi, q), b = __fadd_rn(sum, -hi);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fadd_rn(hi, -__fadd_rn(sum, -b)), __fadd_rn(q, -b)), w));
    hi = sum;
  });
  double d = (double)hi + (double)lo;
  if (!isfinite(hi)) {
    d = 0.;
    walk([&](float v) { d += isfinite(__fmul_rn(v, v)) ? (double)v * (double)v : (double)__fmul_rn(v, v); });
  }
  for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) d += red[w];
    part[blockIdx.x] = d;
  }
}

__global__ void __launch_bounds__(256) k_norm(const double* part, int n, float* norm, int* err) {
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
  if (threadIdx.x == 0) {
    *norm = (float)sqrt(red[0]);
    *err = 0;
  }
}

}  // namespace

int adamw_ctas(int64_t units) { return (int)std::min<int64_t>(units, (int64_t)sm_count() * 8); }

cudaError_t launch_adamw_begin(const AdamStep& c, int64_t* step, const float* norm, AdamScalars* s, int* err, cudaStream_t st) {
  return launch_pdl(k_adamw_begin, dim3(1), dim3(1), 0, st, c, step, norm, s, err);
}

template <int N>
cudaError_t launch_adamw(const AdamTable<N>& t, const AdamScalars* s, cudaStream_t st) {
  return launch_pdl(k_adamw<N>, dim3((unsigned)adamw_ctas(t.units)), dim3(256), 0, st, t, s);
}
template <int N>
cudaError_t launch_sumsq(const AdamTable<N>& t, double* part, cudaStream_t st) {
  return launch_pdl(k_sumsq<N>, dim3((unsigned)adamw_ctas(t.units)), dim3(256), 0, st, t, part);
}
cudaError_t launch_norm(const double* part, int n, float* norm, int* err, cudaStream_t st) {
  return launch_pdl(k_norm, dim3(1), dim3(256), 0, st, part, n, norm, err);
}
template cudaError_t launch_adamw<kAdamFew>(const AdamTable<kAdamFew>&, const AdamScalars*, cudaStream_t);
template cudaError_t launch_adamw<kAdamMany>(const AdamTable<kAdamMany>&, const AdamScalars*, cudaStream_t);
template cudaError_t launch_sumsq<kAdamFew>(const AdamTable<kAdamFew>&, double*, cudaStream_t);
template cudaError_t launch_sumsq<kAdamMany>(const AdamTable<kAdamMany>&, double*, cudaStream_t);

}  // namespace gbla
