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

// t in [0, 448] to an e4m3 magnitude, 16 random bits d: at the normal values (t >= 2^-6) the fraction's lower 20 bits,
// below them the fixed step 2^-9, floor(512 t + d 2^-16) (512 t is exact; floor by an addition rounded down at 2^23).
__device__ __forceinline__ uint32_t e4m3_up(float t, uint32_t d) {
  const uint32_t n = ((__float_as_uint(t) + (d << 4)) >> 20) - (120u << 3);
  const float u = __uint_as_float(0x3F800000u | d << 7) - 1.f;  // d 2^-16
  const uint32_t s = __float_as_uint(__fadd_rd(__fmaf_rn(t, 512.f, u), 8388608.f)) & 15u;
  return t >= 0x1p-6f ? n : s;
}
// Two e4m3 values (exact in fp16 and fp32).
__device__ __forceinline__ float2 e4m3x2(uint32_t w) {
  uint32_t h;
  float2 o;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  asm("{\n .reg .f16 l, g;\n mov.b32 {l, g}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, g;\n}" : "=f"(o.x), "=f"(o.y) : "r"(h));
  return o;
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

// One value: m, root = sqrt(v) and p moved by g.
__device__ __forceinline__ void move(float g, float& m, float& v, float& root, float& p, const AdamScalars& s, float keep) {
  g = __fmul_rn(g, s.clip);
  m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.c1, g));
  v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(__fmul_rn(s.c2, g), g));
  root = __fsqrt_rn(v);
  p = p * keep - s.step * __fdividef(m, fmaf(root, s.inv, s.eps));
}

// Four values at p from element e on: in one access where the tensor is aligned and all are there, else the nv there are.
__device__ __forceinline__ void load4(float (&o)[4], const void* p, int64_t e, bool b16, bool wide, int nv) {
  if (wide) {
    if (b16) {
      const uint2 w = __ldcs((const uint2*)((const bf16*)p + e));
      o[0] = bf_lo(w.x); o[1] = bf_hi(w.x); o[2] = bf_lo(w.y); o[3] = bf_hi(w.y);
    } else {
      const float4 w = __ldcs((const float4*)((const float*)p + e));
      o[0] = w.x; o[1] = w.y; o[2] = w.z; o[3] = w.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = j >= nv ? 0.f : b16 ? to_f(((const bf16*)p)[e + j]) : ((const float*)p)[e + j];
}
__device__ __forceinline__ void store4(const float (&v)[4], void* p, int64_t e, bool b16, bool wide, int nv) {
  if (wide) {
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
__device__ __forceinline__ uint32_t load4b(const void* p, int64_t e, bool wide, int nv) {
  if (wide) return __ldcs((const uint32_t*)((const uint8_t*)p + e));
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < nv) w |= (uint32_t)((const uint8_t*)p)[e + j] << 8 * j;
  return w;
}
__device__ __forceinline__ void store4b(uint32_t w, void* p, int64_t e, bool wide, int nv) {
  if (wide) {
    __stcs((uint32_t*)((uint8_t*)p + e), w);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < nv) ((uint8_t*)p)[e + j] = (uint8_t)(w >> 8 * j);
}

// One pass over every tensor: bound by memory.  A warp takes a block of 256 values at a time, lane l those at 4 l .. 4 l + 3
// of either half: 16-byte accesses of fp32, and the block's largest magnitudes by one warp reduction each.
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
    const bool q8 = t.ms != nullptr, pb = t.pb && !t.master;  // pb: updated in bf16
    const int64_t blk = e0 / kAdamBlock;
    void* src = t.master ? (void*)t.master : t.param;
    float g[2][4], p[2][4], m[2][4], r[2][4];
    uint32_t wm[2], wv[2];
    int64_t e[2];
    int nv[2];
    bool wide[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      e[h] = e0 + 128 * h + 4 * lane;
      nv[h] = (int)max((int64_t)0, min((int64_t)4, t.n - e[h]));
      wide[h] = t.vec && nv[h] == 4;
      load4(g[h], t.grad, e[h], t.gb, wide[h], nv[h]);
      load4(p[h], src, e[h], pb, wide[h], nv[h]);
      if (q8) {
        wm[h] = load4b(t.m, e[h], wide[h], nv[h]);
        wv[h] = load4b(t.v, e[h], wide[h], nv[h]);
      } else {
        load4(m[h], t.m, e[h], false, wide[h], nv[h]);
        load4(r[h], t.v, e[h], false, wide[h], nv[h]);
      }
    }
    if (q8) {
      const float sm = t.ms[blk], sv = t.vs[blk];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 a = e4m3x2(wm[h]), b = e4m3x2(wm[h] >> 16), c = e4m3x2(wv[h]), d = e4m3x2(wv[h] >> 16);
        m[h][0] = __fmul_rn(a.x, sm); m[h][1] = __fmul_rn(a.y, sm); m[h][2] = __fmul_rn(b.x, sm); m[h][3] = __fmul_rn(b.y, sm);
        r[h][0] = __fmul_rn(c.x, sv); r[h][1] = __fmul_rn(c.y, sv); r[h][2] = __fmul_rn(d.x, sv); r[h][3] = __fmul_rn(d.y, sv);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[h][j] = __fmul_rn(r[h][j], r[h][j]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float root;
        move(g[h][j], m[h][j], r[h][j], root, p[h][j], s, t.keep);
        if (q8) r[h][j] = root;
      }
      store4(p[h], src, e[h], pb, wide[h], nv[h]);
      if (t.master) store4(p[h], t.param, e[h], true, wide[h], nv[h]);
      if (!q8) {
        store4(m[h], t.m, e[h], false, wide[h], nv[h]);
        store4(r[h], t.v, e[h], false, wide[h], nv[h]);
      }
    }
    if (!q8) continue;
    // the largest magnitudes as bit patterns: a NaN or infinity is the largest of all (values past the end do not count)
    uint32_t tm = 0, tv = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < nv[h]) {
          tm = max(tm, __float_as_uint(m[h][j]) & 0x7fffffffu);
          tv = max(tv, __float_as_uint(r[h][j]) & 0x7fffffffu);
        }
    tm = __reduce_max_sync(FULL, tm);
    tv = __reduce_max_sync(FULL, tv);
    const float fm = __uint_as_float(tm), fv = __uint_as_float(tv);
    const bool badm = tm >= 0x7f800000u, badv = tv >= 0x7f800000u;
    const float im = fm >= 0x1p-100f ? __fmul_rn(__frcp_rn(fm), 448.f) : 0.f;
    const float iv = fv >= 0x1p-100f ? __fmul_rn(__frcp_rn(fv), 448.f) : 0.f;
    __syncwarp();  // every lane has read the block's scales
    if (lane == 0) {
      t.ms[blk] = badm ? __uint_as_float(0x7fc00000u) : fm >= 0x1p-100f ? __fmul_rn(fm, 1.f / 448.f) : 0.f;
      t.vs[blk] = badv ? __uint_as_float(0x7fc00000u) : fv >= 0x1p-100f ? __fmul_rn(fv, 1.f / 448.f) : 0.f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t cm = 0, cv = 0;
      const uint64_t place = (uint64_t)(t.place + e[h]);
      const uint32_t base = (uint32_t)place * 0x9E3779B9u + (uint32_t)(place >> 32) * 0xBB67AE85u + s.key;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // (four neighbours share the place's upper word: places of blocks are multiples of 256)
        const uint32_t z = mix32(base + j * 0x9E3779B9u);
        const float xm = fminf(__fmul_rn(fabsf(m[h][j]), im), 448.f), xv = fminf(__fmul_rn(r[h][j], iv), 448.f);
        const uint32_t a = e4m3_up(xm, z & 0xffffu) | (__float_as_uint(m[h][j]) >> 31 << 7);
        uint32_t b = e4m3_up(xv, z >> 16);
        if (xv > 0.f) b = max(b, 1u);
        cm |= a << 8 * j;
        cv |= b << 8 * j;
      }
      store4b(badm ? 0x7f7f7f7fu : cm, t.m, e[h], wide[h], nv[h]);
      store4b(badv ? 0x7f7f7f7fu : cv, t.v, e[h], wide[h], nv[h]);
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
    float g[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t e = (int64_t)(u - t.first) * kAdamUnit + 1024 * h + 4 * threadIdx.x;
      const int nv = (int)max((int64_t)0, min((int64_t)4, t.n - e));
      load4(g[h], t.grad, e, t.gb, t.vec && nv == 4, nv);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = g[h][j], q = __fmul_rn(v, v), w = __fmaf_rn(v, v, -q);
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
