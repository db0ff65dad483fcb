// svla_op_adamw: one AdamW step over many tensors (see the declaration in
// svla.h), with the moments in 32 bits or in 8, and the clip by the global
// gradient norm. The update half of the expert's fine-tune, whose loss and
// gradients svla_train_step computes.
//
// Per element, the moments' products and sums rounded to fp32 one by one (no
// fused multiply-add), so what is stored does not depend on how the compiler
// contracts the expression:
//   g' = g c,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   p  = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// The tensors' table travels in the kernel's parameters: nothing is copied to
// the device and nothing is kept between calls. A warp takes 256 consecutive
// elements of one tensor, the block that shares a scale in the 8-bit states, 8
// consecutive ones a lane.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <exception>
#include <string>
#include <utility>
#include <vector>

#include "common.cuh"
#include "elements.cuh"
#include "philox.cuh"

svla_status svla_internal_fail(svla_status s, const char* msg);

namespace svla {
namespace {

constexpr int ADAMW_BLOCK = 256;   // elements of a warp's task = elements that share a scale
constexpr int ADAMW_CAP = 400;     // tensors of one launch (27.6 KB of the 32,764 bytes of kernel parameters)
constexpr int ADAMW_THREADS = 256;
constexpr int ADAMW_WARPS = ADAMW_THREADS / 32;
constexpr int NORM_BLOCKS = 592;   // blocks (and partial sums) of one launch of the norm: 4 on each of 148 SMs

struct AdamwEntry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint16_t* copy;
  long long n;
};

struct AdamwTable {
  AdamwEntry e[ADAMW_CAP];
  uint32_t first[ADAMW_CAP + 1];  // first 256-element block of each tensor; first[count] = all blocks
  uint8_t flags[ADAMW_CAP];       // 1: weight decay, 2: every pointer allows the vector accesses
  int count;
};
constexpr uint8_t AF_DECAY = 1, AF_VEC = 2;

struct AdamwCoefs {
  float b1, c1, b2, c2, eps;
  float keep;       // 1 - lr wd
  float step_size;  // lr / (1 - b1^t)
  float isb2;       // 1 / sqrt(1 - b2^t)
  float minus0;     // -0 (product2)
  double max_norm;  // 0: no clip
  uint32_t k0, k1, step, tensor0;
  // read on the device instead of the host's numbers, where given
  const long long* step_dev;
  const double* lr_dev;
  double lr, beta1, beta2, wd;
};

// tensor of block `blk`: the last t with first[t] <= blk (empty tensors have no block)
SVLA_DEV int find_tensor(const AdamwTable& t, uint32_t blk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= blk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Two fp32 values in one register pair: the packed operations round each half
// like the scalar ones and take half the issue slots.
typedef unsigned long long f32x2;
SVLA_DEV f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
SVLA_DEV float2 halves(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
SVLA_DEV f32x2 both(float x) { return pair(x, x); }
SVLA_DEV f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SVLA_DEV f32x2 mul2_ftz(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SVLA_DEV f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SVLA_DEV f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A product that is rounded before it is added to: the compiler fuses a packed
// product and sum even where both are .rn, but not two fused operations. The
// addend -0 changes no product; it comes from the kernel's arguments, so that
// the compiler does not know it.
SVLA_DEV f32x2 product2(f32x2 a, f32x2 b, f32x2 minus0) { return fma2(a, b, minus0); }

// two 8-bit codes -> two floats (exact; through fp16, which holds both formats:
// an e5m2 code is the upper byte of its fp16 value)
SVLA_DEV float2 decode_m2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
template <int K>
SVLA_DEV float2 decode_v2(uint32_t four) {
  const uint32_t h = __byte_perm(four, 0, K ? 0x3424 : 0x1404);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// two values that the formats hold -> their codes (lo in the low byte)
SVLA_DEV uint32_t code_m2(f32x2 x) {
  uint16_t r;
  const float2 f = halves(x);
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(f.y), "f"(f.x));
  return r;
}
SVLA_DEV uint32_t code_v2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 elements of this lane from a warp's 256, raw, packed into words. `vec`: the
// consecutive elements lane * 8 .., one 32-byte (fp32), 16-byte (bf16) or 8-byte
// (codes) access; else (a tensor's last, shorter block, or a tensor at an odd
// address) the elements lane, lane + 32, .., zeros past the tensor's end.
template <typename E>
struct Raw8 {
  uint32_t w[2 * sizeof(E)];
};
template <typename E>
SVLA_DEV void raw_load(const E* p, bool vec, int left, int lane, Raw8<E>& r) {
  if (vec) {
    if constexpr (sizeof(E) == 4) {
      ld_global_v8(p + lane * 8, r.w);
    } else if constexpr (sizeof(E) == 2) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + lane * 8);
      r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p + lane * 8);
      r.w[0] = q.x, r.w[1] = q.y;
    }
    return;
  }
  uint32_t x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (sizeof(E) == 4)
      x[j] = j * 32 + lane < left ? __float_as_uint(p[j * 32 + lane]) : 0u;
    else
      x[j] = j * 32 + lane < left ? p[j * 32 + lane] : 0u;
  }
  constexpr int PER = 4 / sizeof(E);  // elements of a word
#pragma unroll
  for (int k = 0; k < 8 / PER; ++k) {
    r.w[k] = x[PER * k];
#pragma unroll
    for (int q = 1; q < PER; ++q) r.w[k] |= x[PER * k + q] << (8 * sizeof(E) * q);
  }
}
template <typename E>
SVLA_DEV void raw_store(E* p, bool vec, int left, int lane, const Raw8<E>& r) {
  if (vec) {
    if constexpr (sizeof(E) == 4)
      st_global_v8(p + lane * 8, r.w);
    else if constexpr (sizeof(E) == 2)
      *reinterpret_cast<uint4*>(p + lane * 8) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else
      *reinterpret_cast<uint2*>(p + lane * 8) = make_uint2(r.w[0], r.w[1]);
    return;
  }
  constexpr int PER = 4 / sizeof(E);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j * 32 + lane < left) {
      const uint32_t x = r.w[j / PER] >> (8 * sizeof(E) * (j % PER));
      if constexpr (sizeof(E) == 4)
        p[j * 32 + lane] = __uint_as_float(x);
      else
        p[j * 32 + lane] = (E)x;
    }
}
SVLA_DEV float value(const Raw8<float>& r, int j) { return __uint_as_float(r.w[j]); }
SVLA_DEV float value(const Raw8<uint16_t>& r, int j) {
  return __uint_as_float((j & 1) ? (r.w[j >> 1] & 0xffff0000u) : (r.w[j >> 1] << 16));
}
SVLA_DEV void pack(const float (&x)[8], Raw8<float>& r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) r.w[j] = __float_as_uint(x[j]);
}
SVLA_DEV void pack(const float (&x)[8], Raw8<uint16_t>& r) {
#pragma unroll
  for (int j = 0; j < 4; ++j) r.w[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
}

// Codes of the 8-bit moments: the top bits of the fp32 magnitude, its exponent
// counted from a power of two that the block's largest finite magnitude sets.
// u20 (16 random bits << 4) enters at the top of the dropped bits: the code is
// rounded up with the probability of its distance to the lower code, so the
// stored moment is right in the mean. Nearest rounding would hold v where it
// is: a step moves v by (1 - b2) ~ 1e-3 of itself and the codes lie 1/8 to 1/4
// apart.
//   m: e4m3, largest magnitude in [2^7, 2^8) of the scale; below 2^-6 -> 0
//   v: e5m2, largest in [2^14, 2^15); 0 < v below 2^-14 -> 2^-14, so no
//      gradient is ever divided by a vanished v
// Subnormal codes are not made. Values that are not finite are put in later.
SVLA_DEV uint32_t encode_m(float x, uint32_t u20, uint32_t low) {
  const uint32_t bits = __float_as_uint(x);
  const int code = (int)(((bits & 0x7fffffffu) + u20) >> 20) - (int)low;
  return code < 8 ? 0u : (uint32_t)code | ((bits >> 24) & 0x80u);
}
SVLA_DEV uint32_t encode_v(float x, uint32_t u20, uint32_t low) {
  const uint32_t mag = __float_as_uint(x);
  const int code = max((int)(((mag >> 1) + u20) >> 20) - (int)low, 4);
  return mag == 0 ? 0u : (uint32_t)code;
}
SVLA_DEV uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t INF_MAG = 0x7f800000u;

// One element: the moments, each product and sum rounded to fp32 by itself, and
// the parameter.
SVLA_DEV void update1(const AdamwCoefs& c, float keep, float g, float& p, float& m, float& v) {
  m = __fadd_rn(__fmul_rn(m, c.b1), __fmul_rn(g, c.c1));
  v = __fadd_rn(__fmul_rn(v, c.b2), __fmul_rn(__fmul_rn(g, g), c.c2));
  const float q = __fdiv_rn(m, __fmaf_rn(__fsqrt_rn(v), c.isb2, c.eps));
  p = __fmaf_rn(-q, c.step_size, p * keep);
}

// The 8-bit step of a warp's block whatever its values: a zero v, moments near
// the ends of fp32's range, or ones that are not finite (they take the NaN
// code; the scales are those of the finite ones).
template <typename TP, typename TG>
SVLA_DEV void general8(const AdamwCoefs& c, float keep, float clip, const TP* pp, const TG* gp, const uint8_t* mp,
                       const uint8_t* vp, bool vec, int left, int lane, float ms, float vs, const uint32_t (&r)[4],
                       float (&p)[8], Raw8<uint8_t>& rm, Raw8<uint8_t>& rv, uint32_t& mx, uint32_t& vx) {
  Raw8<TP> rp;
  Raw8<TG> rg;
  raw_load(pp, vec, left, lane, rp);
  raw_load(gp, vec, left, lane, rg);
  raw_load(mp, vec, left, lane, rm);
  raw_load(vp, vec, left, lane, rv);
  float m[8], v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = decode_m2((rm.w[k >> 1] >> (16 * (k & 1))) & 0xffffu);
    const float2 y = k & 1 ? decode_v2<1>(rv.w[k >> 1]) : decode_v2<0>(rv.w[k >> 1]);
    m[2 * k] = __fmul_rn(x.x, ms), m[2 * k + 1] = __fmul_rn(x.y, ms);
    v[2 * k] = __fmul_rn(y.x, vs), v[2 * k + 1] = __fmul_rn(y.y, vs);
  }
  mx = vx = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j] = value(rp, j);
    update1(c, keep, __fmul_rn(value(rg, j), clip), p[j], m[j], v[j]);
    if (magnitude(m[j]) < INF_MAG) mx = max(mx, magnitude(m[j]));
    if (magnitude(v[j]) < INF_MAG) vx = max(vx, magnitude(v[j]));
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  vx = __reduce_max_sync(0xffffffffu, vx);
  const uint32_t em = (uint32_t)max((int)(mx >> 23) - 14, 0), ev = (uint32_t)max((int)(vx >> 23) - 29, 0);
  uint32_t mc[8], vc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u20 = (j & 1) ? (r[j >> 1] >> 12) & 0xffff0u : (r[j >> 1] & 0xffffu) << 4;
    mc[j] = magnitude(m[j]) >= INF_MAG ? 0x7fu : encode_m(m[j], u20, em << 3);
    vc[j] = magnitude(v[j]) >= INF_MAG ? 0x7fu : encode_v(v[j], u20, ev << 2);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    rm.w[k] = mc[4 * k] | mc[4 * k + 1] << 8 | mc[4 * k + 2] << 16 | mc[4 * k + 3] << 24;
    rv.w[k] = vc[4 * k] | vc[4 * k + 1] << 8 | vc[4 * k + 2] << 16 | vc[4 * k + 3] << 24;
  }
}

// The usual case of the 8-bit step: v below 2^100 (its product with 2^24 is
// finite), |m| below 2^13 (the factor 2^-120 / m_scale is a normal number).
constexpr uint32_t VX_USUAL = (127u + 100u) << 23, MX_USUAL = (127u + 13u) << 23;
SVLA_DEV float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
SVLA_DEV float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---------------------------------------------------------------------------
// Sum of squares of the gradients: fp64 throughout, so the norm (and with it
// the clip factor's fp32 rounding) does not depend on the order of the sum in
// practice; fixed order all the same. partial[blockIdx.x] of this launch.
// ---------------------------------------------------------------------------
template <typename TG>
__global__ void __launch_bounds__(ADAMW_THREADS) grad_norm_kernel(const __grid_constant__ AdamwTable tab,
                                                                  double* __restrict__ partial) {
  __shared__ double part[ADAMW_WARPS];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t nb = tab.first[tab.count], stride = gridDim.x * ADAMW_WARPS;
  double acc[2] = {0.0, 0.0};
  uint32_t blk = blockIdx.x * ADAMW_WARPS + warp;
  int t = blk < nb ? find_tensor(tab, blk) : 0;
  for (; blk < nb; blk += stride) {
    while (blk >= tab.first[t + 1]) ++t;
    const AdamwEntry& e = tab.e[t];
    const long long base = (long long)(blk - tab.first[t]) * ADAMW_BLOCK;
    const int left = (int)min(e.n - base, (long long)ADAMW_BLOCK);
    Raw8<TG> r;
    raw_load(reinterpret_cast<const TG*>(e.g) + base, (tab.flags[t] & AF_VEC) && left == ADAMW_BLOCK, left, lane, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j & 1] = fma((double)value(r, j), (double)value(r, j), acc[j & 1]);
  }
  double s = acc[0] + acc[1];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) part[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (int w = 0; w < ADAMW_WARPS; ++w) all += part[w];
    partial[blockIdx.x] = all;
  }
}

// ---------------------------------------------------------------------------
// The step. With a clip every block first sums the norm's partial sums itself
// (a few KB from L2): no third launch and no counter. The blocks of the table
// are walked from its end, where the norm's pass over the gradients has just
// been: the part of them that L2 still holds is not read from memory again.
// ---------------------------------------------------------------------------
#ifndef MINB32
#define MINB32 3
#define MINB8 3
#endif
template <typename TP, typename TG, int BITS>
__global__ void __launch_bounds__(ADAMW_THREADS, BITS == 32 ? MINB32 : MINB8) adamw_kernel(const __grid_constant__ AdamwTable tab,
                                                              const __grid_constant__ AdamwCoefs c0,
                                                              const double* __restrict__ partial, int n_partial,
                                                              float* __restrict__ grad_norm) {
  __shared__ double part[ADAMW_WARPS];
  __shared__ float s_clip;
  __shared__ float s_coef[3];
  __shared__ __align__(16) uint16_t rnd[BITS == 8 ? ADAMW_WARPS : 1][ADAMW_BLOCK];
  // no early launch of dependents: what is written here may be a weight, which other kernels fetch before their wait
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  AdamwCoefs c = c0;
  float clip = 1.f;
  if (c.step_dev || c.lr_dev) {
    if (threadIdx.x == 0) {
      const double t = c.step_dev ? (double)*c.step_dev : (double)c.step;
      const double lr = c.lr_dev ? *c.lr_dev : c.lr;
      s_coef[0] = (float)(1.0 - lr * c.wd);
      s_coef[1] = (float)(lr / (1.0 - pow(c.beta1, t)));
      s_coef[2] = (float)(1.0 / sqrt(1.0 - pow(c.beta2, t)));
    }
    if (c.step_dev) c.step = (uint32_t)*c.step_dev;
    __syncthreads();
    c.keep = s_coef[0];
    c.step_size = s_coef[1];
    c.isb2 = s_coef[2];
  }
  if (c.max_norm > 0.0) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n_partial; i += ADAMW_THREADS) s += partial[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) part[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      double all = 0.0;
      for (int w = 0; w < ADAMW_WARPS; ++w) all += part[w];
      const double norm = sqrt(all);
      if (blockIdx.x == 0 && grad_norm) *grad_norm = (float)norm;
      // a norm that is not finite: 0 marks the step as skipped
      s_clip = norm <= 1.7976931348623157e308 ? (float)fmin(1.0, c.max_norm / (norm + 1e-6)) : -1.f;
    }
    __syncthreads();
    clip = s_clip;
    if (clip < 0.f) return;
  }
  const uint32_t nb = tab.first[tab.count], stride = gridDim.x * ADAMW_WARPS;
  uint32_t i = blockIdx.x * ADAMW_WARPS + warp;
  int t = i < nb ? find_tensor(tab, nb - 1 - i) : 0;
  for (; i < nb; i += stride) {
    const uint32_t blk = nb - 1 - i;
    while (blk < tab.first[t]) --t;
    const AdamwEntry& e = tab.e[t];
    const uint32_t tb = blk - tab.first[t];  // block of the tensor
    const long long base = (long long)tb * ADAMW_BLOCK;
    const int left = (int)min(e.n - base, (long long)ADAMW_BLOCK);
    const bool vec = (tab.flags[t] & AF_VEC) && left == ADAMW_BLOCK;
    const float keep = (tab.flags[t] & AF_DECAY) ? c.keep : 1.f;
    TP* pp = reinterpret_cast<TP*>(e.p) + base;
    const TG* gp = reinterpret_cast<const TG*>(e.g) + base;
    Raw8<TP> rp;
    Raw8<TG> rg;
    raw_load(pp, vec, left, lane, rp);
    raw_load(reinterpret_cast<const TG*>(e.g) + base, vec, left, lane, rg);
    float p[8];
    if constexpr (BITS == 32) {
      float m[8], v[8];
      float* mp = reinterpret_cast<float*>(e.m) + base;
      float* vp = reinterpret_cast<float*>(e.v) + base;
      Raw8<float> rm, rv;
      raw_load(mp, vec, left, lane, rm);
      raw_load(vp, vec, left, lane, rv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = value(rp, j);
        m[j] = value(rm, j);
        v[j] = value(rv, j);
        update1(c, keep, __fmul_rn(value(rg, j), clip), p[j], m[j], v[j]);
      }
      pack(m, rm);
      pack(v, rv);
      raw_store(mp, vec, left, lane, rm);
      raw_store(vp, vec, left, lane, rv);
    } else {
      uint8_t* mp = reinterpret_cast<uint8_t*>(e.m) + base;
      uint8_t* vp = reinterpret_cast<uint8_t*>(e.v) + base;
      const float ms = e.ms[tb], vs = e.vs[tb];
      Raw8<uint8_t> rm, rv;
      raw_load(mp, vec, left, lane, rm);
      raw_load(vp, vec, left, lane, rv);
      // 16 random bits of element k: half k % 8 of the draw of its octet k / 8; both moments take the same bits
      // (each is right in the mean by itself, and the ratio's error is smaller when they round the same way)
      const unsigned long long oct = (unsigned long long)tb * 32 + lane;
      uint32_t r[4] = {(uint32_t)oct, (uint32_t)(oct >> 32), c.step, c.tensor0 + (uint32_t)t};
      philox4x32_10(r, c.k0, c.k1);
      if (!vec) {  // to the lanes that hold the elements
        __syncwarp();
        *reinterpret_cast<uint4*>(&rnd[warp][lane * 8]) = make_uint4(r[0], r[1], r[2], r[3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = rnd[warp][2 * k * 32 + lane] | (uint32_t)rnd[warp][(2 * k + 1) * 32 + lane] << 16;
      }
      // the usual case, two elements at a time: no zero and no large v, all finite
      const f32x2 z = both(c.minus0);
      f32x2 m2[4], v2[4], p2[4], nan2 = both(0.f);
      float mx = 0.f;
      uint32_t vx = 0, vmin = 0xffffffffu;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = decode_m2((rm.w[k >> 1] >> (16 * (k & 1))) & 0xffffu);
        const float2 y = k & 1 ? decode_v2<1>(rv.w[k >> 1]) : decode_v2<0>(rv.w[k >> 1]);
        const f32x2 g2 = mul2(pair(value(rg, 2 * k), value(rg, 2 * k + 1)), both(clip));
        m2[k] = add2(product2(mul2(pair(x.x, x.y), both(ms)), both(c.b1), z), product2(g2, both(c.c1), z));
        v2[k] = add2(product2(mul2(pair(y.x, y.y), both(vs)), both(c.b2), z), product2(mul2(g2, g2), both(c.c2), z));
        nan2 = fma2(m2[k], both(0.f), nan2);  // NaN if an m is not finite
        const float2 mm = halves(m2[k]), vv = halves(v2[k]);
        mx = fmaxf(mx, fmaxf(fabsf(mm.x), fabsf(mm.y)));
        vx = max(vx, max(__float_as_uint(vv.x), __float_as_uint(vv.y)));
        vmin = min(vmin, min(__float_as_uint(vv.x), __float_as_uint(vv.y)));
        // v 2^24 is a normal number whatever v > 0, and finite: v < 2^100 here
        const float2 s2 = halves(mul2(v2[k], both(16777216.f)));
        const float2 root = make_float2(sqrt_approx(s2.x), sqrt_approx(s2.y));
        const float2 den = halves(fma2(pair(root.x, root.y), both(c.isb2 * 0x1p-12f), both(c.eps)));
        const f32x2 q = mul2(m2[k], pair(rcp_approx(den.x), rcp_approx(den.y)));
        p2[k] = fma2(q, both(-c.step_size), mul2(pair(value(rp, 2 * k), value(rp, 2 * k + 1)), both(keep)));
      }
      const float2 nn = halves(nan2);
      uint32_t mxb = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
      vx = __reduce_max_sync(0xffffffffu, vx);
      const bool odd = vmin == 0 || !(nn.x + nn.y == 0.f);
      if (!__any_sync(0xffffffffu, odd) && vx < VX_USUAL && mxb < MX_USUAL) {
        const uint32_t em = (uint32_t)max((int)(mxb >> 23) - 14, 0), ev = (uint32_t)max((int)(vx >> 23) - 29, 0);
        // m / m_scale in two steps: the first takes the smallest normal code to 2^-126, so that what is below it is
        // flushed to zero; the second back into the format's range (and -0 to 0)
        const f32x2 down = both(__uint_as_float((127u + 127u - 120u - em - 7u) << 23)), up = both(0x1p120f);
        const f32x2 vinv = both(__uint_as_float((254u - ev - 15u) << 23));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t u0 = (r[k] & 0xffffu) << 4, u1 = (r[k] >> 12) & 0xffff0u;
          const float2 mm = halves(m2[k]), vv = halves(v2[k]);
          const f32x2 mt = pair(__uint_as_float((__float_as_uint(mm.x) + u0) & 0xfff00000u),
                                __uint_as_float((__float_as_uint(mm.y) + u1) & 0xfff00000u));
          const f32x2 vt = pair(__uint_as_float((__float_as_uint(vv.x) + 2 * u0) & 0xffe00000u),
                                __uint_as_float((__float_as_uint(vv.y) + 2 * u1) & 0xffe00000u));
          const uint32_t mc = code_m2(fma2(mul2_ftz(mt, down), up, both(0.f)));
          const float2 vy = halves(mul2(vt, vinv));
          const uint32_t vc = code_v2(fmaxf(vy.x, 0x1p-14f), fmaxf(vy.y, 0x1p-14f));
          rm.w[k >> 1] = k & 1 ? rm.w[k >> 1] | mc << 16 : mc;
          rv.w[k >> 1] = k & 1 ? rv.w[k >> 1] | vc << 16 : vc;
          const float2 pp2 = halves(p2[k]);
          p[2 * k] = pp2.x;
          p[2 * k + 1] = pp2.y;
        }
      } else {
        general8(c, keep, clip, pp, gp, mp, vp, vec, left, lane, ms, vs, r, p, rm, rv, mxb, vx);
      }
      if (lane == 0) {
        e.ms[tb] = mxb ? __uint_as_float((uint32_t)(max((int)(mxb >> 23) - 14, 0) + 7) << 23) : 0.f;
        e.vs[tb] = vx ? __uint_as_float((uint32_t)(max((int)(vx >> 23) - 29, 0) + 15) << 23) : 0.f;
      }
      raw_store(mp, vec, left, lane, rm);
      raw_store(vp, vec, left, lane, rv);
    }
    pack(p, rp);
    raw_store(pp, vec, left, lane, rp);
    if (e.copy) {
      Raw8<uint16_t> rc;
      pack(p, rc);
      raw_store(e.copy + base, vec, left, lane, rc);
    }
  }
  __threadfence();
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
template <typename... KArgs, typename... Args>
cudaError_t launch(bool pdl, void (*kernel)(KArgs...), unsigned grid, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(ADAMW_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

typedef void (*AdamwFn)(const AdamwTable, const AdamwCoefs, const double*, int, float*);
template <typename TP, typename TG>
AdamwFn pick_bits(int bits) {
  return bits == 32 ? adamw_kernel<TP, TG, 32> : adamw_kernel<TP, TG, 8>;
}
AdamwFn pick(int pt, int gt, int bits) {
  if (pt == SVLA_TYPE_F32) return gt == SVLA_TYPE_F32 ? pick_bits<float, float>(bits) : pick_bits<float, uint16_t>(bits);
  return gt == SVLA_TYPE_F32 ? pick_bits<uint16_t, float>(bits) : pick_bits<uint16_t, uint16_t>(bits);
}

size_t launches_of(int n_tensors) { return ((size_t)n_tensors + ADAMW_CAP - 1) / ADAMW_CAP; }

svla_status bad(svla_status s, int i, const char* why) {
  return svla_internal_fail(s, ((i < 0 ? std::string("workspace or grad_norm") : "tensor " + std::to_string(i)) + ": " + why).c_str());
}

svla_status adamw_checked(const svla_adamw_tensor* ts, int n, const svla_adamw_args* a, void* workspace,
                          size_t workspace_bytes, float* grad_norm, cudaStream_t stream) {
  if (!a || n < 0 || (n > 0 && !ts)) return svla_internal_fail(SVLA_ERR_ARG, "null argument or negative tensor count");
  if ((a->param_type != SVLA_TYPE_F32 && a->param_type != SVLA_TYPE_BF16) ||
      (a->grad_type != SVLA_TYPE_F32 && a->grad_type != SVLA_TYPE_BF16))
    return svla_internal_fail(SVLA_ERR_ARG, "param_type and grad_type must be SVLA_TYPE_F32 or SVLA_TYPE_BF16");
  if (a->state_bits != 32 && a->state_bits != 8) return svla_internal_fail(SVLA_ERR_ARG, "state_bits must be 32 or 8");
  if (!(a->lr >= 0.0) || !std::isfinite(a->lr) || !(a->beta1 >= 0.0 && a->beta1 < 1.0) ||
      !(a->beta2 >= 0.0 && a->beta2 < 1.0) || !((float)a->eps > 0.f) || !std::isfinite((float)a->eps) ||
      !(a->weight_decay >= 0.0) || !std::isfinite(a->weight_decay) || !(a->max_norm >= 0.0))
    return svla_internal_fail(SVLA_ERR_ARG, "lr, weight_decay, max_norm >= 0, 0 <= beta < 1 and eps > 0 (in float32)");
  if (!a->step_device && a->step < 1) return svla_internal_fail(SVLA_ERR_ARG, "step counts from 1");
  const bool clip = a->max_norm > 0.0;
  const size_t pb = a->param_type == SVLA_TYPE_F32 ? 4 : 2, gb = a->grad_type == SVLA_TYPE_F32 ? 4 : 2;
  const size_t sb = a->state_bits / 8;
  if (clip) {
    if (!workspace || workspace_bytes < svla_op_adamw_workspace_bytes(n))
      return svla_internal_fail(SVLA_ERR_ARG, "the clip needs a workspace of svla_op_adamw_workspace_bytes(n_tensors)");
    if ((uintptr_t)workspace & 7) return svla_internal_fail(SVLA_ERR_ARG, "the workspace must be 8-byte aligned");
  }
  // every written range must be apart from every other range
  struct Range {
    uintptr_t at, end;
    int tensor;
    bool written;
  };
  std::vector<Range> ranges;
  ranges.reserve((size_t)n * 7 + 2);
  for (int i = 0; i < n; ++i) {
    const svla_adamw_tensor& t = ts[i];
    if (t.n < 0) return bad(SVLA_ERR_SHAPE, i, "negative size");
    if (t.n == 0) continue;
    if (t.n > ((int64_t)1 << 40)) return bad(SVLA_ERR_SHAPE, i, "more than 2^40 elements");
    if (!t.param || !t.grad || !t.m || !t.v) return bad(SVLA_ERR_ARG, i, "null param, grad, m or v");
    if (a->state_bits == 8 && (!t.m_scale || !t.v_scale)) return bad(SVLA_ERR_ARG, i, "8-bit states need m_scale and v_scale");
    if ((uintptr_t)t.param % pb || (uintptr_t)t.grad % gb || (uintptr_t)t.m % sb || (uintptr_t)t.v % sb ||
        (uintptr_t)t.copy % 2 || (a->state_bits == 8 && (((uintptr_t)t.m_scale | (uintptr_t)t.v_scale) & 3)))
      return bad(SVLA_ERR_ARG, i, "a pointer is not aligned to its element type");
    const size_t n_el = (size_t)t.n, blocks = (n_el + ADAMW_BLOCK - 1) / ADAMW_BLOCK;
    auto put = [&](const void* p, size_t bytes, bool w) {
      if (p) ranges.push_back(Range{(uintptr_t)p, (uintptr_t)p + bytes, i, w});
    };
    put(t.param, n_el * pb, true);
    put(t.grad, n_el * gb, false);
    put(t.m, n_el * sb, true);
    put(t.v, n_el * sb, true);
    put(t.copy, n_el * 2, true);
    if (a->state_bits == 8) {
      put(t.m_scale, blocks * 4, true);
      put(t.v_scale, blocks * 4, true);
    }
  }
  if (clip) ranges.push_back(Range{(uintptr_t)workspace, (uintptr_t)workspace + svla_op_adamw_workspace_bytes(n), -1, true});
  if (clip && grad_norm) ranges.push_back(Range{(uintptr_t)grad_norm, (uintptr_t)grad_norm + 4, -1, true});
  std::sort(ranges.begin(), ranges.end(), [](const Range& x, const Range& y) { return x.at < y.at; });
  uintptr_t end_written = 0, end_any = 0;
  for (const Range& r : ranges) {
    if (r.at < end_written || (r.written && r.at < end_any))
      return bad(SVLA_ERR_ARG, r.tensor, "overlaps memory that the step writes");
    if (r.written) end_written = std::max(end_written, r.end);
    end_any = std::max(end_any, r.end);
  }

  if (std::all_of(ts, ts + n, [](const svla_adamw_tensor& t) { return t.n == 0; })) {  // nothing to update
    if (!clip || !grad_norm) return SVLA_OK;
    const cudaError_t e = cudaMemsetAsync(grad_norm, 0, sizeof(float), stream);
    return e == cudaSuccess ? SVLA_OK : svla_internal_fail(SVLA_ERR_CUDA, cudaGetErrorString(e));
  }

  AdamwCoefs c = {};
  c.b1 = (float)a->beta1;
  c.c1 = (float)(1.0 - a->beta1);
  c.b2 = (float)a->beta2;
  c.c2 = (float)(1.0 - a->beta2);
  c.eps = (float)a->eps;
  c.minus0 = -0.f;
  c.max_norm = a->max_norm;
  c.k0 = (uint32_t)a->seed;
  c.k1 = (uint32_t)(a->seed >> 32);
  c.step = (uint32_t)a->step;
  c.step_dev = reinterpret_cast<const long long*>(a->step_device);
  c.lr_dev = a->lr_device;
  c.lr = a->lr;
  c.beta1 = a->beta1;
  c.beta2 = a->beta2;
  c.wd = a->weight_decay;
  if (!a->step_device) {
    c.keep = (float)(1.0 - a->lr * a->weight_decay);
    c.step_size = (float)(a->lr / (1.0 - std::pow(a->beta1, (double)a->step)));
    c.isb2 = (float)(1.0 / std::sqrt(1.0 - std::pow(a->beta2, (double)a->step)));
  }

  const AdamwFn fn = pick(a->param_type, a->grad_type, a->state_bits);
  int per_sm = 0, dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, ADAMW_THREADS, 0);
  if (e != cudaSuccess || per_sm < 1)
    return svla_internal_fail(SVLA_ERR_CUDA, (std::string("adamw: ") + cudaGetErrorString(e)).c_str());

  // with a clip: pass 0 sums the squares of every launch's gradients, pass 1 updates
  std::vector<AdamwTable> one(1);
  AdamwTable& tab = one[0];
  const int launches = (int)launches_of(n);
  int n_partial = 0;
  bool pdl = false;
  for (int pass = clip ? 0 : 1; pass < 2; ++pass) {
    for (int l = 0; l < launches; ++l) {
      tab.count = std::min(ADAMW_CAP, n - l * ADAMW_CAP);
      unsigned long long nb = 0;
      for (int k = 0; k < tab.count; ++k) {
        const svla_adamw_tensor& t = ts[l * ADAMW_CAP + k];
        tab.e[k] = AdamwEntry{t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, reinterpret_cast<uint16_t*>(t.copy),
                              (long long)t.n};
        const bool vec = ((uintptr_t)t.param & (8 * pb - 1)) == 0 && ((uintptr_t)t.grad & (8 * gb - 1)) == 0 &&
                         ((uintptr_t)t.copy & 15) == 0 && (((uintptr_t)t.m | (uintptr_t)t.v) & (8 * sb - 1)) == 0;
        tab.flags[k] = (uint8_t)((t.decay ? AF_DECAY : 0) | (vec ? AF_VEC : 0));
        tab.first[k] = (uint32_t)nb;
        nb += (unsigned long long)((t.n + ADAMW_BLOCK - 1) / ADAMW_BLOCK);
      }
      if (nb > 0x7fffffffull) return svla_internal_fail(SVLA_ERR_SHAPE, "more than 2^39 elements in 400 tensors");
      tab.first[tab.count] = (uint32_t)nb;
      const unsigned need = (unsigned)std::max(1ull, (nb + ADAMW_WARPS - 1) / ADAMW_WARPS);
      if (pass == 0) {
        const unsigned grid = std::min(need, (unsigned)NORM_BLOCKS);
        double* part = reinterpret_cast<double*>(workspace) + n_partial;
        e = a->grad_type == SVLA_TYPE_F32 ? launch(false, grad_norm_kernel<float>, grid, stream, tab, part)
                                          : launch(false, grad_norm_kernel<uint16_t>, grid, stream, tab, part);
        n_partial += (int)grid;
        pdl = true;
      } else {
        c.tensor0 = (uint32_t)(l * ADAMW_CAP);
        e = launch(pdl, fn, std::min(need, (unsigned)(per_sm * sms)), stream, tab, c,
                   reinterpret_cast<const double*>(workspace), n_partial, l == 0 ? grad_norm : nullptr);
        pdl = true;
      }
      if (e != cudaSuccess)
        return svla_internal_fail(SVLA_ERR_CUDA, (std::string("adamw launch: ") + cudaGetErrorString(e)).c_str());
    }
  }
  return SVLA_OK;
}

}  // namespace
}  // namespace svla

extern "C" {

size_t svla_op_adamw_workspace_bytes(int n_tensors) {
  return n_tensors < 0 ? 0 : std::max<size_t>(1, svla::launches_of(n_tensors)) * svla::NORM_BLOCKS * sizeof(double);
}

svla_status svla_op_adamw(const svla_adamw_tensor* tensors, int n_tensors, const svla_adamw_args* args,
                          void* workspace, size_t workspace_bytes, float* grad_norm, void* stream) {
  try {
    return svla::adamw_checked(tensors, n_tensors, args, workspace, workspace_bytes, grad_norm,
                               reinterpret_cast<cudaStream_t>(stream));
  } catch (const std::exception& x) {  // host memory ran out
    return svla_internal_fail(SVLA_ERR_OOM, "adamw: out of host memory");
  }
}

}  // extern "C"
