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
//
// Measured (a step of 153 tensors, 99.8 M fp32 values with a bf16 copy): 32-bit
// moments 463 us (6.5 TB/s, the rate of a copy), 540 with the clip, whose pass
// over the gradients is 61 us of reading; 8-bit moments 300 and 378 us (6.0
// TB/s without the clip). 144 tensors, 157 M bf16 values, 8-bit moments: 384 us,
// 4.1 TB/s, and neither limit is reached: memory alone would take 241 us, the
// 268.5 M warp instructions (55 a value) 231 us of the schedulers (1965 MHz).
// A warp loads, computes and stores its values in turn, and the 29 warps an SM
// overlap the two too little (DRAM 48 %, issue 63 %); the 64 registers that let
// four blocks on an SM also spill 32 bytes a thread.
// Values whose second moment is 0 cost more (general8): with no gradient
// anywhere 100 M fp32 values take 632 us (273 without such blocks, 440 with a
// third of them), bf16 589 (239, 373).
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <exception>
#include <memory>
#include <string>
#include <type_traits>
#include <utility>
#include <vector>

#include "common.cuh"
#include "pairs.cuh"
#include "philox.cuh"

svla_status svla_internal_fail(svla_status s, const char* msg);

namespace svla {
namespace {

constexpr int ADAMW_BLOCK = 256;   // elements of a warp's task = elements that share a scale
constexpr int ADAMW_CAP = 400;     // tensors of one launch (28.1 KB of the 32,764 bytes of kernel parameters)
// Tensors of a launch of a short list: the parameters are copied at every launch (with the clip, 27 tensors 21.2 us a call
// and 32 tensors 23.4; with the long table 23.4 and 25.3. A longer short table would serve more lists: one of 128 took 33
// tensors in 22.4 us a call, the long one 26.6).
constexpr int ADAMW_FEW = 32;
constexpr int ADAMW_HINTS = 256;   // spans of chunks whose first tensor the table names
constexpr int ADAMW_THREADS = 256;
constexpr int ADAMW_WARPS = ADAMW_THREADS / 32;
constexpr int ADAMW_CHUNK = ADAMW_WARPS * ADAMW_BLOCK;  // elements of a block's task, of one tensor
constexpr int NORM_THREADS = 512;
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

template <int CAP>
struct AdamwTable {
  AdamwEntry e[CAP];
  uint32_t first[CAP + 1];  // first chunk of each tensor; first[count] = all chunks
  uint16_t hint[ADAMW_HINTS + 1]; // tensor of chunk k << shift (the last one for chunks past the end)
  uint8_t flags[CAP];             // 1: weight decay, 2: every pointer allows the vector accesses
  int count, shift;
};
constexpr uint8_t AF_DECAY = 1, AF_VEC = 2;

struct AdamwCoefs {
  // pairs of equal values, operands of the packed arithmetic straight from the constant bank
  unsigned long long b1_2, c1_2, b2_2, c2_2, eps_2, minus0_2, two24_2;
  uint32_t key[20];  // Philox round keys
  float b1, c1, b2, c2, eps;
  float keep;       // 1 - lr wd
  float step_size;  // lr / (1 - b1^t)
  float isb2;       // 1 / sqrt(1 - b2^t)
  double max_norm;  // 0: no clip
  uint32_t step, tensor0;  // the random bits' counter takes the low word of the step number
  double t;                // the bias corrections the whole of it
  uint32_t usual;          // bits of the magnitude that the usual case of the 8-bit step stays below
  // read on the device instead of the host's numbers, where given
  const long long* step_dev;
  const double* lr_dev;
  double lr, beta1, beta2, wd;
};

// tensor of a chunk: the last t with first[t] <= chunk (empty tensors have none),
// searched between the tensors of its span's ends
template <int CAP>
SVLA_DEV int find_tensor(const AdamwTable<CAP>& t, uint32_t chunk) {
  int lo = t.hint[chunk >> t.shift], hi = t.hint[(chunk >> t.shift) + 1];
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
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
// Two values -> fp16, the mantissa cut off (lo in the low half).
SVLA_DEV uint32_t cut_f16x2(f32x2 x) {
  uint32_t r;
  const float2 f = halves(x);
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f.y), "f"(f.x));
  return r;
}
// Codes of two moments that are divided by their scale, with the random bits
// added below what the code keeps.
//   m, further divided by 2^8: cut to 3 mantissa bits; what is below 2^-6 of the
//   scale is a subnormal fp16 number here, and the product with 2^8 flushes it
//   (and makes a -0 0).
//   v: an e5m2 code is the upper byte of an fp16 number, at least 2^-14 here.
SVLA_DEV uint32_t code_m2(f32x2 x) {
  uint32_t h;
  uint16_t r;
  asm("fma.rn.ftz.f16x2 %0, %1, %2, %3;" : "=r"(h) : "r"(cut_f16x2(x) & 0xff80ff80u), "r"(0x5c005c00u), "r"(0u));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
SVLA_DEV uint32_t half_v2(f32x2 x) {
  uint32_t h;
  asm("max.f16x2 %0, %1, %2;" : "=r"(h) : "r"(cut_f16x2(x)), "r"(0x04000400u));
  return h;
}
// the larger (smaller) of three, NaN if one is NaN
SVLA_DEV float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
SVLA_DEV float min3(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 8 elements of this lane from its warp's 256 of a chunk, raw, packed into words.
// `vec`: the consecutive elements from `at`, one 32-byte (fp32), 16-byte (bf16) or 8-byte
// (codes) access; else (a tensor's last, shorter block, or a tensor at an odd
// address) every 32nd element of the warp's, of which `left` exist; zeros past them.
template <typename E>
struct Raw8 {
  uint32_t w[2 * sizeof(E)];
};
template <typename E>
SVLA_DEV void raw_load(const E* p, bool vec, int left, int at, Raw8<E>& r) {
  if (vec) {
    if constexpr (sizeof(E) == 4) {
      ld_global_v8(p + at, r.w);
    } else if constexpr (sizeof(E) == 2) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + at);
      r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p + at);
      r.w[0] = q.x, r.w[1] = q.y;
    }
    return;
  }
  const int lane = (at >> 3) & 31;
  p += at - lane * 8;
  uint32_t x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (left >= ADAMW_BLOCK || j * 32 + lane < left) {
      if constexpr (sizeof(E) == 4)
        x[j] = __float_as_uint(p[j * 32 + lane]);
      else
        x[j] = p[j * 32 + lane];
    } else {
      x[j] = 0u;
    }
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
SVLA_DEV void raw_store(E* p, bool vec, int left, int at, const Raw8<E>& r) {
  if (vec) {
    if constexpr (sizeof(E) == 4)
      st_global_v8(p + at, r.w);
    else if constexpr (sizeof(E) == 2)
      *reinterpret_cast<uint4*>(p + at) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else
      *reinterpret_cast<uint2*>(p + at) = make_uint2(r.w[0], r.w[1]);
    return;
  }
  constexpr int PER = 4 / sizeof(E);
  const int lane = (at >> 3) & 31;
  p += at - lane * 8;
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
// rounded up with the probability of its distance to the lower code, so a
// stored moment of the codes' range is right in the mean. Nearest rounding would
// hold v where it is: a step moves v by (1 - b2) ~ 1e-3 of itself and the codes
// lie 1/8 to 1/4 apart.
//   m: e4m3, largest magnitude in [2^7, 2^8) of the scale; below 2^-6 -> 0
//   v: e5m2, largest in [2^14, 2^15); 0 < v below 2^-14 -> 2^-14, so no
//      gradient is ever divided by a vanished v
// Below the range there is a bias: an m of less than 2^-13 or so of its block's
// largest keeps no momentum (its step is that of 1 - b1 of the gradient while
// that lasts), a v of less than 2^-28 or so of it is too large.
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
SVLA_DEV void update1(const AdamwCoefs& c, float keep, float isb2, float step_size, float g, float& p, float& m, float& v) {
  m = __fadd_rn(__fmul_rn(m, c.b1), __fmul_rn(g, c.c1));
  v = __fadd_rn(__fmul_rn(v, c.b2), __fmul_rn(__fmul_rn(g, g), c.c2));
  const float q = __fdiv_rn(m, __fmaf_rn(__fsqrt_rn(v), isb2, c.eps));
  p = __fmaf_rn(-q, step_size, p * keep);
}

// Where a warp's 256 elements lie: the arrays from the chunk's first element, the
// block's scales, and what all of its elements share.
template <typename TP, typename TG, typename TS>
struct Place {
  TP* p;
  const TG* g;
  TS *m, *v;
  uint16_t* copy;
  float *ms, *vs;
  int left, at;  // elements of this warp; this lane's first one of the chunk (vector accesses)
  bool vec;      // all there, and the tensor's pointers allow the wide accesses
  float keep, clip, isb2, step_size;
};
template <typename TP, typename TG, typename TS>
struct Loaded {
  Raw8<TP> p;
  Raw8<TG> g;
  Raw8<TS> m, v;
  SVLA_DEV void load(const Place<TP, TG, TS>& a) {
    if (a.vec) {
      raw_load(a.p, true, 0, a.at, p);
      raw_load(a.g, true, 0, a.at, g);
      raw_load(a.m, true, 0, a.at, m);
      raw_load(a.v, true, 0, a.at, v);
    } else if (a.left >= ADAMW_BLOCK) {  // all 256 at an odd address: no test an element (30 M fp32 with 8-bit states 127 -> 112 us)
      raw_load(a.p, false, ADAMW_BLOCK, a.at, p);
      raw_load(a.g, false, ADAMW_BLOCK, a.at, g);
      raw_load(a.m, false, ADAMW_BLOCK, a.at, m);
      raw_load(a.v, false, ADAMW_BLOCK, a.at, v);
    } else {
      raw_load(a.p, false, a.left, a.at, p);
      raw_load(a.g, false, a.left, a.at, g);
      raw_load(a.m, false, a.left, a.at, m);
      raw_load(a.v, false, a.left, a.at, v);
    }
  }
};
template <typename TP, typename TG, typename TS>
SVLA_DEV void store_all(const Place<TP, TG, TS>& a, const float (&p)[8], const Raw8<TS>& m, const Raw8<TS>& v) {
  Raw8<TP> rp;
  Raw8<uint16_t> rc;
  pack(p, rp);
  pack(p, rc);
  if (a.vec) {
    raw_store(a.m, true, 0, a.at, m);
    raw_store(a.v, true, 0, a.at, v);
    raw_store(a.p, true, 0, a.at, rp);
    if (a.copy) raw_store(a.copy, true, 0, a.at, rc);
  } else {
    raw_store(a.m, false, a.left, a.at, m);
    raw_store(a.v, false, a.left, a.at, v);
    raw_store(a.p, false, a.left, a.at, rp);
    if (a.copy) raw_store(a.copy, false, a.left, a.at, rc);
  }
}
// fields of the block scales from the largest magnitudes' bits
SVLA_DEV uint32_t m_field(uint32_t mx) { return (uint32_t)max((int)(mx >> 23) - 14, 0); }
SVLA_DEV uint32_t v_field(uint32_t vx) { return (uint32_t)max((int)(vx >> 23) - 29, 0); }

// The 8-bit step of a warp's block whatever its values: a zero v, moments near
// the ends of fp32's range, or ones that are not finite (they take the NaN
// code, and so would a negative v; the scales are those of the others).
template <typename TP, typename TG>
SVLA_DEV void general8(const AdamwCoefs& c, const Place<TP, TG, uint8_t>& a, const uint32_t (&r)[4]) {
  Loaded<TP, TG, uint8_t> in;
  in.load(a);
  const float ms = *a.ms, vs = *a.vs;
  float p[8], m[8], v[8];
  uint32_t mx = 0, vx = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = decode_m2((in.m.w[k >> 1] >> (16 * (k & 1))) & 0xffffu);
    const float2 y = k & 1 ? decode_v2<1>(in.v.w[k >> 1]) : decode_v2<0>(in.v.w[k >> 1]);
    m[2 * k] = __fmul_rn(x.x, ms), m[2 * k + 1] = __fmul_rn(x.y, ms);
    v[2 * k] = __fmul_rn(y.x, vs), v[2 * k + 1] = __fmul_rn(y.y, vs);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j] = value(in.p, j);
    update1(c, a.keep, a.isb2, a.step_size, __fmul_rn(value(in.g, j), a.clip), p[j], m[j], v[j]);
    if (magnitude(m[j]) < INF_MAG) mx = max(mx, magnitude(m[j]));
    if (v[j] >= 0.f && magnitude(v[j]) < INF_MAG) vx = max(vx, magnitude(v[j]));
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  vx = __reduce_max_sync(0xffffffffu, vx);
  const uint32_t em = m_field(mx), ev = v_field(vx);
  uint32_t mc[8], vc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u20 = (j & 1) ? (r[j >> 1] >> 12) & 0xffff0u : (r[j >> 1] & 0xffffu) << 4;
    mc[j] = magnitude(m[j]) >= INF_MAG ? 0x7fu : encode_m(m[j], u20, em << 3);
    vc[j] = v[j] >= 0.f && magnitude(v[j]) < INF_MAG ? encode_v(v[j], u20, ev << 2) : 0x7fu;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    in.m.w[k] = mc[4 * k] | mc[4 * k + 1] << 8 | mc[4 * k + 2] << 16 | mc[4 * k + 3] << 24;
    in.v.w[k] = vc[4 * k] | vc[4 * k + 1] << 8 | vc[4 * k + 2] << 16 | vc[4 * k + 3] << 24;
  }
  store_all(a, p, in.m, in.v);
  __syncwarp();  // every lane has read the scales
  if ((threadIdx.x & 31) == 0) {
    *a.ms = mx ? __uint_as_float((em + 7) << 23) : 0.f;
    *a.vs = vx ? __uint_as_float((ev + 15) << 23) : 0.f;
  }
}

// The usual case of the 8-bit step has |m| and v below 2^100: v's product with 2^24 is finite, and the reciprocals of
// the scales are normal numbers. So is that of the denominator, with an eps below 2^100 (AdamwCoefs::usual: 0 with a
// larger one).
constexpr uint32_t USUAL_MAG = (127u + 100u) << 23;
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
// practice; fixed order all the same. partial[blockIdx.x] of this launch. Bound
// by its reads (99.8 M fp32 gradients: about 70 us, 61 at the rate of a copy).
// ---------------------------------------------------------------------------
template <typename TG, int CAP>
__global__ void __launch_bounds__(NORM_THREADS) grad_norm_kernel(const __grid_constant__ AdamwTable<CAP> tab,
                                                                 double* __restrict__ partial) {
  __shared__ double part[NORM_THREADS / 32];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wc = warp % ADAMW_WARPS;  // place in the chunk: the block takes NORM_THREADS / ADAMW_THREADS chunks at a time
  const uint32_t chunks = tab.first[tab.count], stride = gridDim.x * (NORM_THREADS / ADAMW_THREADS);
  double acc[2] = {0.0, 0.0};
#pragma unroll 2
  for (uint32_t chunk = blockIdx.x * (NORM_THREADS / ADAMW_THREADS) + warp / ADAMW_WARPS; chunk < chunks; chunk += stride) {
    const int t = find_tensor(tab, chunk);
    const AdamwEntry& e = tab.e[t];
    const long long base = (long long)(chunk - tab.first[t]) * ADAMW_CHUNK;
    const int left = (int)min(e.n - base, (long long)ADAMW_CHUNK) - wc * ADAMW_BLOCK;
    Raw8<TG> r;
    raw_load(reinterpret_cast<const TG*>(e.g) + base, (tab.flags[t] & AF_VEC) && left >= ADAMW_BLOCK, left,
             wc * ADAMW_BLOCK + lane * 8, r);
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
    for (int w = 0; w < NORM_THREADS / 32; ++w) all += part[w];
    partial[blockIdx.x] = all;
  }
}

template <typename TP, typename TG>
SVLA_DEV void update32(const AdamwCoefs& c, const Place<TP, TG, float>& a) {
  Loaded<TP, TG, float> in;
  in.load(a);
  float p[8], m[8], v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j] = value(in.p, j);
    m[j] = value(in.m, j);
    v[j] = value(in.v, j);
    update1(c, a.keep, a.isb2, a.step_size, __fmul_rn(value(in.g, j), a.clip), p[j], m[j], v[j]);
  }
  pack(m, in.m);
  pack(v, in.v);
  store_all(a, p, in.m, in.v);
}

// The usual case in packed pairs: every v positive, v, |m| and eps below 2^100.
// Else the block is done by general8.
template <typename TP, typename TG>
SVLA_DEV void update8(const AdamwCoefs& c, const Place<TP, TG, uint8_t>& a, uint32_t block, uint32_t step, uint32_t tensor,
                      int lane, uint16_t* rnd) {
  Loaded<TP, TG, uint8_t> in;
  in.load(a);
  const float ms = *a.ms, vs = *a.vs;
  // 16 random bits of element k: half k % 8 of the draw of its octet k / 8; both moments take the same bits
  // (each is right in the mean by itself in the codes' range, and the ratio's error is smaller when they round the same
  // way)
  const unsigned long long oct = (unsigned long long)block * 32 + lane;
  uint32_t r[4] = {(uint32_t)oct, (uint32_t)(oct >> 32), step, tensor};
#pragma unroll
  for (int k = 0; k < 10; ++k) philox_round(r, c.key[2 * k], c.key[2 * k + 1]);
  if (!a.vec) {  // to the lanes that hold the elements
    __syncwarp();
    *reinterpret_cast<uint4*>(&rnd[lane * 8]) = make_uint4(r[0], r[1], r[2], r[3]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = rnd[2 * k * 32 + lane] | (uint32_t)rnd[(2 * k + 1) * 32 + lane] << 16;
  }
  const f32x2 z = c.minus0_2;
  f32x2 m2[4], v2[4];
  float mx = 0.f, vx = 0.f, vmin = INFINITY;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = decode_m2((in.m.w[k >> 1] >> (16 * (k & 1))) & 0xffffu);
    const float2 y = k & 1 ? decode_v2<1>(in.v.w[k >> 1]) : decode_v2<0>(in.v.w[k >> 1]);
    const f32x2 g2 = mul2(pair(value(in.g, 2 * k), value(in.g, 2 * k + 1)), both(a.clip));
    m2[k] = add2(product2(mul2(pair(x.x, x.y), both(ms)), c.b1_2, z), product2(g2, c.c1_2, z));
    v2[k] = add2(product2(mul2(pair(y.x, y.y), both(vs)), c.b2_2, z), product2(mul2(g2, g2), c.c2_2, z));
    const float2 mm = halves(m2[k]), vv = halves(v2[k]);
    mx = max3_abs(mx, mm.x, mm.y);
    vx = max3_abs(vx, vv.x, vv.y);
    vmin = min3(vmin, vv.x, vv.y);
  }
  const uint32_t mxb = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
  const uint32_t vxb = __reduce_max_sync(0xffffffffu, __float_as_uint(vx));
  if (!__all_sync(0xffffffffu, vmin > 0.f && mxb < c.usual && vxb < c.usual)) {
    general8(c, a, r);
    return;
  }
  float p[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // v 2^24 is a normal number whatever v > 0, and finite: v < 2^100 here
    const float2 s2 = halves(mul2(v2[k], c.two24_2));
    const float2 root = make_float2(sqrt_approx(s2.x), sqrt_approx(s2.y));
    const float2 den = halves(fma2(pair(root.x, root.y), both(a.isb2 * 0x1p-12f), c.eps_2));
    const f32x2 q = mul2(m2[k], pair(rcp_approx(den.x), rcp_approx(den.y)));
    const float2 pn = halves(fma2(q, both(-a.step_size), mul2(pair(value(in.p, 2 * k), value(in.p, 2 * k + 1)), both(a.keep))));
    p[2 * k] = pn.x;
    p[2 * k + 1] = pn.y;
  }
  const uint32_t em = m_field(mxb), ev = v_field(vxb);
  const f32x2 minv = both(__uint_as_float((254u - 7u - 8u - em) << 23));  // 2^-8 / scale of m
  const f32x2 vinv = both(__uint_as_float((254u - 15u - ev) << 23));
  uint32_t vh[4], mc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u0 = r[k] & 0xffffu, u1 = r[k] >> 16;
    const float2 mm = halves(m2[k]), vv = halves(v2[k]);
    mc[k] = code_m2(mul2(pair(__uint_as_float(__float_as_uint(mm.x) + u0 * 16u),
                              __uint_as_float(__float_as_uint(mm.y) + u1 * 16u)), minv));
    vh[k] = half_v2(mul2(pair(__uint_as_float(__float_as_uint(vv.x) + u0 * 32u),
                              __uint_as_float(__float_as_uint(vv.y) + u1 * 32u)), vinv));
  }
  in.m.w[0] = __byte_perm(mc[0], mc[1], 0x5410);
  in.m.w[1] = __byte_perm(mc[2], mc[3], 0x5410);
  in.v.w[0] = __byte_perm(vh[0], vh[1], 0x7531);
  in.v.w[1] = __byte_perm(vh[2], vh[3], 0x7531);
  store_all(a, p, in.m, in.v);
  if (lane == 0) {
    *a.ms = mxb ? __uint_as_float((em + 7) << 23) : 0.f;
    *a.vs = __uint_as_float((ev + 15) << 23);
  }
}

// ---------------------------------------------------------------------------
// The step. With a clip every block first sums the norm's partial sums itself
// (a few KB from L2): no third launch and no counter. The blocks of the table
// are walked from its end, where the norm's pass over the gradients has just
// been: the part of them that L2 still holds is not read from memory again.
// ---------------------------------------------------------------------------
// Ask for the cache lines of a warp's 256 elements, of which `left` exist, to be in L2.
template <typename E>
SVLA_DEV void prefetch_l2(const E* p, int left, int lane) {
  if (lane * 128 < left * (int)sizeof(E)) asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(p) + lane * 128) : "memory");
}

template <typename TP, typename TG, int BITS, int CAP>
__global__ void __launch_bounds__(ADAMW_THREADS, BITS == 8 && sizeof(TP) == 2 ? 4 : 3) adamw_kernel(const __grid_constant__ AdamwTable<CAP> tab,
                                                              const __grid_constant__ AdamwCoefs c,
                                                              const double* __restrict__ partial, int n_partial,
                                                              float* __restrict__ grad_norm) {
  typedef typename std::conditional<BITS == 32, float, uint8_t>::type TS;
  // the next turn's data on its way to L2: what it saves of the loads' latency is more than its instructions cost
  // where the parameters are fp32 (99.8 M values: 379 us, 413 without), not in bf16 (157 M: 413 us, 381 without)
  constexpr bool PREFETCH = BITS == 8 && sizeof(TP) == 4;
  __shared__ double part[ADAMW_WARPS];
  __shared__ float s_clip;
  __shared__ float s_coef[3];
  __shared__ __align__(16) uint16_t rnd[BITS == 8 ? ADAMW_WARPS : 1][ADAMW_BLOCK];
  // no early launch of dependents: what is written here may be a weight, which kernels fetch before their wait
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float clip = 1.f, keep_all = c.keep, step_size = c.step_size, isb2 = c.isb2;
  uint32_t step = c.step;
  if (c.step_dev || c.lr_dev) {
    if (threadIdx.x == 0) {
      const double t = c.step_dev ? (double)*c.step_dev : c.t;
      const double lr = c.lr_dev ? *c.lr_dev : c.lr;
      s_coef[0] = (float)(1.0 - lr * c.wd);
      s_coef[1] = (float)(lr / (1.0 - pow(c.beta1, t)));
      s_coef[2] = (float)(1.0 / sqrt(1.0 - pow(c.beta2, t)));
    }
    if (c.step_dev) step = (uint32_t)*c.step_dev;
    __syncthreads();
    keep_all = s_coef[0];
    step_size = s_coef[1];
    isb2 = s_coef[2];
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
      // a norm that is not finite: -1 marks the step as skipped
      s_clip = norm <= 1.7976931348623157e308 ? (float)fmin(1.0, c.max_norm / (norm + 1e-6)) : -1.f;
    }
    __syncthreads();
    clip = s_clip;
    if (clip < 0.f) return;
  }
  const uint32_t chunks = tab.first[tab.count];
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    if (PREFETCH && chunks - i > gridDim.x) {
      const uint32_t chunk = chunks - 1 - i - gridDim.x;
      const int t = find_tensor(tab, chunk);
      const AdamwEntry& e = tab.e[t];
      const long long base = (long long)(chunk - tab.first[t]) * ADAMW_CHUNK + warp * ADAMW_BLOCK;
      const int left = (int)max(min(e.n - base, (long long)ADAMW_BLOCK), 0ll);
      prefetch_l2(reinterpret_cast<const TP*>(e.p) + base, left, lane);
      prefetch_l2(reinterpret_cast<const TG*>(e.g) + base, left, lane);
      prefetch_l2(reinterpret_cast<const TS*>(e.m) + base, left, lane);
      prefetch_l2(reinterpret_cast<const TS*>(e.v) + base, left, lane);
    }
    // the tensor and the chunk are the block's: they and the pointers stay in uniform registers
    const uint32_t chunk = chunks - 1 - i;
    const int t = find_tensor(tab, chunk);
    const AdamwEntry& e = tab.e[t];
    const uint32_t tc = chunk - tab.first[t];  // chunk of the tensor
    const long long base = (long long)tc * ADAMW_CHUNK;
    const uint8_t flags = tab.flags[t];
    Place<TP, TG, TS> a;
    a.left = (int)min(e.n - base, (long long)ADAMW_CHUNK) - warp * ADAMW_BLOCK;
    if (a.left <= 0) continue;
    a.at = warp * ADAMW_BLOCK + lane * 8;
    a.vec = (flags & AF_VEC) && a.left >= ADAMW_BLOCK;
    a.p = reinterpret_cast<TP*>(e.p) + base;
    a.g = reinterpret_cast<const TG*>(e.g) + base;
    a.m = reinterpret_cast<TS*>(e.m) + base;
    a.v = reinterpret_cast<TS*>(e.v) + base;
    a.copy = e.copy ? e.copy + base : nullptr;
    a.keep = (flags & AF_DECAY) ? keep_all : 1.f;
    a.clip = clip;
    a.isb2 = isb2;
    a.step_size = step_size;
    if constexpr (BITS == 32) {
      update32(c, a);
    } else {
      const uint32_t block = tc * ADAMW_WARPS + warp;  // of the tensor
      a.ms = e.ms + block;
      a.vs = e.vs + block;
      update8(c, a, block, step, c.tensor0 + (uint32_t)t, lane, rnd[warp]);
    }
  }
  __threadfence();
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
template <typename... KArgs, typename... Args>
cudaError_t launch(bool pdl, void (*kernel)(KArgs...), unsigned grid, unsigned threads, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <int CAP>
using AdamwFn = void (*)(const AdamwTable<CAP>, const AdamwCoefs, const double*, int, float*);
template <int CAP, typename TP, typename TG>
AdamwFn<CAP> pick_bits(int bits) {
  return bits == 32 ? adamw_kernel<TP, TG, 32, CAP> : adamw_kernel<TP, TG, 8, CAP>;
}
template <int CAP>
AdamwFn<CAP> pick(int pt, int gt, int bits) {
  if (pt == SVLA_TYPE_F32)
    return gt == SVLA_TYPE_F32 ? pick_bits<CAP, float, float>(bits) : pick_bits<CAP, float, uint16_t>(bits);
  return gt == SVLA_TYPE_F32 ? pick_bits<CAP, uint16_t, float>(bits) : pick_bits<CAP, uint16_t, uint16_t>(bits);
}

// Blocks of a kernel that a device holds at once, asked for once a kernel and device.
template <typename Fn>
cudaError_t resident_blocks(Fn fn, int slot, unsigned* blocks) {
  static std::atomic<unsigned> known[16][64];
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*blocks = known[slot][dev].load()) != 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, ADAMW_THREADS, 0);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  *blocks = (unsigned)(per_sm * sms);
  if (dev < 64) known[slot][dev].store(*blocks);
  return cudaSuccess;
}

// Blocks of a step over `chunks`: what is resident at once, in as many waves as
// leave every block 8 chunks, up to 16, with 32-bit moments: blocks that start
// in order keep their accesses close together in memory, where ones that stay
// drift apart (99.8 M values: 463 us in 13 waves, 509 in one). One wave with
// 8-bit moments: the arithmetic bounds that step, and a block's start costs it
// about 2 us (157 M bf16 values: 381 us in one wave, 409 in 4).
unsigned step_blocks(unsigned chunks, unsigned resident, int bits) {
  const unsigned waves = bits == 32 ? std::min(chunks / (8 * resident), 16u) : 1;
  return std::min(chunks, resident * std::max(waves, 1u));
}

size_t launches_of(int n_tensors) { return ((size_t)n_tensors + ADAMW_CAP - 1) / ADAMW_CAP; }

// The launches of a step: with a clip, pass 0 sums the squares of every launch's gradients; pass 1 updates.
template <int CAP>
svla_status adamw_launches(const svla_adamw_tensor* ts, int n, const svla_adamw_args* a, AdamwCoefs& c, double* workspace,
                           float* grad_norm, cudaStream_t stream) {
  const size_t pb = a->param_type == SVLA_TYPE_F32 ? 4 : 2, gb = a->grad_type == SVLA_TYPE_F32 ? 4 : 2;
  const size_t sb = a->state_bits / 8;
  const AdamwFn<CAP> fn = pick<CAP>(a->param_type, a->grad_type, a->state_bits);
  unsigned resident = 0;
  cudaError_t e = resident_blocks(fn, (CAP == ADAMW_FEW ? 8 : 0) | (pb == 2 ? 4 : 0) | (gb == 2 ? 2 : 0) | (sb == 1), &resident);
  if (e != cudaSuccess) return svla_internal_fail(SVLA_ERR_CUDA, (std::string("adamw: ") + cudaGetErrorString(e)).c_str());
  const std::unique_ptr<AdamwTable<CAP>> table(new AdamwTable<CAP>);
  AdamwTable<CAP>& tab = *table;
  const int launches = (n + CAP - 1) / CAP;
  int n_partial = 0;
  bool pdl = false;
  for (int pass = a->max_norm > 0.0 ? 0 : 1; pass < 2; ++pass) {
    for (int l = 0; l < launches; ++l) {
      tab.count = std::min(CAP, n - l * CAP);
      unsigned long long nb = 0;
      for (int k = 0; k < tab.count; ++k) {
        const svla_adamw_tensor& t = ts[l * CAP + k];
        tab.e[k] = AdamwEntry{t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, reinterpret_cast<uint16_t*>(t.copy),
                              (long long)t.n};
        const bool vec = ((uintptr_t)t.param & (8 * pb - 1)) == 0 && ((uintptr_t)t.grad & (8 * gb - 1)) == 0 &&
                         ((uintptr_t)t.copy & 15) == 0 && (((uintptr_t)t.m | (uintptr_t)t.v) & (8 * sb - 1)) == 0;
        tab.flags[k] = (uint8_t)((t.decay ? AF_DECAY : 0) | (vec ? AF_VEC : 0));
        tab.first[k] = (uint32_t)nb;
        nb += (unsigned long long)((t.n + ADAMW_CHUNK - 1) / ADAMW_CHUNK);
      }
      if (nb > 0x7fffffffull) return svla_internal_fail(SVLA_ERR_SHAPE, "more than 2^42 elements in 400 tensors");
      tab.first[tab.count] = (uint32_t)nb;
      for (tab.shift = 0; (nb >> tab.shift) >= ADAMW_HINTS; ++tab.shift) {
      }
      for (int k = 0, at = 0; k <= ADAMW_HINTS; ++k) {
        while (at + 1 < tab.count && tab.first[at + 1] <= (unsigned long long)k << tab.shift) ++at;
        tab.hint[k] = (uint16_t)at;
      }
      const unsigned need = (unsigned)std::max(1ull, nb);
      if (pass == 0) {
        const unsigned grid = std::min((need + NORM_THREADS / ADAMW_THREADS - 1) / (NORM_THREADS / ADAMW_THREADS), (unsigned)NORM_BLOCKS);
        double* part = workspace + n_partial;
        e = a->grad_type == SVLA_TYPE_F32 ? launch(false, grad_norm_kernel<float, CAP>, grid, NORM_THREADS, stream, tab, part)
                                          : launch(false, grad_norm_kernel<uint16_t, CAP>, grid, NORM_THREADS, stream, tab, part);
        n_partial += (int)grid;
        pdl = true;
      } else {
        c.tensor0 = (uint32_t)(l * CAP);
        e = launch(pdl, fn, step_blocks(need, resident, a->state_bits), ADAMW_THREADS, stream, tab, c,
                   (const double*)workspace, n_partial, l == 0 ? grad_norm : nullptr);
        pdl = true;
      }
      if (e != cudaSuccess)
        return svla_internal_fail(SVLA_ERR_CUDA, (std::string("adamw launch: ") + cudaGetErrorString(e)).c_str());
    }
  }
  return SVLA_OK;
}

svla_status bad(svla_status s, int i, const char* why) {
  return svla_internal_fail(s, ((i < 0 ? std::string("workspace, grad_norm, step_device or lr_device")
                                       : "tensor " + std::to_string(i)) + ": " + why).c_str());
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
  if ((clip && (uintptr_t)grad_norm & 3) || ((uintptr_t)a->step_device | (uintptr_t)a->lr_device) & 7)
    return bad(SVLA_ERR_ARG, -1, "a pointer is not aligned to its element type");
  // every written range must be apart from every other range
  struct Range {
    uintptr_t at, end;
    int tensor;
    bool written;
  };
  std::vector<Range> ranges;
  ranges.reserve((size_t)n * 7 + 4);
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
  if (a->step_device) ranges.push_back(Range{(uintptr_t)a->step_device, (uintptr_t)a->step_device + 8, -1, false});
  if (a->lr_device) ranges.push_back(Range{(uintptr_t)a->lr_device, (uintptr_t)a->lr_device + 8, -1, false});
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
  const auto two = [](float x) {
    uint32_t b;
    memcpy(&b, &x, 4);
    return (unsigned long long)b << 32 | b;
  };
  c.b1_2 = two(c.b1);
  c.c1_2 = two(c.c1);
  c.b2_2 = two(c.b2);
  c.c2_2 = two(c.c2);
  c.eps_2 = two(c.eps);
  c.minus0_2 = two(-0.f);
  c.two24_2 = two(16777216.f);
  for (uint32_t r = 0; r < 10; ++r) {
    c.key[2 * r] = (uint32_t)a->seed + r * 0x9E3779B9u;
    c.key[2 * r + 1] = (uint32_t)(a->seed >> 32) + r * 0xBB67AE85u;
  }
  c.max_norm = a->max_norm;
  c.step = (uint32_t)a->step;
  c.t = (double)a->step;
  c.usual = c.eps < 0x1p100f ? USUAL_MAG : 0u;
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

  double* ws = reinterpret_cast<double*>(workspace);
  return n <= ADAMW_FEW ? adamw_launches<ADAMW_FEW>(ts, n, a, c, ws, grad_norm, stream)
                        : adamw_launches<ADAMW_CAP>(ts, n, a, c, ws, grad_norm, stream);
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
