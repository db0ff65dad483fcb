// svla_op_adamw: one AdamW step over many tensors (see the declaration in
// svla.h), with the moments in 32 bits or in 8, and the clip by the global
// gradient norm. The update half of the expert's fine-tune, whose loss and
// gradients svla_train_step computes.
//
// Per element, every product and sum rounded to fp32 by itself (no fused
// multiply-add), so the stored moments do not depend on how the compiler
// contracts the expression:
//   g' = g c,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   p  = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// The tensors' table travels in the kernel's parameters: nothing is copied to
// the device and nothing is kept between calls. A warp takes 256 consecutive
// elements of one tensor, the block that shares a scale in the 8-bit states;
// lanes hold 8 consecutive elements (16- and 32-byte accesses) where every
// pointer of the tensor allows it, else every 32nd one.
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

// two 8-bit codes -> two floats (exact; through fp16, which holds both formats)
template <bool E5M2>
SVLA_DEV float2 decode2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, E5M2 ? __NV_E5M2 : __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Codes of the 8-bit moments: the top bits of the fp32 magnitude, its exponent
// counted from a power of two that the block's largest finite magnitude sets.
// rnd16 enters at the top of the dropped bits: the code is rounded up with the
// probability of its distance to the lower code, so the stored moment is right
// in the mean. Nearest rounding would hold v where it is: a step moves v by
// (1 - b2) ~ 1e-3 of itself and the codes lie 1/8 to 1/4 apart.
//   m: e4m3, largest magnitude in [2^7, 2^8) of the scale; below 2^-6 -> 0
//   v: e5m2, largest in [2^14, 2^15); 0 < v below 2^-14 -> 2^-14, so no
//      gradient is ever divided by a vanished v
// Subnormal codes are not made. A value that is not finite has the NaN code.
SVLA_DEV uint32_t encode_m(float x, uint32_t rnd16, uint32_t low) {
  const uint32_t bits = __float_as_uint(x), mag = bits & 0x7fffffffu;
  const int code = (int)((mag + (rnd16 << 4)) >> 20) - (int)low;
  const uint32_t c = code < 8 ? 0u : (uint32_t)code | ((bits >> 24) & 0x80u);
  return mag >= 0x7f800000u ? 0x7fu : c;
}
SVLA_DEV uint32_t encode_v(float x, uint32_t rnd16, uint32_t low) {
  const uint32_t mag = __float_as_uint(x);
  const int code = (int)((mag + (rnd16 << 5)) >> 21) - (int)low;
  const uint32_t c = mag == 0 ? 0u : (uint32_t)max(code, 4);
  return mag >= 0x7f800000u ? 0x7fu : c;
}
SVLA_DEV uint32_t finite_mag(float x) {
  const uint32_t mag = __float_as_uint(x) & 0x7fffffffu;
  return mag >= 0x7f800000u ? 0u : mag;
}

// one element, both moments in fp32
SVLA_DEV void update1(const AdamwCoefs& c, float keep, float g, float& p, float& m, float& v) {
  m = __fadd_rn(__fmul_rn(m, c.b1), __fmul_rn(g, c.c1));
  v = __fadd_rn(__fmul_rn(v, c.b2), __fmul_rn(__fmul_rn(g, g), c.c2));
  const float denom = __fadd_rn(__fmul_rn(__fsqrt_rn(v), c.isb2), c.eps);
  p = __fsub_rn(__fmul_rn(p, keep), __fmul_rn(__fdiv_rn(m, denom), c.step_size));
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
    const TG* g = reinterpret_cast<const TG*>(e.g) + base;
    const long long left = e.n - base;
    float x[8];
    if ((tab.flags[t] & AF_VEC) && left >= ADAMW_BLOCK) {
      load8(g + lane * 8, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = j * 32 + lane < left ? load1(g + j * 32 + lane) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j & 1] = fma((double)x[j], (double)x[j], acc[j & 1]);
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
template <typename TP, typename TG, int BITS>
__global__ void __launch_bounds__(ADAMW_THREADS) adamw_kernel(const __grid_constant__ AdamwTable tab,
                                                              const __grid_constant__ AdamwCoefs c0,
                                                              const double* __restrict__ partial, int n_partial,
                                                              float* __restrict__ grad_norm) {
  __shared__ double part[ADAMW_WARPS];
  __shared__ float s_clip;
  __shared__ float s_coef[3];
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
    const long long left = e.n - base;
    const bool vec = (tab.flags[t] & AF_VEC) && left >= ADAMW_BLOCK;
    const float keep = (tab.flags[t] & AF_DECAY) ? c.keep : 1.f;
    TP* pp = reinterpret_cast<TP*>(e.p) + base;
    const TG* gp = reinterpret_cast<const TG*>(e.g) + base;
    uint16_t* cp = e.copy ? e.copy + base : nullptr;
    float p[8], g[8], m[8], v[8];
    // element of this lane's slot j: lane * 8 + j (vector accesses), else j * 32 + lane
    if (vec) {
      load8(pp + lane * 8, p);
      load8(gp + lane * 8, g);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = j * 32 + lane < left;
        p[j] = in ? load1(pp + j * 32 + lane) : 0.f;
        g[j] = in ? load1(gp + j * 32 + lane) : 0.f;
      }
    }
    if constexpr (BITS == 32) {
      float* mp = reinterpret_cast<float*>(e.m) + base;
      float* vp = reinterpret_cast<float*>(e.v) + base;
      if (vec) {
        load8(mp + lane * 8, m);
        load8(vp + lane * 8, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = j * 32 + lane < left;
          m[j] = in ? mp[j * 32 + lane] : 0.f;
          v[j] = in ? vp[j * 32 + lane] : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) update1(c, keep, __fmul_rn(g[j], clip), p[j], m[j], v[j]);
      if (vec) {
        store8(mp + lane * 8, m);
        store8(vp + lane * 8, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j * 32 + lane < left) {
            mp[j * 32 + lane] = m[j];
            vp[j * 32 + lane] = v[j];
          }
      }
    } else {
      uint8_t* mp = reinterpret_cast<uint8_t*>(e.m) + base;
      uint8_t* vp = reinterpret_cast<uint8_t*>(e.v) + base;
      const float ms = e.ms[tb], vs = e.vs[tb];
      uint32_t mc[8], vc[8];
      if (vec) {
        const uint2 a = *reinterpret_cast<const uint2*>(mp + lane * 8);
        const uint2 b = *reinterpret_cast<const uint2*>(vp + lane * 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = decode2<false>(((j < 2 ? a.x : a.y) >> (16 * (j & 1))) & 0xffffu);
          const float2 y = decode2<true>(((j < 2 ? b.x : b.y) >> (16 * (j & 1))) & 0xffffu);
          m[2 * j] = x.x, m[2 * j + 1] = x.y;
          v[2 * j] = y.x, v[2 * j + 1] = y.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = j * 32 + lane < left;
          m[j] = in ? decode2<false>(mp[j * 32 + lane]).x : 0.f;
          v[j] = in ? decode2<true>(vp[j * 32 + lane]).x : 0.f;
        }
      }
      uint32_t mx = 0, vx = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = __fmul_rn(m[j], ms);
        v[j] = __fmul_rn(v[j], vs);
        update1(c, keep, __fmul_rn(g[j], clip), p[j], m[j], v[j]);
        mx = max(mx, finite_mag(m[j]));
        vx = max(vx, finite_mag(v[j]));
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      vx = __reduce_max_sync(0xffffffffu, vx);
      const uint32_t em = (uint32_t)max((int)(mx >> 23) - 14, 0), ev = (uint32_t)max((int)(vx >> 23) - 29, 0);
      // 16 random bits of element k: half k % 8 of the draw of its octet k / 8; both moments take the same bits
      // (each is right in the mean by itself, and the ratio's error is smaller when they round the same way)
      const unsigned long long oct = (unsigned long long)tb * 32 + lane;
      uint32_t r[4] = {(uint32_t)oct, (uint32_t)(oct >> 32), c.step, c.tensor0 + (uint32_t)t};
      philox4x32_10(r, c.k0, c.k1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t u;
        if (vec) {
          u = (r[j >> 1] >> (16 * (j & 1))) & 0xffffu;
        } else {
          const int src = j * 4 + (lane >> 3);
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = __shfl_sync(0xffffffffu, r[k], src);
          const uint32_t a = (lane & 2) ? w[1] : w[0], b = (lane & 2) ? w[3] : w[2];
          u = (((lane & 4) ? b : a) >> (16 * (lane & 1))) & 0xffffu;
        }
        mc[j] = encode_m(m[j], u, em << 3);
        vc[j] = encode_v(v[j], u, ev << 2);
      }
      if (vec) {
        *reinterpret_cast<uint2*>(mp + lane * 8) =
            make_uint2(mc[0] | mc[1] << 8 | mc[2] << 16 | mc[3] << 24, mc[4] | mc[5] << 8 | mc[6] << 16 | mc[7] << 24);
        *reinterpret_cast<uint2*>(vp + lane * 8) =
            make_uint2(vc[0] | vc[1] << 8 | vc[2] << 16 | vc[3] << 24, vc[4] | vc[5] << 8 | vc[6] << 16 | vc[7] << 24);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j * 32 + lane < left) {
            mp[j * 32 + lane] = (uint8_t)mc[j];
            vp[j * 32 + lane] = (uint8_t)vc[j];
          }
      }
      if (lane == 0) {
        e.ms[tb] = mx ? __uint_as_float((em + 7) << 23) : 0.f;
        e.vs[tb] = vx ? __uint_as_float((ev + 15) << 23) : 0.f;
      }
    }
    if (vec) {
      store8(pp + lane * 8, p);
      if (cp) store8(cp + lane * 8, p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j * 32 + lane < left) {
          store1(pp + j * 32 + lane, p[j]);
          if (cp) store1(cp + j * 32 + lane, p[j]);
        }
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
        const bool vec = (((uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.copy) & 15) == 0 &&
                         (((uintptr_t)t.m | (uintptr_t)t.v) & (a->state_bits == 32 ? 15 : 7)) == 0;
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
