// svla_op_layernorm and svla_op_layernorm_backward (see the declarations in
// svla.h): the norm of the vision side's layers, beside the RMSNorm of the
// language side, with the gradients that training them needs.
//
//   mu = mean(x), var = mean((x - mu)^2), r = 1 / sqrt(var + eps)
//   y  = (x - mu) r gamma + beta
//   backward, xh = (x - mu) r and w = dy gamma:
//   dx = r (w - mean(w) - xh mean(w xh)),  dgamma = sum dy xh,  dbeta = sum dy
//
// Both passes read each row once into registers: T threads hold NU units of 8
// elements each, T = 32 up to 1024 columns (the row's sums are shuffles of one
// warp), else the fewest warps that hold a row in two units a thread. With VEC
// a unit is 8 consecutive columns (16- and 32-byte accesses); else (an odd
// width, stride or address) every 32nd one of its warp's 256.
#include <algorithm>
#include <exception>
#include <string>
#include <utility>

#include "common.cuh"
#include "elements.cuh"

svla_status svla_internal_fail(svla_status s, const char* msg);

namespace svla {
namespace {

constexpr int LN_MAX_D = 16384;
constexpr int LN_BWD_BLOCKS = 296;  // blocks (partial sums of dgamma and dbeta): 2 on each of 148 SMs
constexpr int LN_SMEM_ACC_D = 8192; // wider rows keep the column sums in shared memory

struct LnPlan {
  int T, NU, R, threads;  // threads a row, units a thread, rows a block, threads a block
};

LnPlan ln_plan(int D, bool backward) {
  LnPlan p;
  const int units = (D + 7) / 8;
  if (units <= 128) {
    p.T = 32;
    p.NU = (units + 31) / 32;
  } else if (backward && D > LN_SMEM_ACC_D) {
    p.T = 512;
    p.NU = 4;
  } else {
    p.T = 32 * ((units + 63) / 64);
    p.NU = 2;
  }
  p.R = std::max(1, 256 / p.T);
  p.threads = p.R * p.T;
  return p;
}

int ln_bwd_blocks(int M, const LnPlan& p) { return std::min((M + p.R - 1) / p.R, LN_BWD_BLOCKS); }

struct LnArgs {
  const void* x;
  const void* dy;
  const void* gamma;
  const void* beta;
  void* out;  // y or dx
  long long ldx, lddy, ldo;
  float* mean;
  float* rstd;
  float* dgamma;
  float* dbeta;
  float* partial;  // [blocks][2][slots] where more than one block sums
  int M, D, T;
  float eps, inv_d;
};

// column of element k of unit u of this thread
template <bool VEC>
SVLA_DEV int column(int u, int k, int T, int tid) {
  return VEC ? (u * T + tid) * 8 + k : (u * T + (tid & ~31)) * 8 + k * 32 + (tid & 31);
}

// one row's elements of this thread as they lie in memory (zeros past the width)
template <typename E, int NU, bool VEC>
struct RowRegs;
template <int NU>
struct RowRegs<float, NU, true> {
  float4 q[2 * NU];
  SVLA_DEV void load(const float* p, int D, int T, int tid) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int c = (u * T + tid) * 8;
      q[2 * u] = q[2 * u + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < D) {
        q[2 * u] = *reinterpret_cast<const float4*>(p + c);
        q[2 * u + 1] = *reinterpret_cast<const float4*>(p + c + 4);
      }
    }
  }
  SVLA_DEV float get(int u, int k) const {
    const float4& f = q[2 * u + (k >> 2)];
    return (k & 3) == 0 ? f.x : (k & 3) == 1 ? f.y : (k & 3) == 2 ? f.z : f.w;
  }
};
template <int NU>
struct RowRegs<uint16_t, NU, true> {
  uint4 q[NU];
  SVLA_DEV void load(const uint16_t* p, int D, int T, int tid) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int c = (u * T + tid) * 8;
      q[u] = make_uint4(0u, 0u, 0u, 0u);
      if (c < D) q[u] = *reinterpret_cast<const uint4*>(p + c);
    }
  }
  SVLA_DEV float get(int u, int k) const {
    const uint32_t w = (k >> 1) == 0 ? q[u].x : (k >> 1) == 1 ? q[u].y : (k >> 1) == 2 ? q[u].z : q[u].w;
    return __uint_as_float((k & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <typename E, int NU>
struct RowRegs<E, NU, false> {
  E q[NU * 8];
  SVLA_DEV void load(const E* p, int D, int T, int tid) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int c = column<false>(u, 0, T, tid);
#pragma unroll
      for (int k = 0; k < 8; ++k) q[u * 8 + k] = c + k * 32 < D ? p[c + k * 32] : E(0);
    }
  }
  SVLA_DEV float get(int u, int k) const { return load1(&q[u * 8 + k]); }
};

// columns of a vector of weights into 8 floats of unit u
template <typename TW, bool VEC>
SVLA_DEV void load_unit(const TW* w, int u, int D, int T, int tid, float (&x)[8]) {
  if constexpr (VEC) {
    const int c = (u * T + tid) * 8;
    if (c < D) load8(w + c, x);
  } else {
    const int c = column<false>(u, 0, T, tid);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = c + k * 32 < D ? load1(w + c + k * 32) : 0.f;
  }
}

// Sums over the T threads of a row: a butterfly of the warp, then (T > 32) one
// of the warps' sums, which every warp reads from shared memory. red: one float2
// a warp of the block.
template <int N>
SVLA_DEV void row_sums(float (&s)[N], int T, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (T == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = T >> 5, first = warp / per * per;
  if (lane == 0) red[warp] = make_float2(s[0], N > 1 ? s[N - 1] : 0.f);
  __syncthreads();
  const float2 v = lane < per ? red[first + lane] : make_float2(0.f, 0.f);
  s[0] = v.x;
  if (N > 1) s[N - 1] = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < per)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = __shfl_sync(0xffffffffu, s[i], 0);
}

// ---------------------------------------------------------------------------
// forward: one row a group of T threads; mean first, then the squares of the
// differences from registers (no cancellation of two large sums)
// ---------------------------------------------------------------------------
template <typename TX, typename TY, typename TW, int NU, bool VEC>
__global__ void __launch_bounds__(NU == 2 ? 1024 : 256) layernorm_kernel(const LnArgs a) {
  __shared__ float2 red[2][32];
  griddep_launch_dependents();
  griddep_wait();  // nothing is read before: the weights may come from an optimiser step
  const int T = a.T, tid = threadIdx.x % T, D = a.D;
  const long long row = (long long)blockIdx.x * (blockDim.x / T) + threadIdx.x / T;
  const bool active = row < a.M;
  RowRegs<TX, NU, VEC> x;
  x.load(reinterpret_cast<const TX*>(a.x) + (active ? row : 0) * a.ldx, D, T, tid);
  float s[1] = {0.f};
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += x.get(u, k);
  row_sums(s, T, red[0]);
  const float mean = s[0] * a.inv_d;
  s[0] = 0.f;
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = x.get(u, k) - mean;
      if (column<VEC>(u, k, T, tid) < D) s[0] = fmaf(d, d, s[0]);
    }
  row_sums(s, T, red[1]);
  const float rstd = rsqrtf(s[0] * a.inv_d + a.eps);
  if (!active) return;
  TY* y = reinterpret_cast<TY*>(a.out) + row * a.ldo;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    float g[8], b[8] = {}, o[8];
    load_unit<TW, VEC>(reinterpret_cast<const TW*>(a.gamma), u, D, T, tid, g);
    if (a.beta) load_unit<TW, VEC>(reinterpret_cast<const TW*>(a.beta), u, D, T, tid, b);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = fmaf((x.get(u, k) - mean) * rstd, g[k], b[k]);
    if constexpr (VEC) {
      const int c = (u * T + tid) * 8;
      if (c < D) store8(y + c, o);
    } else {
      const int c = column<false>(u, 0, T, tid);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k * 32 < D) store1(y + c + k * 32, o[k]);
    }
  }
  if (tid == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// ---------------------------------------------------------------------------
// backward: each group of T threads walks rows blockIdx.x * R + group, + grid *
// R, .. and keeps its columns' sums of dgamma and dbeta; the next row is on its
// way (VEC) while the current one is reduced. At the end the groups' sums are
// added in order and go to `partial` (or to dgamma and dbeta, where there is one
// block). Column sums are kept by slot, (u * 8 + k) * T + thread for element k
// of unit u, so that neighbouring threads have neighbouring words.
// ---------------------------------------------------------------------------
template <bool VEC>
SVLA_DEV int slot_column(int slot, int T) {
  const int q = slot / T;
  return column<VEC>(q >> 3, q & 7, T, slot - q * T);
}

template <typename TX, typename TY, typename TW, int NU, bool VEC, bool SMEM_ACC>
__global__ void __launch_bounds__(SMEM_ACC ? 512 : NU > 2 ? 256 : 512, SMEM_ACC ? 1 : NU > 2 ? 2 : 1)
    layernorm_bwd_kernel(const LnArgs a) {
  extern __shared__ __align__(16) float cols[];  // [R][2][slots] column sums (SMEM_ACC: [2][slots])
  __shared__ float2 red[2][16];
  // the next row's registers, where they leave two blocks an SM (16 warps)
  constexpr int ROW = NU * 2 * (int)(sizeof(TX) + sizeof(TY));
  constexpr bool PREFETCH = VEC && !SMEM_ACC && 2 * ROW + 16 * NU <= 96;
  griddep_launch_dependents();
  griddep_wait();
  const int T = a.T, tid = threadIdx.x % T, D = a.D, R = blockDim.x / T, group = threadIdx.x / T;
  const int W = NU * 8 * T;  // slots
  const TX* xp = reinterpret_cast<const TX*>(a.x);
  const TY* dyp = reinterpret_cast<const TY*>(a.dy);
  float ag[SMEM_ACC ? 1 : NU * 8], ab[SMEM_ACC ? 1 : NU * 8];
  if constexpr (SMEM_ACC) {
    for (int c = threadIdx.x; c < 2 * W; c += blockDim.x) cols[c] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int j = 0; j < NU * 8; ++j) ag[j] = ab[j] = 0.f;
  }
  const long long stride = (long long)gridDim.x * R;
  long long row0 = (long long)blockIdx.x * R;
  RowRegs<TX, NU, VEC> x;
  RowRegs<TY, NU, VEC> dy;
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](long long row, RowRegs<TX, NU, VEC>& fx, RowRegs<TY, NU, VEC>& fy, float& m, float& r) {
    const bool in = row < a.M;
    const long long at = in ? row : 0;
    fx.load(xp + at * a.ldx, in ? D : 0, T, tid);
    fy.load(dyp + at * a.lddy, in ? D : 0, T, tid);
    m = in ? a.mean[at] : 0.f;
    r = in ? a.rstd[at] : 0.f;
  };
  if (PREFETCH) fetch(row0 + group, x, dy, mean, rstd);
  for (int it = 0; row0 < a.M; row0 += stride, ++it) {
    const long long row = row0 + group;
    RowRegs<TX, NU, VEC> nx;
    RowRegs<TY, NU, VEC> ndy;
    float nmean = 0.f, nrstd = 0.f;
    if (PREFETCH) {
      if (row0 + stride < a.M) fetch(row + stride, nx, ndy, nmean, nrstd);
    } else {
      fetch(row, x, dy, mean, rstd);
    }
    float s[2] = {0.f, 0.f};  // sums of w and of w xh
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      float g[8] = {};
      load_unit<TW, VEC>(reinterpret_cast<const TW*>(a.gamma), u, D, T, tid, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = dy.get(u, k), xh = (x.get(u, k) - mean) * rstd, w = d * g[k];
        s[0] += w;
        s[1] = fmaf(w, xh, s[1]);
        if constexpr (SMEM_ACC) {
          float* c = cols + (u * 8 + k) * T + tid;
          c[0] = fmaf(d, xh, c[0]);
          c[W] += d;
        } else {
          ag[u * 8 + k] = fmaf(d, xh, ag[u * 8 + k]);
          ab[u * 8 + k] += d;
        }
      }
    }
    row_sums(s, T, red[it & 1]);
    const float s0 = s[0] * a.inv_d, s1 = s[1] * a.inv_d;
    if (row < a.M) {
      TX* dx = reinterpret_cast<TX*>(a.out) + row * a.ldo;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        float g[8] = {}, o[8];
        load_unit<TW, VEC>(reinterpret_cast<const TW*>(a.gamma), u, D, T, tid, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xh = (x.get(u, k) - mean) * rstd, w = dy.get(u, k) * g[k];
          o[k] = rstd * (w - s0 - xh * s1);
        }
        if constexpr (VEC) {
          const int c = (u * T + tid) * 8;
          if (c < D) store8(dx + c, o);
        } else {
          const int c = column<false>(u, 0, T, tid);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k * 32 < D) store1(dx + c + k * 32, o[k]);
        }
      }
    }
    if (PREFETCH) {
      x = nx;
      dy = ndy;
      mean = nmean;
      rstd = nrstd;
    }
  }
  if (!a.dgamma && !a.dbeta) return;
  if constexpr (!SMEM_ACC) {
    float* mine = cols + (size_t)group * 2 * W + tid;
#pragma unroll
    for (int j = 0; j < NU * 8; ++j) {
      mine[j * T] = ag[j];
      mine[W + j * T] = ab[j];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * W; c += blockDim.x) {
    float v = cols[c];
    if constexpr (!SMEM_ACC)
      for (int r = 1; r < R; ++r) v += cols[(size_t)r * 2 * W + c];
    if (gridDim.x > 1) {
      a.partial[(size_t)blockIdx.x * 2 * W + c] = v;
    } else {
      const int col = slot_column<VEC>(c < W ? c : c - W, T);
      float* out = c < W ? a.dgamma : a.dbeta;
      if (out && col < D) out[col] = v;
    }
  }
}

// dgamma and dbeta: the blocks' partial sums added per slot. A block of 32
// slots; thread row j adds the blocks j, j + 32, .. and the 32 sums are added in
// order.
template <bool VEC>
__global__ void __launch_bounds__(1024) layernorm_cols_kernel(const float* partial, int blocks, int D, int W, int T,
                                                              float* dgamma, float* dbeta) {
  __shared__ float part[32][33];
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
#pragma unroll 10
  for (int b = threadIdx.y; b < blocks; b += 32) s += partial[(size_t)b * 2 * W + c];
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0) {
    s = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) s += part[j][threadIdx.x];
    const int col = slot_column<VEC>(c < W ? c : c - W, T);
    float* out = c < W ? dgamma : dbeta;
    if (out && col < D) out[col] = s;
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
typedef void (*LnFn)(const LnArgs);

template <typename TX, typename TY, typename TW, bool VEC>
LnFn pick_fwd(int NU) {
  switch (NU) {
    case 1: return layernorm_kernel<TX, TY, TW, 1, VEC>;
    case 2: return layernorm_kernel<TX, TY, TW, 2, VEC>;
    case 3: return layernorm_kernel<TX, TY, TW, 3, VEC>;
    default: return layernorm_kernel<TX, TY, TW, 4, VEC>;
  }
}
template <typename TX, typename TY, typename TW, bool VEC>
LnFn pick_bwd(int NU, bool smem) {
  if (smem) return layernorm_bwd_kernel<TX, TY, TW, 4, VEC, true>;
  switch (NU) {
    case 1: return layernorm_bwd_kernel<TX, TY, TW, 1, VEC, false>;
    case 2: return layernorm_bwd_kernel<TX, TY, TW, 2, VEC, false>;
    case 3: return layernorm_bwd_kernel<TX, TY, TW, 3, VEC, false>;
    default: return layernorm_bwd_kernel<TX, TY, TW, 4, VEC, false>;
  }
}
template <typename TX, typename TY, typename TW>
LnFn pick_v(bool bwd, bool vec, int NU, bool smem) {
  if (bwd) return vec ? pick_bwd<TX, TY, TW, true>(NU, smem) : pick_bwd<TX, TY, TW, false>(NU, smem);
  return vec ? pick_fwd<TX, TY, TW, true>(NU) : pick_fwd<TX, TY, TW, false>(NU);
}
LnFn pick(int xt, int yt, int wt, bool bwd, bool vec, int NU, bool smem) {
  typedef uint16_t h;
  const int k = (xt == SVLA_TYPE_BF16 ? 4 : 0) | (yt == SVLA_TYPE_BF16 ? 2 : 0) | (wt == SVLA_TYPE_BF16 ? 1 : 0);
  switch (k) {
    case 0: return pick_v<float, float, float>(bwd, vec, NU, smem);
    case 1: return pick_v<float, float, h>(bwd, vec, NU, smem);
    case 2: return pick_v<float, h, float>(bwd, vec, NU, smem);
    case 3: return pick_v<float, h, h>(bwd, vec, NU, smem);
    case 4: return pick_v<h, float, float>(bwd, vec, NU, smem);
    case 5: return pick_v<h, float, h>(bwd, vec, NU, smem);
    case 6: return pick_v<h, h, float>(bwd, vec, NU, smem);
    default: return pick_v<h, h, h>(bwd, vec, NU, smem);
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

svla_status arg(const char* why) { return svla_internal_fail(SVLA_ERR_ARG, why); }
svla_status shape(const char* why) { return svla_internal_fail(SVLA_ERR_SHAPE, why); }
bool known(int t) { return t == SVLA_TYPE_F32 || t == SVLA_TYPE_BF16; }
size_t bytes_of(int t) { return t == SVLA_TYPE_F32 ? 4 : 2; }

// a [M, D] matrix with rows ld apart
struct Mat {
  const void* p;
  long long ld;
  int type;
  uintptr_t begin() const { return (uintptr_t)p; }
  uintptr_t end(int M, int D) const { return (uintptr_t)p + ((size_t)(M - 1) * ld + D) * bytes_of(type); }
  bool vec() const { return (((uintptr_t)p | (uintptr_t)(ld * bytes_of(type))) & 15) == 0; }
  bool same(const Mat& o) const { return p == o.p && ld == o.ld && type == o.type; }
};
bool overlap(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) { return a0 < b1 && b0 < a1; }
// an output may be an input matrix itself (each row is read before it is written), not a part of it
bool clash(const Mat& out, const Mat& in, int M, int D) {
  return !out.same(in) && overlap(out.begin(), out.end(M, D), in.begin(), in.end(M, D));
}
bool clash(const Mat& out, const void* v, size_t bytes, int M, int D) {
  return v && overlap(out.begin(), out.end(M, D), (uintptr_t)v, (uintptr_t)v + bytes);
}

svla_status run(LnArgs& a, int xt, int yt, int wt, bool bwd, bool vec, cudaStream_t s) {
  const LnPlan p = ln_plan(a.D, bwd);
  a.T = p.T;
  a.inv_d = (float)(1.0 / a.D);
  const bool smem_acc = bwd && a.D > LN_SMEM_ACC_D;
  const LnFn fn = pick(xt, yt, wt, bwd, vec, p.NU, smem_acc);
  const int blocks = bwd ? ln_bwd_blocks(a.M, p) : (a.M + p.R - 1) / p.R;
  const int W = p.NU * 8 * p.T;
  const size_t smem = bwd && (smem_acc || a.dgamma || a.dbeta) ? (size_t)(smem_acc ? 1 : p.R) * 2 * W * sizeof(float) : 0;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = launch(fn, dim3(blocks), dim3(p.threads), smem, s, a);
  if (e == cudaSuccess && bwd && blocks > 1 && (a.dgamma || a.dbeta))
    e = launch(vec ? layernorm_cols_kernel<true> : layernorm_cols_kernel<false>, dim3(2 * W / 32), dim3(32, 32), 0, s,
               (const float*)a.partial, blocks, a.D, W, p.T, a.dgamma, a.dbeta);
  if (e != cudaSuccess)
    return svla_internal_fail(SVLA_ERR_CUDA, (std::string("layernorm launch: ") + cudaGetErrorString(e)).c_str());
  return SVLA_OK;
}

}  // namespace
}  // namespace svla

extern "C" {

svla_status svla_op_layernorm(const void* x, int x_type, int ldx, const void* gamma, const void* beta, int w_type,
                              int M, int D, float eps, void* y, int y_type, int ldy, float* mean, float* rstd,
                              void* stream) {
  using namespace svla;
  if (!known(x_type) || !known(y_type) || !known(w_type)) return arg("unknown element type");
  if (M < 0 || D < 1 || D > LN_MAX_D || ldx < D || ldy < D || !(eps > 0.f))
    return shape("M >= 0, 1 <= D <= 16384, strides >= D and eps > 0");
  if (!gamma || (M > 0 && (!x || !y))) return arg("null pointer");
  const size_t wb = bytes_of(w_type);
  if ((uintptr_t)x % bytes_of(x_type) || (uintptr_t)y % bytes_of(y_type) || (uintptr_t)gamma % wb ||
      (uintptr_t)beta % wb || (((uintptr_t)mean | (uintptr_t)rstd) & 3))
    return arg("a pointer is not aligned to its element type");
  if (M == 0) return SVLA_OK;
  const Mat mx{x, ldx, x_type}, my{y, ldy, y_type};
  const size_t col = (size_t)M * 4;
  bool inner = mean && rstd && overlap((uintptr_t)mean, (uintptr_t)mean + col, (uintptr_t)rstd, (uintptr_t)rstd + col);
  for (const float* v : {mean, rstd}) {
    if (!v) continue;
    const uintptr_t v0 = (uintptr_t)v, v1 = v0 + col;
    inner = inner || clash(mx, v, col, M, D) || overlap(v0, v1, (uintptr_t)gamma, (uintptr_t)gamma + D * wb) ||
            (beta && overlap(v0, v1, (uintptr_t)beta, (uintptr_t)beta + D * wb));
  }
  if (inner) return arg("mean or rstd overlaps another argument");
  if (clash(my, mx, M, D) || clash(my, gamma, D * wb, M, D) || clash(my, beta, D * wb, M, D) ||
      clash(my, mean, col, M, D) || clash(my, rstd, col, M, D))
    return arg("y overlaps another argument (it may be x itself, with its type and stride)");
  LnArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.gamma = gamma;
  a.beta = beta;
  a.out = y;
  a.ldo = ldy;
  a.mean = mean;
  a.rstd = rstd;
  a.M = M;
  a.D = D;
  a.eps = eps;
  const bool vec = D % 8 == 0 && mx.vec() && my.vec() && (((uintptr_t)gamma | (uintptr_t)beta) & 15) == 0;
  return run(a, x_type, y_type, w_type, false, vec, reinterpret_cast<cudaStream_t>(stream));
}

size_t svla_op_layernorm_backward_workspace_bytes(int M, int D) {
  if (M < 1 || D < 1 || D > svla::LN_MAX_D) return 0;
  const svla::LnPlan p = svla::ln_plan(D, true);
  const int blocks = svla::ln_bwd_blocks(M, p);
  return blocks > 1 ? (size_t)blocks * 2 * p.NU * 8 * p.T * sizeof(float) : 0;
}

svla_status svla_op_layernorm_backward(const void* dy, int y_type, int lddy, const void* x, int x_type, int ldx,
                                       const void* gamma, int w_type, const float* mean, const float* rstd, int M,
                                       int D, void* dx, int lddx, float* dgamma, float* dbeta, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  using namespace svla;
  if (!known(x_type) || !known(y_type) || !known(w_type)) return arg("unknown element type");
  if (M < 0 || D < 1 || D > LN_MAX_D || lddy < D || ldx < D || lddx < D)
    return shape("M >= 0, 1 <= D <= 16384 and strides >= D");
  if (!gamma || (M > 0 && (!x || !dy || !dx || !mean || !rstd))) return arg("null pointer");
  if ((uintptr_t)x % bytes_of(x_type) || (uintptr_t)dx % bytes_of(x_type) || (uintptr_t)dy % bytes_of(y_type) ||
      (uintptr_t)gamma % bytes_of(w_type) ||
      (((uintptr_t)mean | (uintptr_t)rstd | (uintptr_t)dgamma | (uintptr_t)dbeta) & 3))
    return arg("a pointer is not aligned to its element type");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {  // no rows: the gradients are zero
    cudaError_t e = cudaSuccess;
    if (dgamma) e = cudaMemsetAsync(dgamma, 0, (size_t)D * 4, s);
    if (e == cudaSuccess && dbeta) e = cudaMemsetAsync(dbeta, 0, (size_t)D * 4, s);
    if (e != cudaSuccess) return svla_internal_fail(SVLA_ERR_CUDA, cudaGetErrorString(e));
    return SVLA_OK;
  }
  const size_t need = dgamma || dbeta ? svla_op_layernorm_backward_workspace_bytes(M, D) : 0;
  if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 3)))
    return arg("workspace missing, too small (svla_op_layernorm_backward_workspace_bytes) or not 4-byte aligned");
  const Mat mx{x, ldx, x_type}, mdy{dy, lddy, y_type}, mdx{dx, lddx, x_type};
  struct Vec {
    const void* p;
    size_t bytes;
  };
  const Vec in[] = {{gamma, D * bytes_of(w_type)}, {mean, (size_t)M * 4}, {rstd, (size_t)M * 4}};
  const Vec out[] = {{dgamma, (size_t)D * 4}, {dbeta, (size_t)D * 4}, {need ? workspace : nullptr, need}};
  bool bad = clash(mdx, mx, M, D) || clash(mdx, mdy, M, D);
  for (const Vec& v : in) bad = bad || clash(mdx, v.p, v.bytes, M, D);
  for (int i = 0; i < 3 && !bad; ++i) {
    const Vec& o = out[i];
    if (!o.p) continue;
    bad = clash(mdx, o.p, o.bytes, M, D) || clash(mx, o.p, o.bytes, M, D) || clash(mdy, o.p, o.bytes, M, D);
    const uintptr_t o0 = (uintptr_t)o.p, o1 = o0 + o.bytes;
    for (const Vec& v : in) bad = bad || overlap(o0, o1, (uintptr_t)v.p, (uintptr_t)v.p + v.bytes);
    for (int j = 0; j < i; ++j) bad = bad || (out[j].p && overlap(o0, o1, (uintptr_t)out[j].p, (uintptr_t)out[j].p + out[j].bytes));
  }
  if (bad) return arg("an output overlaps another argument (dx may be x or dy itself, with its type and stride)");
  LnArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.dy = dy;
  a.lddy = lddy;
  a.gamma = gamma;
  a.out = dx;
  a.ldo = lddx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.partial = reinterpret_cast<float*>(workspace);
  a.M = M;
  a.D = D;
  const bool vec = D % 8 == 0 && mx.vec() && mdy.vec() && mdx.vec() && ((uintptr_t)gamma & 15) == 0;
  return run(a, x_type, y_type, w_type, true, vec, s);
}

}  // extern "C"
