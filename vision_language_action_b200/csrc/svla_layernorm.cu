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
// elements each. Narrow rows (up to 128 columns) take a part of a warp, T = 1 to
// 16; wider ones whole warps. With VEC a unit is 8 consecutive columns (16- and
// 32-byte accesses); else (an odd width, stride or address) every 32nd (narrow:
// T-th) one.
//
// Both are bound by memory where there are many rows, by latency where there are
// few. Measured: forward of 65536 x 768, fp32 in and bf16 out, 51.5 us (5.9
// TB/s); backward of 16384 rows, bf16: 768 wide 22 us (3.4 TB/s), 4096 wide 82
// us (4.9 TB/s); of 4000 rows 12288 wide 75 us (3.9 TB/s), 16384 wide 117 us (3.4
// TB/s). One row 3.1 us, 50 rows backward 6.1 us: a launch.
#include <algorithm>
#include <atomic>
#include <exception>
#include <string>
#include <utility>

#include "common.cuh"
#include "elements.cuh"
#include "pairs.cuh"

svla_status svla_internal_fail(svla_status s, const char* msg);

namespace svla {
namespace {

constexpr int LN_MAX_D = 16384;
constexpr int LN_SMS = 148;
constexpr int LN_BWD_PER_SM = 4;  // blocks an SM at most (each has partial sums of dgamma and dbeta)
// Up to this many blocks form a cluster and add their column sums through each other's shared memory: one launch, not
// two, and no workspace (50 rows of 720, bf16: 10.3 us a call, 15.4 with the second launch; in a graph 5.8 and 5.6).
constexpr int LN_CLUSTER = 8;

struct LnPlan {
  int T, NU, R, threads;  // threads a row, units a thread, rows a block, threads a block
  bool smem_acc;          // the backward's column sums in shared memory
};

// max_nu: units a thread may hold (the registers of its row, and in the backward of its columns' sums)
LnPlan ln_plan(int D, int max_nu, int max_t) {
  LnPlan p;
  const int units = (D + 7) / 8;
  p.smem_acc = false;
  if (units <= 16) {
    p.T = 1;
    while (p.T < units) p.T *= 2;
    p.NU = 1;
  } else {
    p.T = 32 * ((units + 32 * max_nu - 1) / (32 * max_nu));
    p.NU = (units + p.T - 1) / p.T;
    if (p.T > max_t) {
      p.T = max_t;
      p.NU = 4;  // 4 units x 512 threads hold the widest row
      p.smem_acc = true;
    }
  }
  p.R = std::max(1, 256 / p.T);
  p.threads = p.R * p.T;
  return p;
}
// Forward: one warp a row up to 1024 columns, then four units a thread: the fewer threads share a row, the more rows
// are on their way at once (4000 bf16 rows of 12288: 58 us with four units, 94 with two; 16384 of 4096: 62 and 73).
// Without the wide accesses two (fp32) or, from 257 columns up, one (bf16: the number of 2-byte accesses in flight bounds
// those; 30000 rows of 1283: 79 us, 116 with two).
LnPlan ln_fwd_plan(int D, bool vec, bool bf16_x) {
  if (!vec && bf16_x && D > 256) return ln_plan(D, D <= 8192 ? 1 : 2, 1024);
  return ln_plan(D, vec || D <= 1024 ? 4 : 2, 1024);
}
// Backward: 16 sums and, per unit, 4 (bf16) or 8 (fp32) registers of x and of dy have to fit beside the rest in the 128
// registers of 512 threads an SM. One warp a row up to 768 columns (three units a thread); then two units while 512
// threads hold the row so (the next row's registers fit beside it: 16384 bf16 rows of 4096 in 81 us; three units 94),
// then three (which do not quite fit: 36 to 144 bytes of spills a thread with the wide accesses, 120 to 248 without). What
// is wider than 12288 keeps its columns' sums in shared memory.
LnPlan ln_bwd_plan(int D) { return D <= 768 ? ln_plan(D, 3, 32) : ln_plan(D, D <= 8192 ? 2 : 3, 512); }

int ln_bwd_blocks(int M, const LnPlan& p, int per_sm) {
  return std::min((M - 1) / p.R + 1, LN_SMS * std::min(per_sm, LN_BWD_PER_SM));
}
size_t ln_bwd_workspace(int M, int D) {
  const LnPlan p = ln_bwd_plan(D);
  const int blocks = ln_bwd_blocks(M, p, LN_BWD_PER_SM);
  return blocks > LN_CLUSTER ? (size_t)blocks * 2 * p.NU * 8 * p.T * sizeof(float) : 0;
}

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
  float* partial;  // [blocks][2][slots] where more blocks sum than form a cluster
  int M, D, T;
  int cluster;     // the blocks are one cluster
  float eps, inv_d;
};

// Column of element k of unit u of this thread. STEP: 0 with VEC; else the
// distance of a thread's columns, 32, or T where T is below 32 (STEP 1).
enum { VEC8 = 0, STEP_T = 1, STEP_32 = 2 };
template <int STEP>
SVLA_DEV int column(int u, int k, int T, int tid) {
  if constexpr (STEP == VEC8) return (u * T + tid) * 8 + k;
  if constexpr (STEP == STEP_T) return k * T + tid;
  return (u * T + (tid & ~31)) * 8 + k * 32 + (tid & 31);
}

// One row's elements of this thread (or the weights of its columns) as they lie in
// memory, from unit u0 on, zeros past the width.
template <typename E, int NU, int STEP>
struct RowRegs;
template <int NU>
struct RowRegs<float, NU, VEC8> {
  float4 q[2 * NU];
  SVLA_DEV void load(const float* p, int D, int T, int tid, int u0 = 0) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int c = ((u0 + u) * T + tid) * 8;
      q[2 * u] = q[2 * u + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < D) {
        q[2 * u] = *reinterpret_cast<const float4*>(p + c);
        q[2 * u + 1] = *reinterpret_cast<const float4*>(p + c + 4);
      }
    }
  }
  // elements 2 j and 2 j + 1 of unit u
  SVLA_DEV f32x2 get2(int u, int j) const {
    const float4& f = q[2 * u + (j >> 1)];
    return j & 1 ? pair(f.z, f.w) : pair(f.x, f.y);
  }
};
template <int NU>
struct RowRegs<uint16_t, NU, VEC8> {
  uint4 q[NU];
  SVLA_DEV void load(const uint16_t* p, int D, int T, int tid, int u0 = 0) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int c = ((u0 + u) * T + tid) * 8;
      q[u] = make_uint4(0u, 0u, 0u, 0u);
      if (c < D) q[u] = *reinterpret_cast<const uint4*>(p + c);
    }
  }
  SVLA_DEV f32x2 get2(int u, int j) const {
    const uint32_t w = j == 0 ? q[u].x : j == 1 ? q[u].y : j == 2 ? q[u].z : q[u].w;
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <typename E, int NU, int STEP>
struct RowRegs {
  E q[NU * 8];
  SVLA_DEV void load(const E* p, int D, int T, int tid, int u0 = 0) {
    const int step = STEP == STEP_T ? T : 32;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int c = column<STEP>(u0 + u, 0, T, tid);
#pragma unroll
      for (int k = 0; k < 8; ++k) q[u * 8 + k] = c + k * step < D ? p[c + k * step] : E(0);
    }
  }
  SVLA_DEV f32x2 get2(int u, int j) const { return pair(load1(&q[u * 8 + 2 * j]), load1(&q[u * 8 + 2 * j + 1])); }
};

template <typename E, int STEP>
SVLA_DEV void store_unit(E* p, int u, int D, int T, int tid, const float (&x)[8]) {
  const int c = column<STEP>(u, 0, T, tid);
  if constexpr (STEP == VEC8) {
    if (c < D) store8(p + c, x);
  } else {
    const int step = STEP == STEP_T ? T : 32;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k * step < D) store1(p + c + k * step, x[k]);
  }
}

// Ask for the cache lines of a row's D elements to be in L2, by its T threads.
template <typename E>
SVLA_DEV void prefetch_row(const E* p, int D, int T, int tid) {
  for (int at = tid * 128; at < D * (int)sizeof(E); at += T * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(p) + at) : "memory");
}

// Sums over the T threads of a row: a butterfly of the warp or of its part, then
// (T > 32) one of the warps' sums, which every warp reads from shared memory.
// red: one float2 a warp of the block.
SVLA_DEV void row_sums(float& s0, float& s1, int T, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < T) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
  if (T <= 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = T >> 5, first = warp / per * per;
  if (lane == 0) red[warp] = make_float2(s0, s1);
  __syncthreads();
  const float2 v = lane < per ? red[first + lane] : make_float2(0.f, 0.f);
  s0 = v.x;
  s1 = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < per) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
  s0 = __shfl_sync(0xffffffffu, s0, 0);
  s1 = __shfl_sync(0xffffffffu, s1, 0);
}

// Mean and sum of squared differences of two sets of values from theirs (Chan,
// Golub and LeVeque 1979): no cancellation of large sums, in one pass.
struct Moments {
  float n, mean, m2;
  SVLA_DEV void merge(const Moments& o) {
    const float all = n + o.n, part = all > 0.f ? __fdividef(o.n, all) : 0.f, d = o.mean - mean;
    mean = fmaf(d, part, mean);
    m2 = m2 + o.m2 + d * (d * (n * part));  // n part first: 0 with an empty set, however large the other's mean
    n = all;
  }
  SVLA_DEV void merge_lanes(int from, int below) {  // butterfly over distances from .. 1 that are below `below`
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o <= from && o < below) {
        Moments x;
        x.n = __shfl_xor_sync(0xffffffffu, n, o);
        x.mean = __shfl_xor_sync(0xffffffffu, mean, o);
        x.m2 = __shfl_xor_sync(0xffffffffu, m2, o);
        merge(x);
      }
  }
};

// ---------------------------------------------------------------------------
// forward: one row a group of T threads. A row of one warp or a part of one:
// mean first, then the squares of the differences from registers. Of several
// warps: each warp so for its columns, then the warps' moments merged, for one
// barrier a row.
// ---------------------------------------------------------------------------
template <typename TX, typename TY, typename TW, int NU, int STEP>
__global__ void __launch_bounds__(NU <= 2 ? 1024 : 512) layernorm_kernel(const LnArgs a) {
  __shared__ Moments red[32];
  // no early launch of dependents: y may be a weight of what follows, and kernels fetch weights before their wait
  griddep_wait();  // nothing is read before: the weights may come from an optimiser step
  const int T = a.T, tid = threadIdx.x % T, D = a.D;
  const long long row = (long long)blockIdx.x * (blockDim.x / T) + threadIdx.x / T;
  const bool active = row < a.M;
  RowRegs<TX, NU, STEP> x;
  // the row's loads before the count of columns where they are narrow (30000 fp32 rows of 1283: 66 us, 69 behind it),
  // behind it where they are wide (16384 bf16 rows of 4096: 61 us, 69 before it)
  const TX* xp = reinterpret_cast<const TX*>(a.x) + (active ? row : 0) * a.ldx;
  if (STEP != VEC8) x.load(xp, D, T, tid);
  // columns of this thread's warp (or part of one): whole units of 256, the last one cut
  const int width = min(T, 32);
  float cnt = (float)D, inv_cnt = a.inv_d;
  if (T > 32) {
    int mine = 0;
#pragma unroll
    for (int u = 0; u < NU; ++u) mine += max(0, min(256, D - (u * T + (tid & ~31)) * 8));
    cnt = (float)mine;
    inv_cnt = mine ? 1.f / cnt : 0.f;
  }
  if (STEP == VEC8) x.load(xp, D, T, tid);
  f32x2 s2 = both(0.f);
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) s2 = add2(s2, x.get2(u, j));
  float s = halves(s2).x + halves(s2).y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < width) s += __shfl_xor_sync(0xffffffffu, s, o);
  float mean = s * inv_cnt;
  s2 = both(0.f);
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x2 d = add2(x.get2(u, j), both(-mean));
      if (STEP != VEC8) {
        const float2 h = halves(d);
        d = pair(column<STEP>(u, 2 * j, T, tid) < D ? h.x : 0.f, column<STEP>(u, 2 * j + 1, T, tid) < D ? h.y : 0.f);
      }
      if (STEP != VEC8 || column<STEP>(u, 0, T, tid) < D) s2 = fma2(d, d, s2);
    }
  float m2 = halves(s2).x + halves(s2).y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < width) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
  if (T > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = T >> 5, first = warp / per * per;
    if (lane == 0) red[warp] = Moments{cnt, mean, m2};
    __syncthreads();
    Moments all = lane < per ? red[first + lane] : Moments{0.f, 0.f, 0.f};
    all.merge_lanes(16, per);
    mean = __shfl_sync(0xffffffffu, all.mean, 0);
    m2 = __shfl_sync(0xffffffffu, all.m2, 0);
  }
  const float rstd = rsqrtf(m2 * a.inv_d + a.eps);
  if (!active) return;
  TY* y = reinterpret_cast<TY*>(a.out) + row * a.ldo;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    RowRegs<TW, 1, STEP> g, b;
    g.load(reinterpret_cast<const TW*>(a.gamma), D, T, tid, u);
    b.load(reinterpret_cast<const TW*>(a.beta ? a.beta : a.gamma), a.beta ? D : 0, T, tid, u);
    float o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 h = halves(fma2(mul2(add2(x.get2(u, j), both(-mean)), both(rstd)), g.get2(0, j), b.get2(0, j)));
      o[2 * j] = h.x;
      o[2 * j + 1] = h.y;
    }
    store_unit<TY, STEP>(y, u, D, T, tid, o);
  }
  if (tid == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// ---------------------------------------------------------------------------
// backward: each group of T threads walks rows blockIdx.x * R + group, + grid *
// R, .. and keeps its columns' sums of dgamma and dbeta; the next row is on its
// way while the current one is reduced. At the end the groups' sums are
// added in order and go to `partial`, or to dgamma and dbeta where there is one
// block or one cluster of blocks. Column sums are kept by slot, (u * 8 + k) * T + thread for element k
// of unit u, so that neighbouring threads have neighbouring words.
// ---------------------------------------------------------------------------
template <int STEP>
SVLA_DEV int slot_column(int slot, int T) {
  const int q = slot / T;
  return column<STEP>(q >> 3, q & 7, T, slot - q * T);
}

template <typename TX, typename TY, typename TW, int NU, int STEP, bool SMEM_ACC>
__global__ void __launch_bounds__(STEP == STEP_T ? 256 : 512)
    layernorm_bwd_kernel(const LnArgs a) {
  extern __shared__ __align__(16) float cols[];  // [R][2][slots] column sums (SMEM_ACC: [2][slots])
  __shared__ float2 red[2][16];
  // the next row in registers where that leaves two blocks an SM (16384 bf16 rows of 4096: 81 us, 90 without); else on
  // its way to L2 (16384 x 2048 fp32: 70 us, 77 without)
  constexpr int ROW = NU * 2 * (int)(sizeof(TX) + sizeof(TY));
  constexpr bool PREFETCH = STEP == VEC8 && !SMEM_ACC && 2 * ROW + 16 * NU <= 80;
  if (gridDim.x > 1 && !a.cluster && (a.dgamma || a.dbeta)) griddep_launch_dependents();  // layernorm_cols_kernel, which waits first
  griddep_wait();
  const int T = a.T, tid = threadIdx.x % T, D = a.D, R = blockDim.x / T, group = threadIdx.x / T;
  const int W = NU * 8 * T;  // slots
  const TX* xp = reinterpret_cast<const TX*>(a.x);
  const TY* dyp = reinterpret_cast<const TY*>(a.dy);
  f32x2 ag[SMEM_ACC ? 1 : NU * 4], ab[SMEM_ACC ? 1 : NU * 4];
  // the weights stay in registers where they take no more than 16
  constexpr bool KEEP = NU * 2 * sizeof(TW) <= 16;
  RowRegs<TW, KEEP ? NU : 1, STEP> g;
  if (KEEP) g.load(reinterpret_cast<const TW*>(a.gamma), D, T, tid);
  if constexpr (SMEM_ACC) {
    for (int c = threadIdx.x; c < 2 * W; c += blockDim.x) cols[c] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int j = 0; j < NU * 4; ++j) ag[j] = ab[j] = both(0.f);
  }
  const long long stride = (long long)gridDim.x * R;
  long long row0 = (long long)blockIdx.x * R;
  RowRegs<TX, NU, STEP> x;
  RowRegs<TY, NU, STEP> dy;
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](long long row, RowRegs<TX, NU, STEP>& fx, RowRegs<TY, NU, STEP>& fy, float& m, float& r) {
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
    RowRegs<TX, NU, STEP> nx;
    RowRegs<TY, NU, STEP> ndy;
    float nmean = 0.f, nrstd = 0.f;
    if (PREFETCH) {
      if (row0 + stride < a.M) fetch(row + stride, nx, ndy, nmean, nrstd);
    } else {
      fetch(row, x, dy, mean, rstd);
    }
    if (!PREFETCH && row + stride < a.M) {
      prefetch_row(xp + (row + stride) * a.ldx, D, T, tid);
      prefetch_row(dyp + (row + stride) * a.lddy, D, T, tid);
    }
    f32x2 w2 = both(0.f), x2 = both(0.f);  // sums of w and of w xh
    f32x2 xhs[NU * 4], ws[NU * 4];         // kept for dx (4000 bf16 rows of 12288: 75 us, 82 computed twice, which spills less)
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if (!KEEP) g.load(reinterpret_cast<const TW*>(a.gamma), D, T, tid, u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 d = dy.get2(u, j), xh = mul2(add2(x.get2(u, j), both(-mean)), both(rstd)), w = mul2(d, g.get2(KEEP ? u : 0, j));
        xhs[u * 4 + j] = xh;
        ws[u * 4 + j] = w;
        w2 = add2(w2, w);
        x2 = fma2(w, xh, x2);
        if constexpr (SMEM_ACC) {
          const float2 dh = halves(d), xx = halves(xh);
          float* c = cols + (u * 8 + 2 * j) * T + tid;
          c[0] = fmaf(dh.x, xx.x, c[0]);
          c[T] = fmaf(dh.y, xx.y, c[T]);
          c[W] += dh.x;
          c[W + T] += dh.y;
        } else {
          ag[u * 4 + j] = fma2(d, xh, ag[u * 4 + j]);
          ab[u * 4 + j] = add2(ab[u * 4 + j], d);
        }
      }
    }
    float s0 = halves(w2).x + halves(w2).y, s1 = halves(x2).x + halves(x2).y;
    row_sums(s0, s1, T, red[it & 1]);
    s0 *= a.inv_d;
    s1 *= a.inv_d;
    if (row < a.M) {
      TX* dx = reinterpret_cast<TX*>(a.out) + row * a.ldo;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 h = halves(mul2(add2(fma2(xhs[u * 4 + j], both(-s1), ws[u * 4 + j]), both(-s0)), both(rstd)));
          o[2 * j] = h.x;
          o[2 * j + 1] = h.y;
        }
        store_unit<TX, STEP>(dx, u, D, T, tid, o);
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
    for (int j = 0; j < NU * 4; ++j) {
      mine[2 * j * T] = halves(ag[j]).x;
      mine[(2 * j + 1) * T] = halves(ag[j]).y;
      mine[W + 2 * j * T] = halves(ab[j]).x;
      mine[W + (2 * j + 1) * T] = halves(ab[j]).y;
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * W; c += blockDim.x) {
    float v = cols[c];
    if constexpr (!SMEM_ACC)
      for (int r = 1; r < R; ++r) v += cols[(size_t)r * 2 * W + c];
    if (a.cluster) {
      cols[c] = v;
    } else if (gridDim.x > 1) {
      a.partial[(size_t)blockIdx.x * 2 * W + c] = v;
    } else {
      const int col = slot_column<STEP>(c < W ? c : c - W, T);
      float* out = c < W ? a.dgamma : a.dbeta;
      if (out && col < D) out[col] = v;
    }
  }
  if (a.cluster) {
    cluster_sync();
    const uint32_t own = smem_u32(cols);
    for (int c = (int)(blockIdx.x * blockDim.x + threadIdx.x); c < 2 * W; c += (int)(gridDim.x * blockDim.x)) {
      float v = 0.f;
      for (uint32_t b = 0; b < gridDim.x; ++b) v += ld_dsmem_f(dsmem_addr(own + c * 4, b));
      const int col = slot_column<STEP>(c < W ? c : c - W, T);
      float* out = c < W ? a.dgamma : a.dbeta;
      if (out && col < D) out[col] = v;
    }
    cluster_sync();  // no block ends while another reads its sums
  }
}

// dgamma and dbeta: the blocks' partial sums added per slot. A block of 32
// slots; thread row j adds the blocks j, j + 32, .. and the 32 sums are added in
// order.
template <int STEP>
__global__ void __launch_bounds__(1024) layernorm_cols_kernel(const float* partial, int blocks, int D, int W, int T,
                                                              float* dgamma, float* dbeta) {
  __shared__ float part[32][33];
  griddep_wait();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < 2 * W) {
#pragma unroll 10
    for (int b = threadIdx.y; b < blocks; b += 32) s += partial[(size_t)b * 2 * W + c];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < 2 * W) {
    s = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) s += part[j][threadIdx.x];
    const int col = slot_column<STEP>(c < W ? c : c - W, T);
    float* out = c < W ? dgamma : dbeta;
    if (out && col < D) out[col] = s;
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
typedef void (*LnFn)(const LnArgs);

template <typename TX, typename TY, typename TW, int STEP>
LnFn pick_fwd(int NU) {
  if constexpr (STEP == STEP_T) {
    return layernorm_kernel<TX, TY, TW, 1, STEP>;
  } else {
    switch (NU) {
      case 1: return layernorm_kernel<TX, TY, TW, 1, STEP>;
      case 2: return layernorm_kernel<TX, TY, TW, 2, STEP>;
      case 3: return layernorm_kernel<TX, TY, TW, 3, STEP>;
      default: return layernorm_kernel<TX, TY, TW, 4, STEP>;
    }
  }
}
template <typename TX, typename TY, typename TW, int STEP>
LnFn pick_bwd(int NU, bool smem) {
  if constexpr (STEP == STEP_T) {
    return layernorm_bwd_kernel<TX, TY, TW, 1, STEP, false>;
  } else {
    if (smem) return layernorm_bwd_kernel<TX, TY, TW, 4, STEP, true>;
    switch (NU) {
      case 1: return layernorm_bwd_kernel<TX, TY, TW, 1, STEP, false>;
      case 2: return layernorm_bwd_kernel<TX, TY, TW, 2, STEP, false>;
      default: return layernorm_bwd_kernel<TX, TY, TW, 3, STEP, false>;
    }
  }
}
template <typename TX, typename TY, typename TW>
LnFn pick_v(bool bwd, int step, const LnPlan& p) {
  if (step == VEC8) return bwd ? pick_bwd<TX, TY, TW, VEC8>(p.NU, p.smem_acc) : pick_fwd<TX, TY, TW, VEC8>(p.NU);
  if (step == STEP_T) return bwd ? pick_bwd<TX, TY, TW, STEP_T>(p.NU, false) : pick_fwd<TX, TY, TW, STEP_T>(p.NU);
  return bwd ? pick_bwd<TX, TY, TW, STEP_32>(p.NU, p.smem_acc) : pick_fwd<TX, TY, TW, STEP_32>(p.NU);
}
LnFn pick(int xt, int yt, int wt, bool bwd, int step, const LnPlan& p) {
  typedef uint16_t h;
  const int k = (xt == SVLA_TYPE_BF16 ? 4 : 0) | (yt == SVLA_TYPE_BF16 ? 2 : 0) | (wt == SVLA_TYPE_BF16 ? 1 : 0);
  switch (k) {
    case 0: return pick_v<float, float, float>(bwd, step, p);
    case 1: return pick_v<float, float, h>(bwd, step, p);
    case 2: return pick_v<float, h, float>(bwd, step, p);
    case 3: return pick_v<float, h, h>(bwd, step, p);
    case 4: return pick_v<h, float, float>(bwd, step, p);
    case 5: return pick_v<h, float, h>(bwd, step, p);
    case 6: return pick_v<h, h, float>(bwd, step, p);
    default: return pick_v<h, h, h>(bwd, step, p);
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, bool cluster, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = grid.x;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
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
// rows of one pitch that lie between each other's rows, as the halves of a wider matrix do
bool between(const Mat& a, const Mat& b, int D) {
  const size_t pitch = a.ld * bytes_of(a.type);
  if (pitch != b.ld * bytes_of(b.type)) return false;
  const size_t from = a.begin() <= b.begin() ? (b.begin() - a.begin()) % pitch : (pitch - (a.begin() - b.begin()) % pitch) % pitch;
  return from >= D * bytes_of(a.type) && from + D * bytes_of(b.type) <= pitch;
}
// an output may be an input matrix itself (each row is read before it is written), not a part of it
bool clash(const Mat& out, const Mat& in, int M, int D) {
  return !out.same(in) && overlap(out.begin(), out.end(M, D), in.begin(), in.end(M, D)) && !between(out, in, D);
}
bool clash(const Mat& out, const void* v, size_t bytes, int M, int D) {
  return v && overlap(out.begin(), out.end(M, D), (uintptr_t)v, (uintptr_t)v + bytes);
}

// Blocks of a kernel that an SM holds, asked for once a kernel: the backward's rows are walked by what is resident.
cudaError_t resident_per_sm(LnFn fn, int slot, int threads, size_t smem, int* blocks) {
  static std::atomic<int> known[8 * 3 * 17 * 4];  // by types, way of access, threads a row and units a thread
  if ((*blocks = known[slot].load()) != 0) return cudaSuccess;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, fn, threads, smem);
  if (e != cudaSuccess) return e;
  if (*blocks < 1) return cudaErrorInvalidConfiguration;
  known[slot].store(*blocks);
  return cudaSuccess;
}

// Shared memory that the backward's kernel of NU units may take: the column sums of rows on 512 threads (more, narrower
// rows a block take less). The limit is set once a kernel and device, to this: set to each call's own size, a call of
// another thread could lower it before the launch.
constexpr int ln_bwd_smem_max(int NU) { return 2 * NU * 8 * 512 * (int)sizeof(float); }
cudaError_t allow_bwd_smem(LnFn fn, int slot, int NU) {
  static std::atomic<bool> done[8 * 3 * 17 * 4][64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[slot][dev].load())) return e;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, ln_bwd_smem_max(NU));
  if (e == cudaSuccess && dev < 64) done[slot][dev].store(true);
  return e;
}

svla_status run(LnArgs& a, int xt, int yt, int wt, bool bwd, bool vec, cudaStream_t s) {
  const LnPlan p = bwd ? ln_bwd_plan(a.D) : ln_fwd_plan(a.D, vec, xt == SVLA_TYPE_BF16);
  a.T = p.T;
  a.inv_d = (float)(1.0 / a.D);
  const int step = vec ? VEC8 : p.T < 32 ? STEP_T : STEP_32;
  const LnFn fn = pick(xt, yt, wt, bwd, step, p);
  const int W = p.NU * 8 * p.T;
  const size_t full = bwd ? (size_t)(p.smem_acc ? 1 : p.R) * 2 * W * sizeof(float) : 0;
  const size_t smem = p.smem_acc || a.dgamma || a.dbeta ? full : 0;
  int blocks = (a.M - 1) / p.R + 1;
  cudaError_t e = cudaSuccess;
  const int kind = (xt == SVLA_TYPE_BF16 ? 4 : 0) | (yt == SVLA_TYPE_BF16 ? 2 : 0) | (wt == SVLA_TYPE_BF16 ? 1 : 0);
  const int slot = ((kind * 3 + step) * 17 + p.T / 32) * 4 + p.NU - 1;
  if (full > 40 * 1024) e = allow_bwd_smem(fn, slot, p.NU);
  if (e == cudaSuccess && bwd && blocks > 1) {
    int per_sm = 0;
    e = resident_per_sm(fn, slot, p.threads, full, &per_sm);
    if (e == cudaSuccess) blocks = ln_bwd_blocks(a.M, p, per_sm);
  }
  a.cluster = bwd && blocks > 1 && blocks <= LN_CLUSTER && (a.dgamma || a.dbeta);
  if (e == cudaSuccess) e = launch(fn, dim3(blocks), dim3(p.threads), smem, a.cluster != 0, s, a);
  if (e == cudaSuccess && bwd && blocks > 1 && !a.cluster && (a.dgamma || a.dbeta))
    e = launch(step == VEC8 ? layernorm_cols_kernel<VEC8> : step == STEP_T ? layernorm_cols_kernel<STEP_T> : layernorm_cols_kernel<STEP_32>,
               dim3((2 * W + 31) / 32), dim3(32, 32), 0, false, s, (const float*)a.partial, blocks, a.D, W, p.T, a.dgamma, a.dbeta);
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
  return svla::ln_bwd_workspace(M, D);
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
