// Layer norm with the residual add in front of it, forward and backward.
//
//   forward   r = round(x + res), mean and variance of r over its D columns,
//             y = (r - mean) rstd gamma + beta
//   backward  xh = (r - mean) rstd, a = dy gamma,
//             dx = rstd (a - avg(a) - xh avg(a xh)) + dres,
//             dgamma = sum_rows dy xh, dbeta = sum_rows dy
//
// Both directions are bound by HBM: each row is read once, held in registers
// (or in the thread's own shared-memory slots) between its statistics and its
// output, and written once.  The variance is taken in a second pass over the
// registers, sum (r - mean)^2, which costs no memory and loses nothing to an
// offset of the row.  32768 x 2816 bf16 with a residual (738 MB each way) takes
// 110 us forward and 117 us backward, 0.99 and 0.93 of a copy's rate; a few
// rows are bound by the launch and two sums' latency (1 x 7168: 2.9 us).
//
// Rows of whole, aligned 16-byte vectors move in such vectors.  Rows that
// start inside a 16-byte unit, or end inside one (odd widths), do so too where
// all arrays of the call lie alike (SHIFT): every 8th row (fp32: every 4th)
// starts at the same place of its unit, so a block that walks rows by a
// multiple of 8 keeps its threads' vectors at fixed columns, shifted by that
// place, and only a row's first and last vector need care.  Rows that lie
// unlike each other move element by element, which takes two to three times
// as long (32768 x 1407 bf16: 138 us forward and 256 backward, against 86
// and 84).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "layer.h"
#include "layer_common.cuh"

namespace moe {
namespace {

template <typename T>
struct NormArgs {
  const T *x, *res, *rin;
  const void *gamma, *beta;
  T *r, *y;
  float *mean, *rstd;
  float* partials;
  void *dgamma, *dbeta;  // backward by one block
  int64_t ldx, ldres, ldr, ldy, rows;
  float eps, inv_d;
  int D, nvec;
};

// Sum over the TPR threads of a row: within the warp, then (rows wider than
// one warp own the whole block) over the warps' sums in shared memory.
// `slot` alternates so that one barrier per sum is enough.
template <bool ONE_WARP, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N], int nwarps) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (!ONE_WARP) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[warp][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float p = (threadIdx.x & 31) < nwarps ? red[threadIdx.x & 31][i] : 0.0f;
      v[i] = warp_sum(p);
    }
  }
}

constexpr int kMaxThreads = 512;  // threads of a row at most: 128 registers each
constexpr int kMaxD = 8192;
constexpr int kRowsPerBlock = 4;  // rows of one warp each

// One row per block of blockDim.x threads, or (ONE_WARP) one row per warp.
template <typename T, typename W, int VEC, int NV, bool ONE_WARP>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const NormArgs<T> p) {
  __shared__ float red[2][32][1];
  const int tpr = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = ONE_WARP
                          ? static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5)
                          : static_cast<int64_t>(blockIdx.x);
  if (ONE_WARP && row >= p.rows) return;
  const int nwarps = blockDim.x >> 5;
  const W* gamma = static_cast<const W*>(p.gamma);
  const W* beta = static_cast<const W*>(p.beta);
  const T* x = p.x + row * p.ldx;
  Raw<T, VEC> a[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * tpr + t;
    if (c < p.nvec) a[i].load(x, c);
  }
  if (p.res != nullptr) {
    const T* res = p.res + row * p.ldres;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + t;
      if (c < p.nvec) b[i].load(res, c);
    }
    T* r = p.r + row * p.ldr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + t;
      if (c < p.nvec) {
        float f[VEC], g[VEC];
        a[i].unpack(f);
        b[i].unpack(g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] += g[j];
        a[i].pack(f);  // the stored row is what is normalised
        a[i].store(r, c);
      }
    }
  }
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * tpr + t < p.nvec) {
      float f[VEC];
      a[i].unpack(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum[0] += f[j];
    }
  }
  row_sums<ONE_WARP, 1>(sum, red[0], nwarps);
  const float mean = sum[0] * p.inv_d;
  float sq[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * tpr + t < p.nvec) {
      float f[VEC];
      a[i].unpack(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sq[0] += (f[j] - mean) * (f[j] - mean);
    }
  }
  row_sums<ONE_WARP, 1>(sq, red[1], nwarps);
  const float rstd = 1.0f / sqrtf(sq[0] * p.inv_d + p.eps);
  if (t == 0 && p.mean != nullptr) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  T* y = p.y + row * p.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * tpr + t;
    if (c < p.nvec) {
      float f[VEC], g[VEC], h[VEC];
      a[i].unpack(f);
      load_weights<W, VEC>(gamma, c, g);
      load_weights<W, VEC>(beta, c, h);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = (f[j] - mean) * rstd * g[j] + h[j];
      a[i].pack(f);
      a[i].store(y, c);
    }
  }
}

// ------------------------------------------------------------ shifted rows
// Vector c of a row that starts `e` elements into its first 16-byte unit: its
// elements [lo, hi) are the row's.
template <int VEC>
struct Edge {
  int lo, hi;
  __device__ __forceinline__ Edge(int c, int e, int D) : lo(c == 0 ? e : 0), hi(min(VEC, e + D - c * VEC)) {}
  __device__ __forceinline__ bool whole() const { return lo == 0 && hi == VEC; }
};
template <typename T>
__device__ __forceinline__ int unit_offset(const T* row) {  // in elements
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / static_cast<int>(sizeof(T));
}
// The vector's 16-byte unit up to the row's end, zeros behind.  Ahead of the
// row's start it reads the rest of the unit, which is the same allocation's
// (allocations start at such units), whatever it holds.
template <typename T, int VEC>
__device__ __forceinline__ void copy_unit(void* slot, const T* unit, const Edge<VEC>& g) {
  cp_async16_zfill(slot, unit, g.hi * static_cast<int>(sizeof(T)));
}
template <typename T, int VEC>
__device__ __forceinline__ void store_part(const float (&f)[VEC], T* unit, const Edge<VEC>& g) {
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (j >= g.lo && j < g.hi) unit[j] = from_f32<T>(f[j]);
}
template <typename W, int VEC>
__device__ __forceinline__ void load_shifted_weights(const W* w, int c, int e, int D, float (&f)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int col = c * VEC + j - e;
    f[j] = col >= 0 && col < D ? to_f32<W>(__ldg(w + col)) : 0.0f;
  }
}

// The forward of shifted rows: as norm_fwd_kernel, but a group of threads
// walks rows, whose copies come `steps` - 1 ahead into the threads' own slots
// (as in the backward below), and keeps the weights of its columns.
template <typename T, typename W, int VEC, int NV, bool ONE_WARP>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_fwd_shift_kernel(const NormArgs<T> p, const int steps) {
  using Q = Raw<T, VEC>;
  __shared__ float red[2][32][1];
  extern __shared__ __align__(16) unsigned char stage_mem[];
  const int tpr = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int groups = ONE_WARP ? (blockDim.x >> 5) : 1;
  const int nwarps = blockDim.x >> 5, bd = blockDim.x;
  const bool has_res = p.res != nullptr;
  const int stage_slots = (has_res ? 2 : 1) * NV * bd;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + (ONE_WARP ? (threadIdx.x >> 5) : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int n = first < p.rows ? static_cast<int>((p.rows - 1 - first) / step) + 1 : 0;
  const int e = unit_offset(p.x + first * p.ldx), nvec = (e + p.D + VEC - 1) / VEC;
  typename Q::Store* const slots = reinterpret_cast<typename Q::Store*>(stage_mem) + threadIdx.x;
  const T* x_at = p.x + first * p.ldx - e;
  const T* s_at = has_res ? p.res + first * p.ldres - e : nullptr;
  T* y_at = p.y + first * p.ldy - e;
  T* r_at = has_res ? p.r + first * p.ldr - e : nullptr;
  int fetched = 0;
  auto fetch = [&](int stage) {
    if (fetched < n) {
      typename Q::Store* to = slots + stage * stage_slots;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * tpr + t;
        if (c < nvec) {
          const Edge<VEC> g(c, e, p.D);
          copy_unit(to + i * bd, x_at + c * VEC, g);
          if (has_res) copy_unit(to + (NV + i) * bd, s_at + c * VEC, g);
        }
      }
      x_at += step * p.ldx;
      if (has_res) s_at += step * p.ldres;
    }
    ++fetched;
    cp_async_commit();
  };
  for (int q = 0; q < steps - 1; ++q) fetch(q);
  float gm[NV][VEC], bt[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_shifted_weights(static_cast<const W*>(p.gamma), i * tpr + t, e, p.D, gm[i]);
    load_shifted_weights(static_cast<const W*>(p.beta), i * tpr + t, e, p.D, bt[i]);
  }
  int stage = 0;
  for (int k = 0; k < n; ++k) {
    fetch(stage == 0 ? steps - 1 : stage - 1);
    if (steps == 3) cp_async_wait_group<2>();
    else cp_async_wait_group<1>();
    const typename Q::Store* from = slots + stage * stage_slots;
    float f[NV][VEC], sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + t;
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i][j] = 0.0f;
      if (c < nvec) {
        const Edge<VEC> g(c, e, p.D);
        Q a;
        a.v = from[i * bd];
        a.unpack(f[i]);
        if (has_res) {
          float h[VEC];
          a.v = from[(NV + i) * bd];
          a.unpack(h);
#pragma unroll
          for (int j = 0; j < VEC; ++j) f[i][j] += h[j];
          if (g.whole()) {
            a.pack(f[i]);
            a.store(r_at + c * VEC, 0);
            a.unpack(f[i]);  // the stored row is what is normalised
          } else {
            store_part<T, VEC>(f[i], r_at + c * VEC, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[i][j] = to_f32<T>(from_f32<T>(f[i][j]));
          }
        }
        if (!g.whole()) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (j < g.lo || j >= g.hi) f[i][j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[0] += f[i][j];
      }
    }
    row_sums<ONE_WARP, 1>(sum, red[0], nwarps);
    const float mean = sum[0] * p.inv_d;
    float sq[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + t;
      if (c < nvec) {
        const Edge<VEC> g(c, e, p.D);
        if (!g.whole()) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (j < g.lo || j >= g.hi) f[i][j] = mean;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) sq[0] += (f[i][j] - mean) * (f[i][j] - mean);
      }
    }
    row_sums<ONE_WARP, 1>(sq, red[1], nwarps);
    const float rstd = 1.0f / sqrtf(sq[0] * p.inv_d + p.eps);
    if (t == 0 && p.mean != nullptr) {
      p.mean[first + k * step] = mean;
      p.rstd[first + k * step] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + t;
      if (c < nvec) {
        const Edge<VEC> g(c, e, p.D);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[i][j] = (f[i][j] - mean) * rstd * gm[i][j] + bt[i][j];
        if (g.whole()) {
          Q a;
          a.pack(f[i]);
          a.store(y_at + c * VEC, 0);
        } else {
          store_part<T, VEC>(f[i], y_at + c * VEC, g);
        }
      }
    }
    y_at += step * p.ldy;
    if (has_res) r_at += step * p.ldr;
    if (++stage == steps) stage = 0;
  }
  cp_async_wait_all();
}

// ---------------------------------------------------------------- backward
// A block takes R rows at a time (R = 2 where they fit) so that their two sums
// each share one pass through the warps and one barrier: with one row at a
// time the chain from a row's load to its store, not HBM, set the rate
// (32768 x 2816 bf16: 141 us).  Each thread copies its own vectors of a row
// into its own shared-memory slots with cp.async, one or two steps ahead, and
// reads back only what it copied: the copies need no barrier, and the bytes
// in flight do not depend on registers.  A block walks rows with the grid's
// stride and keeps its columns' weight-gradient sums in registers; at the end
// they become one row of `partials` ([blocks][2][D]: dgamma, dbeta).
constexpr int64_t kOneBlockRows = 8;
constexpr int kBwdGroups = 4;  // ONE_WARP: warps of a block, each on rows of its own

template <typename T, int VEC>
__device__ __forceinline__ void copy_async(void* dst, const T* src) {
  if constexpr (VEC * sizeof(T) == 16) {
    cp_async16(dst, src);
  } else if constexpr (sizeof(T) == 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
  } else {
    *static_cast<T*>(dst) = *src;  // two bytes: below cp.async's smallest copy
  }
}

// Sums of N = 2 or 4 values over the threads of a row group.  Within a warp
// the lanes first halve the values they carry (16, then 8 lanes to a value),
// so that four values cost 6 exchanges instead of 20; across warps through
// `red`, which the caller alternates, so that one barrier is enough.
template <bool ONE_WARP, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float (*red)[4], int nwarps) {
  static_assert(N == 2 || N == 4, "two sums for each of one or two rows");
  constexpr int kLanes = 32 / N;  // lanes that end up with one value
  const int lane = threadIdx.x & 31;
  float c;
  if constexpr (N == 4) {
    const bool hi = lane & 16, h8 = lane & 8;
    float a0 = hi ? v[2] : v[0], a1 = hi ? v[3] : v[1];
    a0 += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
    a1 += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
    c = h8 ? a1 : a0;
    c += __shfl_xor_sync(0xffffffffu, h8 ? a0 : a1, 8);
  } else {
    const bool hi = lane & 16;
    c = hi ? v[1] : v[0];
    c += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 16);
    c += __shfl_xor_sync(0xffffffffu, c, 8);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  const int which = lane / kLanes, part = lane % kLanes;
  if constexpr (!ONE_WARP) {
    if (part == 0) red[threadIdx.x >> 5][which] = c;
    __syncthreads();
    c = 0.0f;
    for (int w = part; w < nwarps; w += kLanes) c += red[w][which];
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, c, i * kLanes);
}

// Slots of a thread; slot u of all threads lies together, so that a warp's
// copy fills whole lines (with each thread's slots together instead, the same
// copies took 192 us where these took 130).
template <int NV, bool RES, int R>
__host__ __device__ constexpr int bwd_slots(int steps) { return steps * R * (RES ? 3 : 2) * NV; }

template <typename T, typename W, int VEC, int NV, bool ONE_WARP, bool RES, int R, bool SHIFT>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_bwd_kernel(const NormArgs<T> p, const int steps) {
  using Q = Raw<T, VEC>;
  using N = Nums<VEC>;
  using F = typename N::F;
  constexpr int kArr = RES ? 3 : 2, kN = N::kN, kPerStep = R * kArr * NV;
  __shared__ float red[2][kMaxThreads / 32][4];
  extern __shared__ __align__(16) unsigned char stage_mem[];
  const int tpr = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int groups = ONE_WARP ? (blockDim.x >> 5) : 1;
  const int group = ONE_WARP ? (threadIdx.x >> 5) : 0;
  const int nwarps = blockDim.x >> 5;
  const int bd = blockDim.x;
  typename Q::Store* const slots = reinterpret_cast<typename Q::Store*>(stage_mem) + threadIdx.x;
  // this group's rows: first, first + step, ... (n of them)
  const int first = blockIdx.x * groups + group, step = gridDim.x * groups;
  const int n = first < p.rows ? static_cast<int>((p.rows - 1 - first) / step) + 1 : 0;
  const int64_t sx = step * p.ldx, sr = step * p.ldr, ss = step * p.ldres, sy = step * p.ldy;
  const int e = SHIFT ? unit_offset(p.x + first * p.ldx) : 0;
  const int nvec = SHIFT ? (e + p.D + VEC - 1) / VEC : p.nvec;
  const T* dy_at = p.x + first * p.ldx - e + t * VEC;  // of the next row to fetch
  const T* r_at = p.rin + first * p.ldr - e + t * VEC;
  const T* s_at = RES ? p.res + first * p.ldres - e + t * VEC : nullptr;
  T* y_at = p.y + first * p.ldy - e + t * VEC;
  int fetched = 0;
  auto fetch = [&](int stage) {
    typename Q::Store* to = slots + stage * kPerStep * bd;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (fetched + r < n) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i * tpr + t < nvec) {
            const auto copy = [&](int q, const T* at) {
              auto* slot = to + ((r * kArr + q) * NV + i) * bd;
              if constexpr (SHIFT) copy_unit(slot, at, Edge<VEC>(i * tpr + t, e, p.D));
              else copy_async<T, VEC>(slot, at);
            };
            copy(0, dy_at + i * tpr * VEC);
            copy(1, r_at + i * tpr * VEC);
            if constexpr (RES) copy(2, s_at + i * tpr * VEC);
          }
        }
      }
      dy_at += sx;
      r_at += sr;
      if constexpr (RES) s_at += ss;
    }
    fetched += R;
    cp_async_commit();
  };
  for (int q = 0; q < steps - 1; ++q) fetch(q);

  const W* gamma = static_cast<const W*>(p.gamma);
  F g[NV][kN], dg[NV][kN], db[NV][kN];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = 0.0f;
    if constexpr (SHIFT) load_shifted_weights(gamma, i * tpr + t, e, p.D, w);
    else if (i * tpr + t < nvec) load_weights<W, VEC>(gamma, i * tpr + t, w);
    N::gather(w, g[i]);
#pragma unroll
    for (int j = 0; j < kN; ++j) dg[i][j] = db[i][j] = N::splat(0.0f);
  }
  // The rows' statistics: every 32 rows a lane reads those of one of them.
  // (Read one step ahead by every thread, they were waited for in that step
  // all the same: 8192 x 5632 bf16 took 111 us so, and takes 71.)
  const int lane = threadIdx.x & 31;
  float lane_mean = 0.0f, lane_rstd = 0.0f;
  int stage = 0, par = 0;
  for (int k = 0; k < n; k += R) {
    fetch(stage == 0 ? steps - 1 : stage - 1);
    if ((k & 31) == 0 && k + lane < n) {
      const int64_t at = first + static_cast<int64_t>(k + lane) * step;
      lane_mean = __ldg(p.mean + at);
      lane_rstd = __ldg(p.rstd + at);
    }
    float rstd[R];
    F away[R];  // minus the mean
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = __shfl_sync(0xffffffffu, lane_rstd, (k + r) & 31);
      away[r] = N::splat(-__shfl_sync(0xffffffffu, lane_mean, (k + r) & 31));
    }
    if (steps == 3) cp_async_wait_group<2>();
    else cp_async_wait_group<1>();
    const typename Q::Store* from = slots + stage * kPerStep * bd;
    Q raw[R][kArr][NV];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int q = 0; q < kArr; ++q)
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[r][q][i].v = from[((r * kArr + q) * NV + i) * bd];
    F a[R][NV][kN], xh[R][NV][kN];
    float sums[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      F s1 = N::splat(0.0f), s2 = s1;
      const F rs = N::splat(rstd[r]);
      if (r == 0 || k + r < n) {  // past the last row the slots hold nothing
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i * tpr + t < nvec) {
            float f[VEC];
            if constexpr (SHIFT) {  // ahead of the row's start the unit may hold anything
              if (i == 0 && t == 0 && e > 0) {
                raw[r][0][i].clear_below(e);
                raw[r][1][i].clear_below(e);
              }
            }
            raw[r][0][i].unpack(f);
            N::gather(f, a[r][i]);
            raw[r][1][i].unpack(f);
            N::gather(f, xh[r][i]);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              const F dy = a[r][i][j];
              xh[r][i][j] = fmul(fadd(xh[r][i][j], away[r]), rs);
              dg[i][j] = ffma(dy, xh[r][i][j], dg[i][j]);
              db[i][j] = fadd(db[i][j], dy);
              a[r][i][j] = fmul(dy, g[i][j]);
              s1 = fadd(s1, a[r][i][j]);
              s2 = ffma(a[r][i][j], xh[r][i][j], s2);
            }
          }
        }
      }
      sums[2 * r] = fold(s1);
      sums[2 * r + 1] = fold(s2);
    }
    group_sums<ONE_WARP, 2 * R>(sums, red[par], nwarps);
    par ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r == 0 || k + r < n) {
        // dx = rstd a - (rstd m1 + xh rstd m2) + dres
        const F rs = N::splat(rstd[r]), c1 = N::splat(-rstd[r] * (sums[2 * r] * p.inv_d)),
                c2 = N::splat(-rstd[r] * (sums[2 * r + 1] * p.inv_d));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i * tpr + t < nvec) {
            Q u;
            float f[VEC];
            F d[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) d[j] = ffma(a[r][i][j], rs, ffma(xh[r][i][j], c2, c1));
            if constexpr (RES) {
              F e[kN];
              raw[r][kArr - 1][i].unpack(f);
              N::gather(f, e);
#pragma unroll
              for (int j = 0; j < kN; ++j) d[j] = fadd(d[j], e[j]);
            }
            N::scatter(d, f);
            if constexpr (SHIFT) {
              const Edge<VEC> part(i * tpr + t, e, p.D);
              if (!part.whole()) {
                store_part<T, VEC>(f, y_at + i * tpr * VEC, part);
                continue;
              }
            }
            u.pack(f);
            u.store(y_at + i * tpr * VEC, 0);
          }
        }
      }
      y_at += sy;
    }
    if (++stage == steps) stage = 0;
  }
  cp_async_wait_all();
  let_next_launch();
  if (p.partials == nullptr && p.dgamma == nullptr) return;
  // one block alone writes the gradients themselves
  W* dgamma = static_cast<W*>(p.dgamma);
  W* dbeta = static_cast<W*>(p.dbeta);
  float* part = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
  auto put = [&](int col, float vg, float vb) {
    if (dgamma != nullptr) {
      dgamma[col] = from_f32<W>(vg);
      dbeta[col] = from_f32<W>(vb);
    } else {
      part[col] = vg;
      part[p.D + col] = vb;
    }
  };
  float fg[NV][VEC], fb[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    N::scatter(dg[i], fg[i]);
    N::scatter(db[i], fb[i]);
  }
  if constexpr (ONE_WARP) {
    // join the warps' sums in shared memory, in the warps' order
    float* acc = reinterpret_cast<float*>(stage_mem);  // [groups][2][NV * VEC][32]
    __syncthreads();
    if constexpr (SHIFT) {  // the warps' columns differ: [groups][2][column]
      constexpr int kRow = NV * VEC * 32;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int col = (i * 32 + t) * VEC + j - e;
          if (col < 0 || col >= p.D) continue;
          acc[group * 2 * kRow + col] = fg[i][j];
          acc[(group * 2 + 1) * kRow + col] = fb[i][j];
        }
      __syncthreads();
      for (int col = threadIdx.x; col < p.D; col += blockDim.x) {
        float sg = 0.0f, sb = 0.0f;
        for (int gq = 0; gq < groups; ++gq) {
          sg += acc[gq * 2 * kRow + col];
          sb += acc[(gq * 2 + 1) * kRow + col];
        }
        put(col, sg, sb);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        acc[((group * 2 + 0) * NV * VEC + i * VEC + j) * 32 + t] = fg[i][j];
        acc[((group * 2 + 1) * NV * VEC + i * VEC + j) * 32 + t] = fb[i][j];
      }
    __syncthreads();
    for (int k = threadIdx.x; k < NV * VEC * 32; k += blockDim.x) {
      float sg = 0.0f, sb = 0.0f;
      for (int gq = 0; gq < groups; ++gq) {
        sg += acc[gq * 2 * NV * VEC * 32 + k];
        sb += acc[(gq * 2 + 1) * NV * VEC * 32 + k];
      }
      const int el = k / 32, c = (el / VEC) * 32 + (k & 31);
      if (c < nvec) put(c * VEC + el % VEC, sg, sb);
    }
  } else if constexpr (SHIFT) {
    // by way of shared memory (2 D floats: no more than the slots, which hold
    // two steps of two rows' vectors or more), so that neighbouring threads
    // write neighbouring columns
    float* acc = reinterpret_cast<float*>(stage_mem);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int col = (i * tpr + t) * VEC + j - e;
        if (col < 0 || col >= p.D) continue;
        acc[col] = fg[i][j];
        acc[p.D + col] = fb[i][j];
      }
    __syncthreads();
    for (int k = t; k < 2 * p.D; k += tpr) part[k] = acc[k];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + t;
      if (c >= nvec) break;
      if constexpr (VEC > 1) {
        if (dgamma == nullptr) {
#pragma unroll
          for (int j = 0; j < VEC; j += 4) {
            float* at = part + c * VEC + j;
            *reinterpret_cast<float4*>(at) = make_float4(fg[i][j], fg[i][j + 1], fg[i][j + 2], fg[i][j + 3]);
            *reinterpret_cast<float4*>(at + p.D) = make_float4(fb[i][j], fb[i][j + 1], fb[i][j + 2], fb[i][j + 3]);
          }
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) put(c * VEC + j, fg[i][j], fb[i][j]);
    }
  }
}

// Column sums of partials [P][C]: 16 columns x 64 rows of threads per block,
// each thread adding every 64th row, then the 64 partial sums in a fixed order.
// The kernel may be resident while the one before it still writes `part`, so
// the sums are read from L2 by ordinary loads (see wait_for_previous).
constexpr int kJoinCols = 16, kJoinRows = 64;
template <typename O>
__global__ void __launch_bounds__(kJoinCols* kJoinRows)
    join_partials_kernel(const float* part, int P, int64_t C, int64_t split, O* out0, O* out1) {
  __shared__ float acc[kJoinRows][kJoinCols + 1];
  wait_for_previous();
  const int tx = threadIdx.x % kJoinCols, ty = threadIdx.x / kJoinCols;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kJoinCols + tx;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int r = ty; r < P; r += kJoinRows) s += __ldcg(part + static_cast<int64_t>(r) * C + c);
  }
  acc[ty][tx] = s;
  __syncthreads();
  // warp w < 16 sums column w of the block
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (w >= kJoinCols) return;
  s = warp_sum(acc[lane][w] + acc[lane + 32][w]);
  const int64_t cw = static_cast<int64_t>(blockIdx.x) * kJoinCols + w;
  if (lane == 0 && cw < C) {
    if (cw < split) out0[cw] = from_f32<O>(s);
    else out1[cw - split] = from_f32<O>(s);
  }
}

int round32(int64_t v) { return static_cast<int>((v + 31) / 32 * 32); }

template <typename T>
NormArgs<T> make_args(const NormCall& c, int vec) {
  NormArgs<T> a{};
  a.x = static_cast<const T*>(c.x);
  a.res = static_cast<const T*>(c.res);
  a.rin = static_cast<const T*>(c.r_in);
  a.gamma = c.gamma;
  a.beta = c.beta;
  a.r = static_cast<T*>(c.r);
  a.y = static_cast<T*>(c.y);
  a.mean = c.mean;
  a.rstd = c.rstd;
  a.partials = c.partials;
  a.ldx = c.ldx;
  a.ldres = c.ldres;
  a.ldr = c.ldr;
  a.ldy = c.ldy;
  a.rows = c.rows;
  a.eps = c.eps;
  a.inv_d = 1.0f / static_cast<float>(c.D);
  a.D = c.D;
  a.nvec = c.D / vec;
  return a;
}

// Whether every row of the call starts on a 16-byte boundary and holds whole
// 16-byte vectors.
bool vector_rows(const NormCall& c, size_t elem) {
  const auto ok = [&](const void* p, int64_t ld) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (static_cast<uint64_t>(ld) * elem)) & 15u) == 0;
  };
  return (static_cast<size_t>(c.D) * elem) % 16 == 0 && ok(c.x, c.ldx) && ok(c.res, c.ldres) &&
         ok(c.r, c.ldr) && ok(c.r_in, c.ldr) && ok(c.y, c.ldy) && ok(c.gamma, 0) && ok(c.beta, 0);
}

// Whether the arrays' rows lie alike within their 16-byte units, and the most
// vectors that such a row touches.
bool alike_rows(const NormCall& c, size_t elem) {
  const auto place = [&](const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) | ((static_cast<uint64_t>(ld) * elem & 15u) << 4);
  };
  const auto ok = [&](const void* p, int64_t ld) { return p == nullptr || place(p, ld) == place(c.x, c.ldx); };
  return ok(c.res, c.ldres) && ok(c.r, c.ldr) && ok(c.r_in, c.ldr) && ok(c.y, c.ldy);
}
int shifted_vectors(int D, int vec) { return (D + 2 * vec - 2) / vec; }

// A number of blocks whose groups walk rows by a multiple of `period` (the
// rows after which a shifted row's place repeats), if they walk at all.
int64_t walk_blocks(int64_t blocks, int groups, int64_t rows, int period) {
  if (blocks * groups >= rows) return blocks;
  const int64_t unit = std::max(1, period / groups);
  return std::max(unit, blocks / unit * unit);
}

// Blocks that an SM holds: a warp's registers (in units of 8 per thread) lie
// in one of its four partitions of 512 per lane, 16 warps' places each.
int resident_blocks(int threads, int regs) {
  return std::max(1, std::min(64, 4 * (512 / ((regs + 7) / 8 * 8))) / (threads / 32));
}

template <typename T, typename W, int VEC, int NV>
cudaError_t fwd_nv(const NormCall& c, cudaStream_t s) {
  const NormArgs<T> a = make_args<T>(c, VEC);
  const int tpr = round32((a.nvec + NV - 1) / NV);
  if (tpr == 32) {
    const int64_t blocks = (c.rows + kRowsPerBlock - 1) / kRowsPerBlock;
    norm_fwd_kernel<T, W, VEC, NV, true><<<static_cast<unsigned>(blocks), 32 * kRowsPerBlock, 0, s>>>(a);
  } else {
    norm_fwd_kernel<T, W, VEC, NV, false><<<static_cast<unsigned>(c.rows), tpr, 0, s>>>(a);
  }
  return cudaGetLastError();
}

// Calls go(n) with the smallest of the compiled vector counts per thread
// that is at least `want` and covers nvec with kMaxThreads threads.
template <int VEC, int MOST_WANTED, class Go>
cudaError_t pick_nv(int nvec, int want, Go go) {
  const int n = std::max(want, (nvec + kMaxThreads - 1) / kMaxThreads);
  using std::integral_constant;
  if constexpr (VEC == 1) {
    if (n <= 4) return go(integral_constant<int, 4>{});
    return go(integral_constant<int, 16>{});
  } else {
    if (n <= 1) return go(integral_constant<int, 1>{});
    constexpr int kNeeded = kMaxD / VEC / kMaxThreads;
    if constexpr (std::max(kNeeded, MOST_WANTED) > 2)
      if (n > 2) return go(integral_constant<int, 4>{});
    return go(integral_constant<int, 2>{});
  }
}

// Vectors per thread: four keep enough bytes in flight per thread when there
// are rows for every SM; a few rows are bound by latency and get as many
// threads as their vectors.
template <typename T, typename W, int VEC>
cudaError_t fwd_vec(const NormCall& c, cudaStream_t s) {
  const int nvec = c.D / VEC;
  const bool many = c.rows >= 4 * static_cast<int64_t>(sm_count());
  const int want = many ? std::min(4, (nvec + 31) / 32) : 1;
  return pick_nv<VEC, 4>(nvec, want, [&](auto n) { return fwd_nv<T, W, VEC, decltype(n)::value>(c, s); });
}
// What the launch of a walking kernel needs to know of it, looked up once
// per device: a captured launch then makes no such call.
struct KernelLimits {
  std::atomic<int> regs[64];  // 0: not looked up
};
constexpr size_t kMaxDynamicSmem = 220 * 1024;

template <class K>
cudaError_t kernel_regs(K kern, KernelLimits& lim, int* regs) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  *regs = lim.regs[dev].load(std::memory_order_acquire);
  if (*regs > 0) return cudaSuccess;
  cudaFuncAttributes at{};
  err = cudaFuncGetAttributes(&at, kern);
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kMaxDynamicSmem));
  if (err != cudaSuccess) return err;
  *regs = std::max(at.numRegs, 1);
  lim.regs[dev].store(*regs, std::memory_order_release);
  return cudaSuccess;
}

template <typename T, typename W, int VEC, int NV, bool ONE_WARP>
cudaError_t fwd_shift_launch(const NormCall& c, cudaStream_t s) {
  const int groups = ONE_WARP ? kRowsPerBlock : 1;
  const int threads = ONE_WARP ? 32 * groups : round32((shifted_vectors(c.D, VEC) + NV - 1) / NV);
  auto kern = norm_fwd_shift_kernel<T, W, VEC, NV, ONE_WARP>;
  static KernelLimits limits;
  int regs = 0;
  const cudaError_t err = kernel_regs(kern, limits, &regs);
  if (err != cudaSuccess) return err;
  int per_sm = resident_blocks(threads, regs);
  const size_t stage = static_cast<size_t>(c.res != nullptr ? 2 : 1) * NV * threads * 16;
  const int steps = (3 * stage + 2048) * per_sm <= kMaxDynamicSmem ? 3 : 2;
  const size_t bytes = steps * stage;
  per_sm = std::min(per_sm, static_cast<int>(228 * 1024 / (bytes + 2048)));
  const int64_t blocks = walk_blocks(
      std::min<int64_t>(static_cast<int64_t>(sm_count()) * per_sm, (c.rows + groups - 1) / groups),
      groups, c.rows, VEC);
  kern<<<static_cast<unsigned>(blocks), threads, bytes, s>>>(make_args<T>(c, VEC), steps);
  return cudaGetLastError();
}
template <typename T, typename W, int VEC>
cudaError_t fwd_shift(const NormCall& c, cudaStream_t s) {
  const int nvec = shifted_vectors(c.D, VEC);
  return pick_nv<VEC, 1>(nvec, 1, [&](auto n) {
    constexpr int NV = decltype(n)::value;
    if constexpr (NV == 1)
      if (nvec <= 32 * NV) return fwd_shift_launch<T, W, VEC, NV, true>(c, s);
    return fwd_shift_launch<T, W, VEC, NV, false>(c, s);
  });
}

enum class Rows { kVectors, kShifted, kElements };
template <typename T>
Rows kind_of_rows(const NormCall& c) {
  constexpr int VEC = 16 / sizeof(T);
  if (vector_rows(c, sizeof(T))) return Rows::kVectors;
  // narrow rows and few of them are left to single elements: 32768 x 63 bf16
  // takes 8 us so forward (19 shifted) and 13 backward (15), 1000 x 1001
  // backward 8.8 (12.4); 20000 x 201 takes 16.4 and 25 (13.4 and 14)
  const bool worth = c.D > 128 && c.rows >= 16 * static_cast<int64_t>(sm_count());
  return worth && alike_rows(c, sizeof(T)) && shifted_vectors(c.D, VEC) <= kMaxD / VEC ? Rows::kShifted
                                                                                      : Rows::kElements;
}

template <typename T, typename W>
cudaError_t fwd_type(const NormCall& c, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  switch (kind_of_rows<T>(c)) {
    case Rows::kVectors: return fwd_vec<T, W, VEC>(c, s);
    case Rows::kShifted: return fwd_shift<T, W, VEC>(c, s);
    default: return fwd_vec<T, W, 1>(c, s);
  }
}

template <typename T, typename W, int VEC, int NV, bool ONE_WARP, bool RES, int R, bool SHIFT>
cudaError_t bwd_launch(const NormCall& c, cudaStream_t s) {
  NormArgs<T> a = make_args<T>(c, VEC);
  const int nvec = SHIFT ? shifted_vectors(c.D, VEC) : a.nvec;
  const int threads = ONE_WARP ? 32 * kBwdGroups : round32((nvec + NV - 1) / NV);
  const int groups = ONE_WARP ? kBwdGroups : 1;
  auto kern = norm_bwd_kernel<T, W, VEC, NV, ONE_WARP, RES, R, SHIFT>;
  static KernelLimits limits;
  int regs = 0;
  cudaError_t err = kernel_regs(kern, limits, &regs);
  if (err != cudaSuccess) return err;
  // two steps ahead where shared memory (1 KB more per block is the system's)
  // keeps the number of blocks that an SM holds, else one
  int per_sm = resident_blocks(threads, regs);
  const auto slot_bytes = [&](int steps) {
    return static_cast<size_t>(bwd_slots<NV, RES, R>(steps)) * threads * sizeof(T) * VEC;
  };
  const int steps = (slot_bytes(3) + 2048) * per_sm <= kMaxDynamicSmem ? 3 : 2;
  size_t bytes = slot_bytes(steps);
  if (ONE_WARP) bytes = std::max(bytes, static_cast<size_t>(groups) * 2 * NV * VEC * 32 * 4);
  per_sm = std::min(per_sm, static_cast<int>(228 * 1024 / (bytes + 2048)));
  int64_t blocks = static_cast<int64_t>(sm_count()) * std::max(per_sm, 1);
  blocks = std::min({blocks, (c.rows + groups * R - 1) / (groups * R), kPartialRows});
  // few rows: one block, which needs no second launch
  if (c.rows <= kOneBlockRows) blocks = 1;
  if (SHIFT) blocks = walk_blocks(blocks, groups, c.rows, VEC);
  if (blocks == 1) {
    a.partials = nullptr;
    a.dgamma = c.dgamma;
    a.dbeta = c.dbeta;
  }
  kern<<<static_cast<unsigned>(blocks), threads, bytes, s>>>(a, steps);
  err = cudaGetLastError();
  if (err != cudaSuccess || c.dgamma == nullptr || blocks == 1) return err;
  return launch_join_partials(c.partials, static_cast<int>(blocks), 2 * static_cast<int64_t>(c.D),
                              c.D, c.dgamma, c.dbeta, c.wtype, s);
}

template <typename T, typename W, int VEC, int NV, bool ONE_WARP, int R, bool SHIFT>
cudaError_t bwd_res(const NormCall& c, cudaStream_t s) {
  return c.res != nullptr ? bwd_launch<T, W, VEC, NV, ONE_WARP, true, R, SHIFT>(c, s)
                          : bwd_launch<T, W, VEC, NV, ONE_WARP, false, R, SHIFT>(c, s);
}

// Two rows at a time where a thread holds up to eight columns; with sixteen
// (the widest rows) two would not fit its registers.
template <typename T, typename W, int VEC, bool SHIFT>
cudaError_t bwd_vec(const NormCall& c, cudaStream_t s) {
  const int nvec = SHIFT ? shifted_vectors(c.D, VEC) : c.D / VEC;
  return pick_nv<VEC, 1>(nvec, 1, [&](auto n) {
    constexpr int NV = decltype(n)::value;
    constexpr int R = NV * VEC <= 8 ? 2 : 1;
    if constexpr (NV == (VEC == 1 ? 4 : 1)) {  // more vectors per thread are only taken by wide rows
      if (nvec <= 32 * NV) return bwd_res<T, W, VEC, NV, true, R, SHIFT>(c, s);
    }
    return bwd_res<T, W, VEC, NV, false, R, SHIFT>(c, s);
  });
}
template <typename T, typename W>
cudaError_t bwd_type(const NormCall& c, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  switch (kind_of_rows<T>(c)) {
    case Rows::kVectors: return bwd_vec<T, W, VEC, false>(c, s);
    case Rows::kShifted: return bwd_vec<T, W, VEC, true>(c, s);
    default: return bwd_vec<T, W, 1, false>(c, s);
  }
}

template <template <typename, typename> class F>
cudaError_t by_type(const NormCall& c, cudaStream_t s) {
  const bool w32 = c.wtype == MOE_FP32;
  switch (c.type) {
    case MOE_BF16:
      return w32 ? F<__nv_bfloat16, float>::go(c, s) : F<__nv_bfloat16, __nv_bfloat16>::go(c, s);
    case MOE_FP16:
      return w32 ? F<__half, float>::go(c, s) : F<__half, __half>::go(c, s);
    default:
      return F<float, float>::go(c, s);
  }
}
template <typename T, typename W>
struct Fwd {
  static cudaError_t go(const NormCall& c, cudaStream_t s) { return fwd_type<T, W>(c, s); }
};
template <typename T, typename W>
struct Bwd {
  static cudaError_t go(const NormCall& c, cudaStream_t s) { return bwd_type<T, W>(c, s); }
};

}  // namespace

cudaError_t launch_layer_norm(const NormCall& c, cudaStream_t s) { return by_type<Fwd>(c, s); }
cudaError_t launch_layer_norm_bwd(const NormCall& c, cudaStream_t s) { return by_type<Bwd>(c, s); }

cudaError_t launch_join_partials(const float* partials, int P, int64_t C, int64_t split, void* out0,
                                 void* out1, moe_dtype type, cudaStream_t s) {
  cudaLaunchAttribute overlap = overlap_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((C + kJoinCols - 1) / kJoinCols));
  cfg.blockDim = dim3(kJoinCols * kJoinRows);
  cfg.stream = s;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  switch (type) {
    case MOE_BF16:
      return cudaLaunchKernelEx(&cfg, join_partials_kernel<__nv_bfloat16>, partials, P, C, split,
                                static_cast<__nv_bfloat16*>(out0), static_cast<__nv_bfloat16*>(out1));
    case MOE_FP16:
      return cudaLaunchKernelEx(&cfg, join_partials_kernel<__half>, partials, P, C, split,
                                static_cast<__half*>(out0), static_cast<__half*>(out1));
    default:
      return cudaLaunchKernelEx(&cfg, join_partials_kernel<float>, partials, P, C, split,
                                static_cast<float*>(out0), static_cast<float*>(out1));
  }
}

}  // namespace moe
