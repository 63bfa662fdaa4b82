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
// offset of the row.
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

// ---------------------------------------------------------------- backward
// Each thread copies its own vectors of a row into its own shared-memory
// slots with cp.async, up to three rows ahead, and reads back only what it
// copied: the copies need no barrier, and the bytes in flight do not depend
// on registers.  A block walks rows with the grid's stride and keeps its
// columns' weight-gradient sums in registers; at the end they become one row
// of `partials` ([blocks][2][D]: dgamma, dbeta).
constexpr int kBwdGroups = 4;  // rows of one warp each per block

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

template <typename T, typename W, int VEC, int NV, bool ONE_WARP, bool RES>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormArgs<T> p, const int stages) {
  using R = Raw<T, VEC>;
  constexpr int kArr = RES ? 3 : 2;
  __shared__ float red[2][32][2];
  extern __shared__ __align__(16) unsigned char stage_mem[];
  const int tpr = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int groups = ONE_WARP ? (blockDim.x >> 5) : 1;
  const int group = ONE_WARP ? (threadIdx.x >> 5) : 0;
  const int nwarps = blockDim.x >> 5;
  using Slot = typename R::Store;
  Slot* slots = reinterpret_cast<Slot*>(stage_mem) + threadIdx.x;
  auto slot = [&](int stage, int arr, int i) -> Slot* {
    return slots + ((stage * kArr + arr) * NV + i) * static_cast<int>(blockDim.x);
  };
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * tpr + t;
        if (c < p.nvec) {
          copy_async<T, VEC>(slot(stage, 0, i), p.x + row * p.ldx + c * VEC);
          copy_async<T, VEC>(slot(stage, 1, i), p.rin + row * p.ldr + c * VEC);
          if constexpr (RES) copy_async<T, VEC>(slot(stage, 2, i), p.res + row * p.ldres + c * VEC);
        }
      }
    }
    cp_async_commit();
  };
  for (int q = 0; q < stages - 1; ++q) fetch(first + q * step, q);

  const W* gamma = static_cast<const W*>(p.gamma);
  float g[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[i][j] = dg[i][j] = db[i][j] = 0.0f;
    if (i * tpr + t < p.nvec) load_weights<W, VEC>(gamma, i * tpr + t, g[i]);
  }
  int stage = 0, par = 0;
  for (int64_t row = first; row < p.rows; row += step) {
    fetch(row + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    if (stages == 4) cp_async_wait_group<3>();
    else cp_async_wait_group<1>();
    float dy[NV][VEC], xh[NV][VEC];
    float sums[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * tpr + t < p.nvec) {
        R u;
        u.v = *slot(stage, 0, i);
        u.unpack(dy[i]);
        u.v = *slot(stage, 1, i);
        u.unpack(xh[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[i][j] = (xh[i][j] - mean) * rstd;
          dg[i][j] += dy[i][j] * xh[i][j];
          db[i][j] += dy[i][j];
          dy[i][j] *= g[i][j];  // a
          sums[0] += dy[i][j];
          sums[1] += dy[i][j] * xh[i][j];
        }
      }
    }
    row_sums<ONE_WARP, 2>(sums, red[par], nwarps);
    par ^= 1;
    const float m1 = sums[0] * p.inv_d, m2 = sums[1] * p.inv_d;
    T* dx = p.y + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + t;
      if (c < p.nvec) {
        float f[VEC];
        if constexpr (RES) {
          R u;
          u.v = *slot(stage, 2, i);
          u.unpack(f);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = rstd * (dy[i][j] - m1 - xh[i][j] * m2);
          f[j] = RES ? d + f[j] : d;
        }
        R u;
        u.pack(f);
        u.store(dx, c);
      }
    }
    if (++stage == stages) stage = 0;
  }
  cp_async_wait_all();
  if (p.partials == nullptr) return;
  float* part = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
  if constexpr (ONE_WARP) {
    // join the warps' sums in shared memory, in the warps' order
    float* acc = reinterpret_cast<float*>(stage_mem);  // [groups][2][NV * VEC][32]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        acc[((group * 2 + 0) * NV * VEC + i * VEC + j) * 32 + t] = dg[i][j];
        acc[((group * 2 + 1) * NV * VEC + i * VEC + j) * 32 + t] = db[i][j];
      }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * NV * VEC * 32; k += blockDim.x) {
      float s = 0.0f;
      for (int gq = 0; gq < groups; ++gq) s += acc[gq * 2 * NV * VEC * 32 + k];
      const int which = k / (NV * VEC * 32), e = (k / 32) % (NV * VEC), lane = k & 31;
      const int c = (e / VEC) * 32 + lane;
      if (c < p.nvec) part[which * p.D + c * VEC + e % VEC] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + t;
      if (c < p.nvec) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          part[c * VEC + j] = dg[i][j];
          part[p.D + c * VEC + j] = db[i][j];
        }
      }
    }
  }
}

// Column sums of partials [P][C]: 32 columns x 32 rows of threads per block,
// each thread adding every 32nd row, then the 32 partial sums in order.
constexpr int kJoinRows = 32;
template <typename O>
__global__ void __launch_bounds__(32 * kJoinRows)
    join_partials_kernel(const float* __restrict__ part, int P, int64_t C, int64_t split, O* out0,
                         O* out1) {
  __shared__ float acc[kJoinRows][33];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 4
    for (int r = threadIdx.y; r < P; r += kJoinRows) s += part[static_cast<int64_t>(r) * C + c];
  }
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // warp y sums column y of the block over the 32 row groups
  s = warp_sum(acc[threadIdx.x][threadIdx.y]);
  const int64_t cw = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && cw < C) {
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
template <typename T, typename W>
cudaError_t fwd_type(const NormCall& c, cudaStream_t s) {
  return vector_rows(c, sizeof(T)) ? fwd_vec<T, W, 16 / sizeof(T)>(c, s) : fwd_vec<T, W, 1>(c, s);
}

// What the launch of a backward needs to know of its kernel, looked up once
// per device: a captured launch then makes no such call.
struct KernelLimits {
  std::atomic<int> regs[64];  // 0: not looked up
};
constexpr int kMaxDynamicSmem = 220 * 1024;

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
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicSmem);
  if (err != cudaSuccess) return err;
  *regs = std::max(at.numRegs, 1);
  lim.regs[dev].store(*regs, std::memory_order_release);
  return cudaSuccess;
}

template <typename T, typename W, int VEC, int NV, bool ONE_WARP, bool RES>
cudaError_t bwd_launch(const NormCall& c, cudaStream_t s) {
  NormArgs<T> a = make_args<T>(c, VEC);
  const int threads = ONE_WARP ? 32 * kBwdGroups : round32((a.nvec + NV - 1) / NV);
  const int groups = ONE_WARP ? kBwdGroups : 1;
  // four rows of slots, or two where four do not fit (wide fp32 rows)
  const size_t row_bytes = static_cast<size_t>(RES ? 3 : 2) * NV * threads * sizeof(T) * VEC;
  const int stages = 4 * row_bytes <= kMaxDynamicSmem ? 4 : 2;
  size_t bytes = stages * row_bytes;
  if (ONE_WARP) bytes = std::max(bytes, static_cast<size_t>(groups) * 2 * NV * VEC * 32 * 4);
  auto kern = norm_bwd_kernel<T, W, VEC, NV, ONE_WARP, RES>;
  static KernelLimits limits;
  int regs = 0;
  cudaError_t err = kernel_regs(kern, limits, &regs);
  if (err != cudaSuccess) return err;
  // blocks that can be resident: by threads, registers (in units of 8 per
  // thread) and shared memory (1 KB more per block is the system's)
  const int per_sm = std::min({2048 / threads, 65536 / ((regs + 7) / 8 * 8 * threads),
                               static_cast<int>(228 * 1024 / (bytes + 2048))});
  int64_t blocks = static_cast<int64_t>(sm_count()) * std::max(per_sm, 1);
  blocks = std::min({blocks, (c.rows + groups - 1) / groups, kPartialRows});
  kern<<<static_cast<unsigned>(blocks), threads, bytes, s>>>(a, stages);
  err = cudaGetLastError();
  if (err != cudaSuccess || c.dgamma == nullptr) return err;
  return launch_join_partials(c.partials, static_cast<int>(blocks), 2 * static_cast<int64_t>(c.D),
                              c.D, c.dgamma, c.dbeta, c.wtype, s);
}

template <typename T, typename W, int VEC, int NV>
cudaError_t bwd_nv(const NormCall& c, cudaStream_t s) {
  const bool one = (c.D / VEC + NV - 1) / NV <= 32;
  if (one)
    return c.res != nullptr ? bwd_launch<T, W, VEC, NV, true, true>(c, s)
                            : bwd_launch<T, W, VEC, NV, true, false>(c, s);
  return c.res != nullptr ? bwd_launch<T, W, VEC, NV, false, true>(c, s)
                          : bwd_launch<T, W, VEC, NV, false, false>(c, s);
}

template <typename T, typename W, int VEC>
cudaError_t bwd_vec(const NormCall& c, cudaStream_t s) {
  return pick_nv<VEC, 1>(c.D / VEC, 1, [&](auto n) { return bwd_nv<T, W, VEC, decltype(n)::value>(c, s); });
}
template <typename T, typename W>
cudaError_t bwd_type(const NormCall& c, cudaStream_t s) {
  return vector_rows(c, sizeof(T)) ? bwd_vec<T, W, 16 / sizeof(T)>(c, s) : bwd_vec<T, W, 1>(c, s);
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
  const dim3 grid(static_cast<unsigned>((C + 31) / 32)), block(32, kJoinRows);
  switch (type) {
    case MOE_BF16:
      join_partials_kernel<<<grid, block, 0, s>>>(partials, P, C, split,
                                                  static_cast<__nv_bfloat16*>(out0),
                                                  static_cast<__nv_bfloat16*>(out1));
      break;
    case MOE_FP16:
      join_partials_kernel<<<grid, block, 0, s>>>(partials, P, C, split, static_cast<__half*>(out0),
                                                  static_cast<__half*>(out1));
      break;
    default:
      join_partials_kernel<<<grid, block, 0, s>>>(partials, P, C, split, static_cast<float*>(out0),
                                                  static_cast<float*>(out1));
  }
  return cudaGetLastError();
}

}  // namespace moe
