// What the kernels that normalise rows share: sums over a row's threads, rows
// that start or end inside a 16-byte unit, and the host's choice of threads,
// vectors and blocks.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "layer_common.cuh"

namespace moe {

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

// --------------------------------------------------------------- host side
inline int round32(int64_t v) { return static_cast<int>((v + 31) / 32 * 32); }

inline int shifted_vectors(int D, int vec) { return (D + 2 * vec - 2) / vec; }

// A number of blocks whose groups walk rows by a multiple of `period` (the
// rows after which a shifted row's place repeats), if they walk at all.
inline int64_t walk_blocks(int64_t blocks, int groups, int64_t rows, int period) {
  if (blocks * groups >= rows) return blocks;
  const int64_t unit = std::max(1, period / groups);
  return std::max(unit, blocks / unit * unit);
}

// Blocks that an SM holds: a warp's registers (in units of 8 per thread) lie
// in one of its four partitions of 512 per lane, 16 warps' places each.
inline int resident_blocks(int threads, int regs) {
  return std::max(1, std::min(64, 4 * (512 / ((regs + 7) / 8 * 8))) / (threads / 32));
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

}  // namespace moe
