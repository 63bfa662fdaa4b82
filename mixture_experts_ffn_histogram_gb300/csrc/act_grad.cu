// dz = dy * act'(z) and its column sums, the first step of the linear
// layer's backward.  dz is rounded to 16 bits because the tensor core takes
// both products' operands in one 16-bit type; in bf16 that puts dw 2.35e-3 of
// its norm from 64 bits, where rounding dw alone is 1.66e-3 (dx 1.74e-3 and
// 1.66e-3; 8192 x 7168 x 2048, SiLU).  Bound by HBM: dy and z are read once, dz is written
// once, 16 bytes per access.  The column sums are of the unrounded fp32 dz;
// each block leaves one row of partial sums per stretch of rows, joined in a
// fixed order.  27688 x 3136: 66 us for the sums alone (347 MB, 51 us of HBM).
#include <algorithm>

#include "activation.cuh"
#include "kernels.h"
#include "layer.h"
#include "layer_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Two rows' loads under way per thread and four resident blocks per SM.  Four
// rows take the registers of two blocks, and a grid of more than one wave only
// lengthens the partial sums and their join: the column sums alone of
// 27688 x 3136 take 66.8 us, of 1012 x 1288 5.3 us; with four rows and a grid
// of eight blocks per SM 95 and 8.8 us.
constexpr int kRows = 2;
constexpr int kBlocksPerSm = 4;
constexpr int64_t kOneBlockRows = 64;

template <typename T, typename Y>
struct ActGradArgs {
  const Y* dy;
  const T* z;
  T* dz;
  float* partials;
  int64_t lddy, ldz, M, N, rows_per_block;
  int act, col_threads;
};

template <typename Y>
__device__ __forceinline__ void load8(const Y* p, float (&f)[8]) {
  if constexpr (sizeof(Y) == 4) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    Raw<Y, 8> r;
    r.load(p, 0);
    r.unpack(f);
  }
}

// g *= act'(z), with one branch on the activation.
template <int ACT>
__device__ __forceinline__ void slope_run(const float (&z)[8], float (&g)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] *= act_slope<false>(z[j], ACT);
}
__device__ __forceinline__ void slope_all(const float (&z)[8], float (&g)[8], int act) {
  switch (act) {
    case MOE_ACT_RELU: slope_run<MOE_ACT_RELU>(z, g); break;
    case MOE_ACT_GELU: slope_run<MOE_ACT_GELU>(z, g); break;
    case MOE_ACT_GELU_TANH: slope_run<MOE_ACT_GELU_TANH>(z, g); break;
    default: slope_run<MOE_ACT_SILU>(z, g); break;
  }
}

// Blocks of col_threads x (kThreads / col_threads) threads, eight columns a thread.
template <typename T, typename Y>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) act_grad_kernel(const ActGradArgs<T, Y> p) {
  __shared__ float red[kThreads][9];
  const int tx = threadIdx.x % p.col_threads, ty = threadIdx.x / p.col_threads;
  const int nrow = kThreads / p.col_threads;
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * p.col_threads + tx) * 8;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * p.rows_per_block;
  const int64_t r1 = min(p.M, r0 + p.rows_per_block);
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  if (col < p.N) {
    for (int64_t r = r0 + ty; r < r1; r += kRows * nrow) {
      float g[kRows][8], z[kRows][8];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t rk = min(r + k * nrow, p.M - 1);
        load8<Y>(p.dy + rk * p.lddy + col, g[k]);
        if (p.act != MOE_ACT_NONE) load8<T>(p.z + rk * p.ldz + col, z[k]);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (r + k * nrow >= r1) break;
        if (p.act != MOE_ACT_NONE) slope_all(z[k], g[k], p.act);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += g[k][j];
        if (p.dz != nullptr) {
          Raw<T, 8> o;
          o.pack(g[k]);
          o.store(p.dz + (r + k * nrow) * p.N + col, 0);
        }
      }
    }
  }
  let_next_launch();
  if (p.partials == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) red[threadIdx.x][j] = sum[j];
  __syncthreads();
  for (int i = threadIdx.x; i < p.col_threads * 8; i += kThreads) {
    const int c = i / 8, j = i % 8;
    float s = 0.0f;
    for (int y = 0; y < nrow; ++y) s += red[y * p.col_threads + c][j];
    const int64_t cc = (static_cast<int64_t>(blockIdx.x) * p.col_threads + c) * 8 + j;
    if (cc < p.N) p.partials[static_cast<int64_t>(blockIdx.y) * p.N + cc] = s;  // (the sums themselves for one block)
  }
}

template <typename T, typename Y>
cudaError_t launch_t(const ActGradCall& c, cudaStream_t s) {
  ActGradArgs<T, Y> a{};
  a.dy = static_cast<const Y*>(c.dy);
  a.z = static_cast<const T*>(c.z);
  a.dz = static_cast<T*>(c.dz);
  a.partials = c.db != nullptr ? c.partials : nullptr;
  a.lddy = c.lddy;
  a.ldz = c.ldz;
  a.M = c.M;
  a.N = c.N;
  a.act = c.act;
  int ct = 32;
  while (ct > 1 && ct / 2 * 8 >= c.N) ct /= 2;
  a.col_threads = ct;
  const int64_t gx = (c.N + ct * 8 - 1) / (ct * 8);
  // one wave of resident blocks, whole passes of the block's rows each
  const int64_t pass = kThreads / ct;
  int64_t gy = std::max<int64_t>(1, static_cast<int64_t>(sm_count()) * kBlocksPerSm / gx);
  // few rows: one block down the rows writes the sums themselves, which
  // saves the second launch
  gy = c.M <= kOneBlockRows ? 1 : std::min({gy, (c.M + pass - 1) / pass, kPartialRows});
  a.rows_per_block = ((c.M + gy - 1) / gy + pass - 1) / pass * pass;
  gy = (c.M + a.rows_per_block - 1) / a.rows_per_block;
  if (gy == 1 && c.db != nullptr) a.partials = c.db;
  act_grad_kernel<T, Y><<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kThreads, 0, s>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || c.db == nullptr || gy == 1) return err;
  return launch_join_partials(c.partials, static_cast<int>(gy), c.N, c.N, c.db, nullptr, MOE_FP32, s);
}

}  // namespace

cudaError_t launch_act_grad(const ActGradCall& c, cudaStream_t s) {
  const bool f32 = c.dy_type == MOE_FP32;
  if (c.type == MOE_BF16)
    return f32 ? launch_t<__nv_bfloat16, float>(c, s) : launch_t<__nv_bfloat16, __nv_bfloat16>(c, s);
  return f32 ? launch_t<__half, float>(c, s) : launch_t<__half, __half>(c, s);
}

}  // namespace moe
