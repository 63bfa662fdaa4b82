// RMS norms after and before a block, with its gate and residual scale between
// them, forward and backward.  Per row, with q = post + offset and so on:
//
//   forward   yh = y / rms(y),  r = round(res + s t gate q_post yh),
//             rh = r / rms(r),  u = round(q_pre rh)
//             (s the scale, t the token's gate; any of the norms and gates may
//             be left out)
//   backward  a = du q_pre,  m = avg(a rh),  d = dr + (a - m rh) / rms(r)   -> dres
//             g = s gate q_post,  b = sum_d g yh d                          -> dtoken_gate
//             dy = (t g d - t b yh / D) / rms(y)
//             dpre = sum_rows du rh,  e = sum_rows t d yh,
//             dpost = s gate e,  dgate = s q_post e
//
// One pass over the row's data in each direction: bound by HBM, like the layer
// norm, with four arrays forward and six backward.  Backward, b needs d and d
// needs m; but b = sum g yh (dr + a / rms(r)) - m / rms(r) sum g yh rh, so that
// all three sums are taken together and a row costs one exchange between its
// threads.  dpost and dgate have one sum over the rows in common.
//
// Rows of whole, aligned 16-byte vectors move in such vectors, rows that lie
// alike within their 16-byte units shifted by their place in it, other rows
// element by element (row_common.cuh).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "layer.h"
#include "layer_common.cuh"
#include "row_common.cuh"

namespace moe {
namespace {

template <typename T, typename W>
struct Args {
  const T *y, *res, *rin, *du, *dr;
  T *r, *u, *dres, *dy;
  const W *post, *pre, *gate;
  const float* token_gate;
  float *rstd_y, *rstd_r, *dtoken_gate;
  float* partials;            // [blocks][2][D]: dpre, e
  W *dpost, *dpre, *dgate;    // backward by one block
  int64_t ldy, ldres, ldr, ldu, lddu, lddr, lddres, lddy, rows;
  float eps, scale, offset, inv_d;
  int D, nvec;
};

// Weights of a vector's columns: w + offset, or (w not given) ones.
template <typename W, int VEC, bool SHIFT>
__device__ __forceinline__ void weights_or_one(const W* w, float offset, int c, int e, int D, float (&f)[VEC]) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = 1.0f;
    return;
  }
  if constexpr (SHIFT) load_shifted_weights(w, c, e, D, f);
  else load_weights<W, VEC>(w, c, f);
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] += offset;
}
template <int VEC>
__device__ __forceinline__ float square_sum(const float (&f)[VEC]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < VEC; ++j) s += f[j] * f[j];
  return s;
}

// ---------------------------------------------------------------- forward
// One row per block of blockDim.x threads, or (ONE_WARP) one row per warp.
template <typename T, typename W, int VEC, int NV, bool ONE_WARP>
__global__ void __launch_bounds__(kMaxThreads, NV <= 2 ? 3 : NV == 4 ? 2 : 1) block_norm_kernel(const Args<T, W> p) {
  using N = Nums<VEC>;
  using F = typename N::F;
  constexpr int kN = N::kN;
  __shared__ float red[2][32][1];
  const int tpr = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = ONE_WARP ? static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5)
                               : static_cast<int64_t>(blockIdx.x);
  if (ONE_WARP && row >= p.rows) return;
  const int nwarps = blockDim.x >> 5;
  const auto values = [](const Raw<T, VEC>& raw, F (&v)[kN]) {
    float f[VEC];
    raw.unpack(f);
    N::gather(f, v);
  };
  const auto weights = [&](const W* w, float offset, int at, F (&v)[kN]) {
    float f[VEC];
    weights_or_one<W, VEC, false>(w, offset, at, 0, p.D, f);
    N::gather(f, v);
  };
  // of the row whose vectors are in x
  const auto rstd_of = [&](const Raw<T, VEC> (&x)[NV], float (*slots)[1]) {
    F s = N::splat(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * tpr + t < p.nvec) {
        F v[kN];
        values(x[i], v);
#pragma unroll
        for (int j = 0; j < kN; ++j) s = ffma(v[j], v[j], s);
      }
    }
    float sum[1] = {fold(s)};
    row_sums<ONE_WARP, 1>(sum, slots, nwarps);
    return 1.0f / sqrtf(sum[0] * p.inv_d + p.eps);
  };
  const auto put = [&](const F (&v)[kN], Raw<T, VEC>& raw, T* to, int at) {
    float f[VEC];
    N::scatter(v, f);
    raw.pack(f);
    raw.store(to, at);
  };
  Raw<T, VEC> a[NV], b[NV];
  const T* res = p.res + row * p.ldres;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i * tpr + t < p.nvec) b[i].load(res, i * tpr + t);
  if (p.y != nullptr) {
    const T* y = p.y + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * tpr + t < p.nvec) a[i].load(y, i * tpr + t);
    float c = p.token_gate != nullptr ? p.scale * __ldg(p.token_gate + row) : p.scale;
    if (p.post != nullptr) {
      const float rstd = rstd_of(a, red[0]);
      if (t == 0 && p.rstd_y != nullptr) p.rstd_y[row] = rstd;
      c *= rstd;
    }
    T* r = p.r + row * p.ldr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = i * tpr + t;
      if (at < p.nvec) {
        F f[kN], g[kN], w[kN];
        values(a[i], f);
        values(b[i], g);
        weights(p.post, p.offset, at, w);
        if (p.gate != nullptr) {
          F m[kN];
          weights(p.gate, 0.0f, at, m);
#pragma unroll
          for (int j = 0; j < kN; ++j) w[j] = fmul(w[j], m[j]);
        }
#pragma unroll
        for (int j = 0; j < kN; ++j) g[j] = ffma(fmul(f[j], N::splat(c)), w[j], g[j]);
        put(g, b[i], r, at);  // the stored row is what is normalised next
      }
    }
  }
  if (p.pre == nullptr) return;
  const float rstd = rstd_of(b, red[1]);
  if (t == 0 && p.rstd_r != nullptr) p.rstd_r[row] = rstd;
  T* u = p.u + row * p.ldu;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = i * tpr + t;
    if (at < p.nvec) {
      F g[kN], w[kN];
      values(b[i], g);
      weights(p.pre, p.offset, at, w);
#pragma unroll
      for (int j = 0; j < kN; ++j) g[j] = fmul(fmul(g[j], N::splat(rstd)), w[j]);
      put(g, b[i], u, at);
    }
  }
}

// Shifted rows: a group of threads walks rows, whose copies come `steps` - 1
// ahead into the threads' own slots, and keeps the weights of its columns.
// (Bound by instructions and by what is under way: held to 40 registers more
// rows are (32768 x 1407 bf16 114 us, 119 without); two rows to a barrier
// changed nothing, since few blocks then fit.)
template <typename T, typename W, int VEC, int NV, bool ONE_WARP>
__global__ void __launch_bounds__(kMaxThreads, NV == 1 ? (ONE_WARP ? 2 : 3) : 1) block_norm_shift_kernel(const Args<T, W> p, const int steps) {
  using Q = Raw<T, VEC>;
  __shared__ float red[2][32][1];
  extern __shared__ __align__(16) unsigned char stage_mem[];
  const int tpr = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int groups = ONE_WARP ? (blockDim.x >> 5) : 1;
  const int nwarps = blockDim.x >> 5, bd = blockDim.x;
  const bool has_y = p.y != nullptr;
  const int stage_slots = 2 * NV * bd;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + (ONE_WARP ? (threadIdx.x >> 5) : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int n = first < p.rows ? static_cast<int>((p.rows - 1 - first) / step) + 1 : 0;
  const int e = unit_offset(p.res + first * p.ldres), nvec = (e + p.D + VEC - 1) / VEC;
  typename Q::Store* const slots = reinterpret_cast<typename Q::Store*>(stage_mem) + threadIdx.x;
  const T* s_at = p.res + first * p.ldres - e;
  const T* y_at = has_y ? p.y + first * p.ldy - e : nullptr;
  T* r_at = has_y ? p.r + first * p.ldr - e : nullptr;
  T* u_at = p.pre != nullptr ? p.u + first * p.ldu - e : nullptr;
  int fetched = 0;
  auto fetch = [&](int stage) {
    if (fetched < n) {
      typename Q::Store* to = slots + stage * stage_slots;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * tpr + t;
        if (c < nvec) {
          const Edge<VEC> g(c, e, p.D);
          copy_unit(to + i * bd, s_at + c * VEC, g);
          if (has_y) copy_unit(to + (NV + i) * bd, y_at + c * VEC, g);
        }
      }
      s_at += step * p.ldres;
      if (has_y) y_at += step * p.ldy;
    }
    ++fetched;
    cp_async_commit();
  };
  for (int q = 0; q < steps - 1; ++q) fetch(q);
  float wy[NV][VEC], wu[NV][VEC];  // of the branch, of u
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float m[VEC];
    weights_or_one<W, VEC, true>(p.post, p.offset, i * tpr + t, e, p.D, wy[i]);
    weights_or_one<W, VEC, true>(p.gate, 0.0f, i * tpr + t, e, p.D, m);
    weights_or_one<W, VEC, true>(p.pre, p.offset, i * tpr + t, e, p.D, wu[i]);
#pragma unroll
    for (int j = 0; j < VEC; ++j) wy[i][j] *= m[j];
  }
  int stage = 0, par = 0;  // sums take turns in `red`: one barrier each
  for (int k = 0; k < n; ++k) {
    fetch(stage == 0 ? steps - 1 : stage - 1);
    if (steps == 3) cp_async_wait_group<2>();
    else cp_async_wait_group<1>();
    const int64_t row = first + k * step;
    const typename Q::Store* from = slots + stage * stage_slots;
    const auto outside_zero = [](float (&f)[VEC], const Edge<VEC>& g) {
      if (!g.whole()) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (j < g.lo || j >= g.hi) f[j] = 0.0f;
      }
    };
    float f[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i][j] = 0.0f;
      if (i * tpr + t < nvec) {
        Q a;
        a.v = from[i * bd];
        a.unpack(f[i]);
      }
    }
    if (has_y) {
      float h[NV][VEC], sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[i][j] = 0.0f;
        if (i * tpr + t < nvec) {
          Q a;
          a.v = from[(NV + i) * bd];
          a.unpack(h[i]);
          outside_zero(h[i], Edge<VEC>(i * tpr + t, e, p.D));
          sum[0] += square_sum(h[i]);
        }
      }
      float c = p.token_gate != nullptr ? p.scale * __ldg(p.token_gate + row) : p.scale;
      if (p.post != nullptr) {
        row_sums<ONE_WARP, 1>(sum, red[par], nwarps);
        par ^= 1;
        const float rstd = 1.0f / sqrtf(sum[0] * p.inv_d + p.eps);
        if (t == 0 && p.rstd_y != nullptr) p.rstd_y[row] = rstd;
        c *= rstd;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i * tpr + t < nvec) {
          const Edge<VEC> g(i * tpr + t, e, p.D);
#pragma unroll
          for (int j = 0; j < VEC; ++j) f[i][j] = fmaf(h[i][j] * c, wy[i][j], f[i][j]);
          if (g.whole()) {
            Q a;
            a.pack(f[i]);
            a.store(r_at + (i * tpr + t) * VEC, 0);
            a.unpack(f[i]);  // the stored row is what is normalised next
          } else {
            store_part<T, VEC>(f[i], r_at + (i * tpr + t) * VEC, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[i][j] = to_f32<T>(from_f32<T>(f[i][j]));
          }
        }
      }
      r_at += step * p.ldr;
    }
    if (p.pre != nullptr) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i * tpr + t < nvec) {
          outside_zero(f[i], Edge<VEC>(i * tpr + t, e, p.D));
          sum[0] += square_sum(f[i]);
        }
      }
      row_sums<ONE_WARP, 1>(sum, red[par], nwarps);
      par ^= 1;
      const float rstd = 1.0f / sqrtf(sum[0] * p.inv_d + p.eps);
      if (t == 0 && p.rstd_r != nullptr) p.rstd_r[row] = rstd;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i * tpr + t < nvec) {
          const Edge<VEC> g(i * tpr + t, e, p.D);
#pragma unroll
          for (int j = 0; j < VEC; ++j) f[i][j] = f[i][j] * rstd * wu[i][j];
          if (g.whole()) {
            Q a;
            a.pack(f[i]);
            a.store(u_at + (i * tpr + t) * VEC, 0);
          } else {
            store_part<T, VEC>(f[i], u_at + (i * tpr + t) * VEC, g);
          }
        }
      }
      u_at += step * p.ldu;
    }
    if (++stage == steps) stage = 0;
  }
  cp_async_wait_all();
}

// ---------------------------------------------------------------- backward
// A block takes R rows at a time, whose copies come a step or two ahead into
// the threads' own shared-memory slots (no barrier: a thread reads what it
// copied), walks rows with the grid's stride and keeps its columns' weight
// gradients in registers; at the end they become one row of `partials`.

// Sums of N = 4 or 8 values over the threads of a row: within a warp the lanes
// first halve the values that they carry; across warps through `red`, which
// the caller alternates, so that one barrier is enough.
template <bool ONE_WARP, int N>
__device__ __forceinline__ void sums_of(float (&v)[N], float (*red)[8], int nwarps) {
  constexpr int kLanes = 32 / N;  // lanes that end up with one value
  const int lane = threadIdx.x & 31;
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = v[i];
#pragma unroll
  for (int n = N / 2, h = 16; n >= 1; n /= 2, h /= 2) {
    const bool hi = lane & h;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = hi ? a[i + n] : a[i], give = hi ? a[i] : a[i + n];
      a[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  float c = a[0];
#pragma unroll
  for (int o = kLanes / 2; o > 0; o /= 2) c += __shfl_xor_sync(0xffffffffu, c, o);
  if constexpr (!ONE_WARP) {
    const int which = lane / kLanes, part = lane % kLanes;
    if (part == 0) red[threadIdx.x >> 5][which] = c;
    __syncthreads();
    c = 0.0f;
    for (int w = part; w < nwarps; w += kLanes) c += red[w][which];
#pragma unroll
    for (int o = kLanes / 2; o > 0; o /= 2) c += __shfl_xor_sync(0xffffffffu, c, o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, c, i * kLanes);
}

constexpr int kBwdGroups = 4;  // ONE_WARP: warps of a block, each on rows of its own
// Rows that one block takes, which needs no kernel to join sums (bf16, one block
// against several and the join: 2 x 7168 9.5 us and 10.9, 4 x 2816 6.8 and 7.0, 4 x 7168
// 13.5 and 11.1, 8 x 2816 9.6 and 7.0, 8 x 7168 21.1 and 11.2; 256 columns are equal).
constexpr int64_t kOneBlockRows = 2;
enum { kDu, kR, kDr, kY, kArrays };  // arrays of a row, each in its own slots

// FULL: every array is given and all have the same ld, as between two blocks
// of a contiguous model.  A row's place is then one offset, and no array is
// asked for; where a thread has eight columns at most (HOLD) it keeps its
// values between the sums and the gradients instead of unpacking them again.
// (32768 x 2816 bf16 with neither: 460 instructions of a warp for a vector and
// 262 us.)
template <typename T, typename W, int VEC, int NV, bool ONE_WARP, int R, bool SHIFT, bool FULL>
__global__ void __launch_bounds__(kMaxThreads, 1) block_norm_bwd_kernel(const Args<T, W> p, const int steps) {
  using Q = Raw<T, VEC>;
  using N = Nums<VEC>;
  using F = typename N::F;
  constexpr int kN = N::kN, kPerStep = R * kArrays * NV, kSums = 4 * R;
  constexpr bool HOLD = FULL && NV * VEC <= 8;
  __shared__ float red[2][kMaxThreads / 32][8];
  extern __shared__ __align__(16) unsigned char stage_mem[];
  const int tpr = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int groups = ONE_WARP ? (blockDim.x >> 5) : 1;
  const int group = ONE_WARP ? (threadIdx.x >> 5) : 0;
  const int nwarps = blockDim.x >> 5, bd = blockDim.x;
  typename Q::Store* const slots = reinterpret_cast<typename Q::Store*>(stage_mem) + threadIdx.x;
  const int first = blockIdx.x * groups + group, step = gridDim.x * groups;  // this group's rows
  const int n = first < p.rows ? static_cast<int>((p.rows - 1 - first) / step) + 1 : 0;
  const T* const base[kArrays] = {p.du, p.rin, p.dr, p.y};
  const int64_t ld[kArrays] = {p.lddu, p.ldr, p.lddr, p.ldy};
  const int e = SHIFT ? unit_offset(p.dres + first * p.lddres) : 0;
  const int nvec = SHIFT ? (e + p.D + VEC - 1) / VEC : p.nvec;
  // (Addresses are made from the row's number each time: pointers kept for six
  // arrays cost 16 registers.)
  const auto place = [&](int64_t ld0, int k) {
    return (first + static_cast<int64_t>(k) * step) * ld0 + (t * VEC - e);
  };
  int fetched = 0;
  auto fetch = [&](int stage) {
    typename Q::Store* to = slots + stage * kPerStep * bd;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (fetched + r >= n) break;
      int64_t off = FULL ? place(p.lddres, fetched + r) : 0;
#pragma unroll
      for (int q = 0; q < kArrays; ++q) {
        if constexpr (!FULL) {
          if (base[q] == nullptr) continue;
          off = place(ld[q], fetched + r);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i * tpr + t < nvec) {
            auto* slot = to + ((r * kArrays + q) * NV + i) * bd;
            if constexpr (SHIFT) copy_unit(slot, base[q] + off + i * tpr * VEC, Edge<VEC>(i * tpr + t, e, p.D));
            else copy_async<T, VEC>(slot, base[q] + off + i * tpr * VEC);
          }
        }
      }
    }
    fetched += R;
    cp_async_commit();
  };
  for (int q = 0; q < steps - 1; ++q) fetch(q);

  F wa[NV][kN], wg[NV][kN], sp[NV][kN], se[NV][kN];  // q_pre, g; sums: dpre, e
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[VEC], b[VEC], m[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) a[j] = b[j] = m[j] = 0.0f;
    if (i * tpr + t < nvec) {
      weights_or_one<W, VEC, SHIFT>(p.pre, p.offset, i * tpr + t, e, p.D, a);
      weights_or_one<W, VEC, SHIFT>(p.post, p.offset, i * tpr + t, e, p.D, b);
      weights_or_one<W, VEC, SHIFT>(p.gate, 0.0f, i * tpr + t, e, p.D, m);
#pragma unroll
      for (int j = 0; j < VEC; ++j) b[j] *= m[j] * p.scale;
    }
    N::gather(a, wa[i]);
    N::gather(b, wg[i]);
#pragma unroll
    for (int j = 0; j < kN; ++j) sp[i][j] = se[i][j] = N::splat(0.0f);
  }
  const int lane = threadIdx.x & 31;
  float lane_y = 1.0f, lane_r = 0.0f, lane_t = 1.0f;  // every 32 rows a lane reads those of one
  int stage = 0, par = 0;
  for (int k = 0; k < n; k += R) {
    fetch(stage == 0 ? steps - 1 : stage - 1);
    if ((k & 31) == 0 && k + lane < n) {
      const int64_t row = first + static_cast<int64_t>(k + lane) * step;
      if (p.post != nullptr) lane_y = __ldg(p.rstd_y + row);
      if (p.pre != nullptr) lane_r = __ldg(p.rstd_r + row);
      if (p.token_gate != nullptr) lane_t = __ldg(p.token_gate + row);
    }
    if (steps == 3) cp_async_wait_group<2>();
    else if (steps == 2) cp_async_wait_group<1>();
    else cp_async_wait_group<0>();
    const typename Q::Store* from = slots + stage * kPerStep * bd;
    // of vector i of row r of the step: du q_pre as `a` (and du, if asked for),
    // rh, yh and dr + a / rms(r)
    const auto load = [&](int r, int i, float ry, float rr, F (&du)[kN], F (&a)[kN], F (&rh)[kN], F (&yh)[kN],
                          F (&d)[kN]) {
      const auto get = [&](int q, F (&v)[kN]) {
        if (FULL || base[q] != nullptr) {
          Q raw;
          raw.v = from[((r * kArrays + q) * NV + i) * bd];
          // ahead of the row's start the unit may hold anything
          if constexpr (SHIFT)
            if (i == 0 && t == 0 && e > 0) raw.clear_below(e);
          float f[VEC];
          raw.unpack(f);
          N::gather(f, v);
        } else {
#pragma unroll
          for (int j = 0; j < kN; ++j) v[j] = N::splat(0.0f);
        }
      };
      get(kDu, du);
      get(kR, rh);
      get(kDr, d);
      get(kY, yh);
      const F sr = N::splat(rr), sy = N::splat(ry);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        a[j] = fmul(du[j], wa[i][j]);
        rh[j] = fmul(rh[j], sr);
        yh[j] = fmul(yh[j], sy);
        d[j] = ffma(a[j], sr, d[j]);
      }
    };
    float ry[R], rr[R], tg[R], sums[kSums];
    F rh[HOLD ? R : 1][NV][kN], yh[HOLD ? R : 1][NV][kN], d[HOLD ? R : 1][NV][kN];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = HOLD ? r : 0;
      ry[r] = __shfl_sync(0xffffffffu, lane_y, (k + r) & 31);
      rr[r] = __shfl_sync(0xffffffffu, lane_r, (k + r) & 31);
      tg[r] = __shfl_sync(0xffffffffu, lane_t, (k + r) & 31);
      F s1 = N::splat(0.0f), s2 = s1, s3 = s1;
      if (r == 0 || k + r < n) {  // past the last row the slots hold nothing
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i * tpr + t < nvec) {
            F du[kN], a[kN];
            load(r, i, ry[r], rr[r], du, a, rh[h][i], yh[h][i], d[h][i]);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              const F gy = fmul(wg[i][j], yh[h][i][j]);
              sp[i][j] = ffma(du[j], rh[h][i][j], sp[i][j]);
              s1 = ffma(a[j], rh[h][i][j], s1);
              s2 = ffma(gy, d[h][i][j], s2);
              s3 = ffma(gy, rh[h][i][j], s3);
            }
          }
        }
      }
      sums[4 * r] = fold(s1);
      sums[4 * r + 1] = fold(s2);
      sums[4 * r + 2] = fold(s3);
      sums[4 * r + 3] = 0.0f;
    }
    sums_of<ONE_WARP, kSums>(sums, red[par], nwarps);
    par ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = HOLD ? r : 0;
      if (r == 0 || k + r < n) {
        const float m = rr[r] * (sums[4 * r] * p.inv_d);
        const float b = sums[4 * r + 1] - m * sums[4 * r + 2];
        if (t == 0 && p.dtoken_gate != nullptr) p.dtoken_gate[first + static_cast<int64_t>(k + r) * step] = b;
        const float cy = p.post != nullptr ? tg[r] * b * p.inv_d : 0.0f;
        const F nm = N::splat(-m), ts = N::splat(tg[r]), nc = N::splat(-cy * ry[r]), sy = N::splat(ry[r]);
        const int64_t off = place(p.lddres, k + r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i * tpr + t < nvec) {
            F g[kN];
            if constexpr (!HOLD) {
              F a[kN];
              load(r, i, ry[r], rr[r], g, a, rh[0][i], yh[0][i], d[0][i]);
            }
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              d[h][i][j] = ffma(rh[h][i][j], nm, d[h][i][j]);
              const F dt = fmul(d[h][i][j], ts);
              se[i][j] = ffma(dt, yh[h][i][j], se[i][j]);
              g[j] = ffma(fmul(wg[i][j], dt), sy, fmul(yh[h][i][j], nc));
            }
            const auto put = [&](const F (&v)[kN], T* to) {
              float f[VEC];
              N::scatter(v, f);
              if constexpr (SHIFT) {
                const Edge<VEC> part(i * tpr + t, e, p.D);
                if (!part.whole()) {
                  store_part<T, VEC>(f, to, part);
                  return;
                }
              }
              Q u;
              u.pack(f);
              u.store(to, 0);
            };
            put(d[h][i], p.dres + off + i * tpr * VEC);
            if constexpr (FULL) put(g, p.dy + off + i * tpr * VEC);
            else if (p.dy != nullptr) put(g, p.dy + place(p.lddy, k + r) + i * tpr * VEC);
          }
        }
      }
    }
    if (++stage == steps) stage = 0;
  }
  cp_async_wait_all();
  let_next_launch();
  const bool alone = p.dpost != nullptr || p.dpre != nullptr || p.dgate != nullptr;
  if (p.partials == nullptr && !alone) return;
  float* part = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
  const auto put = [&](int col, float dpre, float se_) {
    if (alone) {  // this block is the only one: it writes the gradients themselves
      const float post = p.post != nullptr ? to_f32<W>(p.post[col]) + p.offset : 1.0f;
      const float gate = p.gate != nullptr ? to_f32<W>(p.gate[col]) : 1.0f;
      if (p.dpre != nullptr) p.dpre[col] = from_f32<W>(dpre);
      if (p.dpost != nullptr) p.dpost[col] = from_f32<W>(p.scale * gate * se_);
      if (p.dgate != nullptr) p.dgate[col] = from_f32<W>(p.scale * post * se_);
    } else {
      part[col] = dpre;
      part[p.D + col] = se_;
    }
  };
  // by way of shared memory, column by column, the warps' sums (ONE_WARP: each
  // had rows of its own) added in their order
  float* acc = reinterpret_cast<float*>(stage_mem);  // [groups][2][D]
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float fp[VEC], fe[VEC];
    N::scatter(sp[i], fp);
    N::scatter(se[i], fe);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int col = (i * tpr + t) * VEC + j - e;
      if (col < 0 || col >= p.D) continue;
      acc[group * 2 * p.D + col] = fp[j];
      acc[(group * 2 + 1) * p.D + col] = fe[j];
    }
  }
  __syncthreads();
  for (int col = threadIdx.x; col < p.D; col += bd) {
    float a = 0.0f, b = 0.0f;
    for (int g = 0; g < groups; ++g) {
      a += acc[g * 2 * p.D + col];
      b += acc[(g * 2 + 1) * p.D + col];
    }
    put(col, a, b);
  }
}

// Sums the blocks' partial rows, 16 columns x 64 rows of threads to a block, in
// a fixed order, and makes the three gradients of them.  (Resident while the
// kernel before it still writes: ordinary loads, see wait_for_previous.)
constexpr int kJoinCols = 16, kJoinRows = 64;
template <typename W>
struct JoinArgs {
  const float* part;
  const W *post, *gate;
  W *dpost, *dpre, *dgate;
  float scale, offset;
  int P, D;
};
template <typename W>
__global__ void __launch_bounds__(kJoinCols* kJoinRows) block_norm_join_kernel(const JoinArgs<W> p) {
  __shared__ float acc[kJoinRows][kJoinCols + 1];
  wait_for_previous();
  const int tx = threadIdx.x % kJoinCols, ty = threadIdx.x / kJoinCols;
  const int64_t C = 2 * static_cast<int64_t>(p.D), c = static_cast<int64_t>(blockIdx.x) * kJoinCols + tx;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int r = ty; r < p.P; r += kJoinRows) s += __ldcg(p.part + r * C + c);
  }
  acc[ty][tx] = s;
  __syncthreads();
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;  // warp w < 16 sums column w of the block
  if (w >= kJoinCols) return;
  s = warp_sum(acc[lane][w] + acc[lane + 32][w]);
  const int64_t cw = static_cast<int64_t>(blockIdx.x) * kJoinCols + w;
  if (lane != 0 || cw >= C) return;
  if (cw < p.D) {
    if (p.dpre != nullptr) p.dpre[cw] = from_f32<W>(s);
    return;
  }
  const int64_t d = cw - p.D;
  const float post = p.post != nullptr ? to_f32<W>(p.post[d]) + p.offset : 1.0f;
  const float gate = p.gate != nullptr ? to_f32<W>(p.gate[d]) : 1.0f;
  if (p.dpost != nullptr) p.dpost[d] = from_f32<W>(p.scale * gate * s);
  if (p.dgate != nullptr) p.dgate[d] = from_f32<W>(p.scale * post * s);
}

// --------------------------------------------------------------- host side
template <typename T, typename W>
Args<T, W> make_args(const BlockNormCall& c, int vec) {
  Args<T, W> a{};
  a.y = static_cast<const T*>(c.y);
  a.res = static_cast<const T*>(c.res);
  a.rin = static_cast<const T*>(c.r_in);
  a.du = static_cast<const T*>(c.du);
  a.dr = static_cast<const T*>(c.dr);
  a.r = static_cast<T*>(c.r);
  a.u = static_cast<T*>(c.u);
  a.dres = static_cast<T*>(c.dres);
  a.dy = static_cast<T*>(c.dy);
  a.post = static_cast<const W*>(c.post);
  a.pre = static_cast<const W*>(c.pre);
  a.gate = static_cast<const W*>(c.gate);
  a.token_gate = c.token_gate;
  a.rstd_y = c.rstd_y;
  a.rstd_r = c.rstd_r;
  a.dtoken_gate = c.dtoken_gate;
  a.partials = c.partials;
  a.ldy = c.ldy;
  a.ldres = c.ldres;
  a.ldr = c.ldr;
  a.ldu = c.ldu;
  a.lddu = c.lddu;
  a.lddr = c.lddr;
  a.lddres = c.lddres;
  a.lddy = c.lddy;
  a.rows = c.d.rows;
  a.eps = c.d.eps;
  a.scale = c.d.scale;
  a.offset = c.d.offset;
  a.inv_d = 1.0f / static_cast<float>(c.d.D);
  a.D = c.d.D;
  a.nvec = c.d.D / vec;
  return a;
}

// How the call's rows can be moved (row_common.cuh): all arrays that it gives
// have to agree.
enum class Rows { kVectors, kShifted, kElements };
template <typename T>
Rows kind_of_rows(const BlockNormCall& c) {
  constexpr int VEC = 16 / sizeof(T);
  const struct {
    const void* p;
    int64_t ld;
  } rows[] = {{c.y, c.ldy},   {c.res, c.ldres}, {c.r, c.ldr},       {c.r_in, c.ldr}, {c.u, c.ldu},
              {c.du, c.lddu}, {c.dr, c.lddr},   {c.dres, c.lddres}, {c.dy, c.lddy}};
  const auto place = [](const void* p, int64_t ld) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) |
                            ((static_cast<uint64_t>(ld) * sizeof(T) & 15u) << 4));
  };
  int common = -1;
  bool alike = true;
  for (const auto& q : rows) {
    if (q.p == nullptr) continue;
    if (common < 0) common = place(q.p, q.ld);
    alike = alike && place(q.p, q.ld) == common;
  }
  const auto whole = [](const void* w) { return (reinterpret_cast<uintptr_t>(w) & 15u) == 0; };
  if (alike && common == 0 && c.d.D % VEC == 0 && whole(c.post) && whole(c.pre) && whole(c.gate))
    return Rows::kVectors;
  // narrow rows and few of them are left to single elements, as for the layer norm
  const bool worth = c.d.D > 128 && c.d.rows >= 16 * static_cast<int64_t>(sm_count());
  return worth && alike && shifted_vectors(c.d.D, VEC) <= kMaxD / VEC ? Rows::kShifted : Rows::kElements;
}

template <typename T, typename W, int VEC>
cudaError_t fwd_rows(const BlockNormCall& c, cudaStream_t s) {
  const int nvec = c.d.D / VEC;
  // Where there are rows for every SM, four vectors a thread for wide rows, two
  // for others (32768 x 2816 bf16: 125 us against 129; 1408 columns: 68 against
  // 64); a few rows are bound by latency and get as many threads as vectors.
  const bool many = c.d.rows >= 4 * static_cast<int64_t>(sm_count());
  const int want = many ? std::min(nvec > 256 ? 4 : 2, (nvec + 31) / 32) : 1;
  return pick_nv<VEC, 4>(nvec, want, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    const Args<T, W> a = make_args<T, W>(c, VEC);
    const int tpr = round32((nvec + NV - 1) / NV);
    if (tpr == 32) {
      const int64_t blocks = (c.d.rows + kRowsPerBlock - 1) / kRowsPerBlock;
      block_norm_kernel<T, W, VEC, NV, true><<<static_cast<unsigned>(blocks), 32 * kRowsPerBlock, 0, s>>>(a);
    } else {
      block_norm_kernel<T, W, VEC, NV, false><<<static_cast<unsigned>(c.d.rows), tpr, 0, s>>>(a);
    }
    return cudaGetLastError();
  });
}

template <typename T, typename W, int VEC, int NV, bool ONE_WARP>
cudaError_t fwd_shift_launch(const BlockNormCall& c, cudaStream_t s) {
  const int groups = ONE_WARP ? kRowsPerBlock : 1;
  const int threads = ONE_WARP ? 32 * groups : round32((shifted_vectors(c.d.D, VEC) + NV - 1) / NV);
  auto kern = block_norm_shift_kernel<T, W, VEC, NV, ONE_WARP>;
  static KernelLimits limits;
  int regs = 0;
  const cudaError_t err = kernel_regs(kern, limits, &regs);
  if (err != cudaSuccess) return err;
  int per_sm = resident_blocks(threads, regs);
  const size_t stage = static_cast<size_t>(2) * NV * threads * 16;
  const int steps = (3 * stage + 2048) * per_sm <= kMaxDynamicSmem ? 3 : 2;
  const size_t bytes = steps * stage;
  per_sm = std::min(per_sm, static_cast<int>(228 * 1024 / (bytes + 2048)));
  const int64_t blocks =
      walk_blocks(std::min<int64_t>(static_cast<int64_t>(sm_count()) * per_sm, (c.d.rows + groups - 1) / groups),
                  groups, c.d.rows, VEC);
  kern<<<static_cast<unsigned>(blocks), threads, bytes, s>>>(make_args<T, W>(c, VEC), steps);
  return cudaGetLastError();
}
template <typename T, typename W, int VEC>
cudaError_t fwd_shift(const BlockNormCall& c, cudaStream_t s) {
  const int nvec = shifted_vectors(c.d.D, VEC);
  return pick_nv<VEC, 1>(nvec, 1, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if constexpr (NV == 1)
      if (nvec <= 32) return fwd_shift_launch<T, W, VEC, NV, true>(c, s);
    return fwd_shift_launch<T, W, VEC, NV, false>(c, s);
  });
}

template <typename T, typename W, int VEC, int NV, bool ONE_WARP, int R, bool SHIFT, bool FULL>
cudaError_t bwd_launch(const BlockNormCall& c, cudaStream_t s) {
  Args<T, W> a = make_args<T, W>(c, VEC);
  const int nvec = SHIFT ? shifted_vectors(c.d.D, VEC) : a.nvec;
  const int threads = ONE_WARP ? 32 * kBwdGroups : round32((nvec + NV - 1) / NV);
  const int groups = ONE_WARP ? kBwdGroups : 1;
  auto kern = block_norm_bwd_kernel<T, W, VEC, NV, ONE_WARP, R, SHIFT, FULL>;
  static KernelLimits limits;
  int regs = 0;
  cudaError_t err = kernel_regs(kern, limits, &regs);
  if (err != cudaSuccess) return err;
  int per_sm = resident_blocks(threads, regs);
  const auto slot_bytes = [&](int steps) {
    return static_cast<size_t>(steps) * R * kArrays * NV * threads * sizeof(T) * VEC;
  };
  // one step alone where two do not fit: fp32 rows of more than some 6900 columns
  const int steps = (slot_bytes(3) + 2048) * per_sm <= kMaxDynamicSmem ? 3 : slot_bytes(2) <= kMaxDynamicSmem ? 2 : 1;
  const size_t bytes = std::max(slot_bytes(steps), static_cast<size_t>(groups) * 2 * c.d.D * sizeof(float));
  per_sm = std::min(per_sm, static_cast<int>(228 * 1024 / (bytes + 2048)));
  int64_t blocks = static_cast<int64_t>(sm_count()) * std::max(per_sm, 1);
  blocks = std::min({blocks, (c.d.rows + groups * R - 1) / (groups * R), kPartialRows});
  const bool weights = c.dpost != nullptr || c.dpre != nullptr || c.dgate != nullptr;
  if (weights && c.d.rows <= kOneBlockRows) blocks = 1;  // few rows: no second launch
  if (SHIFT) blocks = walk_blocks(blocks, groups, c.d.rows, VEC);
  if (!weights || blocks == 1) {
    a.partials = nullptr;
    a.dpost = static_cast<W*>(c.dpost);
    a.dpre = static_cast<W*>(c.dpre);
    a.dgate = static_cast<W*>(c.dgate);
  }
  kern<<<static_cast<unsigned>(blocks), threads, bytes, s>>>(a, steps);
  err = cudaGetLastError();
  if (err != cudaSuccess || !weights || blocks == 1) return err;
  JoinArgs<W> j{};
  j.part = c.partials;
  j.post = static_cast<const W*>(c.post);
  j.gate = static_cast<const W*>(c.gate);
  j.dpost = static_cast<W*>(c.dpost);
  j.dpre = static_cast<W*>(c.dpre);
  j.dgate = static_cast<W*>(c.dgate);
  j.scale = c.d.scale;
  j.offset = c.d.offset;
  j.P = static_cast<int>(blocks);
  j.D = c.d.D;
  cudaLaunchAttribute overlap = overlap_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((2 * static_cast<int64_t>(c.d.D) + kJoinCols - 1) / kJoinCols));
  cfg.blockDim = dim3(kJoinCols * kJoinRows);
  cfg.stream = s;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_norm_join_kernel<W>, j);
}

template <typename T, typename W, int VEC, int NV, bool ONE_WARP, int R, bool SHIFT>
cudaError_t bwd_full(const BlockNormCall& c, cudaStream_t s) {
  if constexpr (VEC > 1) {
    bool full = true;
    for (const void* p : {c.du, c.r_in, c.dr, c.y, static_cast<const void*>(c.dy)}) full = full && p != nullptr;
    for (int64_t ld : {c.lddu, c.ldr, c.lddr, c.ldy, c.lddy}) full = full && ld == c.lddres;
    if (full) return bwd_launch<T, W, VEC, NV, ONE_WARP, R, SHIFT, true>(c, s);
  }
  return bwd_launch<T, W, VEC, NV, ONE_WARP, R, SHIFT, false>(c, s);
}
// Two rows at a time where a thread holds up to eight columns (one against two:
// 32768 x 2816 bf16 202 us and 172, x 1407 134 and 125, 4099 x 1001 fp32 22.1 and 21.0;
// even rows of fp32 are better off with one, 8192 x 2048 64.4 and 68.5, but wide ones
// of odd length and all of 16 bits are not).
template <typename T, typename W, int VEC, bool SHIFT>
cudaError_t bwd_rows(const BlockNormCall& c, cudaStream_t s) {
  const int nvec = SHIFT ? shifted_vectors(c.d.D, VEC) : c.d.D / VEC;
  return pick_nv<VEC, 1>(nvec, 1, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    constexpr int R = NV * VEC <= 8 ? 2 : 1;
    if constexpr (NV == (VEC == 1 ? 4 : 1)) {  // more vectors per thread are only taken by wide rows
      if (nvec <= 32 * NV) return bwd_full<T, W, VEC, NV, true, R, SHIFT>(c, s);
    }
    return bwd_full<T, W, VEC, NV, false, R, SHIFT>(c, s);
  });
}

template <typename T, typename W>
cudaError_t go(const BlockNormCall& c, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  const Rows kind = kind_of_rows<T>(c);
  if (c.dres == nullptr) {
    if (kind == Rows::kVectors) return fwd_rows<T, W, VEC>(c, s);
    if (kind == Rows::kShifted) return fwd_shift<T, W, VEC>(c, s);
    return fwd_rows<T, W, 1>(c, s);
  }
  if (kind == Rows::kVectors) return bwd_rows<T, W, VEC, false>(c, s);
  if (kind == Rows::kShifted) return bwd_rows<T, W, VEC, true>(c, s);
  return bwd_rows<T, W, 1, false>(c, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormCall& c, cudaStream_t s) {
  const bool w32 = c.d.wtype == MOE_FP32;
  switch (c.d.type) {
    case MOE_BF16:
      return w32 ? go<__nv_bfloat16, float>(c, s) : go<__nv_bfloat16, __nv_bfloat16>(c, s);
    case MOE_FP16:
      return w32 ? go<__half, float>(c, s) : go<__half, __half>(c, s);
    default:
      return go<float, float>(c, s);
  }
}

}  // namespace moe
