// Expert selection with a balance bias and group-limited top-k, and its
// backward.
//
//   s_e = sigmoid(l_e) or softmax(l)_e;  sel_e = s_e + bias_e (without a bias
//   the logits themselves order the experts);  the top_groups best groups
//   (by the sum of their group_top best) stay;  ids = the K largest sel left;
//   w_k = scale s_k (/ sum_k s_k).
//   backward: dlogits from dw through the weights (the selection has none).
//
// One warp per token, lane i holding experts [i VPL, (i+1) VPL) in registers:
// the row is read once with 16-byte loads, and each of the K rounds takes the
// largest key of the warp with one warp-wide maximum (the lowest lane, and in
// it the lowest index, wins a tie, which is the lowest expert id).
//
// The selection compares fp32 scores, which a rounding can swap.  Each
// comparison that decides something (neighbours in the list, the last expert
// taken against the first left out, the last group taken against the first
// left out) is therefore checked against the error bound of the two scores;
// where they lie too near, the warp selects the token again in fp64.  With
// scores spread as in training this happens to a token in some thousands.
#include <cuda.h>

#include <algorithm>

#include "kernels.h"
#include "layer.h"
#include "layer_common.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTopkWarps = 4;
constexpr float kNegInf = -INFINITY;

struct TopkArgs {
  const float *logits, *bias;
  int32_t* ids;
  float* w;
  moe_topk_dims d;
};

// fp32 -> a 32-bit key of the same order (0 lies below every key).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 and +0 tie
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// The two largest of (a1 >= a2) and (b1 >= b2).
template <typename F>
__device__ __forceinline__ void merge_top2(F& a1, F& a2, F b1, F b2) {
  const F hi = a1 > b1 ? a1 : b1, lo = a1 > b1 ? b1 : a1;
  const F m2 = a2 > b2 ? a2 : b2;
  a1 = hi;
  a2 = lo > m2 ? lo : m2;
}
// A group's score from its two best: masked experts (-inf) add nothing to
// one that has others.
template <typename F>
__device__ __forceinline__ F group_score(F t1, F t2, int group_top) {
  return (group_top == 2 && t2 > static_cast<F>(kNegInf)) ? t1 + t2 : t1;
}

// e^(l - m), with the limit at l = m = +inf and 0 for a masked logit.
__device__ __forceinline__ float soft_num(float l, float m) {
  return l == kNegInf ? 0.0f : (l == m ? 1.0f : expf(l - m));
}

// The selection of one token in fp64, over the whole warp; returns the id of
// slot `lane` (lane < K).
template <int VPL, bool SOFTMAX>
__device__ __noinline__ int select_fp64(const float* row, const float* bias, const moe_topk_dims& d,
                                        int lane) {
  double sel[VPL], s[VPL];
  const double ninf = -INFINITY;
  double m = ninf;
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    float l = e < d.E ? row[e] : kNegInf;
    if (!(l > kNegInf)) l = kNegInf;
    s[i] = l;
    m = fmax(m, s[i]);
  }
  if (SOFTMAX) {
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, o));
    double total = 0.0;
    for (int i = 0; i < VPL; ++i) {
      sel[i] = s[i];
      s[i] = s[i] == ninf ? 0.0 : (s[i] == m ? 1.0 : exp(s[i] - m));
      total += s[i];
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    for (int i = 0; i < VPL; ++i) s[i] = total > 0.0 ? s[i] / total : 0.0;
  } else {
    for (int i = 0; i < VPL; ++i) {
      sel[i] = s[i];
      s[i] = s[i] == ninf ? 0.0 : 1.0 / (1.0 + exp(-s[i]));
    }
  }
  const bool by_s = bias == nullptr && d.group_top == 2;  // groups scored by s
  if (bias != nullptr)
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (sel[i] != ninf) sel[i] = s[i] + static_cast<double>(bias[e]);
    }
  uint32_t used = 0;  // bit i: expert i of this lane is out
  for (int i = 0; i < VPL; ++i)
    if (lane * VPL + i >= d.E) used |= 1u << i;
  if (d.groups > 1) {
    const int gs = d.E / d.groups;
    double mine = ninf;
    for (int g = 0; g < d.groups; ++g) {
      double t1 = ninf, t2 = ninf;
      for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        if (e < d.E && e / gs == g)
          merge_top2(t1, t2, sel[i] == ninf ? ninf : (by_s ? s[i] : sel[i]), ninf);
      }
      for (int o = 16; o > 0; o >>= 1) {
        const double b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
        merge_top2(t1, t2, b1, b2);
      }
      if (lane == g) mine = group_score(t1, t2, d.group_top);
    }
    int rank = 0;
    for (int g = 0; g < d.groups; ++g) {
      const double other = __shfl_sync(kAll, mine, g);
      if (other > mine || (other == mine && g < lane)) ++rank;
    }
    const uint32_t stay = __ballot_sync(kAll, lane < d.groups && rank < d.top_groups);
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e < d.E && !((stay >> (e / gs)) & 1u)) used |= 1u << i;
    }
  }
  int mine = 0;
  for (int k = 0; k < d.K; ++k) {
    double best = ninf;
    int id = 1 << 30;  // no expert: behind every id
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (!((used >> i) & 1u) && (id == (1 << 30) || sel[i] > best)) {
        best = sel[i];
        id = e;
      }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const double v = __shfl_xor_sync(kAll, best, o);
      const int j = __shfl_xor_sync(kAll, id, o);
      if (j != (1 << 30) && (id == (1 << 30) || v > best || (v == best && j < id))) {
        best = v;
        id = j;
      }
    }
    if (id / VPL == lane) used |= 1u << (id % VPL);
    if (lane == k) mine = id;
  }
  return mine;
}

// Bounds of the error of a fast score (see fast_score): s (6e-7 + 1.5e-7
// max(-l, 0)) for the sigmoid, from __expf's 2 + 1.17 |x| ulp and
// __fdividef's 2 ulp; for the softmax s (3e-6 + 2e-7 (m - l)), which
// includes the error of the sum over experts.
template <bool SOFTMAX>
__device__ __forceinline__ float score_error(float s, float l, float m) {
  return SOFTMAX ? s * (3e-6f + 2e-7f * fmaxf(m - l, 0.0f)) : s * (6e-7f + 1.5e-7f * fmaxf(-l, 0.0f));
}
constexpr float kSumError = 1.2e-7f;  // of the rounded sum s + bias, relative

template <int VPL, bool SOFTMAX>
__global__ void __launch_bounds__(32 * kTopkWarps) route_topk_kernel(const TopkArgs p) {
  __shared__ float gval[kTopkWarps][VPL * 32];  // only for groups that split a lane's experts
  const moe_topk_dims d = p.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = d.E, K = d.K;
  const bool biased = p.bias != nullptr;
  const bool grouped = d.groups > 1 && d.top_groups < d.groups;
  const bool by_s = !biased && d.group_top == 2;      // groups scored by s
  const bool scored = biased || (grouped && by_s);     // s takes part in the selection
  const bool need_total = SOFTMAX && (scored || !d.renorm);
  const int gs = E / d.groups;
  const int lpg = gs / VPL;  // lanes of a group
  const bool whole_lanes = lpg * VPL == gs && (lpg & (lpg - 1)) == 0;
  const bool vec = VPL % 4 == 0 && E % 4 == 0;
  float b[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    b[i] = biased && e < E ? __ldg(p.bias + e) : 0.0f;
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTopkWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTopkWarps + warp; t < d.T; t += stride) {
    const float* row = p.logits + t * E;
    float l[VPL];
    if (vec) {
#pragma unroll
      for (int i = 0; i + 3 < VPL; i += 4) {
        const int e = lane * VPL + i;
        const float4 v = e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                               : make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
        l[i] = v.x;
        l[i + 1] = v.y;
        l[i + 2] = v.z;
        l[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        l[i] = e < E ? __ldg(row + e) : kNegInf;
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = l[i] > kNegInf ? l[i] : kNegInf;  // NaN too

    float m = 0.0f, inv_total = 0.0f;
    if constexpr (SOFTMAX) {
      float lm = l[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) lm = fmaxf(lm, l[i]);
      m = warp_max(lm);
      if (need_total) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          total += l[i] == kNegInf ? 0.0f : (l[i] == m ? 1.0f : __expf(l[i] - m));
        total = warp_sum(total);
        inv_total = total > 0.0f ? 1.0f / total : 0.0f;
      }
    }
    auto fast_score = [&](float v) -> float {
      if constexpr (SOFTMAX)
        return v == kNegInf ? 0.0f : (v == m ? 1.0f : __expf(v - m)) * inv_total;
      else
        return __fdividef(1.0f, 1.0f + __expf(-v));
    };
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float v = biased && l[i] != kNegInf ? fast_score(l[i]) + b[i] : l[i];
      key[i] = lane * VPL + i < E ? order_key(v) : 0u;
    }
    bool unsure = false;
    if (grouped) {
      float mine = kNegInf;  // the score of group `lane`
      if (whole_lanes) {
        float t1 = kNegInf, t2 = kNegInf;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const float v = by_s ? (l[i] == kNegInf ? kNegInf : fast_score(l[i])) : key_value(key[i]);
          merge_top2(t1, t2, key[i] ? v : kNegInf, kNegInf);
        }
        for (int o = 1; o < lpg; o <<= 1) {
          const float b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
          merge_top2(t1, t2, b1, b2);
        }
        mine = __shfl_sync(kAll, group_score(t1, t2, d.group_top), (lane * lpg) & 31);
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          gval[warp][lane * VPL + i] =
              by_s ? (l[i] == kNegInf ? kNegInf : fast_score(l[i])) : (key[i] ? key_value(key[i]) : kNegInf);
        __syncwarp();
        if (lane < d.groups) {
          float t1 = kNegInf, t2 = kNegInf;
          for (int j = 0; j < gs; ++j) merge_top2(t1, t2, gval[warp][lane * gs + j], kNegInf);
          mine = group_score(t1, t2, d.group_top);
        }
        __syncwarp();
      }
      uint32_t gkey = lane < d.groups ? order_key(mine) : 0u, last = 0u, stay = 0u;
      for (int g = 0; g < d.top_groups; ++g) {
        last = __reduce_max_sync(kAll, gkey);
        const int src = __ffs(__ballot_sync(kAll, gkey == last)) - 1;
        stay |= 1u << src;
        if (lane == src) gkey = 0u;
      }
      if (scored) {
        const float in = key_value(last), out = key_value(__reduce_max_sync(kAll, gkey));
        // two scores a side, each within score_error's largest value
        const float err = SOFTMAX ? 12.5e-6f * inv_total : 2.6e-6f;
        unsure = out > kNegInf && in - out <= err + 2.0f * kSumError * (fabsf(in) + fabsf(out));
      }
      if (whole_lanes) {
        if (!((stay >> (lane / lpg & 31)) & 1u)) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) key[i] = 0u;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = lane * VPL + i;
          if (e < E && !((stay >> (e / gs)) & 1u)) key[i] = 0u;
        }
      }
    }

    // K rounds: the warp's largest key, and its lane's next one
    uint32_t top = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = max(top, key[i]);
    int my_id = 0;
    uint32_t my_key = 0u;
    auto take = [&](uint32_t best) -> int {
      const int src = __ffs(__ballot_sync(kAll, top == best)) - 1;
      int idx = 0;
      if (lane == src) {
        uint32_t rest = 0u;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
          if (key[i] == best) idx = i;  // the lowest such index
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (i == idx) key[i] = 0u;
          rest = max(rest, key[i]);
        }
        top = rest;
      }
      return __shfl_sync(kAll, lane * VPL + idx, src);
    };
    for (int k = 0; k < K; ++k) {
      const uint32_t best = __reduce_max_sync(kAll, top);
      const int id = take(best);
      if (lane == k) {
        my_id = id;
        my_key = best;
      }
    }
    float my_l = lane < K ? __ldg(row + my_id) : kNegInf;
    if (!(my_l > kNegInf)) my_l = kNegInf;
    if (biased) {
      const uint32_t next = __reduce_max_sync(kAll, top);  // the first expert left out
      int next_id = 0;
      float next_l = kNegInf;
      if (next != 0u) {
        next_id = take(next);
        next_l = __ldg(row + next_id);
        if (!(next_l > kNegInf)) next_l = kNegInf;
      }
      const float my_sel = key_value(my_key), my_b = lane < K ? __ldg(p.bias + my_id) : 0.0f;
      float o_sel = __shfl_down_sync(kAll, my_sel, 1);
      float o_l = __shfl_down_sync(kAll, my_l, 1), o_b = __shfl_down_sync(kAll, my_b, 1);
      if (lane == K - 1) {
        o_sel = next != 0u ? key_value(next) : kNegInf;
        o_l = next_l;
        o_b = next != 0u ? __ldg(p.bias + next_id) : 0.0f;
      }
      if (lane < K && o_sel > kNegInf && !(my_l == o_l && my_b == o_b)) {
        const float err = score_error<SOFTMAX>(fast_score(my_l), my_l, m) +
                          score_error<SOFTMAX>(fast_score(o_l), o_l, m) +
                          kSumError * (fabsf(my_sel) + fabsf(o_sel));
        if (my_sel - o_sel <= err) unsure = true;
      }
    }
    if (scored && __any_sync(kAll, unsure)) {
      my_id = select_fp64<VPL, SOFTMAX>(row, p.bias, d, lane);
      my_l = lane < K ? __ldg(row + my_id) : kNegInf;
      if (!(my_l > kNegInf)) my_l = kNegInf;
    }
    float s = 0.0f;
    if (lane < K) {
      if constexpr (SOFTMAX) s = soft_num(my_l, m);
      else s = 1.0f / (1.0f + expf(-my_l));
    }
    if (d.renorm) {
      const float total = warp_sum(s);
      s = total > 0.0f ? s / total : 0.0f;
    } else if constexpr (SOFTMAX) {
      s *= inv_total;
    }
    if (lane < K) {
      p.ids[t * K + lane] = my_id;
      p.w[t * K + lane] = s * d.scale;
    }
  }
}

// ---------------------------------------------------------------- backward
struct TopkBwdArgs {
  const float* logits;
  const int32_t* ids;
  const float* dw;
  float* dlogits;
  moe_topk_dims d;
};

// One warp per token.  Only the softmax without renormalisation has a dense
// gradient (and reads the row); the others write zeros and the K values.
// The K values overwrite the row's after a warp barrier.
template <int VPL, bool DENSE>
__global__ void __launch_bounds__(32 * kTopkWarps) route_topk_bwd_kernel(const TopkBwdArgs p) {
  const moe_topk_dims d = p.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = d.E, K = d.K;
  const bool vec = VPL % 4 == 0 && E % 4 == 0;
  const bool softmax = d.gate == MOE_GATE_SOFTMAX;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTopkWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTopkWarps + warp; t < d.T; t += stride) {
    const float* row = p.logits + t * E;
    float* out = p.dlogits + t * E;
    int id = -1;
    float g = 0.0f, l = kNegInf;
    if (lane < K) {
      id = p.ids[t * K + lane];
      if (id < 0 || id >= E) id = -1;
      if (id >= 0) {
        g = p.dw[t * K + lane] * d.scale;
        l = __ldg(row + id);
        if (!(l > kNegInf)) l = kNegInf;
      }
    }
    float v[VPL];
    float base = 0.0f, value;
    if constexpr (DENSE) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = kNegInf;
      if (vec) {
#pragma unroll
        for (int i = 0; i + 3 < VPL; i += 4) {
          const int e = lane * VPL + i;
          if (e < E) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(row + e));
            v[i] = q.x;
            v[i + 1] = q.y;
            v[i + 2] = q.z;
            v[i + 3] = q.w;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (lane * VPL + i < E) v[i] = __ldg(row + lane * VPL + i);
      }
      float m = kNegInf;
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, v[i]);
      m = warp_max(m);
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        v[i] = v[i] > kNegInf ? soft_num(v[i], m) : 0.0f;
        total += v[i];
      }
      total = warp_sum(total);
      const float inv = total > 0.0f ? 1.0f / total : 0.0f;
      const float s = soft_num(l, m) * inv;
      const float dot = warp_sum(g * s);
      base = -dot * inv;  // times e^(l - m)
      value = s * (g - dot);
    } else if (softmax) {
      // shares of the selected experts: the sum over all others cancels
      const float m = warp_max(l);
      const float e = soft_num(l, m);
      const float total = warp_sum(e);
      const float q = total > 0.0f ? e / total : 0.0f;
      value = q * (g - warp_sum(g * q));
    } else {
      const float s = 1.0f / (1.0f + expf(-l));
      float ds = g;
      if (d.renorm) {
        const float total = warp_sum(s), dot = warp_sum(g * s);
        ds = total > 0.0f ? (g - dot / total) / total : 0.0f;
      }
      value = ds * s * (1.0f / (1.0f + expf(l)));  // 1 - s without cancellation
    }
    if (vec) {
#pragma unroll
      for (int i = 0; i + 3 < VPL; i += 4) {
        const int e = lane * VPL + i;
        if (e < E) {
          float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if constexpr (DENSE)
            q = make_float4(base * v[i], base * v[i + 1], base * v[i + 2], base * v[i + 3]);
          *reinterpret_cast<float4*>(out + e) = q;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        if (e < E) out[e] = DENSE ? base * v[i] : 0.0f;
      }
    }
    __syncwarp();
    if (id >= 0) out[id] = value;
  }
}

unsigned topk_grid(int T) {
  const int64_t want = (static_cast<int64_t>(T) + kTopkWarps - 1) / kTopkWarps;
  return static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(sm_count()) * 16));
}

// Calls go(n) with the experts a lane holds: E / 32 rounded up to a power of two.
template <class Go>
void pick_vpl(int E, Go go) {
  using std::integral_constant;
  if (E <= 32) go(integral_constant<int, 1>{});
  else if (E <= 64) go(integral_constant<int, 2>{});
  else if (E <= 128) go(integral_constant<int, 4>{});
  else if (E <= 256) go(integral_constant<int, 8>{});
  else if (E <= 512) go(integral_constant<int, 16>{});
  else go(integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_route_topk(const float* logits, const float* bias, int32_t* ids, float* w,
                              const moe_topk_dims& d, cudaStream_t s) {
  const TopkArgs a{logits, bias, ids, w, d};
  const unsigned grid = topk_grid(d.T);
  pick_vpl(d.E, [&](auto n) {
    constexpr int VPL = decltype(n)::value;
    if (d.gate == MOE_GATE_SOFTMAX) route_topk_kernel<VPL, true><<<grid, 32 * kTopkWarps, 0, s>>>(a);
    else route_topk_kernel<VPL, false><<<grid, 32 * kTopkWarps, 0, s>>>(a);
  });
  return cudaGetLastError();
}

cudaError_t launch_route_topk_bwd(const float* logits, const int32_t* ids, const float* dw,
                                  float* dlogits, const moe_topk_dims& d, cudaStream_t s) {
  const TopkBwdArgs a{logits, ids, dw, dlogits, d};
  const unsigned grid = topk_grid(d.T);
  const bool dense = d.gate == MOE_GATE_SOFTMAX && !d.renorm;
  pick_vpl(d.E, [&](auto n) {
    constexpr int VPL = decltype(n)::value;
    if (dense) route_topk_bwd_kernel<VPL, true><<<grid, 32 * kTopkWarps, 0, s>>>(a);
    else route_topk_bwd_kernel<VPL, false><<<grid, 32 * kTopkWarps, 0, s>>>(a);
  });
  return cudaGetLastError();
}

}  // namespace moe
