// Expert selection with a balance bias and group-limited top-k, and its
// backward.
//
//   s_e = sigmoid(l_e) or softmax(l)_e;  sel_e = s_e + bias_e (without a bias
//   the logits themselves order the experts);  the top_groups best groups
//   (by the sum of their group_top best) stay;  ids = the K largest sel left;
//   w_k = scale s_k (/ sum_k s_k).
//   backward: dlogits from dw through the weights (the selection has none).
//
// One warp per token; a lane holds up to `vpl` neighbouring experts in
// registers, and `lpg` lanes hold a group.  Selection without K passes over the
// experts: the K-th largest of the lanes' maxima bounds the K-th largest
// expert from below, so the few experts at or above it (a dozen for 8 of 256)
// hold the answer; they are compacted to one per lane, in the order of their
// ids, and each counts those ahead of it.  Where they do not fit a warp (K
// near 32), K rounds take one warp-wide maximum each.  A few tokens are bound
// by the launch and this chain (16 tokens, 256 experts: 4.1 us).
//
// The selection compares fp32 scores, which a rounding can swap.  Each
// comparison that decides something is therefore checked against the error
// bounds of its two sides: neighbours in the sorted list, the last expert
// taken and every one left out, the groups taken and those left.
// Where they lie too near, those experts (one per lane) or those groups are
// evaluated again in fp64.  With scores spread as in training this happens
// to a token in some thousands.
#include <cuda.h>

#include <algorithm>
#include <cfloat>

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

// The two largest of (a1 >= a2) and (b1 >= b2).
template <typename F>
__device__ __forceinline__ void merge_top2(F& a1, F& a2, F b1, F b2) {
  const F hi = a1 > b1 ? a1 : b1, lo = a1 > b1 ? b1 : a1;
  const F m2 = a2 > b2 ? a2 : b2;
  a1 = hi;
  a2 = lo > m2 ? lo : m2;
}
__device__ __forceinline__ void merge_top2(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fmaxf(a2, b2), fminf(a1, b1));
  a1 = fmaxf(a1, b1);
}
// A group's score from its two best: masked experts (-inf) add nothing to
// one that has others.
__device__ __forceinline__ double group_score(double t1, double t2, int group_top) {
  return (group_top == 2 && t2 > static_cast<double>(kNegInf)) ? t1 + t2 : t1;
}
// The same in fp32, where a sum past the largest number stays ahead of a group
// whose experts are all masked (its error, see group_error, covers the rest).
__device__ __forceinline__ float group_score(float t1, float t2, int group_top) {
  return (group_top == 2 && t2 > kNegInf) ? fminf(fmaxf(t1 + t2, -FLT_MAX), FLT_MAX) : t1;
}

// e^(l - m), with the limit at l = m = +inf and 0 for a masked logit.
__device__ __forceinline__ float soft_num(float l, float m) {
  return l == kNegInf ? 0.0f : (l == m ? 1.0f : expf(l - m));
}

// A token's weights are shares of its K scores, which may all lie below what
// fp32 holds.  Where none of the chosen logits lies within kDeep of `base` (0
// for the sigmoid, the row's largest logit for the softmax), the scores are
// taken relative to the largest chosen one instead, which leaves the shares as
// they are.
constexpr float kDeep = 64.0f;
__device__ __forceinline__ bool shallow(float l, float base) { return l - base >= -kDeep || l == base; }
__device__ __forceinline__ float deep_base(float most, float base) {
  return most > kNegInf && base < INFINITY ? most : base;
}
// sigmoid(l) e^-base, base being 0 or below -kDeep (there the sigmoid is e^l to
// fp32's precision, down to the smallest numbers).
__device__ __forceinline__ float sigmoid_num(float l, float base) {
  return l < -kDeep ? expf(l - base) : 1.0f / (1.0f + expf(-l));
}

// Largest value over the warp, in one instruction (no NaN among them).
__device__ __forceinline__ float warp_max_f32(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// A logit with NaN taken as masked (the maximum of NaN and a number is the number).
__device__ __forceinline__ float clean(float l) { return fmaxf(l, kNegInf); }

// The score of one logit in fp64; m and inv_total are the softmax's.
template <bool SOFTMAX>
__device__ __forceinline__ double score_fp64(float l, double m, double inv_total) {
  const double v = l;
  if (l == kNegInf) return 0.0;
  if constexpr (SOFTMAX) return (v == m ? 1.0 : exp(v - m)) * inv_total;
  else return 1.0 / (1.0 + exp(-v));
}
// Largest logit and 1 / sum of e^(l - m) of a row in fp64, over the warp.
__device__ __noinline__ double2 softmax_fp64(const float* row, int E, int lane) {
  double m = -INFINITY, total = 0.0;
  for (int e = lane; e < E; e += 32) m = fmax(m, static_cast<double>(clean(row[e])));
  for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, o));
  for (int e = lane; e < E; e += 32) {
    const double v = clean(row[e]);
    total += v == -INFINITY ? 0.0 : (v == m ? 1.0 : exp(v - m));
  }
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  return make_double2(m, total > 0.0 ? 1.0 / total : 0.0);
}

// Of the groups in `band`, the `need` best in fp64 (ties: the lowest group).
template <bool SOFTMAX>
__device__ __noinline__ uint32_t groups_fp64(const float* row, const float* bias,
                                             const moe_topk_dims& d, uint32_t band, int need,
                                             int lane) {
  double2 st = make_double2(0.0, 0.0);
  if constexpr (SOFTMAX) st = softmax_fp64(row, d.E, lane);
  const int gs = d.E / d.groups;
  double mine = -INFINITY;
  for (uint32_t left = band; left != 0; left &= left - 1) {
    const int g = __ffs(left) - 1;
    double t1 = -INFINITY, t2 = -INFINITY;
    for (int e = g * gs + lane; e < (g + 1) * gs; e += 32) {
      const float l = clean(row[e]);
      if (l == kNegInf) continue;
      const double v = score_fp64<SOFTMAX>(l, st.x, st.y) + (bias != nullptr ? static_cast<double>(bias[e]) : 0.0);
      merge_top2(t1, t2, v, static_cast<double>(-INFINITY));
    }
    for (int o = 16; o > 0; o >>= 1) {
      const double b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
      merge_top2(t1, t2, b1, b2);
    }
    if (lane == g) mine = group_score(t1, t2, d.group_top);
  }
  int rank = 0;
  for (uint32_t left = band; left != 0; left &= left - 1) {
    const int g = __ffs(left) - 1;
    const double other = __shfl_sync(kAll, mine, g);
    if (other > mine || (other == mine && g < lane)) ++rank;
  }
  return __ballot_sync(kAll, ((band >> lane) & 1u) && rank < need);
}

// Rank in fp64 of this lane's expert `id` (logit l) among those of lanes < n,
// which hold them in any order; ties go to the lowest id, masked ones last.
template <bool SOFTMAX>
__device__ __noinline__ int rank_fp64(const float* row, const float* bias, int E, int id, float l, int n,
                                      int lane) {
  double2 st = make_double2(0.0, 0.0);
  if constexpr (SOFTMAX) st = softmax_fp64(row, E, lane);
  const double sel = l == kNegInf ? -INFINITY
                                  : score_fp64<SOFTMAX>(l, st.x, st.y) +
                                        (lane < n ? static_cast<double>(bias[id]) : 0.0);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double other = __shfl_sync(kAll, sel, j);
    const int o_id = __shfl_sync(kAll, id, j);
    if (other > sel || (other == sel && o_id < id)) ++rank;
  }
  return rank;
}

// The selection of one token in fp64, over the whole warp, among the groups
// in `stay`; returns the id of slot `lane` (lane < K).  Used where the
// candidates do not fit one per lane.
template <int VPL, bool SOFTMAX>
__device__ __noinline__ int select_fp64(const float* row, const float* bias, const moe_topk_dims& d,
                                        int first, int mine, uint32_t stay, int lane) {
  double sel[VPL];
  double2 st = make_double2(0.0, 0.0);
  if constexpr (SOFTMAX) st = softmax_fp64(row, d.E, lane);
  const int gs = d.E / d.groups;
  uint32_t used = 0;  // bit i: expert i of this lane is out
  for (int i = 0; i < VPL; ++i) {
    const int e = first + i;
    sel[i] = -INFINITY;
    if (i >= mine || !((stay >> (e / gs)) & 1u)) {
      used |= 1u << i;
    } else {
      const float l = clean(row[e]);
      if (l != kNegInf) sel[i] = score_fp64<SOFTMAX>(l, st.x, st.y) + static_cast<double>(bias[e]);
    }
  }
  int slot = 0;
  for (int k = 0; k < d.K; ++k) {
    double best = -INFINITY;
    int id = 1 << 30;  // no expert: behind every id
    for (int i = 0; i < VPL; ++i) {
      if (!((used >> i) & 1u) && (id == (1 << 30) || sel[i] > best)) {
        best = sel[i];
        id = first + i;
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
    if (id >= first && id < first + mine) used |= 1u << (id - first);
    if (lane == k) slot = id;
  }
  return slot;
}

// Four values in descending order, and the first of them taken off.
__device__ __forceinline__ void sort4(float (&q)[4]) {
  auto order = [&](int x, int y) {
    const float hi = fmaxf(q[x], q[y]);
    q[y] = fminf(q[x], q[y]);
    q[x] = hi;
  };
  order(0, 1);
  order(2, 3);
  order(0, 2);
  order(1, 3);
  order(1, 2);
}
__device__ __forceinline__ void pop4(float (&q)[4]) {
  q[0] = q[1];
  q[1] = q[2];
  q[2] = q[3];
  q[3] = kNegInf;
}

// The score of a logit that is not -inf, fast.
template <bool SOFTMAX>
__device__ __forceinline__ float quick_score(float v, float m, float inv_total) {
  if constexpr (SOFTMAX) return (v == m ? 1.0f : exp2_fast((v - m) * kLog2e)) * inv_total;
  else return rcp_fast(1.0f + exp2_fast(-kLog2e * v));
}

// Bounds of the error of a fast score (see quick_score): s (6e-7 + 1.5e-7
// max(-l, 0)) for the sigmoid, from the exponential's 2 ulp and its rounded
// argument (1.17 |l| ulp) and the reciprocal's ulp; for the softmax
// s (3e-6 + 2e-7 (m - l)), which includes the error of the sum over experts.
template <bool SOFTMAX>
__device__ __forceinline__ float score_error(float s, float l, float m) {
  return SOFTMAX ? s * (3e-6f + 2e-7f * fmaxf(m - l, 0.0f)) : s * (6e-7f + 1.5e-7f * fmaxf(-l, 0.0f));
}
constexpr float kSumError = 1.2e-7f;  // of the rounded sum s + bias, relative
// Of a group's score, the sum of its best two t1 and t2 (or t1 alone): the
// scores' own errors, their sums with the biases rounded at |t1| and |t2|, and
// the last sum.  The terms count, not their sum, which may be far smaller
// (biases of opposite sign).
__device__ __forceinline__ float group_error(float t1, float t2, int group_top, float worst) {
  const float a = t1 > kNegInf ? fabsf(t1) : 0.0f, b = group_top == 2 && t2 > kNegInf ? fabsf(t2) : 0.0f;
  return 2.0f * worst + (kSumError * a + kSumError * b);
}
// Largest score_error of any logit: (1 - s) is folded in for the sigmoid, and
// s e^-x x <= 0.37 for the softmax, relative to the row's largest score.
template <bool SOFTMAX>
__device__ __forceinline__ float worst_error(float largest) {
  return SOFTMAX ? 3.1e-6f * largest : 6.5e-7f;
}

// Of the score v = s + bias of an expert with logit l; a fast score below
// 2^-126 is 0.
template <bool SOFTMAX>
__device__ __forceinline__ float value_error(float v, float bias, float l, float m) {
  return v > kNegInf ? score_error<SOFTMAX>(v - bias, l, m) + (2.0f * kSumError * fabsf(v) + 1.2e-38f) : 0.0f;
}

// Whether a list of n candidates, sorted by v over the lanes, may be out of
// order as far as its first K: each of those against the next, and each one
// left out against the last one taken (one further down may have a larger
// error than the first).  Equal logits under equal biases are equal in fp64.
template <bool SOFTMAX>
__device__ __forceinline__ bool unsure_order(float v, float bias, float l, float m, int n, int K, int lane) {
  const float err = value_error<SOFTMAX>(v, bias, l, m);
  const int other = lane < K - 1 ? lane + 1 : K - 1;
  const float o_v = __shfl_sync(kAll, v, other), o_b = __shfl_sync(kAll, bias, other);
  const float o_l = __shfl_sync(kAll, l, other), o_err = __shfl_sync(kAll, err, other);
  const bool unsure = lane < n && lane != K - 1 && fabsf(v - o_v) <= err + o_err && !(l == o_l && bias == o_b);
  return __any_sync(kAll, unsure);
}

// Whether one of this lane's experts, taken or not, lies within `reach` (and
// its own rounding) of the last one taken without being equal to it.
template <bool SOFTMAX>
__device__ __noinline__ bool others_near(const float* row, const float* bias, int first, int mine, float m,
                                         float inv_total, float last, float last_l, float last_b, float reach) {
  bool near = false;
  for (int e = first; e < first + mine; ++e) {
    const float l = clean(__ldg(row + e)), b = __ldg(bias + e);
    if (l == kNegInf || (l == last_l && b == last_b)) continue;
    const float f = quick_score<SOFTMAX>(l, m, inv_total) + b;
    near = near || fabsf(last - f) <= reach + 2.0f * kSumError * fabsf(f);
  }
  return near;
}

// One token by a whole warp.  vpl: experts a lane holds at most (<= VPL); lpg:
// lanes of a group; cand: room for 32 (value, id) candidates.
template <int VPL, bool SOFTMAX>
struct WarpToken {
  const TopkArgs& p;
  float2* cand;
  int vpl, lpg, lane, first, mine, group, r;
  // tight: the experts to choose from lie on fewer than 2 K lanes, whose maxima
  // alone would leave too many candidates (2400 tokens, 11 of 512 experts in
  // one of 4 groups: 29 us so, 9.0 with four maxima a lane); few: and are 32
  // at most
  bool vec, tight, few;

  __device__ __forceinline__ WarpToken(const TopkArgs& p_, float2* cand_, int vpl_, int lpg_)
      : p(p_), cand(cand_), vpl(vpl_), lpg(lpg_), lane(threadIdx.x & 31) {
    // this lane's experts: `mine` of them from `first`
    const moe_topk_dims& d = p.d;
    const bool grouped = d.groups > 1 && d.top_groups < d.groups;
    const int gs = grouped ? d.E / d.groups : d.E, staying = grouped ? d.top_groups : 1;
    tight = 2 * d.K > staying * ((gs + vpl - 1) / vpl);
    few = tight && staying * gs <= 32;
    group = lane / lpg;
    r = lane - group * lpg;
    first = group * gs + r * vpl;
    mine = group * gs < d.E ? max(0, min(vpl, gs - r * vpl)) : 0;
    vec = VPL % 4 == 0 && vpl % 4 == 0 && gs % 4 == 0 && d.E % 4 == 0;
  }
  __device__ __forceinline__ void load_bias(float (&b)[VPL]) const {
#pragma unroll
    for (int i = 0; i < VPL; ++i) b[i] = p.bias != nullptr && i < mine ? __ldg(p.bias + first + i) : 0.0f;
  }
  __device__ __forceinline__ void load_row(int64_t t, float (&l)[VPL]) const {
    const float* row = p.logits + t * p.d.E;
    if (vec) {
#pragma unroll
      for (int i = 0; i + 3 < VPL; i += 4) {
        float4 v = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
        if (i < mine) v = __ldg(reinterpret_cast<const float4*>(row + first + i));
        l[i] = v.x;
        l[i + 1] = v.y;
        l[i + 2] = v.z;
        l[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = i < mine ? __ldg(row + first + i) : kNegInf;
    }
  }

  // Selects and writes token t from its row l (NaN not yet taken as masked).
  __device__ __forceinline__ void run(int64_t t, float (&l)[VPL], const float (&b)[VPL]) {
  const moe_topk_dims& d = p.d;
  const int E = d.E, K = d.K;
  const bool biased = p.bias != nullptr;
  const bool grouped = d.groups > 1 && d.top_groups < d.groups;
  const bool by_s = grouped && !biased && d.group_top == 2;  // groups scored by s
  const bool need_total = SOFTMAX && (biased || by_s || !d.renorm);
  const bool pow2 = (lpg & (lpg - 1)) == 0;
  const uint32_t below = (1u << lane) - 1u;
    const float* row = p.logits + t * E;
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = clean(l[i]);

    float m = 0.0f, inv_total = 0.0f;
    if constexpr (SOFTMAX) {
      m = l[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
      m = warp_max_f32(m);
      if (need_total) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          total += l[i] == m && l[i] != kNegInf ? 1.0f : exp2_fast((l[i] - m) * kLog2e);
        total = m == kNegInf ? 0.0f : warp_sum(total);
        inv_total = total > 0.0f ? 1.0f / total : 0.0f;
      }
    }
    auto fast_score = [&](float v) -> float { return quick_score<SOFTMAX>(v, m, inv_total); };
    // the value that orders the experts; masked and absent ones are -inf
    if (biased) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = l[i] == kNegInf ? kNegInf : fast_score(l[i]) + b[i];
    }
    const float worst = worst_error<SOFTMAX>(inv_total);

    uint32_t stay = kAll;  // groups that stay
    bool out = false;      // this lane's group does not
    if (grouped) {
      float t1 = kNegInf, t2 = kNegInf;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        t2 = fmaxf(t2, fminf(t1, l[i]));
        t1 = fmaxf(t1, l[i]);
      }
      if (by_s) {  // scores keep the logits' order
        if (t1 != kNegInf) t1 = fast_score(t1);
        if (t2 != kNegInf) t2 = fast_score(t2);
      }
      if (pow2) {
        for (int o = 1; o < lpg; o <<= 1) {
          const float b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
          merge_top2(t1, t2, b1, b2);
        }
      } else {  // the group's other lanes in turn
        const float own1 = t1, own2 = t2;
        for (int o = 1; o < lpg; ++o) {
          const int src = (group * lpg + (r + o) % lpg) & 31;
          const float b1 = __shfl_sync(kAll, own1, src), b2 = __shfl_sync(kAll, own2, src);
          merge_top2(t1, t2, b1, b2);
        }
      }
      // the score of group `lane`
      const float score = __shfl_sync(kAll, group_score(t1, t2, d.group_top), (lane * lpg) & 31);
      uint32_t gkey = lane < d.groups ? order_key(score) : 0u;
      stay = 0u;
      for (int g = 0; g < d.top_groups; ++g) {
        const uint32_t last = __reduce_max_sync(kAll, gkey);
        const int src = __ffs(__ballot_sync(kAll, gkey == last)) - 1;
        stay |= 1u << src;
        if (lane == src) gkey = 0u;
      }
      if (biased || by_s) {
        // the groups taken, each at its least, against those left, each at its
        // most; those that do not clear the other side are taken again in fp64
        const float err = __shfl_sync(kAll, group_error(t1, t2, d.group_top, worst), (lane * lpg) & 31);
        const bool taken = (stay >> lane) & 1u, left = lane < d.groups && !taken;
        const float least = -warp_max_f32(taken ? err - score : kNegInf);
        const float most = warp_max_f32(left ? score + err : kNegInf);
        if (most > kNegInf && least <= most) {
          const uint32_t band = __ballot_sync(kAll, taken ? score - err <= most : left && score + err >= least);
          const uint32_t sure = stay & ~band;
          stay = sure | groups_fp64<SOFTMAX>(row, p.bias, d, band, d.top_groups - __popc(sure), lane);
        }
      }
      out = !((stay >> group) & 1u);
      if (out) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = kNegInf;
      }
    }

    // a lower bound of the K-th value: the K-th largest of the lanes' maxima,
    // or (tight) of the maxima of every fourth of a lane's experts; none where
    // all experts are candidates
    float bound = kNegInf;
    if (!tight) {
      float rest = l[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) rest = fmaxf(rest, l[i]);
      for (int k = 0; k < K; ++k) {
        bound = warp_max_f32(rest);
        if (rest == bound) rest = kNegInf;
      }
    } else if (!few) {
      float q4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
      for (int i = 0; i < VPL; ++i) q4[i % 4] = fmaxf(q4[i % 4], l[i]);
      sort4(q4);
      for (int k = 0; k < K; ++k) {
        bound = warp_max_f32(q4[0]);
        if (q4[0] == bound) pop4(q4);
      }
    }
    if (biased) bound -= 2.0f * (worst + kSumError * fabsf(bound));  // what may still pass it
    int count = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) count += l[i] >= bound && i < mine ? 1 : 0;
    if (out) count = 0;
    // candidates before this lane's, in the order of the ids
    int at = 0, n = 0;
#pragma unroll
    for (int w = 0; (1 << w) <= VPL; ++w) {
      const uint32_t have = __ballot_sync(kAll, (count >> w) & 1);
      at += __popc(have & below) << w;
      n += __popc(have) << w;
    }
    int my_id = 0;
    if ((few || bound > kNegInf) && n >= K && n <= 32) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (l[i] >= bound && i < mine && !out) cand[at++] = make_float2(l[i], __int_as_float(first + i));
      __syncwarp();
      float v = kNegInf;
      int id = 0;
      if (lane < n) {
        const float2 c = cand[lane];
        v = c.x;
        id = __float_as_int(c.y);
      }
      int rank = 0;
      for (int j = 0; j < n; ++j) {
        const float o = __shfl_sync(kAll, v, j);
        rank += (o > v || (o == v && j < lane)) ? 1 : 0;
      }
      __syncwarp();
      if (lane < n) cand[rank] = make_float2(v, __int_as_float(id));
      __syncwarp();
      if (lane < n) {
        const float2 c = cand[lane];
        v = c.x;
        id = __float_as_int(c.y);
      }
      if (biased) {
        const float bs = lane < n ? __ldg(p.bias + id) : 0.0f;
        const float lo = lane < n ? clean(__ldg(row + id)) : kNegInf;
        if (unsure_order<SOFTMAX>(v, bs, lo, m, n, K, lane)) {
          rank = rank_fp64<SOFTMAX>(row, p.bias, E, id, lo, n, lane);
          if (lane < n) cand[rank] = make_float2(v, __int_as_float(id));
          __syncwarp();
          if (lane < n) id = __float_as_int(cand[lane].y);
        }
      }
      my_id = id;
    } else {
      // K rounds: the warp's largest key, and its lane's next one
      uint32_t key[VPL], ktop = 0u, my_key = 0u;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        key[i] = i < mine && !out ? order_key(l[i]) : 0u;
        ktop = max(ktop, key[i]);
      }
      auto take = [&](uint32_t best) -> int {
        const int src = __ffs(__ballot_sync(kAll, ktop == best)) - 1;
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
          ktop = rest;
        }
        return __shfl_sync(kAll, first + idx, src);
      };
      for (int k = 0; k < K; ++k) {
        const uint32_t best = __reduce_max_sync(kAll, ktop);
        const int id = take(best);
        if (lane == k) {
          my_id = id;
          my_key = best;
        }
      }
      if (biased) {
        const float v = lane < K ? key_value(my_key) : kNegInf, bs = lane < K ? __ldg(p.bias + my_id) : 0.0f;
        const float lo = lane < K ? clean(__ldg(row + my_id)) : kNegInf;
        bool unsure = unsure_order<SOFTMAX>(v, bs, lo, m, K, K, lane);
        // the last one taken against every expert that is left
        const float last = __shfl_sync(kAll, v, K - 1), last_b = __shfl_sync(kAll, bs, K - 1);
        const float last_l = __shfl_sync(kAll, lo, K - 1);
        const float reach = worst + value_error<SOFTMAX>(last, last_b, last_l, m);
        const uint32_t next = __reduce_max_sync(kAll, ktop);
        const float most = next != 0u ? key_value(next) : kNegInf;
        if (most > kNegInf && last - most <= reach + 2.0f * kSumError * fabsf(most))
          unsure = unsure || others_near<SOFTMAX>(row, p.bias, first, out ? 0 : mine, m, inv_total, last, last_l,
                                                  last_b, reach);
        if (__any_sync(kAll, unsure))
          my_id = select_fp64<VPL, SOFTMAX>(row, p.bias, d, first, mine, stay, lane);
      }
    }
    const float my_l = lane < K ? clean(__ldg(row + my_id)) : kNegInf;
    float s = 0.0f, base = m;  // (m is 0 for the sigmoid)
    if (d.renorm && __ballot_sync(kAll, lane < K && shallow(my_l, base)) == 0u)
      base = deep_base(warp_max_f32(my_l), base);
    if (lane < K) {
      if constexpr (SOFTMAX) s = soft_num(my_l, base);
      else s = sigmoid_num(my_l, base);
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
};

template <int VPL, bool SOFTMAX>
__global__ void __launch_bounds__(32 * kTopkWarps)
    route_topk_kernel(const __grid_constant__ TopkArgs p, const int vpl, const int lpg) {
  __shared__ float2 cand[kTopkWarps][32];
  const int warp = threadIdx.x >> 5;
  WarpToken<VPL, SOFTMAX> w(p, cand[warp], vpl, lpg);
  float b[VPL];
  w.load_bias(b);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTopkWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kTopkWarps + warp;
  float ahead[VPL];
  if (t < p.d.T) w.load_row(t, ahead);
  for (; t < p.d.T; t += stride) {
    float l[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = ahead[i];
    if (t + stride < p.d.T) w.load_row(t + stride, ahead);  // the next token's row, meanwhile
    w.run(t, l, b);
  }
}

// --------------------------------------------------- several tokens a warp
// The same selection with LANES = 8 or 16 lanes to a token: most of a token's
// instructions are not its experts' but the selection's, which a few lanes
// share as well as thirty-two do.  A lane
// holds up to 32 experts; the bound comes from the best of each quarter of
// a lane's (every fourth expert), and the candidates (up to 32) are ranked through shared memory.  A token whose
// candidates do not fit, and one with near ties, is finished by the whole
// warp.  Bound by latency (96 registers leave 20 warps an SM, which issue in
// half of the cycles).  32768 tokens, 256 experts in 8 groups: 8 taken 27 us,
// 38 us with a token a warp; 16 taken 39 and 46 (5600 tokens: 12.3 and 13.2).
template <int LANES>
__device__ __forceinline__ float sub_max(float v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int LANES>
__device__ __forceinline__ float sub_sum(float v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// A token that the packed kernel leaves to the whole warp, with VPL experts to
// a lane at most.
template <int VPL, bool SOFTMAX>
__device__ __noinline__ void whole_warp_token(const TopkArgs& p, float2* cand, int vpl, int lpg,
                                              int64_t t) {
  WarpToken<VPL, SOFTMAX> w(p, cand, vpl, lpg);
  float b[VPL], l[VPL];
  w.load_bias(b);
  w.load_row(t, l);
  w.run(t, l, b);
}

// The order of a token's n sorted candidates, checked against the bounds of
// their scores and redone in fp64 where that fails.  Whole warp.
template <bool SOFTMAX>
__device__ __noinline__ void settle_order(const float* row, const float* bias, int E, int K, float2* cand,
                                          int n, float m, int lane) {
  float v = kNegInf, bs = 0.0f, lo = kNegInf;
  int id = 0;
  if (lane < n) {
    v = cand[lane].x;
    id = __float_as_int(cand[lane].y);
    bs = __ldg(bias + id);
    lo = clean(__ldg(row + id));
  }
  if (!unsure_order<SOFTMAX>(v, bs, lo, m, n, K, lane)) return;
  const int rank = rank_fp64<SOFTMAX>(row, bias, E, id, lo, n, lane);
  __syncwarp();
  if (lane < n) cand[rank] = make_float2(v, __int_as_float(id));
  __syncwarp();
}

// Experts of a lane when the whole warp takes a token over.
__host__ __device__ constexpr int packed_warp_vpl(int lanes, int vpl) { return lanes == 16 && vpl == 32 ? 16 : 8; }

template <int LANES, int VPL, bool SOFTMAX>
__global__ void __launch_bounds__(32 * kTopkWarps)
    route_topk_packed_kernel(const __grid_constant__ TopkArgs p, const int vpl, const int lpg,
                             const int warp_vpl, const int warp_lpg, const bool few) {
  constexpr int kTokens = 32 / LANES, kEach = 32 / LANES;  // tokens a warp, candidates a lane
  constexpr uint32_t kTokenMask = LANES == 32 ? kAll : (1u << LANES) - 1u;
  constexpr int kRow = VPL + 4;  // a lane's part of a row: 16-byte accesses without bank conflicts
  __shared__ __align__(16) float rows[kTopkWarps][32][kRow];
  __shared__ __align__(16) float bias[LANES][kRow];
  __shared__ float2 cands[kTopkWarps][kTokens][32];
  const moe_topk_dims& d = p.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = lane / LANES, r = lane % LANES;
  const int E = d.E, K = d.K;
  const bool biased = p.bias != nullptr;
  const bool grouped = d.groups > 1 && d.top_groups < d.groups;
  const bool by_s = grouped && !biased && d.group_top == 2;
  const bool need_total = SOFTMAX && (biased || by_s || !d.renorm);
  const int gs = grouped ? E / d.groups : E;
  const int group = r / lpg, part = r - group * lpg;
  const int first = group * gs + part * vpl;
  const int mine = group * gs < E ? max(0, min(vpl, gs - part * vpl)) : 0;
  const bool vec = vpl % 4 == 0 && gs % 4 == 0 && E % 4 == 0;
  if (biased) {
    for (int k = threadIdx.x; k < LANES * VPL; k += 32 * kTopkWarps) {
      const int q = k / VPL, i = k % VPL;
      const int e = (q / lpg) * gs + (q % lpg) * vpl + i;
      bias[q][i] = i < vpl && e < E ? __ldg(p.bias + e) : 0.0f;
    }
    __syncthreads();
  }
  float2* cand = cands[warp][tok];
  float* own_row = rows[warp][lane];
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTopkWarps * kTokens;
  for (int64_t base = (static_cast<int64_t>(blockIdx.x) * kTopkWarps + warp) * kTokens; base < d.T;
       base += stride) {
    const int64_t t = base + tok;
    const bool real = t < d.T;
    const float* row = p.logits + (real ? t : d.T - 1) * E;
    float l[VPL];
    if (vec) {
#pragma unroll
      for (int i = 0; i < VPL; i += 4) {
        float4 v = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
        if (i < mine) v = __ldg(reinterpret_cast<const float4*>(row + first + i));
        l[i] = clean(v.x);
        l[i + 1] = clean(v.y);
        l[i + 2] = clean(v.z);
        l[i + 3] = clean(v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = i < mine ? clean(__ldg(row + first + i)) : kNegInf;
    }
    float m = 0.0f, inv_total = 0.0f;
    if constexpr (SOFTMAX) {
      m = l[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
      m = sub_max<LANES>(m);
      if (need_total) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          total += l[i] == m && l[i] != kNegInf ? 1.0f : exp2_fast((l[i] - m) * kLog2e);
        total = sub_sum<LANES>(total);
        inv_total = m != kNegInf ? 1.0f / total : 0.0f;
      }
    }
    auto fast_score = [&](float v) -> float { return quick_score<SOFTMAX>(v, m, inv_total); };
    if (biased) {
#pragma unroll
      for (int i = 0; i < VPL; i += 4) {
        const float4 b = *reinterpret_cast<const float4*>(&bias[r][i]);
        l[i] = l[i] == kNegInf ? kNegInf : fast_score(l[i]) + b.x;
        l[i + 1] = l[i + 1] == kNegInf ? kNegInf : fast_score(l[i + 1]) + b.y;
        l[i + 2] = l[i + 2] == kNegInf ? kNegInf : fast_score(l[i + 2]) + b.z;
        l[i + 3] = l[i + 3] == kNegInf ? kNegInf : fast_score(l[i + 3]) + b.w;
      }
    }
    const float worst = worst_error<SOFTMAX>(inv_total);

    // the best of each quarter of the lane's experts, then in order
    float q4[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      q4[c] = l[c];
#pragma unroll
      for (int i = c + 4; i < VPL; i += 4) q4[c] = fmaxf(q4[c], l[i]);
    }
    bool out = mine == 0;
    if (grouped) {
      float t1 = kNegInf, t2 = kNegInf;
      if (d.group_top == 2) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          t2 = fmaxf(t2, fminf(t1, l[i]));
          t1 = fmaxf(t1, l[i]);
        }
        if (by_s) {  // scores keep the logits' order
          if (t1 != kNegInf) t1 = fast_score(t1);
          if (t2 != kNegInf) t2 = fast_score(t2);
        }
      } else {
        t1 = fmaxf(fmaxf(q4[0], q4[1]), fmaxf(q4[2], q4[3]));
      }
      for (int o = 1; o < lpg; o <<= 1) {
        const float b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
        merge_top2(t1, t2, b1, b2);
      }
      const float score = group < d.groups ? group_score(t1, t2, d.group_top) : kNegInf;
      int ahead = 0;  // groups before this lane's
      for (int o = lpg; o < LANES; o += lpg) {
        const int q = (r + o) % LANES;
        const float other = __shfl_sync(kAll, score, tok * LANES + q);
        if (q / lpg < d.groups && (other > score || (other == score && q / lpg < group))) ++ahead;
      }
      bool stays = group < d.groups && ahead < d.top_groups;
      if (biased || by_s) {
        const bool left_out = group < d.groups && !stays;
        const float gerr = group_error(t1, t2, d.group_top, worst);
        const float least = -sub_max<LANES>(stays ? gerr - score : kNegInf);
        const float most = sub_max<LANES>(left_out ? score + gerr : kNegInf);
        const bool near = real && most > kNegInf && least <= most;
        uint32_t left = __ballot_sync(kAll, near);
        while (left != 0) {  // a token at a time, by the whole warp
          const int q = (__ffs(left) - 1) / LANES;
          left &= ~(kTokenMask << (q * LANES));
          const bool mineq = tok == q && group < d.groups;
          const bool in_band = mineq && (stays ? score - gerr <= most : score + gerr >= least);
          const uint32_t band = __reduce_or_sync(kAll, in_band ? 1u << group : 0u);
          const uint32_t sure = __reduce_or_sync(kAll, mineq && stays && !in_band ? 1u << group : 0u);
          const uint32_t stay = sure | groups_fp64<SOFTMAX>(p.logits + (base + q) * E, p.bias, d, band,
                                                            d.top_groups - __popc(sure), lane);
          if (mineq) stays = (stay >> group) & 1u;
        }
      }
      out = out || !stays;
    }
    // a lower bound of the K-th value: the K-th largest of the quarters' bests
    // (none where there are fewer of those: then all experts are candidates)
    if (out) q4[0] = q4[1] = q4[2] = q4[3] = kNegInf;
    sort4(q4);
    float bound = kNegInf;
    for (int k = 0; k < K && !few; ++k) {
      bound = sub_max<LANES>(q4[0]);
      if (q4[0] == bound) pop4(q4);
    }
    const bool bounded = few || bound > kNegInf;
    if (biased) bound -= 2.0f * (worst + kSumError * fabsf(bound));
    uint32_t mask = 0u;  // the lane's candidates
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (l[i] >= bound) mask |= 1u << i;
    if (mine < 32) mask &= (1u << mine) - 1u;
    if (out || !bounded) mask = 0u;
    const int count = __popc(mask);
    int upto = count;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
      const int v = __shfl_up_sync(kAll, upto, o, LANES);
      if (r >= o) upto += v;
    }
    const int n = __shfl_sync(kAll, upto, LANES - 1, LANES);
    const bool good = real && bounded && n >= K && n <= 32;
    __syncwarp();
    if (good && mask != 0u) {  // candidates one by one: their values through shared memory
#pragma unroll
      for (int i = 0; i < VPL; i += 4)
        *reinterpret_cast<float4*>(own_row + i) = make_float4(l[i], l[i + 1], l[i + 2], l[i + 3]);
      int at = upto - count;
      while (mask != 0u) {
        const int i = __ffs(mask) - 1;
        mask &= mask - 1u;
        cand[at++] = make_float2(own_row[i], __int_as_float(first + i));
      }
    }
    __syncwarp();
    const int most = __reduce_max_sync(kAll, good ? n : 0);
    float v[kEach];
    int id[kEach], rank[kEach];
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
      v[c] = kNegInf;
      id[c] = rank[c] = 0;
      if (good && c * LANES + r < n) {
        const float2 q = cand[c * LANES + r];
        v[c] = q.x;
        id[c] = __float_as_int(q.y);
      }
    }
    // candidates lie in the order of their ids, so that an equal one counts as
    // ahead exactly where it lies before
#pragma unroll
    for (int w = 0; w < kEach; ++w) {
      if (w * LANES >= most) break;
      const int upper = min(LANES, most - w * LANES);
      for (int j = 0; j < upper; ++j) {
        const float o = w * LANES + j < n ? cand[w * LANES + j].x : kNegInf;
#pragma unroll
        for (int c = 0; c < kEach; ++c) {
          if (c < w) rank[c] += o > v[c] ? 1 : 0;
          else if (c > w) rank[c] += o >= v[c] ? 1 : 0;
          else rank[c] += (o > v[c] || (o == v[c] && j < r)) ? 1 : 0;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kEach; ++c)
      if (good && c * LANES + r < n) cand[rank[c]] = make_float2(v[c], __int_as_float(id[c]));
    __syncwarp();
    if (biased) {
      bool near = false;
      if (good && r < K && r + 1 < n) {
        const float a = cand[r].x, b = cand[r + 1].x;
        near = a - b <= 2.0f * (worst + kSumError * (fabsf(a) + fabsf(b)));
      }
      uint32_t left = __ballot_sync(kAll, near);
      while (left != 0) {
        const int q = (__ffs(left) - 1) / LANES;
        left &= ~(kTokenMask << (q * LANES));
        settle_order<SOFTMAX>(p.logits + (base + q) * E, p.bias, E, K, cands[warp][q],
                              __shfl_sync(kAll, n, q * LANES), __shfl_sync(kAll, m, q * LANES), lane);
      }
    }
    const bool slot = good && r < K;
    const int my_id = slot ? __float_as_int(cand[r].y) : 0;
    const float my_l = slot ? clean(__ldg(row + my_id)) : kNegInf;
    float s = 0.0f, base_l = m;  // (m is 0 for the sigmoid)
    if (d.renorm) {
      const uint32_t some = __ballot_sync(kAll, slot && shallow(my_l, base_l));
      bool all = true;
#pragma unroll
      for (int q = 0; q < kTokens; ++q) all = all && ((some >> (q * LANES)) & kTokenMask) != 0u;
      if (!all) {
        const float most = sub_max<LANES>(my_l);
        if (((some >> (tok * LANES)) & kTokenMask) == 0u) base_l = deep_base(most, base_l);
      }
    }
    if (slot) {
      if constexpr (SOFTMAX) s = soft_num(my_l, base_l);
      else s = sigmoid_num(my_l, base_l);
    }
    if (d.renorm) {
      const float total = sub_sum<LANES>(s);
      s = total > 0.0f ? s / total : 0.0f;
    } else if constexpr (SOFTMAX) {
      s *= inv_total;
    }
    if (slot) {
      p.ids[t * K + r] = my_id;
      p.w[t * K + r] = s * d.scale;
    }
    uint32_t rest = __ballot_sync(kAll, real && !good && r == 0);
    while (rest != 0) {
      const int q = (__ffs(rest) - 1) / LANES;
      rest &= rest - 1u;
      whole_warp_token<packed_warp_vpl(LANES, VPL), SOFTMAX>(p, cands[warp][0], warp_vpl, warp_lpg, base + q);
      __syncwarp();
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
// The K values overwrite the row's after a warp barrier.  The loads of a warp's
// next token are under way while it works on this one; what is left is the
// chain of dependent sums and the gather of the chosen logits (DRAM is busy a
// fifth of the time, issue half): 32768 x 128, softmax, 9.5 us (36 MB, 5.3 us
// of HBM); sigmoid with renorm 10.2 us.
template <int VPL, bool DENSE>
__global__ void __launch_bounds__(32 * kTopkWarps) route_topk_bwd_kernel(const TopkBwdArgs p) {
  const moe_topk_dims d = p.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = d.E, K = d.K;
  const bool vec = VPL % 4 == 0 && E % 4 == 0;
  const bool softmax = d.gate == MOE_GATE_SOFTMAX;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTopkWarps;
  int next_id = -1;
  float next_dw = 0.0f, ahead[VPL];
  auto fetch = [&](int64_t t) {
    if (t >= d.T) return;
    if (lane < K) {
      next_id = __ldg(p.ids + t * K + lane);
      next_dw = __ldg(p.dw + t * K + lane);
    }
    if constexpr (DENSE) {
      const float* row = p.logits + t * E;
      if (vec) {
#pragma unroll
        for (int i = 0; i + 3 < VPL; i += 4) {
          const int e = lane * VPL + i;
          float4 q = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
          if (e < E) q = __ldg(reinterpret_cast<const float4*>(row + e));
          ahead[i] = q.x;
          ahead[i + 1] = q.y;
          ahead[i + 2] = q.z;
          ahead[i + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = lane * VPL + i;
          ahead[i] = e < E ? __ldg(row + e) : kNegInf;
        }
      }
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * kTopkWarps + warp;
  fetch(t);
  for (; t < d.T; t += stride) {
    float* out = p.dlogits + t * E;
    const int id = lane < K && next_id >= 0 && next_id < E ? next_id : -1;
    const float g = id >= 0 ? next_dw * d.scale : 0.0f;
    const float l = id >= 0 ? clean(__ldg(p.logits + t * E + id)) : kNegInf;
    float v[VPL];
    if constexpr (DENSE) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = clean(ahead[i]);
    }
    fetch(t + stride);
    float base = 0.0f, value;
    if constexpr (DENSE) {
      float m = v[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = fmaxf(m, v[i]);
      m = warp_max_f32(m);
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        v[i] = v[i] == m && m != kNegInf ? 1.0f : exp2_fast((v[i] - m) * kLog2e);
        total += v[i];
      }
      total = m == kNegInf ? 0.0f : warp_sum(total);
      const float inv = total > 0.0f ? 1.0f / total : 0.0f;
      const float s = soft_num(l, m) * inv;
      const float dot = warp_sum(g * s);
      base = -dot * inv;  // times e^(l - m)
      value = s * (g - dot);
      if (m == kNegInf) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = 0.0f;
      }
    } else if (softmax) {
      // shares of the selected experts: the sum over all others cancels
      const float m = warp_max_f32(l);
      const float e = soft_num(l, m);
      const float total = warp_sum(e);
      const float q = total > 0.0f ? e / total : 0.0f;
      value = q * (g - warp_sum(g * q));
    } else {
      float top = 0.0f;
      if (d.renorm && __ballot_sync(kAll, shallow(l, top)) == 0u) top = deep_base(warp_max_f32(l), top);
      const float s = sigmoid_num(l, top);
      if (d.renorm) {
        const float total = warp_sum(s);
        const float q = total > 0.0f ? s / total : 0.0f;
        const float dot = warp_sum(g * q);
        value = total > 0.0f ? q * (g - dot) : 0.0f;
      } else {
        value = g * s;
      }
      value *= 1.0f / (1.0f + expf(l));  // 1 - s without cancellation
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

// Blocks: a warp per token, at most per_sm blocks per SM (a warp that takes a
// few tokens reads the next one's row ahead; of 4 to 64 blocks these measured
// best at 32768 tokens).
unsigned topk_grid(int T, int per_sm) {
  const int64_t want = (static_cast<int64_t>(T) + kTopkWarps - 1) / kTopkWarps;
  return static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(sm_count()) * per_sm));
}

// Calls go(n) with the smallest compiled capacity for vpl experts per lane.
template <class Go>
void pick_vpl(int vpl, Go go) {
  using std::integral_constant;
  if (vpl <= 1) go(integral_constant<int, 1>{});
  else if (vpl <= 2) go(integral_constant<int, 2>{});
  else if (vpl <= 4) go(integral_constant<int, 4>{});
  else if (vpl <= 8) go(integral_constant<int, 8>{});
  else if (vpl <= 16) go(integral_constant<int, 16>{});
  else go(integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_route_topk(const float* logits, const float* bias, int32_t* ids, float* w,
                              const moe_topk_dims& d, cudaStream_t s) {
  const TopkArgs a{logits, bias, ids, w, d};
  const bool grouped = d.groups > 1 && d.top_groups < d.groups;
  const int lpg = grouped ? topk_group_lanes(d) : 32;
  const int gs = grouped ? d.E / d.groups : d.E;
  const int vpl = (gs + lpg - 1) / lpg;
  // Several tokens a warp, where the experts, groups and slots fit LANES lanes
  // and the lanes whose groups stay offer K values for the bound (a lane's
  // experts in four quarters) or few enough experts to need none.
  auto packed = [&](auto lanes) -> bool {
    constexpr int LANES = decltype(lanes)::value;
    int lp = LANES;
    if (grouped) {
      lp = d.groups <= LANES ? LANES / d.groups : 0;
      while (lp & (lp - 1)) lp &= lp - 1;  // a power of two
    }
    const int vp = lp > 0 ? (gs + lp - 1) / lp : 33;
    if (vp > 32 || d.K > LANES) return false;
    const int staying = grouped ? d.top_groups : 1;
    int offered = 0;
    for (int r = 0; r < lp; ++r) offered += std::max(0, std::min({4, vp, gs - r * vp}));
    // 32 experts at most to choose from: ranking them all costs less than the
    // bound for more than eight of them (30000 tokens, 16 of one of 4 groups of
    // 32: 26.4 us, 32.1 with it), more for fewer (28006, 5 of 16: 9.4 and 8.1)
    const bool few = staying * gs <= 32 && (LANES == 16 || d.K > staying * offered);
    if (!few && d.K > staying * offered) return false;
    if (vpl > packed_warp_vpl(LANES, vp > 16 ? 32 : 16)) return false;
    const unsigned grid = topk_grid((d.T + 32 / LANES - 1) / (32 / LANES), LANES == 8 ? 12 : 6);
    pick_vpl(vp, [&](auto n) {
      constexpr int VPL = decltype(n)::value < 4 ? 4 : decltype(n)::value;
      if (d.gate == MOE_GATE_SOFTMAX)
        route_topk_packed_kernel<LANES, VPL, true><<<grid, 32 * kTopkWarps, 0, s>>>(a, vp, lp, vpl, lpg, few);
      else
        route_topk_packed_kernel<LANES, VPL, false><<<grid, 32 * kTopkWarps, 0, s>>>(a, vp, lp, vpl, lpg, few);
    });
    return true;
  };
  // below this a token a warp fills the SMs better (256 experts in 8 groups, 8
  // taken: 2400 tokens 7.0 us, 8.2 packed; 4000 9.9 and 9.8; 8000 13.1 and
  // 11.6; 512 experts, 8 taken, 4000: 12.0 and 9.2)
  if (d.T >= 24 * static_cast<int64_t>(sm_count()) &&
      ((d.K <= 8 && packed(std::integral_constant<int, 8>{})) || packed(std::integral_constant<int, 16>{})))
    return cudaGetLastError();
  const unsigned grid = topk_grid(d.T, 12);
  pick_vpl(vpl, [&](auto n) {
    constexpr int VPL = decltype(n)::value;
    if (d.gate == MOE_GATE_SOFTMAX)
      route_topk_kernel<VPL, true><<<grid, 32 * kTopkWarps, 0, s>>>(a, vpl, lpg);
    else
      route_topk_kernel<VPL, false><<<grid, 32 * kTopkWarps, 0, s>>>(a, vpl, lpg);
  });
  return cudaGetLastError();
}

cudaError_t launch_route_topk_bwd(const float* logits, const int32_t* ids, const float* dw,
                                  float* dlogits, const moe_topk_dims& d, cudaStream_t s) {
  const TopkBwdArgs a{logits, ids, dw, dlogits, d};
  const bool dense = d.gate == MOE_GATE_SOFTMAX && !d.renorm;
  const unsigned grid = topk_grid(d.T, dense ? 8 : 12);
  pick_vpl((d.E + 31) / 32, [&](auto n) {
    constexpr int VPL = decltype(n)::value;
    if (dense) route_topk_bwd_kernel<VPL, true><<<grid, 32 * kTopkWarps, 0, s>>>(a);
    else route_topk_bwd_kernel<VPL, false><<<grid, 32 * kTopkWarps, 0, s>>>(a);
  });
  return cudaGetLastError();
}

}  // namespace moe
