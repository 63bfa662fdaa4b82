// The expert layer for a few tokens, in two kernels: routing, FC1 with SwiGLU
// and FC2, then the weighted combine (with a residual).
//
//   ids, p = top-K of the scores, or given     z[t,k] = x[t] . wi[e_tk]
//   h[t,k] = silu(z[:F]) z[F:]                 out[t] = sum_k p_tk h[t,k] . wo[e_tk] + res[t]
//
// With a few tokens the layer is bound by reading the weights of the experts
// that the tokens name, each once.  So the weights' columns are the 128 side
// of the MMA and the expert's tokens its narrow side (up to 64), and the work
// is cut by weight bytes alone: a phase is a list of tiles of 128 weight
// columns (64 of gate and 64 of up, or 128 of wo), expert by expert, each a
// row of 64-deep blocks of 16 KB.  Each of the grid's CTAs (one to an SM)
// takes every so manieth tile as long as there is one for each, so that
// neighbouring columns are read at the same time; the tiles that are left (all
// of them for one token, some 90) are cut into equal runs of blocks, which
// begin and end inside a tile.  Whole tiles alone would leave a tenth to a
// third of the SMs idle in the last wave.  FC2's tiles, where there are several
// for each CTA, are claimed one by one instead: an SM in a large group of SMs
// gets an eighth less of the memory's rate than one in a small group, so that
// equal shares end 20 us apart for 16 tokens, and whoever is done with FC1 early
// makes up for it here.  The CTA that has a tile's first
// part joins the others to it, in their order: it comes to that part last, the
// others to theirs first, so it need not wait, and results do not depend on
// who was faster.  (Joining by whoever adds the last part took 3 us longer from
// the last product to h.)
//
// One ring of shared memory carries both phases' blocks and keeps 128 KB of
// weights under way, 112 beside the routing tables of 2048 slots, 96 with those of
// a thousand experts too (with 32 KB an SM streams at two thirds of the rate): FC2's
// weights start to stream as soon as FC1's have been asked for, and only the
// rows of h wait, block by block, for the flags that FC1's epilogue sets.  The
// launch is cooperative: CTAs wait (bounded) for one another's flags, so all
// have to be resident.
//
// h is rounded to the operands' type: the tensor core multiplies no wider one,
// and its error, half a step on each of F terms of both signs, is about as large
// as the result's own rounding.  Partial sums, routing weights and the combine are fp32.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "layer.h"
#include "layer_common.cuh"
#include "tmem_share.h"
#include "umma_tile.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 128;                         // weight columns of a tile
constexpr int kWeightStage = kCols * kBlockK * 2;  // 16 KB
// Tokens of a tile: an expert with more of them reads its weights again.  Tiles of
// 16 or 32 for calls that need no more leave the ring more stages and are slower
// all the same (4 tokens of 2816 -> 704: 71.0 us with 16, 67.0 with 64; of 7168 ->
// 2048: 391 and 383; only 24 of 512 -> 192 and 256 experts: 41.2 with 32, 42.3), and
// 256 tokens read too much twice (2816 -> 704: 291 us with 16, 255 with 32, 254).
constexpr int kTokens = 64;
constexpr int kStage = kWeightStage + kTokens * kBlockK * 2;  // 24 KB
constexpr int kTmemCols = 2 * kTokens;
constexpr int kMaxStages = 9;
constexpr int kMinStages = 3;
constexpr int kBufLd = kCols + 4;
constexpr int kBufBytes = 16 * kBufLd * 4;  // 16 tokens of a tile
constexpr size_t kSmemLimit = 227 * 1024;
constexpr int kFirstEpiWarp = 4;
constexpr uint16_t kNone = 0xffff;
constexpr int kQueue = 4;
constexpr int kQueueReaders = 1 + 1 + 4;
static_assert(!fits_beside_pair(kMinStages * kStage),
              "CTAs that wait for one another must not fit beside a pair's: tmem_share.h");

// What the combine reads and writes.
struct CombineParams {
  const uint2* slots;  // [n * K]: slot_word, the weight's bits; [n * K].x: virtual experts
  const float *y, *part;
  const void* res;
  void* out;
  int64_t ldres, ldout;
  int n, D, F, K;
  uint32_t grid;  // of the first kernel
};

struct Params {
  const float *logits, *bias, *w_in;
  const int32_t* ids_in;
  int32_t* ids_out;
  float* w_out;
  int n, D, E, K, F;  // n: tokens of this call
  int mode;
  uint32_t k_inverse;  // 2^16 / K, rounded up: slot * k_inverse >> 16 = slot / K for slots below 2048
  int stages;
  uint32_t type;      // of the instruction descriptor
  void* h;            // [n * K][F]
  float* y;           // [n * K][D]: FC2's rows of tiles that one CTA summed alone
  float* part;        // [2 phases][CTA][head, tail][kTokens][128]: sums of parts of tiles
  uint2* slots;       // for the combine's kernel
  int32_t* gids;      // [n * K] and its weights: selections that the CTAs exchange
  float* gw;
  int32_t* claimed;   // tiles of FC2 that CTAs took
  int32_t* leave;     // CTAs that read no more flags
  int32_t* routed;    // tokens whose selection is stored
  int32_t* done;      // [tile of FC1]: its h is stored
  int32_t* stored;    // [CTA]: its part of an FC1 tile that began before its run is stored
  int32_t* status;
  uint64_t limit_ns;
};

struct Ctl {
  uint64_t fullw[kMaxStages];  // a stage's weights landed
  uint64_t fullt[kMaxStages];  // ... and its tokens' rows
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint32_t tmem_base;
  int abort_flag;
  uint2 warp_sums[kThreads / 32];
  uint64_t qfull[kQueue];   // a claimed tile is in the queue
  uint64_t qempty[kQueue];  // ... and has been read by the tokens', products' and epilogue's warps
  uint32_t qtile[kQueue];
};

// The routing, in shared memory.  Slot j = t * K + k.  An expert with more than
// kTokens slots makes several entries of the list that the tiles follow ("virtual
// experts").
struct Route {
  float* w;  // [R]: block 0's weights, or (all blocks', up to kWarps tokens that select) scores
  uint16_t *expert, *rank, *at, *list;       // [R]; at: the slot's virtual expert
  uint16_t *vexp, *vstart, *vcnt;            // [V]
  uint16_t* before;                          // [warps][E]: slots of the expert in the warps ahead
  uint16_t *first, *start;                   // [E]: its first virtual expert, its place in the list
};
constexpr int kWarps = kThreads / 32;
__host__ __device__ inline int most_virtual(int R, int E) {
  const int v = E + R / kTokens;
  return v < R ? v : R;
}
__host__ __device__ inline size_t route_bytes(int R, int E) {
  const size_t half = 4 * static_cast<size_t>(R) + 3 * static_cast<size_t>(most_virtual(R, E)) +
                      (kWarps + 2) * static_cast<size_t>(E);
  return 4 * static_cast<size_t>(R) + (half * 2 + 15) / 16 * 16;
}
__device__ __forceinline__ Route route_at(uint8_t* p, int R, int E) {
  const int V = most_virtual(R, E);
  Route r;
  r.w = reinterpret_cast<float*>(p);
  uint16_t* q = reinterpret_cast<uint16_t*>(p + 4 * static_cast<size_t>(R));
  auto take = [&](int count) {
    uint16_t* a = q;
    q += count;
    return a;
  };
  r.expert = take(R);
  r.rank = take(R);
  r.at = take(R);
  r.list = take(R);
  r.vexp = take(V);
  r.vstart = take(V);
  r.vcnt = take(V);
  r.before = take(kWarps * E);
  r.first = take(E);
  r.start = take(E);
  return r;
}

__device__ __forceinline__ int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(int32_t* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Between generic and asynchronous (TMA) accesses to global memory.
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
// Adds to a counter; what this thread has seen written is written before, and
// what others had written before they added is seen after.
__device__ __forceinline__ int add_acq_rel(int32_t* p, int v) {
  int before;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(before) : "l"(p), "r"(v) : "memory");
  return before;
}

// Waits until *at is `want`, for wc's limit.
__device__ __forceinline__ bool wait_for(const int32_t* at, int want, const WaitCtl& wc) {
  if (ld_acquire(at) == want) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1; it < kMaxWaitIters; ++it) {
    if (ld_acquire(at) == want) return true;
    if ((it & 31u) == 0) {
      if (*wc.abort) return false;
      if (global_timer_ns() - t0 > wc.limit_ns) break;
    }
  }
  *wc.abort = 1;
  report(wc.status, MOE_ERR_TIMEOUT);
  return false;
}

// A slot as the combine reads it: its virtual expert, its row there, and
// whether it names an expert at all.
__device__ __forceinline__ uint32_t slot_word(uint32_t v, uint32_t row) { return 0x80000000u | row << 16 | v; }

// A score as an unsigned number of the same order (-0 as +0).
__device__ __forceinline__ uint32_t order_of(float v) {
  uint32_t u = __float_as_uint(v);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float score_of(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

// The K best of a token's E scores by one warp: K rounds of a maximum over the
// lanes' own best, the lower expert first among equal scores.
// Lane k < K of the warp gets slot k's expert and score.
template <int PER>
__device__ __forceinline__ void select_token(const Params& p, int t, int lane, int* id, float* score) {
  uint32_t key[PER];
  const float* row = p.logits + static_cast<int64_t>(t) * p.E;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0u;  // below every score's; a NaN is taken as 0, like the block's routing takes it
    if (e < p.E) {
      float s = __ldg(row + e);
      if (p.bias != nullptr) s = __fadd_rn(s, __ldg(p.bias + e));
      key[i] = order_of(s == s ? s : 0.0f);
    }
  }
  uint32_t mine = 0u;
  int mine_e = 0;
  for (int k = 0; k < p.K; ++k) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i) {
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int e = static_cast<int>(
        __reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(at * 32 + lane) : 0xffffffffu));
    if ((e & 31) == lane) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == (e >> 5)) key[i] = 0u;
    }
    if (lane == k) {
      mine = top;
      mine_e = e;
    }
  }
  *id = mine_e;
  *score = score_of(mine);
}
__device__ __forceinline__ void select_one(const Params& p, int t, int lane, int* id, float* score) {
  if (p.E <= 128) select_token<4>(p, t, lane, id, score);
  else if (p.E <= 256) select_token<8>(p, t, lane, id, score);
  else select_token<32>(p, t, lane, id, score);
}
// The weights of the K scores that the first lanes hold.
__device__ __forceinline__ float weigh(const Params& p, float v, int lane) {
  const float first = __shfl_sync(0xffffffffu, v, 0);
  float ex = 0.0f;
  if (lane < p.K)
    ex = p.mode == MOE_SCORE_SOFTMAX_TOPK ? expf(v - first) : sigmoid_num(v, first < -kDeep ? first : 0.0f);
  float sum = 0.0f;  // in the slots' order
  for (int k = 0; k < p.K; ++k) sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, ex, k));
  return __fdiv_rn(ex, sum);
}

// Everyone's selection in r.expert (and block 0's r.w).  Up to a token for each of its warps a
// CTA selects all for itself (and leaves the scores in r.w: only the combine
// needs weights, and that is far off); of more tokens each CTA selects its own, and they
// exchange them through global memory (128 tokens of 128 experts: 42 us when
// every CTA selected all; 8 tokens, 2816 -> 704, 102.9 us and 103.9 exchanged, 512 ->
// 192 28.2 and 30.6).  False: a wait gave up.
__device__ __forceinline__ bool select_all(const Params& p, const Route& r, const WaitCtl& wc, int warp, int lane) {
  const int R = p.n * p.K;
  bool ok = true;
  if (p.mode == MOE_SCORE_GIVEN) {
    for (int j = threadIdx.x; j < R; j += kThreads) {
      const int e = __ldg(p.ids_in + j);
      const bool in = e >= 0 && e < p.E;
      r.expert[j] = in ? static_cast<uint16_t>(e) : kNone;
      if (blockIdx.x == 0) r.w[j] = __ldg(p.w_in + j);
      if (!in && blockIdx.x == 0) report(p.status, MOE_ERR_DEVICE);
    }
  } else if (p.n <= kWarps) {
    if (warp < p.n) {
      int e;
      float v;
      select_one(p, warp, lane, &e, &v);
      if (lane < p.K) {
        r.expert[warp * p.K + lane] = static_cast<uint16_t>(e);
        r.w[warp * p.K + lane] = v;
      }
    }
  } else {
    for (int t = blockIdx.x + gridDim.x * warp; t < p.n; t += gridDim.x * kWarps) {
      int e;
      float w;
      select_one(p, t, lane, &e, &w);
      w = weigh(p, w, lane);
      if (lane < p.K) {
        const int j = t * p.K + lane;
        p.gids[j] = e;
        p.gw[j] = w;
        if (p.ids_out != nullptr) p.ids_out[j] = e;
        if (p.w_out != nullptr) p.w_out[j] = w;
      }
      __syncwarp();
      if (lane == 0) (void)add_acq_rel(p.routed, 1);
    }
    if (threadIdx.x == 0) ok = wait_for(p.routed, p.n, wc);
    ok = __syncthreads_and(ok);
    for (int j = threadIdx.x; j < R && ok; j += kThreads) {
      r.expert[j] = static_cast<uint16_t>(__ldcg(p.gids + j));
      if (blockIdx.x == 0) r.w[j] = __ldcg(p.gw + j);
    }
  }
  return ok;
}

// The list of virtual experts, by number of expert; the slots of one in their
// order.  Warp w ranks the slots of the w-th stretch of whole 32, then every
// expert's counts are summed over the warps, then over the experts.
__device__ __forceinline__ int build_list(const Params& p, const Route& r, Ctl& s, int warp, int lane) {
  const int R = p.n * p.K, span = (R + kThreads - 1) / kThreads * 32;
  const int warps = (R + span - 1) / span;  // that have slots
  uint16_t* mine = r.before + warp * p.E;
  if (warp < warps)
    for (int e = lane; e < p.E; e += 32) mine[e] = 0;
  __syncwarp();
  for (int j0 = warp * span; j0 < min(R, (warp + 1) * span); j0 += 32) {
    const int j = j0 + lane;
    const int e = j < R ? r.expert[j] : kNone;
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    const int ahead = e != kNone ? mine[e] : 0;
    __syncwarp();
    if (e != kNone) {
      r.rank[j] = static_cast<uint16_t>(ahead + __popc(peers & ((1u << lane) - 1u)));
      if (lane == __ffs(peers) - 1) mine[e] = static_cast<uint16_t>(ahead + __popc(peers));
    }
    __syncwarp();
  }
  __syncthreads();
  // a thread's experts: counts over the warps become what lies ahead of each
  const int per = (p.E + kThreads - 1) / kThreads, e0 = min(static_cast<int>(threadIdx.x) * per, p.E);
  const int e1 = min(e0 + per, p.E);
  int slots = 0, lists = 0;
  for (int e = e0; e < e1; ++e) {
    int sum = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = r.before[w * p.E + e];
      r.before[w * p.E + e] = static_cast<uint16_t>(sum);
      sum += c;
    }
    r.start[e] = static_cast<uint16_t>(sum);  // the count, until its place is known
    slots += sum;
    lists += (sum + kTokens - 1) / kTokens;
  }
  int ss = slots, sl = lists;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, ss, d), b = __shfl_up_sync(0xffffffffu, sl, d);
    if (lane >= d) {
      ss += a;
      sl += b;
    }
  }
  if (lane == 31) s.warp_sums[warp] = make_uint2(ss, sl);
  __syncthreads();
  int entries = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const uint2 q = s.warp_sums[w];
    if (w < warp) {
      ss += q.x;
      sl += q.y;
    }
    entries += q.y;
  }
  int at = ss - slots, v = sl - lists;
  for (int e = e0; e < e1; ++e) {
    const int count = r.start[e];
    r.start[e] = static_cast<uint16_t>(at);
    r.first[e] = static_cast<uint16_t>(v);
    for (int c = 0; c < count; c += kTokens, ++v) {
      r.vexp[v] = static_cast<uint16_t>(e);
      r.vstart[v] = static_cast<uint16_t>(at + c);
      r.vcnt[v] = static_cast<uint16_t>(min(kTokens, count - c));
    }
    at += count;
  }
  __syncthreads();
  for (int j0 = warp * span; j0 < min(R, (warp + 1) * span); j0 += 32) {
    const int j = j0 + lane;
    if (j >= R) break;
    const int e = r.expert[j];
    if (e != kNone) {
      const uint32_t rank = static_cast<uint32_t>(r.rank[j]) + mine[e];
      r.list[r.start[e] + rank] = static_cast<uint16_t>(j);
      r.at[j] = static_cast<uint16_t>(r.first[e] + rank / kTokens);
      r.rank[j] = static_cast<uint16_t>(rank % kTokens);  // in its virtual expert
    }
  }
  return entries;
}
// Slot j as the combine reads it.
__device__ __forceinline__ uint32_t word_of(const Route& r, int j) {
  return r.expert[j] != kNone ? slot_word(r.at[j], r.rank[j]) : 0u;
}

// What is left of the routing once the tiles are known, by block 0's epilogue
// warps while there is nothing to finish: weights, the caller's copies and the
// combine's table.
__device__ __forceinline__ void finish_routing(const Params& p, const Route& r, int entries, int ew, int lane) {
  const bool raw = p.mode != MOE_SCORE_GIVEN && p.n <= kWarps;  // r.w holds scores
  if (blockIdx.x != 0) return;
  for (int t = ew; t < p.n; t += 4) {
    const int j = t * p.K + lane;
    float w = lane < p.K ? r.w[j] : 0.0f;
    if (raw) w = weigh(p, w, lane);
    if (lane >= p.K) continue;
    p.slots[j] = make_uint2(word_of(r, j), __float_as_uint(w));
    if (raw && p.ids_out != nullptr) p.ids_out[j] = r.expert[j];
    if (raw && p.w_out != nullptr) p.w_out[j] = w;
  }
  if (ew == 0 && lane == 0) p.slots[p.n * p.K] = make_uint2(entries, 0u);
}

// A part of a tile: blocks [k0, k1) of tile `col` of virtual expert `v`.
struct Piece {
  uint32_t tile, v, col;
  int k0, k1;
};

// a / b for a below 2^24 and quotients below 2^20: the fast division is then off
// by one at most.  (The compiler's own takes three times as many instructions,
// and each role's first ones are fetched from far: with these, 2 us fewer lie
// between the routing and the first rows asked for.)
__device__ __forceinline__ uint32_t quotient(uint32_t a, uint32_t b) {
  const uint32_t q = __float2uint_rz(__fdividef(__uint2float_rn(a), __uint2float_rn(b)));
  const int r = static_cast<int>(a - q * b);
  return r < 0 ? q - 1 : r >= static_cast<int>(b) ? q + 1 : q;
}

// One phase's tiles and blocks.  (At most 1056 virtual experts of 256 tiles; the
// blocks cut into runs are of fewer tiles than CTAs: products stay below 2^24.)
// Blocks of a run: shorter ones cost more to join than they save (1 token of 2816 ->
// 704: 40.2 us with one at least, 40.0 with two, 38.0 with four, 37.8 with eight; of
// 256 -> 512: 18.6, 16.6, 14.6, 16.7).
constexpr uint32_t kLeastBlocks = 4;
// FC2's tiles for each CTA, for these to be claimed one by one (2816 -> 704: 8 tokens,
// eight tiles each, 103 us claimed and 109 not; 4 tokens, four each, 67.8 and 71.6; 2
// tokens, two each, 48.7 and 47.4; 1 token, 40.4 and 38.0).
constexpr uint32_t kLeastClaims = 4;
struct Phase {
  uint32_t kb;                       // blocks of a tile
  uint32_t cols;                     // tiles of a virtual expert
  uint32_t grid, tiles;
  bool claims;                       // tiles are claimed, whole
  uint32_t waves;                    // else every CTA takes `waves` whole tiles
  uint32_t blocks, ctas;             // of the tiles behind them; the CTAs that take runs of these
  __device__ __forceinline__ Phase(int D, int F, uint32_t grid, int which, uint32_t entries) : grid(grid) {
    kb = static_cast<uint32_t>(which == 0 ? D : F) / kBlockK;
    cols = static_cast<uint32_t>(which == 0 ? F : D + 64) / (which == 0 ? 64 : kCols);  // D: whole 64s
    tiles = entries * cols;
    claims = which == 1 && tiles >= kLeastClaims * grid;
    waves = quotient(tiles, grid);
    blocks = (tiles - waves * grid) * kb;
    ctas = min(grid, (blocks + kLeastBlocks - 1) / kLeastBlocks);
  }
  __device__ __forceinline__ uint32_t run(uint32_t c) const { return quotient(blocks * c, ctas); }
  __device__ __forceinline__ bool whole(uint32_t tile) const { return claims || tile < waves * grid; }
  __device__ __forceinline__ void place(Piece& q) const;
  // the CTA whose run holds block b
  __device__ __forceinline__ uint32_t owner(uint32_t b) const { return quotient((b + 1) * ctas - 1, blocks); }
};
__device__ __forceinline__ void Phase::place(Piece& q) const {
  q.v = quotient(q.tile, cols);
  q.col = q.tile - q.v * cols;
}
// The CTA's pieces in their order.
struct Walk {
  uint32_t wave, b, end;
  __device__ __forceinline__ explicit Walk(const Phase& f) : wave(0), b(0), end(0) {
    if (blockIdx.x < f.ctas) {
      b = f.run(blockIdx.x);
      end = f.run(blockIdx.x + 1);
    }
  }
  __device__ __forceinline__ bool next(const Phase& f, Piece& q) {
    if (wave < f.waves) {
      q.tile = wave * f.grid + blockIdx.x;
      q.k0 = 0;
      q.k1 = static_cast<int>(f.kb);
      ++wave;
    } else if (b < end) {
      const uint32_t t = quotient(b, f.kb);
      q.tile = f.waves * f.grid + t;
      q.k0 = static_cast<int>(b - t * f.kb);
      q.k1 = static_cast<int>(min(f.kb, q.k0 + (end - b)));
      b += q.k1 - q.k0;
    } else {
      return false;
    }
    f.place(q);
    return true;
  }
};
// Where a role gets its pieces from: the walk, or the queue of claimed tiles.
// `Walk`s end by themselves; a queue ends with a tile past the last.
struct Feed {
  Walk walk;
  uint32_t taken;  // from the queue
  __device__ __forceinline__ explicit Feed(const Phase& f) : walk(f), taken(0) {}

  // by one thread, or (WARP) a whole warp; ok becomes false where a wait gave up
  template <bool WARP>
  __device__ __forceinline__ bool next(const Phase& f, Piece& q, Ctl& s, const WaitCtl& wc, int lane, bool& ok) {
    if (!f.claims) return walk.next(f, q);
    const int slot = taken % kQueue;
    const uint32_t parity = taken / kQueue & 1u;
    ok = WARP ? warp_wait(&s.qfull[slot], parity, wc) : mbar_wait(&s.qfull[slot], parity, wc);
    if (!ok) return false;
    q.tile = s.qtile[slot];
    if (WARP) __syncwarp();
    if (!WARP || lane == 0) mbar_arrive(&s.qempty[slot]);
    ++taken;
    if (q.tile >= f.tiles) return false;
    q.k0 = 0;
    q.k1 = static_cast<int>(f.kb);
    f.place(q);
    return true;
  }
};
// Where CTA c keeps the sums of a part that starts its tile (tail = 1: it is
// the last of the CTA's run) or not (tail = 0: its first).
__device__ __forceinline__ float* part_rows(float* part, uint32_t grid, int phase, uint32_t c, int tail) {
  return part + ((static_cast<int64_t>(phase) * grid + c) * 2 + tail) * kTokens * kCols;
}

template <typename T>
__device__ __forceinline__ void store_h(const Params& p, int slot, int f, const float (&g)[8], const float (&u)[8]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = g[i] * sigmoid_fast(g[i]) * u[i];
  Raw<T, 8> o;
  o.pack(v);
  *reinterpret_cast<uint4*>(static_cast<T*>(p.h) + static_cast<int64_t>(slot) * p.F + f) = o.v;
}
template <bool SHARED>  // or of another CTA's part: never by the read-only path
__device__ __forceinline__ void add8(const float* at, float (&f)[8]) {
  const float4* p = reinterpret_cast<const float4*>(at);
  float4 a, b;
  if constexpr (SHARED) a = p[0], b = p[1];
  else a = __ldcg(p), b = __ldcg(p + 1);
  f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w, f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
}

// out[t, 128 col ..] by one warp, four columns a lane: the token's slots in
// order, each the sum of its tile's parts in the reduction's order.  Lane k < K
// brings slot k's word and weight.
template <typename T>
__device__ __forceinline__ void combine_unit(const CombineParams& p, const Phase& f, int t, int col, int lane,
                                             uint32_t word, float w) {
  constexpr int kAhead = 8;
  const int c4 = col * kCols + lane * 4;
  const bool in = c4 < p.D;
  float r4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.res != nullptr && in) {
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.res) + t * p.ldres + c4);
    const float2 lo = unpack_pair(q.x, T{}), hi = unpack_pair(q.y, T{});
    r4[0] = lo.x, r4[1] = lo.y, r4[2] = hi.x, r4[3] = hi.y;
  }
  // lane k looks at slot k: the CTAs of its tile's first and last part (the
  // same where one summed it alone) and its row in their parts
  uint32_t first = 0, last = 0, row = 0;
  const bool valid = lane < p.K && (word & 0x80000000u) != 0u;
  if (valid) {
    row = (word >> 16) & 0xffu;
    const uint32_t tile = (word & 0xffffu) * f.cols + col;
    if (!f.whole(tile)) {
      const uint32_t b = (tile - f.waves * f.grid) * f.kb;
      first = f.owner(b);
      last = f.owner(b + f.kb - 1);
    }
  }
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const auto part = [&](uint32_t c, int tail, uint32_t at) {
    return __ldcg(reinterpret_cast<const float4*>(part_rows(const_cast<float*>(p.part), p.grid, 1, c, tail) +
                                                  at * kCols + lane * 4));
  };
  for (int k0 = 0; k0 < p.K; k0 += kAhead) {
    float4 a[kAhead], b[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = min(k0 + i, p.K - 1);
      const uint32_t c0 = __shfl_sync(0xffffffffu, first, k), c1 = __shfl_sync(0xffffffffu, last, k);
      const uint32_t at = __shfl_sync(0xffffffffu, row, k);
      const bool named = __shfl_sync(0xffffffffu, valid ? 1 : 0, k) != 0;
      a[i] = b[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (named && in && k0 + i < p.K) {
        if (c0 == c1) {
          a[i] = __ldcg(reinterpret_cast<const float4*>(p.y + (static_cast<int64_t>(t) * p.K + k) * p.D + c4));
        } else {
          a[i] = part(c0, 1, at);
          b[i] = part(c0 + 1, 0, at);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = min(k0 + i, p.K - 1);
      const uint32_t c0 = __shfl_sync(0xffffffffu, first, k), c1 = __shfl_sync(0xffffffffu, last, k);
      const uint32_t at = __shfl_sync(0xffffffffu, row, k);
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const bool named = __shfl_sync(0xffffffffu, valid ? 1 : 0, k) != 0;
      if (!named || k0 + i >= p.K) continue;  // a slot left out: whatever its weight
      float4 s = make_float4(a[i].x + b[i].x, a[i].y + b[i].y, a[i].z + b[i].z, a[i].w + b[i].w);
      for (uint32_t c = c0 + 2; c <= c1 && in; ++c) {
        const float4 q = part(c, 0, at);
        s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
      }
      acc[0] = fmaf(wk, s.x, acc[0]);
      acc[1] = fmaf(wk, s.y, acc[1]);
      acc[2] = fmaf(wk, s.z, acc[2]);
      acc[3] = fmaf(wk, s.w, acc[3]);
    }
  }
  if (!in) return;
  *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + t * p.ldout + c4) =
      make_uint2(pack_pair(acc[0] + r4[0], acc[1] + r4[1], T{}), pack_pair(acc[2] + r4[2], acc[3] + r4[3], T{}));
}

// The combine as a kernel of its own: a warp to a token's 128 columns.  (What
// the first kernel wrote is read by ordinary loads: see wait_for_previous.)
constexpr int kCombineWarps = 4;
template <typename T>
__global__ void __launch_bounds__(32 * kCombineWarps) combine_kernel(const CombineParams p) {
  const int lane = threadIdx.x & 31;
  const int tiles = (p.D + kCols - 1) / kCols;
  const int unit = blockIdx.x * kCombineWarps + (threadIdx.x >> 5);
  const int t = unit / tiles, col = unit - t * tiles;
  wait_for_previous();
  if (t >= p.n) return;
  uint2 slot = make_uint2(0u, 0u);
  if (lane < p.K) slot = __ldcg(p.slots + static_cast<int64_t>(t) * p.K + lane);
  const Phase f(p.D, p.F, p.grid, 1, __ldcg(&p.slots[static_cast<int64_t>(p.n) * p.K].x));
  combine_unit<T>(p, f, t, col, lane, slot.x, __uint_as_float(slot.y));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap map_wi, const __grid_constant__ CUtensorMap map_wo,
                  const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_h,
                  const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* buf = reinterpret_cast<float*>(ring + p.stages * kStage);
  Ctl& s = *reinterpret_cast<Ctl*>(reinterpret_cast<uint8_t*>(buf) + kBufBytes);
  const Route r = route_at(reinterpret_cast<uint8_t*>(&s) + sizeof(Ctl), p.n * p.K, p.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // set up by the last warps, while the first ones select
  if (threadIdx.x == 0) s.abort_flag = 0;
  if (warp == kWarps - 2) {
    tmem_alloc<1>(&s.tmem_base, kTmemCols);
    tmem_relinquish<1>();
  } else if (threadIdx.x == 32 * (kWarps - 1)) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s.fullw[i], 1);
      mbar_init(&s.fullt[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], 4);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&s.qfull[i], 1);
      mbar_init(&s.qempty[i], kQueueReaders);
    }
    mbar_fence_init();
    tma_prefetch_map(&map_wi);
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_wo);
    tma_prefetch_map(&map_h);
  }
  __syncwarp();
  const WaitCtl wc{&s.abort_flag, p.status, p.limit_ns};
  const bool routed = select_all(p, r, wc, warp, lane);
  __syncthreads();
  int entries = 0;
  if (routed) {
    entries = build_list(p, r, s, warp, lane);
  } else if (blockIdx.x == 0) {  // the combine's kernel finds no slot
    for (int j = threadIdx.x; j <= p.n * p.K; j += kThreads) p.slots[j] = make_uint2(0u, 0u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  let_next_launch();  // the combine's blocks: they need what this kernel leaves of an SM
  const uint32_t tmem = s.tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------ weights' producer
    if (elect_one()) {
      int stage = 0, filled = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Phase f(p.D, p.F, gridDim.x, ph, entries);
        Walk walk(f);
        Piece q;
        int ahead = f.claims ? atomicAdd(p.claimed, 1) : 0;  // a tile ahead: its latency is hidden
        for (uint32_t put = 0; ok; ++put) {
          if (f.claims) {
            const int slot = put % kQueue;
            q.tile = static_cast<uint32_t>(ahead);
            if (put >= kQueue) ok = mbar_wait(&s.qempty[slot], (put / kQueue - 1) & 1u, wc);
            if (!ok) break;
            s.qtile[slot] = q.tile;
            mbar_arrive(&s.qfull[slot]);
            if (q.tile >= f.tiles) break;
            ahead = atomicAdd(p.claimed, 1);
            q.k0 = 0;
            q.k1 = static_cast<int>(f.kb);
            f.place(q);
          } else if (!walk.next(f, q)) {
            break;
          }
          const int e = r.vexp[q.v];
          const int c0 = ph == 0 ? q.col * 64 : q.col * kCols;
          const int c1 = ph == 0 ? p.F + c0 : c0 + 64;
          const void* map = ph == 0 ? &map_wi : &map_wo;
          for (int kb = q.k0; kb < q.k1; ++kb) {
            ok = mbar_wait(&s.empty[stage], phase ^ 1u, wc);
            if (!ok) break;
            uint8_t* at = ring + stage * kStage;
            mbar_arrive_expect_tx(&s.fullw[stage], kWeightStage);
            tma_load_3d(at, map, &s.fullw[stage], c0, kb * kBlockK, e);
            tma_load_3d(at + kChunk, map, &s.fullw[stage], c1, kb * kBlockK, e);
            ++filled;
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      if (!ok) {  // copies in flight land before the CTA goes on
        for (int i = 0; i < p.stages; ++i) {
          const int n = filled > i ? (filled - i + p.stages - 1) / p.stages : 0;
          if (n > 0) (void)mbar_wait_drain(&s.fullw[i], (n - 1) & 1, 100000000ull);
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------- tokens' producer
    // Lane i gathers rows 4i .. 4i + 3 of the tile's tokens: of x, then of h
    // once the flag of the block's h is set.  (Rows past the last are the last
    // again; their columns of the product are not read.)
    int stage = 0, filled = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int ph = 0; ph < 2 && ok; ++ph) {
      const Phase f(p.D, p.F, gridDim.x, ph, entries);
      Feed feed(f);
      Piece q;
      const int flags = p.F / 64;  // of a virtual expert
      while (ok && feed.next<true>(f, q, s, wc, lane, ok)) {
        const int cnt = r.vcnt[q.v], groups = (cnt + 3) / 4;
        int row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int slot = r.list[r.vstart[q.v] + min(4 * lane + i, cnt - 1)];
          row[i] = ph == 0 ? static_cast<int>(slot * p.k_inverse >> 16) : slot;
        }
        if (ph == 1) {
          const int32_t* flag = p.done + static_cast<int64_t>(q.v) * flags;
          for (int i = q.k0 + lane; i < q.k1 && ok; i += 32) ok = wait_for(flag + i, 1, wc);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          __syncwarp();  // a lane's rows may lie behind other lanes' flags
          fence_proxy_async_global();
        }
        for (int kb = q.k0; kb < q.k1; ++kb) {
          ok = warp_wait(&s.empty[stage], phase ^ 1u, wc);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&s.fullt[stage], groups * 512);
          __syncwarp();
          if (lane < groups)
            gather4(ring + stage * kStage + kWeightStage + 512 * lane, ph == 0 ? &map_x : &map_h,
                    &s.fullt[stage], kb * kBlockK, row);
          ++filled;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    // This CTA's producer reads no more flags.  The last to say so clears them:
    // each tile's flag was waited for by some CTA's producer, so it has been
    // set, and the parts that were joined before it was are no more waited for.
    int left = 0;
    if (lane == 0) {
      __threadfence();
      left = atomicAdd(p.leave, 1);
    }
    if (__shfl_sync(0xffffffffu, left, 0) == static_cast<int>(gridDim.x) - 1) {
      __threadfence();
      const int n = entries * (p.F / 64);
      for (int i = lane; i < n; i += 32) p.done[i] = 0;
      for (int i = lane; i < static_cast<int>(gridDim.x); i += 32) p.stored[i] = 0;
      if (lane == 0) *p.leave = *p.routed = *p.claimed = 0;
    }
    if (!ok && lane == 0) {
      for (int i = 0; i < p.stages; ++i) {
        const int n = filled > i ? (filled - i + p.stages - 1) / p.stages : 0;
        if (n > 0) (void)mbar_wait_drain(&s.fullt[i], (n - 1) & 1, 100000000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    if (elect_one()) {
      const uint32_t base = smem_u32(ring);
      const Operand weights = operand128<true>(), tokens = operand128<false>();
      int stage = 0, done = 0, piece = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int ph = 0; ph < 2 && ok; ++ph) {
        const Phase f(p.D, p.F, gridDim.x, ph, entries);
        Feed feed(f);
        Piece q;
        for (; ok && feed.next<false>(f, q, s, wc, lane, ok); ++piece) {
          const int slot = piece & 1;
          const uint32_t idesc = dense_idesc(kCols, (r.vcnt[q.v] + 15) & ~15, true, false, p.type);
          if (piece >= 2) ok = mbar_wait(&s.tempty[slot], ((piece >> 1) - 1) & 1, wc);
          tc_fence_after();
          for (int kb = q.k0; kb < q.k1 && ok; ++kb) {
            ok = mbar_wait(&s.fullw[stage], phase, wc) && mbar_wait(&s.fullt[stage], phase, wc);
            if (!ok) break;
            tc_fence_after();
            const uint32_t at = base + stage * kStage;
            issue_block<1>(tmem + slot * kTokens, at, at + kWeightStage, weights, tokens, idesc, kb > q.k0 ? 1u : 0u);
            umma_commit<1>(&s.empty[stage]);
            ++done;
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) umma_commit<1>(&s.tfull[slot]);
        }
      }
      if (!ok && done > 0) {  // issued products end before TMEM is freed
        const int last = (done - 1) % p.stages;
        (void)mbar_wait_drain(&s.empty[last], ((done - last + p.stages - 1) / p.stages - 1) & 1, 100000000ull);
      }
    }
  } else if (warp >= kFirstEpiWarp) {
    // -------------------------------------------------------------- epilogue
    const int tid = threadIdx.x - kFirstEpiWarp * 32, ew = warp - kFirstEpiWarp;
    const int col = (warp & 3) * 32 + lane;  // the tile's column: this thread's TMEM lane
    const uint32_t tq = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    if (routed) finish_routing(p, r, entries, ew, lane);
    int piece = 0;
    bool ok = true;
    for (int ph = 0; ph < 2 && ok; ++ph) {
      const Phase f(p.D, p.F, gridDim.x, ph, entries);
      Feed feed(f);
      Piece q;
      for (;; ++piece) {
        // the four warps meet at barriers below: all go on or none does
        const bool more = feed.next<true>(f, q, s, wc, lane, ok);
        ok = epi_all(ok);
        if (!ok || !more) break;
        const int slot = piece & 1, cnt = r.vcnt[q.v], start = r.vstart[q.v];
        const bool whole = q.k1 - q.k0 == static_cast<int>(f.kb);
        const int i16 = tid / 8, c8 = (tid % 8) * 8;  // FC1: this thread's token of 16, its columns
        // FC1, the tile's first part: the CTAs that have the others
        uint32_t join0 = blockIdx.x + 1, join1 = blockIdx.x;
        if (ph == 0 && q.k0 == 0 && !whole) {
          join1 = f.owner((q.tile - f.waves * f.grid + 1) * f.kb - 1);
          for (uint32_t c = join0 + tid; c <= join1 && ok; c += 128) ok = wait_for(p.stored + c, 1, wc);
        }
        ok = epi_all(ok);
        if (!ok) break;
        const auto joined = [&](int t0, float (&g)[8], float (&u)[8]) {
          for (uint32_t c = join0; c <= join1; ++c) {
            const float* at = part_rows(p.part, gridDim.x, 0, c, 0) + (t0 + i16) * kCols;
            add8<false>(at + c8, g);
            add8<false>(at + 64 + c8, u);
          }
        };
        float g[8] = {}, u[8] = {};
        if (i16 < cnt) joined(0, g, u);  // while the products end
        ok = epi_all(warp_wait(&s.tfull[slot], (piece >> 1) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        float* rows = part_rows(p.part, gridDim.x, ph, blockIdx.x, q.k0 == 0 ? 1 : 0);
        for (int t0 = 0; t0 < cnt; t0 += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(tq + slot * kTokens + t0, v);
          tmem_ld_wait();
          const int m = min(16, cnt - t0);
          if (ph == 0 && q.k0 == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) buf[i * kBufLd + col] = __uint_as_float(v[i]);
            epi_sync();
            if (i16 < m) {
              if (t0 > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = u[i] = 0.0f;
                joined(t0, g, u);
              }
              add8<true>(buf + i16 * kBufLd + c8, g);
              add8<true>(buf + i16 * kBufLd + 64 + c8, u);
              store_h<T>(p, r.list[start + t0 + i16], q.col * 64 + c8, g, u);
            }
            epi_sync();
          } else if (whole) {  // FC2
            const int c = static_cast<int>(q.col) * kCols + col;
            if (c < p.D) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (i < m) __stcg(p.y + static_cast<int64_t>(r.list[start + t0 + i]) * p.D + c, __uint_as_float(v[i]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < m) __stcg(rows + (t0 + i) * kCols + col, __uint_as_float(v[i]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.tempty[slot]);
        if (ph == 1) continue;
        if (q.k0 == 0) fence_proxy_async_global();  // h is read by TMA
        epi_sync();
        if (tid == 0) st_release(q.k0 == 0 ? p.done + q.tile : p.stored + blockIdx.x, 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarps - 2) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, kTmemCols);
  }
}

// 16-bit [outer][mid][inner], boxes of 64 x 64 x 1.  L2 fetches the box's 128
// bytes of a row and no more: the next 128 are another tile's, and gone again by
// its turn (7168 -> 2048, FC1: 366 us with 256 bytes, 280 with 128).
bool map3(CUtensorMap* m, const void* base, uint64_t inner, uint64_t mid, uint64_t outer) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {inner, mid, outer}, strides[2] = {inner * 2, inner * mid * 2};
  const cuuint32_t box[3] = {64, kBlockK, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxGrid = 192;  // CTAs that the workspace has room for: no device of this kind has more SMs
static_assert((32 + kMaxGrid) * 4 <= 1024, "counters and flags ahead of the tiles' flags");
size_t up(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: counters (zero between calls; placed by the capacity, not by a
// call's tokens), then the data.
struct Layout {
  size_t done, slots, gids, gw, h, y, part, all;
  explicit Layout(const moe_dims& d) {
    const size_t R = static_cast<size_t>(d.T) * d.K;
    const size_t tiles = static_cast<size_t>(most_virtual(static_cast<int>(R), d.E)) * (d.F / 64);
    done = 1024;  // behind the three counters and the CTAs' flags
    slots = done + up(tiles * 4);
    gids = slots + up((R + 1) * 8);
    gw = gids + up(R * 4);
    h = gw + up(R * 4);
    y = h + up(R * d.F * 2);
    part = y + up(R * d.D * 4);
    all = part + up(static_cast<size_t>(kMaxGrid) * 4 * kTokens * kCols * 4);
  }
};

template <typename T>
cudaError_t launch_typed(const DecodeCall& c, cudaStream_t s) {
  const moe_dims& d = c.d;
  Params p{};
  p.logits = c.logits;
  p.bias = c.bias;
  p.ids_in = c.ids;
  p.w_in = c.w;
  p.ids_out = c.ids_out;
  p.w_out = c.w_out;
  p.n = c.n;
  p.D = d.D;
  p.E = d.E;
  p.K = d.K;
  p.F = d.F;
  p.mode = c.mode;
  p.k_inverse = static_cast<uint32_t>((65536 + d.K - 1) / d.K);
  p.type = c.type == MOE_BF16 ? 1u : 0u;
  p.status = c.dev_status;
  p.limit_ns = kDefaultWaitLimitNs;
  const int grid = std::min(sm_count(), kMaxGrid);
  const Layout at(d);
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  p.leave = reinterpret_cast<int32_t*>(ws);
  p.done = reinterpret_cast<int32_t*>(ws + at.done);
  p.routed = p.leave + 1;
  p.claimed = p.leave + 2;
  p.stored = p.leave + 32;
  p.slots = reinterpret_cast<uint2*>(ws + at.slots);
  p.gids = reinterpret_cast<int32_t*>(ws + at.gids);
  p.gw = reinterpret_cast<float*>(ws + at.gw);
  p.h = ws + at.h;
  p.y = reinterpret_cast<float*>(ws + at.y);
  p.part = reinterpret_cast<float*>(ws + at.part);
  const size_t R = static_cast<size_t>(c.n) * d.K;
  const size_t fixed = 1024 + kBufBytes + sizeof(Ctl) + route_bytes(static_cast<int>(R), d.E);
  p.stages = static_cast<int>(std::min<size_t>(kMaxStages, (kSmemLimit - fixed) / kStage));
  if (p.stages < kMinStages) return cudaErrorInvalidValue;
  CUtensorMap wi, wo, x, h;
  if (!map3(&wi, c.wi, 2 * static_cast<uint64_t>(d.F), d.D, d.E) || !map3(&wo, c.wo, d.D, d.F, d.E) ||
      !map_rows(&x, c.x, d.D, c.n, c.ldx) || !map_rows(&h, p.h, d.F, R, d.F))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(decode_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSmemLimit));
    if (err != cudaSuccess) return err;
    attr_set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = fixed + p.stages * static_cast<size_t>(kStage);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, decode_kernel<T>, wi, wo, x, h, p);
  if (err != cudaSuccess) return err;
  CombineParams q{};
  q.slots = p.slots;
  q.y = p.y;
  q.part = p.part;
  q.res = c.res;
  q.ldres = c.ldres;
  q.out = c.out;
  q.ldout = c.ldout;
  q.n = c.n;
  q.D = d.D;
  q.F = d.F;
  q.K = d.K;
  q.grid = static_cast<uint32_t>(grid);
  cudaLaunchAttribute overlap = overlap_attribute();
  const int units = c.n * ((d.D + kCols - 1) / kCols);
  cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((units + kCombineWarps - 1) / kCombineWarps));
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.stream = s;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<T>, q);
}

}  // namespace

size_t decode_ws_bytes(const moe_dims& d) { return Layout(d).all; }

cudaError_t launch_decode(const DecodeCall& c, cudaStream_t s) {
  return c.type == MOE_BF16 ? launch_typed<__nv_bfloat16>(c, s) : launch_typed<__half>(c, s);
}

}  // namespace moe
