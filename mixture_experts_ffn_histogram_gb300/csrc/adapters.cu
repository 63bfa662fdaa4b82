// Low-rank adapters of many requests beside a shared projection:
//
//   y[t] = res[t] + scale[s] (x[t] a_s^T) b_s^T,   s = ids[t]   (none: y = res)
//
// a_s [r, K] and b_s [N, r] are one adapter's factors, of up to 1024 kept in a
// pool; a batch's tokens name them in any order.
//
// plan: a stable counting sort of the tokens by adapter, in one block, and the
// list of tiles of up to 128 tokens of one adapter (those without one come
// last).  Made once for a batch: all of its projections share it.
// shrink: v = x a_s^T by tile on the tensor cores.  The tile's tokens are
// copied straight from their places in x as the 128 side, the rank is the narrow
// side, and the reduction over K is cut among CTAs where tiles are few.  Bound by
// reading x; for a few tokens by latency.
// expand: y = res + scale v b_s^T.  Its reduction is the rank, one to eight
// MMAs deep, so that nearly all of it is moving res and y: the products are
// mma.sync's, whose accumulators already lie in the registers that add and
// store (tensor memory would add a round trip to a kernel without a main loop).
// Columns and reduction indices are permuted among the fragments so that every
// access is 8 or 16 contiguous bytes.
//
// v is summed in fp32 (over the cuts in a fixed order, by the CTA that stores a
// tile's last part) and rounded once, with the scale, to the operands' type for
// the second product, as a layer of the model would hand it on: half a step on
// each of r terms, together about what the result's own rounding is.  (What that
// leaves, kept as a second part with products of its own: 73 to 77 us for 32768
// tokens of rank 32, 52 to 55 for 8191 of rank 64, 118 to 141 for 16000 of 128.)
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

constexpr int kTile = 128;  // tokens

// A plan in memory: the header, the tiles, the tokens in their order.
struct PlanHead {
  int32_t n, slots;
  int32_t tiles;  // of tokens with an adapter
  int32_t none;   // tiles behind them, of tokens without
  int32_t live;   // tokens with an adapter: the first ones in the order
  int32_t pad[3];
};
struct PlanTile {
  int32_t adapter, start, count, pad;
};
__host__ __device__ inline int64_t most_tiles(int64_t T, int64_t slots) {
  return T / kTile + (slots + 1 < T ? slots + 1 : T);
}
__host__ __device__ inline size_t plan_order_at(int64_t T, int64_t slots) {
  return sizeof(PlanHead) + static_cast<size_t>(most_tiles(T, slots)) * sizeof(PlanTile);
}

// -------------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;

// Warp w ranks the tokens of the w-th stretch; every adapter's counts are
// summed over the warps, then over the adapters.  Bucket `slots` holds the
// tokens without one.
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int32_t* ids, int n, int slots, PlanHead* head, PlanTile* tiles, int32_t* order, int32_t* status) {
  extern __shared__ int32_t before[];  // [warps][buckets]
  __shared__ int2 warp_sums[kPlanWarps];
  const int buckets = slots + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int span = (n + kPlanThreads - 1) / kPlanThreads * 32;
  const int j0 = min(n, warp * span), j1 = min(n, j0 + span);
  int32_t* mine = before + warp * buckets;
  for (int b = lane; b < buckets; b += 32) mine[b] = 0;
  __syncwarp();
  // the buckets of eight times 32 tokens at a time: eight loads under way
  const auto each = [&](const auto& visit) {
    constexpr int kLoads = 8;
    for (int j = j0; j < j1; j += 32 * kLoads) {
      int id[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = j + 32 * i + lane;
        id[i] = at < j1 ? __ldg(ids + at) : 0;
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = j + 32 * i + lane;
        const int b = at >= j1 ? -1 : id[i] >= 0 && id[i] < slots ? id[i] : slots;
        visit(at, b, id[i]);
      }
    }
  };
  each([&](int, int b, int id) {
    if (b == slots && id != -1) report(status, MOE_ERR_DEVICE);
    if (b >= 0) atomicAdd(mine + b, 1);
  });
  __syncthreads();
  // thread i has bucket i (there are at most 1025: the last thread has two)
  const int per = buckets > kPlanThreads && threadIdx.x == kPlanThreads - 1 ? 2 : 1;
  const int b0 = threadIdx.x, b1 = min(buckets, b0 + per);
  int count[2] = {0, 0}, tokens = 0, lists = 0;
  for (int b = b0; b < b1; ++b) {
    int sum = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = before[w * buckets + b];
      before[w * buckets + b] = sum;
      sum += c;
    }
    count[b - b0] = sum;
    tokens += sum;
    lists += (sum + kTile - 1) / kTile;
  }
  int st = tokens, sl = lists;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, st, d), b = __shfl_up_sync(0xffffffffu, sl, d);
    if (lane >= d) {
      st += a;
      sl += b;
    }
  }
  if (lane == 31) warp_sums[warp] = make_int2(st, sl);
  __syncthreads();
  int all = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    const int2 q = warp_sums[w];
    if (w < warp) {
      st += q.x;
      sl += q.y;
    }
    all += q.y;
  }
  int at = st - tokens, tile = sl - lists;
  for (int b = b0; b < b1; ++b) {
    const int c = count[b - b0];
    for (int w = 0; w < kPlanWarps; ++w) before[w * buckets + b] += at;  // places in the order
    for (int i = 0; i < c; i += kTile)
      tiles[tile++] = PlanTile{b, at + i, min(kTile, c - i), 0};
    if (b == slots) {  // the last bucket
      const int none = (c + kTile - 1) / kTile;
      *head = PlanHead{n, slots, all - none, none, at, {0, 0, 0}};
    }
    at += c;
  }
  __syncthreads();
  each([&](int j, int b, int) {
    const uint32_t peers = __match_any_sync(0xffffffffu, b);
    const int first = b >= 0 ? mine[b] : 0;
    __syncwarp();
    if (b >= 0) {
      order[first + __popc(peers & ((1u << lane) - 1u))] = j;
      if (lane == __ffs(peers) - 1) mine[b] = first + __popc(peers);
    }
    __syncwarp();
  });
}

// ------------------------------------------------------------------ shrink
constexpr int kShrinkThreads = 192;
constexpr int kTokenStage = kTile * kBlockK * 2;  // 16 KB
constexpr int kMaxStages = 8;
constexpr int kMinStages = 3;
// Blocks of a cut of the reduction (8 tokens of 8 adapters, 2816 -> 16 -> 2816: 10.5 us
// with one at least, 9.9 with two, 10.2 with four, 11.4 with eight; 16 tokens of one of
// rank 64: 14.4, 12.5, 12.4, 12.5).
constexpr int kLeastCutBlocks = 4;

// The cuts of a tile's reduction: as many as give every CTA of the grid (two
// to an SM) at most one, of four blocks at least.
__device__ __forceinline__ int cuts_of(int tiles, int grid, int kblocks) {
  return tiles > 0 ? max(1, min(grid / tiles, kblocks / kLeastCutBlocks)) : 1;
}

// Whether tiles are of few tokens, whose latency counts: their rows come by a TMA
// gather for every four, and the CTA that stores a tile's last part joins them
// (61 tokens of 64 adapters: 14.0 us against 15.9 the other way; 2000 of 1024: 100
// against 125).  Else the epilogue's warps copy the rows, and parts are joined by
// a kernel of their own (2000 tokens of 16 adapters: 18 against 23; 32768 of 16:
// 73 against 87, since gathers keep to 31 bytes a ns and SM).
// The border is 32 tokens to a tile (2816 -> 2816, one adapter, of rank 16 and of
// 64: 32 tokens 10.5 and 16.6 us this way, 12.7 and 18.7 the other; 48: 12.4 and
// 20.6, 12.6 and 14.6; 128: 20.2 and 39.3, 14.4 and 18.7).
constexpr int kFewTokens = 32;  // of a tile
// A call of up to 256 tokens and 32 to each of the pool's adapters is taken for
// such a one whatever its plan, and its kernel for parts is not launched (256 of 16
// adapters of rank 16: 12.5 us against 14.6 with it; if they all name one adapter
// 20.6 against 14.4, which is why longer calls leave it to the plan).
constexpr int kFewOfCall = 256;
inline bool few_tokens(int n, int slots) { return n <= kFewOfCall && n <= static_cast<int64_t>(kFewTokens) * slots; }
__device__ __forceinline__ bool few_tokens(const PlanHead& h, bool of_call) {
  return of_call || h.live <= kFewTokens * h.tiles;
}

struct ShrinkParams {
  const void* x;
  int64_t ldx;
  int K;
  const PlanHead* head;
  const PlanTile* tiles;
  const int32_t* order;
  void* v;           // 16-bit [live tokens][width], by place in the order: scaled
  float* parts;      // [cuts][live tokens][width], where there is more than one cut
  int32_t* arrived;  // [tile]: cuts whose part is stored; zero between calls
  const float* scale;
  int n, slots, width, kblocks, stages;  // width: rank in whole 16s
  bool few;  // few_tokens whatever the plan: no kernel for parts
  uint32_t type;
  int32_t* status;
  uint64_t limit_ns;
};
struct ShrinkCtl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t done;     // a unit's products
  uint64_t drained;  // ... have been read
  float4 sums[128];
  uint32_t tmem_base;
  int abort_flag;
  int last;
};
__host__ __device__ constexpr int tmem_width(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : 128; }

// The reduction blocks of unit u, in the order in which they are read: every
// so manieth, from another one on for each unit.
struct Blocks {
  int kb, count, first, step, kblocks;
  __device__ __forceinline__ Blocks(int u, int cuts, int kblocks) : first(u % cuts), step(cuts), kblocks(kblocks) {
    count = (kblocks - first + cuts - 1) / cuts;
    kb = first + u % count * cuts;
  }
  __device__ __forceinline__ void next() {
    kb += step;
    if (kb >= kblocks) kb = first;
  }
};

// v of a tile from its parts.  Tiles of few tokens: by the 128 epilogue threads of the
// CTA that stored the last part, four neighbouring ranks of a token to a thread;
// where there are fewer of those than threads, 2^k threads take the cuts in
// turns and their sums are added in the threads' order.  (61 tokens: 1.2 us,
// about a launch.)  Others: by a kernel of its own, as wide as there are
// values, since the last CTAs' 128 threads took 14 us of 73 for 8191 tokens.
template <typename T>
__device__ __forceinline__ void join_parts(const ShrinkParams& p, const PlanTile& tile, int live, int cuts, int tid,
                                           float4* sums) {
  const int per_row = p.width / 4, quads = tile.count * per_row;
  int share = 1;
  while (share < 32 && quads * share * 2 <= 128 && share * 2 <= cuts) share *= 2;
  const float scale = __ldg(p.scale + tile.adapter);
  const int64_t cut = static_cast<int64_t>(live) * p.width;
  const float* parts = p.parts + static_cast<int64_t>(tile.start) * p.width;
  const auto add = [](float4& f, const float4& d) { f.x += d.x, f.y += d.y, f.z += d.z, f.w += d.w; };
  const auto store = [&](int i, const float4& f) {
    *reinterpret_cast<uint2*>(static_cast<T*>(p.v) + static_cast<int64_t>(tile.start) * p.width + 4 * i) =
        make_uint2(pack_pair(scale * f.x, scale * f.y, T{}), pack_pair(scale * f.z, scale * f.w, T{}));
  };
  if (share > 1) {
    const int sub = tid % share, i = tid / share;
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < quads) {
#pragma unroll 4
      for (int c = sub; c < cuts; c += share) add(f, __ldcg(reinterpret_cast<const float4*>(parts + 4 * i + c * cut)));
    }
    sums[tid] = f;
    epi_sync();
    if (i < quads && sub == 0) {
      for (int k = 1; k < share; ++k) add(f, sums[tid + k]);
      store(i, f);
    }
    return;
  }
  for (int i = tid; i < quads; i += 128) {
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int c = 0; c < cuts; ++c) add(f, __ldcg(reinterpret_cast<const float4*>(parts + 4 * i + c * cut)));
    store(i, f);
  }
}

struct JoinParams {
  const PlanHead* head;
  const PlanTile* tiles;
  const float *parts, *scale;
  void* v;
  int n, slots, width, kblocks, shrink_grid;
};
constexpr int kJoinThreads = 256;
// A block takes a tile at a time.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const JoinParams p) {
  const PlanHead head = *p.head;
  const int cuts = cuts_of(head.tiles, p.shrink_grid, p.kblocks);
  const bool few = few_tokens(head, false), work = head.n == p.n && head.slots == p.slots && cuts > 1 && !few;
  // Of tiles of few tokens, expand's blocks are better let in together once
  // shrink's have gone than one by one between them (2000 tokens of 1024 adapters
  // of rank 64: 188 us against 234; of rank 16: 100 against 99), of others the
  // other way (32768 of 16: 73 against 75).
  if (!few) let_next_launch();
  wait_for_previous();
  if (!work) return;
  const int per_row = p.width / 4;
  const int64_t cut = static_cast<int64_t>(head.live) * per_row;
  const float4* parts = reinterpret_cast<const float4*>(p.parts);
  // a slice of a tile's values to a block
  constexpr int kSlices = 4;
  for (int u = blockIdx.x; u < head.tiles * kSlices; u += gridDim.x) {
    const PlanTile tile = p.tiles[u / kSlices];
    const float scale = p.scale[tile.adapter];
    const int64_t first = static_cast<int64_t>(tile.start) * per_row;
    for (int i = u % kSlices * kJoinThreads + threadIdx.x; i < tile.count * per_row; i += kSlices * kJoinThreads) {
      float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int c = 0; c < cuts; ++c) {
        const float4 d = __ldcg(parts + first + i + c * cut);
        f.x += d.x, f.y += d.y, f.z += d.z, f.w += d.w;
      }
      reinterpret_cast<uint2*>(p.v)[first + i] =
          make_uint2(pack_pair(scale * f.x, scale * f.y, T{}), pack_pair(scale * f.z, scale * f.w, T{}));
    }
  }
}

// Tiles of many tokens: the four epilogue warps copy them, wherever they lie, in
// 16-byte pieces (eight lanes to a row's 128 bytes, swizzled like a TMA box),
// some stages ahead of telling the products: all stages but two, so that a
// stage's products and the word that it is free again take their time while
// others land (all but one: 32768 mixed tokens 81 us against 73).
constexpr int kMostLag = 4;
template <typename T>
struct TokenCopies {
  uint8_t* ring;
  int stage_bytes, q, lane, lag;
  int stage = 0, told = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ TokenCopies(const ShrinkParams& p, uint8_t* ring, int stage_bytes, int q, int lane)
      : ring(ring), stage_bytes(stage_bytes), q(q), lane(lane), lag(min(kMostLag, p.stages - 2)) {}

  __device__ __forceinline__ bool run(const ShrinkParams& p, ShrinkCtl& s, const WaitCtl& wc, const PlanTile& tile,
                                      Blocks blocks) {
    const int piece = lane % 8;
    const T* from[8];  // rows 32 q + 4 i + lane / 8
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 32 * q + 4 * i + lane / 8;
      from[i] = r < tile.count ? static_cast<const T*>(p.x) + __ldg(p.order + tile.start + r) * p.ldx + piece * 8
                               : nullptr;
    }
    for (int i = 0; i < blocks.count + lag; ++i) {
      if (i < blocks.count) {
        if (!warp_wait(&s.empty[stage], phase ^ 1u, wc)) {
          cp_async_wait_all();
          return false;
        }
        uint8_t* to = ring + stage * stage_bytes;
        const int k = blocks.kb * kBlockK;
        const int bytes = k + piece * 8 < p.K ? 16 : 0;  // zeros past the last column
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = 32 * q + 4 * j + lane / 8;
          if (from[j] != nullptr)
            cp_async16_zfill(to + r * 128 + (piece ^ (r & 7)) * 16, bytes != 0 ? from[j] + k : from[j], bytes);
        }
        blocks.next();
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      cp_async_commit();
      if (i >= lag) {
        if (lag == 4) cp_async_wait_group<4>();
        else if (lag == 3) cp_async_wait_group<3>();
        else if (lag == 2) cp_async_wait_group<2>();
        else cp_async_wait_group<1>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.full[told]);
        if (++told == p.stages) told = 0;
      }
    }
    return true;
  }
};

// A CTA takes every so manieth unit (tile, cut): the tile's products over every
// so manieth reduction block, so that a tile's CTAs read neighbouring pieces of
// its rows at the same time.
template <typename T>
__global__ void __launch_bounds__(kShrinkThreads)
    shrink_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
                  const ShrinkParams p) {
  extern __shared__ uint8_t smem_raw[];
  let_next_launch();
  const PlanHead head = *p.head;
  if (head.n != p.n || head.slots != p.slots) {  // another batch's plan
    if (blockIdx.x == 0 && threadIdx.x == 0) report(p.status, MOE_ERR_DEVICE);
    return;
  }
  const int cuts = cuts_of(head.tiles, gridDim.x, p.kblocks), units = head.tiles * cuts;
  if (static_cast<int>(blockIdx.x) >= units) return;
  const bool few = few_tokens(head, p.few);
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int stage_bytes = kTokenStage + p.width * kBlockK * 2;
  ShrinkCtl& s = *reinterpret_cast<ShrinkCtl*>(ring + p.stages * stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cols = tmem_width(p.width);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s.full[i], few ? 1 : 1 + 4);  // warp 0, and the four warps that copy tokens
      mbar_init(&s.empty[i], 1);
    }
    mbar_init(&s.done, 1);
    mbar_init(&s.drained, 4);
    s.abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_a);
  }
  if (warp == 1) {
    tmem_alloc<1>(&s.tmem_base, cols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const WaitCtl wc{&s.abort_flag, p.status, p.limit_ns};

  if (warp == 0) {
    int stage = 0, filled = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const PlanTile tile = p.tiles[u / cuts];
      // Tiles of few tokens: lane i gathers the tile's tokens 4i .. 4i + 3 (past the
      // last: the last again; their rows of the product are not stored).
      const int groups = few ? (tile.count + 3) / 4 : 0;
      int row[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) row[i] = few ? __ldg(p.order + tile.start + min(4 * lane + i, tile.count - 1)) : 0;
      Blocks blocks(u, cuts, p.kblocks);
      for (int i = 0; i < blocks.count; ++i, blocks.next()) {
        ok = warp_wait(&s.empty[stage], phase ^ 1u, wc);
        if (!ok) break;
        uint8_t* to = ring + stage * stage_bytes;
        if (lane == 0) {
          mbar_arrive_expect_tx(&s.full[stage], groups * 512 + p.width * kBlockK * 2);
          tma_load_3d(to + kTokenStage, &map_a, &s.full[stage], blocks.kb * kBlockK, 0, tile.adapter);
        }
        __syncwarp();  // armed before any gather lands
        if (lane < groups) gather4(to + 512 * lane, &map_x, &s.full[stage], blocks.kb * kBlockK, row);
        ++filled;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {  // copies in flight land before the CTA goes on
      for (int i = 0; i < p.stages; ++i) {
        const int f = filled > i ? (filled - i + p.stages - 1) / p.stages : 0;
        if (f > 0) (void)mbar_wait_drain(&s.full[i], (f - 1) & 1, 100000000ull);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = dense_idesc(kTile, p.width, false, false, p.type);
      const uint32_t base = smem_u32(ring);
      const Operand op = operand128<false>();
      int stage = 0, done = 0, unit = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++unit) {
        if (unit > 0) ok = mbar_wait(&s.drained, (unit - 1) & 1, wc);
        tc_fence_after();
        const int count = Blocks(u, cuts, p.kblocks).count;
        for (int i = 0; i < count && ok; ++i) {
          ok = mbar_wait(&s.full[stage], phase, wc);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = base + stage * stage_bytes;
          issue_block<1>(tmem, at, at + kTokenStage, op, op, idesc, i > 0 ? 1u : 0u);
          umma_commit<1>(&s.empty[stage]);
          ++done;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit<1>(&s.done);
      }
      if (!ok && done > 0) {  // issued products end before TMEM is freed
        const int last = (done - 1) % p.stages;
        (void)mbar_wait_drain(&s.empty[last], ((done - last + p.stages - 1) / p.stages - 1) & 1, 100000000ull);
      }
    }
  } else {
    const int q = warp & 3, tid = q * 32 + lane;  // also this thread's token of the tile
    TokenCopies<T> copies(p, ring, stage_bytes, q, lane);
    int unit = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++unit) {
      const PlanTile tile = p.tiles[u / cuts];
      const bool copied = few || copies.run(p, s, wc, tile, Blocks(u, cuts, p.kblocks));
      // the four warps meet at barriers below: all go on or none does
      if (!epi_all(copied && warp_wait(&s.done, unit & 1, wc))) break;
      tc_fence_after();
      const int64_t at = static_cast<int64_t>(tile.start + tid) * p.width;
      const float scale = __ldg(p.scale + tile.adapter);
      for (int c0 = 0; c0 < p.width; c0 += 16) {  // ranks past the last: sums of x times 0
        uint32_t v[16];
        tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c0, v);
        tmem_ld_wait();
        if (tid < tile.count) {
          if (cuts > 1) {
            float* to = p.parts + static_cast<int64_t>(u % cuts) * head.live * p.width + at + c0;
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              __stcg(reinterpret_cast<float4*>(to + j),
                     make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                                 __uint_as_float(v[j + 3])));
          } else {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              w[j] = pack_pair(scale * __uint_as_float(v[2 * j]), scale * __uint_as_float(v[2 * j + 1]), T{});
            uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(p.v) + at + c0);
            to[0] = make_uint4(w[0], w[1], w[2], w[3]);
            to[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.drained);
      if (cuts > 1 && few) {
        epi_sync();
        if (tid == 0) {  // releases the four warps' part, and acquires the others' where it is the last
          int before;
          asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.arrived + u / cuts) : "memory");
          s.last = before == cuts - 1 ? 1 : 0;
        }
        epi_sync();
        if (s.last) {
          join_parts<T>(p, tile, head.live, cuts, tid, s.sums);
          if (tid == 0) p.arrived[u / cuts] = 0;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, cols);
  }
}

// ------------------------------------------------------------------ expand
constexpr int kExpandThreads = 128;
constexpr int kExpandBlocks = 4;                  // to an SM (three of rank 128)
constexpr int kExpandCols = kExpandThreads;       // of a unit: 32 to a warp
constexpr int kExpandTokens = 64;                 // of a unit: half a tile
constexpr int kPieces = kExpandTokens / 8;        // 16-byte pieces of res of a thread
struct ExpandParams {
  const PlanHead* head;
  const PlanTile* tiles;
  const int32_t* order;
  const void* v;
  const void *b, *res;
  void* y;
  int64_t ldres, ldy;
  int n, slots, N, rank, width;
  int halves;    // of a tile: one where no tile can have more tokens than a unit
  bool few;
  bool in_place;  // y is res: nothing to do for tokens without an adapter
};
// Words of a row of v in shared memory: 8 more than whole 32s, so that the
// eight rows of a fragment lie in different banks.
__host__ __device__ constexpr int v_words(int kb) { return 8 * kb + (40 - 8 * kb % 32) % 32; }
__host__ __device__ constexpr size_t expand_smem(int kb) {
  return static_cast<size_t>(2 * kPieces) * kExpandThreads * 16 + static_cast<size_t>(2 * kExpandTokens) * v_words(kb) * 4;
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Units of up to 64 of a tile's tokens by 128 columns, the columns of the same
// tokens one after another; a block takes an equal run of them.  A warp has 32
// columns: it holds its part of b in registers and walks down the tokens, 16 at
// a time.  The next unit's part of res is on its way into the threads' own
// slots of shared memory meanwhile (64 KB to an SM; one unit to a block, with
// its loads, its products and its stores one after another, took 60 us where
// this takes 36, at 32768 tokens of 1536 columns), and so is v where the tokens
// change.  In a fragment, lane 4 g + q holds reduction elements 4 q .. 4 q + 3 of
// each 16 (in both operands), and the columns 8 q .. 8 q + 7 of rows g and g + 8:
// column c of the j-th of its four MMAs is column 8 (c / 2) + 2 j + c % 2 of the
// warp's.
template <typename T, int KB>
__global__ void __launch_bounds__(kExpandThreads, KB > 4 ? 3 : kExpandBlocks) expand_kernel(const ExpandParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* const slots = reinterpret_cast<uint4*>(smem) + threadIdx.x;
  uint32_t* const vs = reinterpret_cast<uint32_t*>(smem + static_cast<size_t>(2 * kPieces) * kExpandThreads * 16);
  constexpr int kWords = v_words(KB);
  // the plan and res are older than the call: no need to wait for those
  const PlanHead head = *p.head;
  const bool mine = head.n == p.n && head.slots == p.slots, early = KB > 1 && !few_tokens(head, p.few);
  const int chunks = (p.N + kExpandCols - 1) / kExpandCols;
  const int64_t units = mine ? static_cast<int64_t>(head.tiles + (p.in_place ? 0 : head.none)) * p.halves * chunks : 0;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;

  // where the next unit lies, and its rows 8 i + g (-1: none)
  int64_t next = u0;
  int t_next = u0 < u1 ? static_cast<int>(u0 / chunks) : 0, c_next = u0 < u1 ? static_cast<int>(u0 % chunks) : 0;
  PlanTile tile_next{};
  int count_next = 0, row_next[kPieces];
  const auto look = [&] {
    tile_next = p.tiles[t_next / p.halves];
    tile_next.start += t_next % p.halves * kExpandTokens;
    count_next = max(0, min(kExpandTokens, tile_next.count - t_next % p.halves * kExpandTokens));
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      row_next[i] = 8 * i + g < count_next ? p.order[tile_next.start + 8 * i + g] : -1;
  };
  // v of the next unit's tokens, by the whole block: 16-byte pieces of rows, and
  // zeros past the ranks that there are (v holds an infinite row's x times 0 there)
  const auto fetch_v = [&](int half) {
    constexpr int kRow = 2 * KB;  // pieces
    const bool named = t_next / p.halves < head.tiles;
    for (int i = threadIdx.x; named && i < count_next * kRow; i += kExpandThreads) {
      const int r = i / kRow, e = i % kRow * 8;
      cp_async16_zfill(vs + (half * kExpandTokens + r) * kWords + e / 2,
                       static_cast<const T*>(p.v) + static_cast<int64_t>(tile_next.start + r) * p.width +
                           (e < p.rank ? e : 0),
                       e < p.rank ? 16 : 0);
    }
  };
  const auto fetch = [&](int buffer) {  // the next unit's part of res
    const int col = c_next * kExpandCols + warp * 32 + 8 * q;
    if (next < u1 && p.res != nullptr && col < p.N) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (row_next[i] >= 0)
          cp_async16(slots + (buffer * kPieces + i) * kExpandThreads,
                     static_cast<const T*>(p.res) + row_next[i] * p.ldres + col);
    }
    cp_async_commit();
  };
  // a unit's part of b, into registers
  uint2 b[4][KB];
  const auto load_b = [&](int adapter, int c0) {
    const T* pool = static_cast<const T*>(p.b) + static_cast<int64_t>(adapter) * p.N * p.rank;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
      for (int k = 0; k < KB; ++k)
        b[j][k] = col < p.N && 16 * k + 4 * q < p.rank
                      ? *reinterpret_cast<const uint2*>(pool + static_cast<int64_t>(col) * p.rank + 16 * k + 4 * q)
                      : make_uint2(0u, 0u);
    }
  };
  if (u0 < u1) look();
  fetch(0);
  wait_for_previous();
  int half = 0, buffer = 0;  // of v's, of res's slots
  if (u0 < u1) fetch_v(0);
  cp_async_commit();
  bool fresh = true;  // this block's other threads have copied v for this unit
  for (int64_t u = u0; u < u1; ++u, buffer ^= 1) {
    const int count = count_next, c0 = c_next * kExpandCols + warp * 32, col = c0 + 8 * q, adapter = tile_next.adapter;
    const bool in = col < p.N, named = t_next / p.halves < head.tiles;
    int row[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) row[i] = row_next[i];
    next = u + 1;
    const bool first = fresh;
    fresh = ++c_next == chunks;
    if (fresh) {
      // the other half of v was read for the tile before this one: ahead of this
      // tile's barrier below, unless that is still to come
      if (first) __syncthreads();
      c_next = 0;
      ++t_next;
      if (next < u1) {
        look();
        fetch_v(half ^ 1);
      }
    }
    fetch(buffer ^ 1);
    // Past rank 16, full tiles' b comes as soon as the unit before has done with
    // its own (32768 tokens of rank 32 69 us, 73 all here); of few tokens, where it
    // comes from HBM, it is better asked for after res (2000 of 1024 adapters 97
    // us, 106 the other way); of rank 16 the further code costs as much as it gives
    // (61 tokens 13.5 us against 14.3 with it, 32000 98 against 96).
    if (named && count > 0 && (!early || u == u0)) load_b(adapter, c0);
    cp_async_wait_group<1>();
    if (first) __syncthreads();  // the same for the whole block
#pragma unroll
    for (int s = 0; s < kPieces / 2; ++s) {
      if (16 * s >= count) break;
      uint4 r[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        r[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p.res != nullptr && in && row[2 * s + i] >= 0)
          r[i] = slots[(buffer * kPieces + 2 * s + i) * kExpandThreads];
      }
      if (named) {
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // the products are added to res
          Raw<T, 8> raw;
          raw.v = r[i];
          float f[8];
          raw.unpack(f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[j][2 * i] = f[2 * j];
            acc[j][2 * i + 1] = f[2 * j + 1];
          }
        }
        // (rows past the tile's last hold anything: their results are dropped)
        const uint32_t* at = vs + (half * kExpandTokens + 16 * s + g) * kWords + 2 * q;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          const uint2 lo = *reinterpret_cast<const uint2*>(at + 8 * k);
          const uint2 hi = *reinterpret_cast<const uint2*>(at + 8 * kWords + 8 * k);
          const uint32_t a[4] = {lo.x, hi.x, lo.y, hi.y};
#pragma unroll
          for (int j = 0; j < 4; ++j) mma16816<T>(acc[j], a, b[j][k].x, b[j][k].y);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[2 * j] = acc[j][2 * i];
            f[2 * j + 1] = acc[j][2 * i + 1];
          }
          Raw<T, 8> raw;
          raw.pack(f);
          r[i] = raw.v;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (in && row[2 * s + i] >= 0)
          *reinterpret_cast<uint4*>(static_cast<T*>(p.y) + row[2 * s + i] * p.ldy + col) = r[i];
    }
    if (fresh) half ^= 1;
    if (early && next < u1 && t_next / p.halves < head.tiles && count_next > 0)
      load_b(tile_next.adapter, c_next * kExpandCols + warp * 32);
  }
  cp_async_wait_all();
}

// --------------------------------------------------------------- host side
// The pool [slots][rank][K] in boxes of 64 elements of all of an adapter's
// rows; rows past the rank and elements past K read as zero.
bool map_pool(CUtensorMap* m, const void* base, uint64_t K, uint64_t rank, uint64_t slots, uint32_t width) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {K, rank, slots}, strides[2] = {K * 2, K * rank * 2};
  const cuuint32_t box[3] = {64, width, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMostSms = 192;  // any device of this kind has fewer
constexpr int kShrinkSmem = 110 * 1024;  // two CTAs to an SM
static_assert(1024 + kMinStages * (kTokenStage + 128 * kBlockK * 2) + sizeof(ShrinkCtl) <= kShrinkSmem, "rank 128");

cudaError_t allow_smem(const void* kern, std::atomic<bool> (&set)[64], int bytes) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) set[dev].store(true, std::memory_order_release);
  return err;
}

template <typename T>
cudaError_t launch_shrink(const ShrinkParams& p, const CUtensorMap& mx, const CUtensorMap& ma, int grid, size_t bytes, cudaStream_t s) {
  static std::atomic<bool> set[64];
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(shrink_kernel<T>), set, kShrinkSmem);
  if (err != cudaSuccess) return err;
  shrink_kernel<T><<<grid, kShrinkThreads, bytes, s>>>(mx, ma, p);
  const cudaError_t launched = cudaGetLastError();
  if (launched != cudaSuccess || p.few) return launched;
  JoinParams j{};
  j.head = p.head;
  j.tiles = p.tiles;
  j.parts = p.parts;
  j.scale = p.scale;
  j.v = p.v;
  j.n = p.n;
  j.slots = p.slots;
  j.width = p.width;
  j.kblocks = p.kblocks;
  j.shrink_grid = grid;
  cudaLaunchAttribute overlap = overlap_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * sm_count()));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T>, j);
}
template <typename T, int KB>
cudaError_t launch_expand(const ExpandParams& p, dim3 grid, cudaStream_t s) {
  static std::atomic<bool> set[64];
  constexpr size_t bytes = expand_smem(KB);
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(expand_kernel<T, KB>), set, static_cast<int>(bytes));
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute overlap = overlap_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kExpandThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, expand_kernel<T, KB>, p);
}
template <typename T>
cudaError_t launch_expand(const ExpandParams& p, dim3 grid, int kb, cudaStream_t s) {
  if (kb <= 1) return launch_expand<T, 1>(p, grid, s);
  if (kb <= 2) return launch_expand<T, 2>(p, grid, s);
  if (kb <= 4) return launch_expand<T, 4>(p, grid, s);
  return launch_expand<T, 8>(p, grid, s);
}

}  // namespace

size_t adapter_plan_bytes(int64_t T, int slots) {
  return plan_order_at(T, slots) + (static_cast<size_t>(T) * 4 + 255) / 256 * 256;
}
// Workspace: the tiles' counters (zero between calls), v, the parts: as many
// cuts as make the tiles of 128 tokens fill the grid.
struct AdapterLayout {
  size_t v, parts, all;
  explicit AdapterLayout(const moe_adapter_dims& d) {
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t width = (d.rank + 15) / 16 * 16;
    v = up(static_cast<size_t>(most_tiles(d.T, d.slots)) * 4);
    parts = v + up(static_cast<size_t>(d.T) * width * 2);
    all = parts + 2 * static_cast<size_t>(kMostSms) * kTile * width * 4;
  }
};
size_t adapter_ws_bytes(const moe_adapter_dims& d) { return AdapterLayout(d).all; }

cudaError_t launch_adapter_plan(const int32_t* ids, int32_t n, int32_t T, int32_t slots, void* plan,
                                int32_t* dev_status, cudaStream_t s) {
  static std::atomic<bool> set[64];
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(plan_kernel), set, kPlanWarps * 1025 * 4);
  if (err != cudaSuccess) return err;
  uint8_t* at = static_cast<uint8_t*>(plan);
  plan_kernel<<<1, kPlanThreads, kPlanWarps * (slots + 1) * 4, s>>>(
      ids, n, slots, reinterpret_cast<PlanHead*>(at), reinterpret_cast<PlanTile*>(at + sizeof(PlanHead)),
      reinterpret_cast<int32_t*>(at + plan_order_at(T, slots)), dev_status);
  return cudaGetLastError();
}

cudaError_t launch_adapters(const AdapterCall& c, cudaStream_t s) {
  const moe_adapter_dims& d = c.d;
  const uint8_t* at = static_cast<const uint8_t*>(c.plan);
  const int64_t most = most_tiles(c.n, d.slots);
  ShrinkParams p{};
  p.x = c.x;
  p.ldx = c.ldx;
  p.K = d.K;
  p.head = reinterpret_cast<const PlanHead*>(at);
  p.tiles = reinterpret_cast<const PlanTile*>(at + sizeof(PlanHead));
  p.order = reinterpret_cast<const int32_t*>(at + plan_order_at(d.T, d.slots));
  const AdapterLayout ws(d);
  uint8_t* scratch = static_cast<uint8_t*>(c.ws);
  p.arrived = reinterpret_cast<int32_t*>(scratch);
  p.v = scratch + ws.v;
  p.parts = reinterpret_cast<float*>(scratch + ws.parts);
  p.scale = c.scale;
  p.n = c.n;
  p.slots = d.slots;
  p.few = few_tokens(c.n, d.slots);
  p.width = (d.rank + 15) / 16 * 16;
  p.kblocks = (d.K + kBlockK - 1) / kBlockK;
  p.type = d.type == MOE_BF16 ? 1u : 0u;
  p.status = c.dev_status;
  p.limit_ns = kDefaultWaitLimitNs;
  const size_t stage = kTokenStage + static_cast<size_t>(p.width) * kBlockK * 2;
  p.stages = static_cast<int>(std::min<size_t>(kMaxStages, (kShrinkSmem - 1024 - sizeof(ShrinkCtl)) / stage));
  const size_t bytes = 1024 + p.stages * stage + sizeof(ShrinkCtl);
  CUtensorMap mx, ma;
  if (!map_rows(&mx, c.x, d.K, c.n, c.ldx) || !map_pool(&ma, c.a, d.K, d.rank, d.slots, p.width)) return cudaErrorInvalidValue;
  // no more CTAs than units of the fewest blocks
  const int grid = static_cast<int>(std::min<int64_t>(
      2 * std::min(sm_count(), kMostSms), most * std::max(1, p.kblocks / kLeastCutBlocks)));
  const cudaError_t err = d.type == MOE_BF16 ? launch_shrink<__nv_bfloat16>(p, mx, ma, grid, bytes, s)
                                             : launch_shrink<__half>(p, mx, ma, grid, bytes, s);
  if (err != cudaSuccess) return err;

  ExpandParams e{};
  e.head = p.head;
  e.tiles = p.tiles;
  e.order = p.order;
  e.v = p.v;
  e.b = c.b;
  e.res = c.res;
  e.ldres = c.ldres;
  e.y = c.y;
  e.ldy = c.ldy;
  e.n = c.n;
  e.slots = d.slots;
  e.N = d.N;
  e.rank = d.rank;
  e.width = p.width;
  e.few = p.few;
  e.halves = c.n <= kExpandTokens ? 1 : kTile / kExpandTokens;
  e.in_place = c.y == c.res && c.ldy == c.ldres;
  const int64_t units = most * e.halves * ((d.N + kExpandCols - 1) / kExpandCols);
  const int kb = p.width / 16, per_sm = kb > 4 ? 3 : kExpandBlocks;
  const dim3 blocks(static_cast<unsigned>(std::min<int64_t>(units, per_sm * sm_count())));
  return d.type == MOE_BF16 ? launch_expand<__nv_bfloat16>(e, blocks, kb, s) : launch_expand<__half>(e, blocks, kb, s);
}

}  // namespace moe
