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
// gathered straight from x (four rows of 128 bytes to a TMA gather) as the 128
// side, the rank is the narrow side, and the reduction over K is cut among
// CTAs where tiles are few.  Bound by reading x; for a few tokens by latency.
// expand: y = res + scale v b_s^T.  Its reduction is the rank, one to eight
// MMAs deep, so that nearly all of it is moving res and y: the products are
// mma.sync's, whose accumulators already lie in the registers that add and
// store (tensor memory would add a round trip to a kernel without a main loop).
// Columns and reduction indices are permuted among the fragments so that every
// access is 8 or 16 contiguous bytes; nothing goes through shared memory.
//
// v is summed in fp32 (over the cuts in their order) and rounded once to the
// operands' type for the second product, with the scale: half a step on each of
// r terms, below the result's own rounding.
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
  int32_t n, slots, tiles, pad;
};
struct PlanTile {
  int32_t adapter, start, count, pad;  // adapter -1: none
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
  const auto bucket_of = [&](int j) {
    if (j >= j1) return -1;
    const int id = __ldg(ids + j);
    return id >= 0 && id < slots ? id : slots;
  };
  for (int j = j0; j < j1; j += 32) {
    const int b = bucket_of(j + lane);
    if (b == slots && __ldg(ids + j + lane) != -1) report(status, MOE_ERR_DEVICE);
    const uint32_t peers = __match_any_sync(0xffffffffu, b);
    if (b >= 0 && lane == __ffs(peers) - 1) mine[b] += __popc(peers);
    __syncwarp();
  }
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
      tiles[tile++] = PlanTile{b < slots ? b : -1, at + i, min(kTile, c - i), 0};
    at += c;
  }
  if (threadIdx.x == 0) *head = PlanHead{n, slots, all, 0};
  __syncthreads();
  for (int j = j0; j < j1; j += 32) {
    const int b = bucket_of(j + lane);
    const uint32_t peers = __match_any_sync(0xffffffffu, b);
    const int first = b >= 0 ? mine[b] : 0;
    __syncwarp();
    if (b >= 0) {
      order[first + __popc(peers & ((1u << lane) - 1u))] = j + lane;
      if (lane == __ffs(peers) - 1) mine[b] = first + __popc(peers);
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------ shrink
constexpr int kShrinkThreads = 192;
constexpr int kTokenStage = kTile * kBlockK * 2;  // 16 KB
constexpr int kMaxStages = 8;

struct ShrinkParams {
  const PlanHead* head;
  const PlanTile* tiles;
  const int32_t* order;
  float* v;             // [splits][n][r]: by place in the order
  int n, slots, rank, width, kblocks, splits, stages;  // width: rank in whole 16s
  uint32_t type;
  int32_t* status;
  uint64_t limit_ns;
};
struct ShrinkCtl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
};
__host__ __device__ constexpr int tmem_width(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : 128; }

// Four rows of a map whose box is 64 columns of one row, into 512 consecutive
// bytes (swizzled by their address like any tile).
__device__ __forceinline__ void gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                        const int (&r)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]),
      "r"(r[3])
      : "memory");
}

// Block (tile, split): the tile's products over the split's reduction blocks.
__global__ void __launch_bounds__(kShrinkThreads)
    shrink_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
                  const ShrinkParams p) {
  extern __shared__ uint8_t smem_raw[];
  let_next_launch();
  const PlanHead head = *p.head;
  if (head.n != p.n || head.slots != p.slots) {  // another batch's plan
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report(p.status, MOE_ERR_DEVICE);
    return;
  }
  if (static_cast<int>(blockIdx.x) >= head.tiles) return;
  const PlanTile tile = p.tiles[blockIdx.x];
  if (tile.adapter < 0) return;
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int stage_bytes = kTokenStage + p.width * kBlockK * 2;
  ShrinkCtl& s = *reinterpret_cast<ShrinkCtl*>(ring + p.stages * stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * blockIdx.y / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (blockIdx.y + 1) / p.splits);
  const int cols = tmem_width(p.width);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    mbar_init(&s.done, 1);
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
    // lane i gathers tokens 4i .. 4i + 3 of the tile (past the last: the last
    // again; their rows of the product are not stored)
    const int groups = (tile.count + 3) / 4;
    int row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = __ldg(p.order + tile.start + min(4 * lane + i, tile.count - 1));
    int stage = 0, filled = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = warp_wait(&s.empty[stage], phase ^ 1u, wc);
      if (!ok) break;
      uint8_t* at = ring + stage * stage_bytes;
      if (lane == 0) {
        mbar_arrive_expect_tx(&s.full[stage], groups * 512 + p.width * kBlockK * 2);
        tma_load_3d(at + kTokenStage, &map_a, &s.full[stage], kb * kBlockK, 0, tile.adapter);
      }
      __syncwarp();  // armed before any gather lands
      if (lane < groups) gather4(at + 512 * lane, &map_x, &s.full[stage], kb * kBlockK, row);
      ++filled;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
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
      int stage = 0, done = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = mbar_wait(&s.full[stage], phase, wc);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = base + stage * stage_bytes;
        issue_block<1>(tmem, at, at + kTokenStage, op, op, idesc, kb > kb0 ? 1u : 0u);
        umma_commit<1>(&s.empty[stage]);
        ++done;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) {
        umma_commit<1>(&s.done);
      } else if (done > 0) {  // issued products end before TMEM is freed
        const int last = (done - 1) % p.stages;
        (void)mbar_wait_drain(&s.empty[last], ((done - last + p.stages - 1) / p.stages - 1) & 1, 100000000ull);
      }
    }
  } else {
    const int q = warp & 3, i = q * 32 + lane;  // this thread's token of the tile
    if (warp_wait(&s.done, 0, wc)) {
      tc_fence_after();
      float* to = p.v + (static_cast<int64_t>(blockIdx.y) * p.n + tile.start + i) * p.rank;
      for (int c0 = 0; c0 < p.width; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c0, v);
        tmem_ld_wait();
        if (i < tile.count) {
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            if (c0 + j < p.rank)
              *reinterpret_cast<float4*>(to + c0 + j) = make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                                                                    __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
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
constexpr int kExpandWarps = 4;
constexpr int kExpandTokens = 32;  // of a block: two MMAs of 16
struct ExpandParams {
  const PlanHead* head;
  const PlanTile* tiles;
  const int32_t* order;
  const float* v;
  const void *b, *res;
  const float* scale;
  void* y;
  int64_t ldres, ldy;
  int n, slots, N, rank, splits, groups;  // groups: of 32 columns, to a warp
};

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

// Block (tile, columns, quarter of the tile): 32 tokens by 4 * groups * 32
// columns, a warp a quarter of these.  In a fragment, lane 4 g + q holds
// reduction elements 4 q .. 4 q + 3 of each 16 (in both operands), and of a
// group of 32 columns the columns 8 q .. 8 q + 7 of rows g and g + 8: column c
// of the j-th of its four MMAs is column 8 (c / 2) + 2 j + c % 2 of the group.
template <typename T, int KB>
__global__ void __launch_bounds__(32 * kExpandWarps) expand_kernel(const ExpandParams p) {
  // the plan is older than the call: no need to wait for that
  const PlanHead head = *p.head;
  if (head.n != p.n || head.slots != p.slots || static_cast<int>(blockIdx.x) >= head.tiles) {
    wait_for_previous();
    return;
  }
  const PlanTile tile = p.tiles[blockIdx.x];
  const int t0 = blockIdx.z * kExpandTokens;
  if (t0 >= tile.count) {
    wait_for_previous();
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int m_tiles = tile.count - t0 > 16 ? 2 : 1;
  const int first = (blockIdx.y * kExpandWarps + warp) * p.groups * 32;  // column
  // rows g and g + 8 of either 16 tokens
  int row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = t0 + 8 * i + g;
    row[i] = at < tile.count ? __ldg(p.order + tile.start + at) : -1;
  }
  uint32_t a[2][KB][4];
  wait_for_previous();
  if (tile.adapter >= 0) {
    const float scale = __ldg(p.scale + tile.adapter);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* at = p.v + static_cast<int64_t>(tile.start + t0 + 8 * i + g) * p.rank + 4 * q;
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row[i] >= 0 && 16 * k + 4 * q < p.rank) {
          for (int sp = 0; sp < p.splits; ++sp) {
            const float4 d = *reinterpret_cast<const float4*>(at + static_cast<int64_t>(sp) * p.n * p.rank + 16 * k);
            f.x += d.x, f.y += d.y, f.z += d.z, f.w += d.w;
          }
        }
        a[i / 2][k][i % 2] = pack_pair(scale * f.x, scale * f.y, T{});
        a[i / 2][k][2 + i % 2] = pack_pair(scale * f.z, scale * f.w, T{});
      }
    }
  }
  const T* b = static_cast<const T*>(p.b) + static_cast<int64_t>(max(tile.adapter, 0)) * p.N * p.rank;
  for (int grp = 0; grp < p.groups; ++grp) {
    const int c0 = first + grp * 32;
    if (c0 >= p.N) break;
    const int col = c0 + 8 * q;  // of this lane's eight results
    uint4 r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.res != nullptr && row[i] >= 0 && col < p.N)
        r[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.res) + row[i] * p.ldres + col);
    }
    float acc[2][4][4];
    if (tile.adapter >= 0) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int bc = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
        const T* at = b + static_cast<int64_t>(bc) * p.rank + 4 * q;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          uint2 w = make_uint2(0u, 0u);
          if (bc < p.N && 16 * k + 4 * q < p.rank) w = __ldg(reinterpret_cast<const uint2*>(at + 16 * k));
          mma16816<T>(acc[0][j], a[0][k], w.x, w.y);
          if (m_tiles > 1) mma16816<T>(acc[1][j], a[1][k], w.x, w.y);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (row[i] < 0 || col >= p.N) continue;
      uint4 out = r[i];
      if (tile.adapter >= 0) {
        Raw<T, 8> raw;
        raw.v = r[i];
        float f[8];
        raw.unpack(f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] += acc[i / 2][j][2 * (i % 2)];
          f[2 * j + 1] += acc[i / 2][j][2 * (i % 2) + 1];
        }
        raw.pack(f);
        out = raw.v;
      }
      *reinterpret_cast<uint4*>(static_cast<T*>(p.y) + row[i] * p.ldy + col) = out;
    }
  }
}

// --------------------------------------------------------------- host side
bool map_gather(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t ld) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {inner, rows}, strides[1] = {ld * 2};
  const cuuint32_t box[2] = {64, 1}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
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

constexpr int kMostSms = 192;       // any device of this kind has fewer
constexpr int kLeastSplitBlocks = 4;

// Cuts of the reduction: CTAs for two to an SM, by the tiles that n tokens
// probably make, and four blocks to a CTA at least.
int shrink_splits(int64_t n, int slots, int kblocks, int sms) {
  const int64_t tiles = std::max<int64_t>((n + kTile - 1) / kTile, std::min<int64_t>(n, slots));
  const int64_t want = 2 * static_cast<int64_t>(sms) / tiles;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, kblocks / kLeastSplitBlocks)));
}

template <typename T>
cudaError_t launch_expand(const ExpandParams& p, dim3 grid, int kb, cudaStream_t s) {
  cudaLaunchAttribute overlap = overlap_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * kExpandWarps);
  cfg.stream = s;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  if (kb <= 1) return cudaLaunchKernelEx(&cfg, expand_kernel<T, 1>, p);
  if (kb <= 2) return cudaLaunchKernelEx(&cfg, expand_kernel<T, 2>, p);
  if (kb <= 4) return cudaLaunchKernelEx(&cfg, expand_kernel<T, 4>, p);
  return cudaLaunchKernelEx(&cfg, expand_kernel<T, 8>, p);
}

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

}  // namespace

size_t adapter_plan_bytes(int64_t T, int slots) {
  return plan_order_at(T, slots) + (static_cast<size_t>(T) * 4 + 255) / 256 * 256;
}
size_t adapter_ws_bytes(const moe_adapter_dims& d) {
  // splits * n rows: splits is 1, or at most 2 SMs' worth over the tiles
  return (static_cast<size_t>(d.T) + 2 * static_cast<size_t>(kMostSms) * kTile) * d.rank * sizeof(float);
}

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
  const auto* head = reinterpret_cast<const PlanHead*>(at);
  const auto* tiles = reinterpret_cast<const PlanTile*>(at + sizeof(PlanHead));
  const auto* order = reinterpret_cast<const int32_t*>(at + plan_order_at(d.T, d.slots));
  const int sms = std::min(sm_count(), kMostSms);
  const unsigned most = static_cast<unsigned>(most_tiles(c.n, d.slots));

  ShrinkParams p{};
  p.head = head;
  p.tiles = tiles;
  p.order = order;
  p.v = static_cast<float*>(c.ws);
  p.n = c.n;
  p.slots = d.slots;
  p.rank = d.rank;
  p.width = (d.rank + 15) / 16 * 16;
  p.kblocks = (d.K + kBlockK - 1) / kBlockK;
  p.splits = shrink_splits(c.n, d.slots, p.kblocks, sms);
  p.type = d.type == MOE_BF16 ? 1u : 0u;
  p.status = c.dev_status;
  p.limit_ns = kDefaultWaitLimitNs;
  const size_t stage = kTokenStage + static_cast<size_t>(p.width) * kBlockK * 2;
  // two CTAs to an SM
  p.stages = static_cast<int>(std::min<size_t>(kMaxStages, (110 * 1024 - 1024 - sizeof(ShrinkCtl)) / stage));
  const size_t bytes = 1024 + p.stages * stage + sizeof(ShrinkCtl);
  static std::atomic<bool> set[64];
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(shrink_kernel), set, 110 * 1024);
  if (err != cudaSuccess) return err;
  CUtensorMap mx, ma;
  if (!map_gather(&mx, c.x, d.K, c.n, c.ldx) || !map_pool(&ma, c.a, d.K, d.rank, d.slots, p.width))
    return cudaErrorInvalidValue;
  shrink_kernel<<<dim3(most, p.splits), kShrinkThreads, bytes, s>>>(mx, ma, p);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;

  ExpandParams e{};
  e.head = head;
  e.tiles = tiles;
  e.order = order;
  e.v = p.v;
  e.b = c.b;
  e.res = c.res;
  e.ldres = c.ldres;
  e.scale = c.scale;
  e.y = c.y;
  e.ldy = c.ldy;
  e.n = c.n;
  e.slots = d.slots;
  e.N = d.N;
  e.rank = d.rank;
  e.splits = p.splits;
  // four groups of 32 columns to a warp where that leaves blocks for all SMs
  const int64_t blocks = (static_cast<int64_t>(c.n) / kExpandTokens + std::min(c.n, d.slots)) * (d.N / 512);
  e.groups = blocks >= 4 * sms ? 4 : 1;
  const unsigned across = static_cast<unsigned>((d.N + 128 * e.groups - 1) / (128 * e.groups));
  const unsigned down = static_cast<unsigned>((std::min(c.n, kTile) + kExpandTokens - 1) / kExpandTokens);
  const dim3 grid(most, across, down);
  const int kb = p.width / 16;
  return d.type == MOE_BF16 ? launch_expand<__nv_bfloat16>(e, grid, kb, s) : launch_expand<__half>(e, grid, kb, s);
}

}  // namespace moe
