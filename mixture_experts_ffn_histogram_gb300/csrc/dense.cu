// Dense products of the linear layer on the fifth-generation tensor cores,
// with its epilogue (bias, activation, residual) in the kernel.
//
//   forward  z = x w + bias, y = act(z) + res     (w [K, N]: its N axis contiguous)
//   dgrad    dx = dz w^T + dx_add
//   wgrad    dw = x^T dz
// Operands are 16-bit, sums fp32 in tensor memory.
//
// split kernel: one 128 x BN tile per cluster, the reduction split over the
// cluster's CTAs.  Each CTA runs a TMA ring over its share of the reduction,
// leaves its fp32 partial tile in its own shared memory, and after a cluster
// barrier every CTA sums one slice of the rows over all partials (in rank
// order, so results are reproducible) and runs the epilogue on it.  Narrow
// tiles swap the roles of the operands (SWAP): the weights' columns are the
// tile's 128 side and 16, 32 or 64 rows its narrow side, so that a handful of
// rows costs a 16-column MMA, the weights are read once by all SMs together,
// and small products have tiles enough for the SMs and short epilogues.
// For fp32 results the accumulators are drained into registers every
// kChunkBlocks reduction blocks: the tensor core's additions truncate, and a
// long chain of them would lose what an fp32 result is asked for.  A 16-bit
// result keeps one chain over the whole reduction: sums of one sign come out
// low by 8e-10 of their value per term (measured: 2.5e-5 at 32768 terms,
// 1.1e-4 at 131072, 4.3e-4 at 524288), below half a step of fp16 to some
// 300,000 terms and of bf16 to some 2,400,000; sums of random signs show
// nothing of it.
// pair kernel: persistent, for products with enough 256 x 256 tiles (or of 192
// or 128 columns) for the SMs.  The CTA pair of a 2-CTA cluster works on one
// tile: each CTA loads its 128 rows of A and half of the columns of B, the even
// CTA issues tcgen05.mma.cta_group::2 (M = 256), and each CTA's tensor memory
// holds its 128 rows twice (the next tile's products overlap the epilogue).
// Sixteen epilogue warps take a quarter of the rows and of the columns each
// (one warp's chain of waits, loads and stores is latency: fewer warps leave
// the epilogue behind short reductions); results, z and the residual move
// through swizzled shared-memory buffers by TMA, the residual of the next tile
// while its products run.
//
// Measured (bf16): 4 x 7168 -> 2048 7.4 us (29 MB of weights: 4.3 us of HBM,
// then launch, set-up and cluster barriers); 8191 x 7168 -> 256 to fp32 33 us
// (bound by what an SM takes in from L2, 32 KB a block); 4096 x 2048 -> 768 with
// GELU and z 19.4 us (one tile a pair, set-up and epilogue not overlapped);
// 32768 x 704 -> 2816 with a residual 108 us (1.2 PFLOP/s beside 370 MB of
// residual and results); dx and dw of 8192 x 7168 x 2048 141 and 129 us (1.71
// and 1.87 PFLOP/s, the tensor rate).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "activation.cuh"
#include "kernels.h"
#include "layer.h"
#include "layer_common.cuh"
#include "tmem_share.h"
#include "umma_tile.cuh"

namespace moe {
namespace {

constexpr int kTileM = 128;
constexpr int kATile = kTileM * kBlockK * 2;     // 16 KB
constexpr int kSplitMaxStages = 12;
constexpr int kChunkBlocks = 8;                  // fp32 results: 512 products per chain
constexpr int kSplitSmemLimit = 220 * 1024;

struct DenseParams {
  const float* bias;
  const void* res;
  void* c;
  void* z;
  int64_t ldres, ldc, ldz;
  int64_t M, N;      // of the output
  int kblocks;       // reduction blocks of 64
  int type, out_type, act;
  int32_t* status;
  uint64_t limit_ns;
};

// Four neighbouring values of an output row, 16-bit or fp32, as they lie in
// memory.
template <typename O>
struct Quad {
  using Store = typename std::conditional<sizeof(O) == 4, float4, uint2>::type;
  Store v;
  __device__ __forceinline__ void load(const O* at) { v = *reinterpret_cast<const Store*>(at); }
  __device__ __forceinline__ float4 get() const {
    if constexpr (sizeof(O) == 4) {
      return v;
    } else {
      const float2 a = unpack_pair(v.x, O{}), b = unpack_pair(v.y, O{});
      return make_float4(a.x, a.y, b.x, b.y);
    }
  }
};
template <typename O>
__device__ __forceinline__ void store4(O* at, const float (&v)[4]) {
  if constexpr (sizeof(O) == 4)
    *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(at) =
        make_uint2(pack_pair(v[0], v[1], O{}), pack_pair(v[2], v[3], O{}));
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// One operand's share of a stage: W rows of 64 reduction elements (K-major,
// one box), or W / 64 chunks of 64 columns (MN-major).
template <bool MN, int W>
__device__ __forceinline__ void operand_load(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int x0,
                                             int k0) {
  if constexpr (!MN) {
    tma_load_2d(dst, map, bar, k0, x0);
  } else {
#pragma unroll
    for (int j = 0; j < W / 64; ++j) tma_load_2d(dst + j * kChunk, map, bar, x0 + 64 * j, k0);
  }
}

// MN-major in 32-wide chunks, 64-byte swizzling (mode 4): eight reduction rows
// of a chunk are 512 bytes.
constexpr int kChunk32 = 32 * kBlockK * 2;
__device__ __forceinline__ Operand operand64() {
  return Operand{(smem_desc_sw128(0, kChunk32, 512) & ~(7ull << 61)) | (4ull << 61), 64};
}
struct SplitCtl {
  uint64_t full[kSplitMaxStages];
  uint64_t empty[kSplitMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint32_t tmem_base;
  int abort_flag;
};

// Columns of a TMEM allocation: a power of two, at least 32.
__host__ __device__ constexpr int tmem_cols(int n) {
  return n <= 32 ? 32 : (n <= 64 ? 64 : (n <= 128 ? 128 : (n <= 256 ? 256 : 512)));
}

// A tile of the split kernel: 128 by BN.  SWAP: the 128 side is the output's
// columns.
constexpr int kSplitThreads = 192;
template <int BN_, bool AMN_, bool BMN_, bool SWAP_>
struct SplitShape {
  static constexpr int BN = BN_;
  static constexpr bool AMN = AMN_, BMN = BMN_, SWAP = SWAP_;
  static constexpr int kStage = kATile + BN * kBlockK * 2;  // operand bytes of a block
  static constexpr int kCols = tmem_cols(2 * BN);
  static constexpr int kRowsOut = SWAP ? BN : kTileM;       // the partial tile
  static constexpr int kColsOut = SWAP ? kTileM : BN;
  static constexpr int kLd = kColsOut + 4;
  static constexpr int kPartial = kRowsOut * kLd * 4;       // laid over the operand ring
  static_assert(!BMN || BN % 64 == 0, "MN-major operands come in 64-wide chunks");
  // The fewest stages: what the partial tile needs, and so many that CTAs that
  // fit an SM's shared memory together never ask for more than its 512
  // tensor-memory columns, beside a kernel of CTA pairs or beside one another
  // (tmem_share.h).
  static constexpr int kOver = 1024 + static_cast<int>(sizeof(SplitCtl));
  static constexpr int stages_of(int bytes) { return (bytes + kStage - 1) / kStage; }
  static constexpr int kFloorBytes = static_cast<int>(kSmSmem) / (kSmTmemCols / kCols + 1) + 1024;
  static constexpr int kBesidePair = static_cast<int>(kSmSmem - kLeastPairSmem - 2 * kBlockSmem) + 1 - kOver;
  static constexpr int kLeast =
      std::max({2, stages_of(kPartial), stages_of(kFloorBytes), stages_of(kBesidePair)});
  static constexpr int kLeastBytes = kLeast * kStage + kOver;
  static_assert(kLeast <= kSplitMaxStages && kLeastBytes <= kSplitSmemLimit, "shared memory");
  static_assert(!fits_beside_pair(kLeastBytes), "a cluster's CTA must not fit beside a pair's");
};

// No mix of split CTAs that fits an SM's shared memory asks for more columns
// than the SM has.
constexpr bool split_mixes_fit() {
  constexpr size_t b16 = SplitShape<16, false, false, true>::kLeastBytes + kBlockSmem;
  constexpr size_t b32 = SplitShape<32, false, false, true>::kLeastBytes + kBlockSmem;
  constexpr size_t b64 = std::min(SplitShape<64, false, false, true>::kLeastBytes,
                                  SplitShape<64, true, true, false>::kLeastBytes) + kBlockSmem;
  constexpr size_t b128 = SplitShape<128, false, false, false>::kLeastBytes + kBlockSmem;
  for (size_t i = 0; i * b16 <= kSmSmem; ++i)
    for (size_t j = 0; i * b16 + j * b32 <= kSmSmem; ++j)
      for (size_t k = 0; i * b16 + j * b32 + k * b64 <= kSmSmem; ++k)
        for (size_t l = 0; i * b16 + j * b32 + k * b64 + l * b128 <= kSmSmem; ++l)
          if (32 * i + 64 * j + 128 * k + 256 * l > kSmTmemCols) return false;
  return true;
}
static_assert(split_mixes_fit(), "split clusters must not wait for each other's columns");

// A CTA's part of a finished tile: rows [r0, r1) of the partial tile that lies
// in shared memory at `ring`, the output's rows from row0 + r0 on.
struct TileEnd {
  int64_t row0, col0;
  int r0, r1;
  uint32_t ring;        // shared address of the partial tile
  const uint8_t* smem;  // ... and its pointer
};

// Sums the partials of the splits (SP or fewer, in rank order) and runs the
// epilogue.  A thread keeps
// to four columns and walks down the rows, G of them at a time: G * SP loads
// are under way together, and addresses advance by constants.
template <class S, typename T, typename O, int G, int SP>
__device__ __forceinline__ void finish_rows(const TileEnd& te, const DenseParams& p, int splits) {
  constexpr bool kExact = sizeof(O) == 4;
  constexpr int kPer = S::kColsOut / 4;          // threads across a row
  constexpr int kDown = kSplitThreads / kPer;    // rows of one pass
  static_assert(kDown * kPer == kSplitThreads, "threads cover whole rows");
  const int cc = (threadIdx.x % kPer) * 4;
  const int64_t col = te.col0 + cc;
  const int64_t last = min(static_cast<int64_t>(te.r1), p.M - te.row0);  // rows below exist
  if (col >= p.N) return;
  int r = te.r0 + threadIdx.x / kPer;
  float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (p.bias != nullptr) bias = __ldg(reinterpret_cast<const float4*>(p.bias + col));
  uint32_t from[SP];
#pragma unroll
  for (int q = 0; q < SP; ++q) {
    const uint32_t at = te.ring + static_cast<uint32_t>(r * S::kLd + cc) * 4;
    from[q] = SP > 1 ? mapa_shared(at, min(q, splits - 1)) : at;
  }
  const int64_t row = te.row0 + r;
  O* c = static_cast<O*>(p.c) + row * p.ldc + col;
  const O* res = p.res != nullptr ? static_cast<const O*>(p.res) + row * p.ldres + col : nullptr;
  T* z = p.z != nullptr ? static_cast<T*>(p.z) + row * p.ldz + col : nullptr;
  for (; r < last; r += G * kDown) {
    // all loads first and without branches: a row past the end reads the
    // last (and is not stored: its residual may already be overwritten)
    float4 f[G][SP];
    Quad<O> e[G];
    int down[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      down[g] = min(g * kDown, static_cast<int>(last - 1) - r);
#pragma unroll
      for (int q = 0; q < SP; ++q) {
        const uint32_t at = from[q] + static_cast<uint32_t>(down[g] * (S::kLd * 4));
        if constexpr (SP > 1) f[g][q] = ld_cluster_f4(at);
        else f[g][q] = *reinterpret_cast<const float4*>(te.smem + (at - te.ring));
      }
    }
    if (res != nullptr) {
#pragma unroll
      for (int g = 0; g < G; ++g) e[g].load(res + down[g] * p.ldres);
    }
    float v[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float4 t = f[g][0];
#pragma unroll
      for (int q = 1; q < SP; ++q) {
        if (q >= splits) break;
        t.x += f[g][q].x;
        t.y += f[g][q].y;
        t.z += f[g][q].z;
        t.w += f[g][q].w;
      }
      v[g][0] = t.x + bias.x;
      v[g][1] = t.y + bias.y;
      v[g][2] = t.z + bias.z;
      v[g][3] = t.w + bias.w;
    }
    if (z != nullptr) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (down[g] == g * kDown) store4<T>(z + down[g] * p.ldz, v[g]);
    }
    act_all<kExact, 4 * G>(&v[0][0], p.act);
    if (res != nullptr) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float4 a = e[g].get();
        v[g][0] += a.x;
        v[g][1] += a.y;
        v[g][2] += a.z;
        v[g][3] += a.w;
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (down[g] == g * kDown) store4<O>(c + down[g] * p.ldc, v[g]);
#pragma unroll
    for (int q = 0; q < SP; ++q) from[q] += G * kDown * S::kLd * 4;
    c += G * kDown * p.ldc;
    if (res != nullptr) res += G * kDown * p.ldres;
    if (z != nullptr) z += G * kDown * p.ldz;
  }
}
template <class S, typename T, typename O>
__device__ __forceinline__ void finish_tile(const TileEnd& te, int splits, const DenseParams& p) {
  if (splits == 1) finish_rows<S, T, O, 4, 1>(te, p, splits);
  else if (splits == 2) finish_rows<S, T, O, 4, 2>(te, p, splits);
  else if (splits <= 4) finish_rows<S, T, O, 2, 4>(te, p, splits);
  else finish_rows<S, T, O, 1, 8>(te, p, splits);
}

template <class S>
__global__ void __launch_bounds__(kSplitThreads)
    dense_split_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, const DenseParams p,
                       const int stages, const int splits, const int chunk_blocks) {
  constexpr int BN = S::BN, kStage = S::kStage;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  SplitCtl& s = *reinterpret_cast<SplitCtl*>(ring + stages * kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int a0 = (blockIdx.x / splits) * kTileM;  // first row of the tile's 128 side
  const int b0 = blockIdx.y * BN;                 // ... of its BN side
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * split / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (split + 1) / splits);
  const int nkb = kb1 - kb0;

  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
    for (int i = 0; i < stages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], 4);
    }
    s.abort_flag = 0;
    mbar_fence_init();
    wait_for_previous();
    // the first stages' operands come while the rest is set up (the barriers
    // are this thread's own so far)
    for (int i = 0; i < min(stages, nkb); ++i) {
      uint8_t* sa = ring + i * kStage;
      mbar_arrive_expect_tx(&s.full[i], kStage);
      operand_load<S::AMN, kTileM>(sa, &map_a, &s.full[i], a0, (kb0 + i) * kBlockK);
      operand_load<S::BMN, BN>(sa + kATile, &map_b, &s.full[i], b0, (kb0 + i) * kBlockK);
    }
  }
  if (warp == 1) {
    tmem_alloc<1>(&s.tmem_base, S::kCols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_for_previous();
  const uint32_t tmem = s.tmem_base;
  const WaitCtl wc{&s.abort_flag, p.status, p.limit_ns};

  if (warp == 0) {
    if (elect_one()) {
      int filled = min(stages, nkb), stage = filled % stages;
      uint32_t phase = filled / stages;
      bool ok = true;
      for (int kb = kb0 + filled; kb < kb1; ++kb) {
        ok = mbar_wait(&s.empty[stage], phase ^ 1u, wc);
        if (!ok) break;
        uint8_t* sa = ring + stage * kStage;
        uint64_t* bar = &s.full[stage];
        mbar_arrive_expect_tx(bar, kStage);
        operand_load<S::AMN, kTileM>(sa, &map_a, bar, a0, kb * kBlockK);
        operand_load<S::BMN, BN>(sa + kATile, &map_b, bar, b0, kb * kBlockK);
        ++filled;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {  // copies in flight land before the CTA goes on
        for (int i = 0; i < stages; ++i) {
          const int f = filled > i ? (filled - i + stages - 1) / stages : 0;
          if (f > 0) (void)mbar_wait_drain(&s.full[i], (f - 1) & 1, 100000000ull);
        }
      }
    }
  } else if (warp == 1) {
    // one thread waits, issues and commits: between two blocks there is
    // nothing for the others to do, and every warp-wide step is latency that
    // the tensor core would idle through
    if (elect_one()) {
      const uint32_t idesc = dense_idesc(kTileM, BN, S::AMN, S::BMN, p.type == MOE_BF16 ? 1u : 0u);
      const uint32_t base = smem_u32(ring);
      int stage = 0, done = 0, left = nkb;
      uint32_t phase = 0;
      bool ok = true;
      for (int chunk = 0; left > 0 && ok; ++chunk) {
        const int n = min(left, chunk_blocks);
        const int slot = chunk & 1;
        if (chunk >= 2) ok = mbar_wait(&s.tempty[slot], ((chunk >> 1) - 1) & 1, wc);
        tc_fence_after();
        uint32_t add = 0u;
        for (int i = 0; i < n && ok; ++i) {
          ok = mbar_wait(&s.full[stage], phase, wc);
          if (!ok) break;
          tc_fence_after();
          issue_block<1>(tmem + slot * BN, base + stage * kStage, base + stage * kStage + kATile,
                         operand128<S::AMN>(), operand128<S::BMN>(), idesc, add);
          add = 1u;
          umma_commit<1>(&s.empty[stage]);
          ++done;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit<1>(&s.tfull[slot]);
        left -= n;
      }
      if (!ok && done > 0) {  // issued products end before TMEM is freed
        const int last = (done - 1) % stages;
        (void)mbar_wait_drain(&s.empty[last], ((done - last + stages - 1) / stages - 1) & 1, 100000000ull);
      }
    }
  } else {
    // drain the accumulators into registers, chunk by chunk
    const int q = warp & 3;  // TMEM lane quarter of this warp
    const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
    float acc[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[j] = 0.0f;
    const int chunks = (nkb + chunk_blocks - 1) / chunk_blocks;
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const int slot = c & 1;
      ok = warp_wait(&s.tfull[slot], (c >> 1) & 1, wc);
      if (!ok) break;
      tc_fence_after();
      if constexpr (BN >= 32) {
#pragma unroll
        for (int j = 0; j < BN; j += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tq + slot * BN + j, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[j + e] += __uint_as_float(v[e]);
        }
      } else {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tq + slot * BN, v);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] += __uint_as_float(v[e]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.tempty[slot]);
    }
    // every product has read its operands: the ring now holds the partial
    // tile, in the output's orientation
    if (ok) {
      float* part = reinterpret_cast<float*>(ring);
      const int r = q * 32 + lane;
      if constexpr (S::SWAP) {
#pragma unroll
        for (int j = 0; j < BN; ++j) part[j * S::kLd + r] = acc[j];
      } else {
#pragma unroll
        for (int j = 0; j < BN; j += 4)
          *reinterpret_cast<float4*>(part + r * S::kLd + j) =
              make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      }
    }
  }
  __syncwarp();
  if (splits > 1) cluster_sync();
  else __syncthreads();
  let_next_launch();

  // this CTA's share of the tile's rows: the sum over the partials of the
  // splits, and the epilogue
  const int r0 = S::kRowsOut * split / splits, r1 = S::kRowsOut * (split + 1) / splits;
  const TileEnd te{S::SWAP ? b0 : a0, S::SWAP ? a0 : b0, r0, r1, smem_u32(ring), ring};
  if (p.out_type == MOE_FP32) {
    if (p.type == MOE_BF16) finish_tile<S, __nv_bfloat16, float>(te, splits, p);
    else finish_tile<S, __half, float>(te, splits, p);
  } else {
    if (p.type == MOE_BF16) finish_tile<S, __nv_bfloat16, __nv_bfloat16>(te, splits, p);
    else finish_tile<S, __half, __half>(te, splits, p);
  }
  tc_fence_before();
  __syncthreads();
  if (splits > 1) cluster_sync();  // the others have read this CTA's partial tile
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, S::kCols);
  }
}

// ------------------------------------------------------------ pair kernel
constexpr int kPairN = 256;
constexpr int kPairEpiWarps = 16;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int kPairStage = 2 * kATile;          // per CTA: 128 A rows, 128 B columns
constexpr int kPairBuf = 32 * 128;              // 32 rows x 64 columns, 16-bit
constexpr int kPairStages = 5;

struct PairCtl {
  uint64_t full[kPairStages];
  uint64_t empty[kPairStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t rbar[kPairEpiWarps];  // a residual chunk landed in the warp's buffer
  uint32_t tmem_base;
  int abort_flag;
};
// The ring takes what the staging buffers leave: with three stages and two
// buffers per warp, 32768 x 704 -> 2816 takes 126 us instead of 108, and
// every longer reduction more.
constexpr size_t kPairSmem = 1024 + static_cast<size_t>(kPairStages) * kPairStage +
                             kPairEpiWarps * kPairBuf + sizeof(PairCtl);
static_assert(kPairSmem <= 227 * 1024, "shared memory");
static_assert(kPairSmem >= kLeastPairSmem, "clusters of other kernels must not fit beside");

struct PairParams {
  const float* bias;
  int64_t M, N;
  int kblocks, m_tiles, n_tiles, act;
  int bn;                  // columns of a tile: 128, 192 or 256
  int b_boxes, stage_bytes;  // boxes of an MN-major B per CTA; bytes of a CTA's stage
  int a_chunks, b_chunks;  // MN-major operands: one box of two 64-wide chunks (3-D map)
  int has_res, has_z;
  const void* res;
  int64_t ldres;
  uint32_t idesc;
  int32_t* status;
  uint64_t limit_ns;
};

// Half h (32 columns) of row `lane` of a 128-byte-swizzled buffer.
__device__ __forceinline__ uint4* buf_unit(uint8_t* buf, int lane, int h, int j) {
  return reinterpret_cast<uint4*>(buf + lane * 128 + (((h * 4 + j) ^ (lane & 7)) << 4));
}
template <typename T>
__device__ __forceinline__ void put32(uint8_t* buf, int lane, int h, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float* f = v + 8 * j;
    *buf_unit(buf, lane, h, j) = make_uint4(pack_pair(f[0], f[1], T{}), pack_pair(f[2], f[3], T{}),
                                            pack_pair(f[4], f[5], T{}), pack_pair(f[6], f[7], T{}));
  }
}
template <typename T>
__device__ __forceinline__ void add32(uint8_t* buf, int lane, int h, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 q = *buf_unit(buf, lane, h, j);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_pair(w[i], T{});
      v[8 * j + 2 * i] += f.x;
      v[8 * j + 2 * i + 1] += f.y;
    }
  }
}

// One operand's share of a stage: up to 128 rows (K-major); or one or two
// 64-wide chunks (two in one box where the map has them), or three 32-wide.
template <bool MN>
__device__ __forceinline__ void pair_load(uint8_t* dst, const CUtensorMap* map, uint32_t bar, int x0,
                                          int k0, int chunked, int boxes) {
  if constexpr (!MN) {
    tma_load_2d_pair(dst, map, bar, k0, x0);
  } else if (chunked) {
    tma_load_3d_pair(dst, map, bar, 0, k0, x0 / 64);
  } else if (boxes == 3) {
#pragma unroll
    for (int i = 0; i < 3; ++i) tma_load_2d_pair(dst + i * kChunk32, map, bar, x0 + 32 * i, k0);
  } else {
    tma_load_2d_pair(dst, map, bar, x0, k0);
    if (boxes == 2) tma_load_2d_pair(dst + kChunk, map, bar, x0 + 64, k0);
  }
}

// FULL: bias, activation and z (the forward); otherwise only a residual.
template <typename T, bool AMN, bool BMN, bool FULL>
__global__ void __launch_bounds__(kPairThreads, 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_c,
                      const __grid_constant__ CUtensorMap map_r,
                      const __grid_constant__ CUtensorMap map_z, const PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* epi = ring + kPairStages * kPairStage;
  PairCtl& s = *reinterpret_cast<PairCtl*>(epi + kPairEpiWarps * kPairBuf);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int units = gridDim.x / 2;
  const int ntiles = p.m_tiles * p.n_tiles;

  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
    tma_prefetch_map(&map_c);
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], 2 * kPairEpiWarps);
    }
    for (int i = 0; i < kPairEpiWarps; ++i) mbar_init(&s.rbar[i], 1);
    s.abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc<2>(&s.tmem_base, 512);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before any remote arrive
  tc_fence_after();
  wait_for_previous();
  const uint32_t tmem = s.tmem_base;
  const WaitCtl wc{&s.abort_flag, p.status, p.limit_ns};

  if (warp == 0) {
    // producer: this CTA's operands; both CTAs' bytes complete on the even
    // CTA's barrier
    if (elect_one()) {
      int stage = 0, filled = 0;
      uint32_t phase = 0;
      const uint32_t full0 = mapa_shared(smem_u32(&s.full[0]), 0);
      bool aborted = false;
      for (int t = blockIdx.x / 2; t < ntiles && !aborted; t += units) {
        const int mt = t / p.n_tiles, nt = t - mt * p.n_tiles;
        const int a0 = mt * 256 + 128 * rank, b0 = nt * p.bn + p.bn / 2 * rank;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!mbar_wait(&s.empty[stage], phase ^ 1u, wc)) {
            aborted = true;
            break;
          }
          uint8_t* sa = ring + stage * kPairStage;
          if (leader) mbar_arrive_expect_tx(&s.full[stage], 2 * p.stage_bytes);
          const uint32_t bar = full0 + stage * static_cast<uint32_t>(sizeof(uint64_t));
          pair_load<AMN>(sa, &map_a, bar, a0, kb * kBlockK, p.a_chunks, 2);
          pair_load<BMN>(sa + kATile, &map_b, bar, b0, kb * kBlockK, p.b_chunks, p.b_boxes);
          ++filled;
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (aborted && leader) {  // copies in flight land before the CTA exits
        for (int i = 0; i < kPairStages; ++i) {
          const int f = filled > i ? (filled - i + kPairStages - 1) / kPairStages : 0;
          if (f > 0) (void)mbar_wait_drain(&s.full[i], (f - 1) & 1, 100000000ull);
        }
      }
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {  // as in the split kernel, one thread
      const uint32_t base = smem_u32(ring);
      const Operand ob = BMN && p.b_boxes == 3 ? operand64() : operand128<BMN>();
      int stage = 0, done = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = blockIdx.x / 2; t < ntiles && ok; t += units) {
        ok = mbar_wait_cluster(&s.tempty[acc], acc_phase ^ 1u, wc);
        if (!ok) break;
        tc_fence_after();
        uint32_t add = 0u;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          ok = mbar_wait_cluster(&s.full[stage], phase, wc);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = base + stage * kPairStage;
          issue_block<2>(tmem + acc * kPairN, a, a + kATile, operand128<AMN>(), ob, p.idesc, add);
          add = 1u;
          umma_commit<2>(&s.empty[stage]);
          ++done;
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit<2>(&s.tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok && done > 0) {  // issued products end before TMEM is freed
        const int last = (done - 1) % kPairStages;
        (void)mbar_wait_drain(&s.empty[last], ((done - last + kPairStages - 1) / kPairStages - 1) & 1,
                              100000000ull);
      }
    }
  } else {
    // epilogue: rows 32 q.. of this CTA's 128, columns 64 part.. of the
    // tile's (narrower tiles leave some of these warps idle).  A residual comes by TMA, one tile ahead, into the buffer
    // from which the result is stored.  With z the buffer is used for z and
    // then for the result, and a residual is read by the threads.
    const int ew = warp - 2, q = warp & 3, part = ew >> 2;
    uint8_t* buf = epi + ew * kPairBuf;
    uint64_t* rbar = &s.rbar[ew];
    const uint32_t tempty_peer = mapa_shared(smem_u32(&s.tempty[0]), 0);
    const bool with_z = FULL && p.has_z;
    const bool res_tma = p.has_res && !with_z;
    const int unit = blockIdx.x / 2;
    auto place = [&](int t, int& y, int64_t& col) -> bool {  // of this warp's chunk of tile t
      const int mt = t / p.n_tiles, nt = t - mt * p.n_tiles;
      y = mt * 256 + 128 * rank + 32 * q;
      col = static_cast<int64_t>(nt) * p.bn + 64 * part;
      return 64 * part < p.bn && y < p.M && col < p.N;
    };
    bool flying = false;  // a residual is under way
    uint32_t rphase = 0;
    auto fetch = [&](int t) {  // the residual of this warp's next chunk, from tile t on
      int y;
      int64_t col;
      while (t < ntiles && !place(t, y, col)) t += units;
      if (t >= ntiles) return;
      if (elect_one()) {
        mbar_arrive_expect_tx(rbar, kPairBuf);
        tma_load_2d(buf, &map_r, rbar, static_cast<int>(col), y);
      }
      __syncwarp();
      flying = true;
    };
    if (res_tma) fetch(unit);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = unit; t < ntiles; t += units) {
      int y;
      int64_t col;
      const bool mine = place(t, y, col);
      float bias[2] = {0.0f, 0.0f};  // of columns col + 32 h + lane, while the products still run
      if (FULL && mine && p.bias != nullptr) {
#pragma unroll
        for (int h = 0; h < 2; ++h) bias[h] = __ldg(p.bias + min(col + 32 * h + lane, p.N - 1));
      }
      ok = warp_wait(&s.tfull[acc], acc_phase, wc);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tbase = tmem + acc * kPairN + 64 * part + (static_cast<uint32_t>(q * 32) << 16);
      if (mine) {
        if (res_tma) {
          ok = warp_wait(rbar, rphase, wc);
          if (!ok) break;
          rphase ^= 1u;
          flying = false;
        } else {
          if (lane == 0) bulk_wait_read<0>();  // the buffer's last store has read it
          __syncwarp();
        }
        auto values = [&](int h, float (&v)[32]) {  // z of half h
          uint32_t raw[32];
          tmem_ld_32x32b_x32(tbase + 32 * h, raw);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
          if (FULL && p.bias != nullptr) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, h == 0 ? bias[0] : bias[1], i);
          }
        };
        auto send = [&](const CUtensorMap* map) {  // the staged chunk
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(map, buf, static_cast<int>(col), y);
            bulk_commit();
          }
        };
        if (with_z) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            values(h, v);
            put32<T>(buf, lane, h, v);
          }
          send(&map_z);
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[32];
          values(h, v);
          if constexpr (FULL) act_all<false, 32>(v, p.act);
          if (res_tma) {
            add32<T>(buf, lane, h, v);
          } else if (p.has_res && y + lane < p.M) {
            const T* r = static_cast<const T*>(p.res) + (y + lane) * p.ldres + col + 32 * h;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (col + 32 * h + 8 * j >= p.N) break;
              const uint4 u = *reinterpret_cast<const uint4*>(r + 8 * j);
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = unpack_pair(w[i], T{});
                v[8 * j + 2 * i] += f.x;
                v[8 * j + 2 * i + 1] += f.y;
              }
            }
          }
          put32<T>(buf, lane, h, v);
        }
        // the accumulator is read: the next tile's products may overwrite it
        tc_fence_before();
        send(&map_c);
      }
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(&s.tempty[acc]);
        else mbar_arrive_remote(tempty_peer + acc * static_cast<uint32_t>(sizeof(uint64_t)));
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
      if (res_tma && mine) {  // once the store has read the buffer
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        fetch(t + units);
      }
    }
    // a residual in flight lands (an abort left it), every store is done
    if (flying) (void)mbar_wait_drain(rbar, rphase, 100000000ull);
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  __syncwarp();
  let_next_launch();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs are done with each other's memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem, 512);
  }
}

// ------------------------------------------------------------- host side
// 16-bit matrix [outer][inner] with `ld` elements between rows, in boxes of
// box_inner x box_outer; what lies outside reads as zero.
bool map2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
           uint32_t box_inner, uint32_t box_outer) {
  // rows of a box as wide as the swizzle: 128 bytes, 64 for boxes of 32
  const CUtensorMapSwizzle swizzle = box_inner == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {ld * 2};
  const cuuint32_t box[2] = {box_inner, box_outer}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An MN-major operand [rows][inner] (inner a multiple of 64) as
// [inner / 64][rows][64]: one box brings two 64-wide chunks of 64 rows.
bool map_chunks(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t ld) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {64, rows, inner / 64};
  const cuuint64_t strides[2] = {ld * 2, 128};
  const cuuint32_t box[3] = {64, kBlockK, 2}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class K>
cudaError_t allow_smem(K kern, std::atomic<bool> (&set)[64], int bytes) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    set[dev].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

DenseParams make_params(const DenseCall& c) {
  DenseParams p{};
  p.bias = c.bias;
  p.res = c.res;
  p.c = c.c;
  p.z = c.z;
  p.ldres = c.ldres;
  p.ldc = c.ldc;
  p.ldz = c.ldz;
  p.M = c.M;
  p.N = c.N;
  p.kblocks = static_cast<int>(cdiv(c.Kred, kBlockK));
  p.type = c.type;
  p.out_type = c.out_type;
  p.act = c.act;
  p.status = c.dev_status;
  p.limit_ns = kDefaultWaitLimitNs;
  return p;
}

// Clusters of 1 to 8 CTAs that find an SM for each CTA (as the driver counts
// them for 152 SMs): a cluster lies within one group of SMs, so that clusters
// of 7 or 8 leave a fifth of the SMs idle or pair up on some.
int64_t lone_clusters(int splits) {
  static const int kOf152[8] = {152, 76, 46, 36, 28, 23, 15, 15};
  return kOf152[splits - 1] * static_cast<int64_t>(sm_count()) / 152;
}

template <class S>
cudaError_t launch_split(const DenseCall& c, int splits, cudaStream_t s) {
  auto kern = dense_split_kernel<S>;
  static std::atomic<bool> attr_set[64];
  cudaError_t err = allow_smem(kern, attr_set, kSplitSmemLimit);
  if (err != cudaSuccess) return err;
  const DenseParams p = make_params(c);
  // the 128 side is A's rows; swapped, that is the output's columns
  const void* a = S::SWAP ? c.b : c.a;
  const void* b = S::SWAP ? c.a : c.b;
  const int64_t lda = S::SWAP ? c.ldb : c.lda, ldb = S::SWAP ? c.lda : c.ldb;
  const int64_t na = S::SWAP ? c.N : c.M, nb = S::SWAP ? c.M : c.N;
  CUtensorMap ma, mb;
  const bool ok = (S::AMN ? map2d(&ma, a, na, c.Kred, lda, 64, kBlockK)
                          : map2d(&ma, a, c.Kred, na, lda, kBlockK, kTileM)) &&
                  (S::BMN ? map2d(&mb, b, nb, c.Kred, ldb, 64, kBlockK)
                          : map2d(&mb, b, c.Kred, nb, ldb, kBlockK, S::BN));
  if (!ok) return cudaErrorInvalidValue;
  // No more stages than reduction blocks.
  // All of an SM's shared memory where every cluster finds SMs of its own: six
  // 32 KB stages instead of three keep a lone CTA's operands coming (8191 x
  // 7168 -> 256: 33.5 us, 48 with three; 203 x 5224 -> 3904 in two splits 19.3
  // and 25.2).  Otherwise two CTAs to an SM, one's epilogue behind the other's
  // products.
  const bool alone = cdiv(na, kTileM) * cdiv(nb, S::BN) <= lone_clusters(splits);
  const int budget = (alone ? kSplitSmemLimit : kSplitSmemLimit / 2) - S::kOver - 1024;
  const int mine = static_cast<int>(cdiv(p.kblocks, splits));
  const int stages = std::max(S::kLeast, std::min({budget / S::kStage, kSplitMaxStages, mine}));
  const size_t bytes = static_cast<size_t>(stages) * S::kStage + S::kOver;
  const int chunk = c.out_type == MOE_FP32 ? kChunkBlocks : p.kblocks;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  unsigned attrs = 0;
  if (c.follows) attr[attrs++] = overlap_attribute();
  if (splits > 1) {
    attr[attrs].id = cudaLaunchAttributeClusterDimension;
    attr[attrs].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[attrs].val.clusterDim.y = 1;
    attr[attrs++].val.clusterDim.z = 1;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(na, kTileM) * splits),
                     static_cast<unsigned>(cdiv(nb, S::BN)), 1);
  cfg.blockDim = dim3(kSplitThreads, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = attrs;
  return cudaLaunchKernelEx(&cfg, kern, ma, mb, p, stages, splits, chunk);
}

template <bool MN>
bool pair_operand(CUtensorMap* m, const void* base, int64_t outer, int64_t Kred, int64_t ld, int rows,
                  int chunked) {
  if (!MN) return map2d(m, base, Kred, outer, ld, kBlockK, rows);
  return chunked ? map_chunks(m, base, outer, Kred, ld)
                 : map2d(m, base, outer, Kred, ld, rows == 96 ? 32 : 64, kBlockK);
}

template <typename T, bool AMN, bool BMN, bool FULL>
cudaError_t launch_pair(const DenseCall& c, int bn, cudaStream_t s) {
  auto kern = dense_pair_kernel<T, AMN, BMN, FULL>;
  static std::atomic<bool> attr_set[64];
  cudaError_t err = allow_smem(kern, attr_set, static_cast<int>(kPairSmem));
  if (err != cudaSuccess) return err;
  PairParams p{};
  p.bias = c.bias;
  p.M = c.M;
  p.N = c.N;
  p.kblocks = static_cast<int>(cdiv(c.Kred, kBlockK));
  p.m_tiles = static_cast<int>(cdiv(c.M, 256));
  p.n_tiles = static_cast<int>(cdiv(c.N, bn));
  p.bn = bn;
  p.b_boxes = bn / 64 == 3 ? 3 : bn / 128;  // a CTA's 64, 96 or 128 columns
  p.stage_bytes = kATile + bn / 2 * kBlockK * 2;
  p.act = c.act;
  p.a_chunks = AMN && c.M % 64 == 0;
  p.b_chunks = BMN && c.N % 64 == 0 && bn == kPairN;
  p.has_res = c.res != nullptr;
  p.has_z = c.z != nullptr;
  p.res = c.res;
  p.ldres = c.ldres;
  p.idesc = dense_idesc(256, bn, AMN, BMN, c.type == MOE_BF16 ? 1u : 0u);
  p.status = c.dev_status;
  p.limit_ns = kDefaultWaitLimitNs;
  CUtensorMap ma, mb, mc, mr, mz;
  bool ok = pair_operand<AMN>(&ma, c.a, c.M, c.Kred, c.lda, 128, p.a_chunks) &&
            pair_operand<BMN>(&mb, c.b, c.N, c.Kred, c.ldb, bn / 2, p.b_chunks) && map2d(&mc, c.c, c.N, c.M, c.ldc, 64, 32);
  mr = mz = mc;
  if (ok && p.has_res) ok = map2d(&mr, c.res, c.N, c.M, c.ldres, 64, 32);
  if (ok && p.has_z) ok = map2d(&mz, c.z, c.N, c.M, c.ldz, 64, 32);
  if (!ok) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[1] = overlap_attribute();
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // pairs that can be resident at once (one CTA per SM), cached per kernel
  static int max_pairs = 0;
  static std::once_flag once;
  std::call_once(once, [&] {
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (sm_count() / 2)), 1, 1);
    int n = 0;
    max_pairs = (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0) ? n : sm_count() / 2;
  });
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(tiles, max_pairs)), 1, 1);
  cfg.numAttrs = c.follows ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, ma, mb, mc, mr, mz, p);
}

template <typename T>
cudaError_t launch_pair_type(const DenseCall& c, int bn, cudaStream_t s) {
  if (c.a_mn) return launch_pair<T, true, true, false>(c, bn, s);
  if (c.b_mn) return launch_pair<T, false, true, true>(c, bn, s);
  return launch_pair<T, false, false, false>(c, bn, s);
}

// The kernel, tile and splits of a product, by an estimate in cycles fitted to
// measurements (bf16, 172 products from 1 x 320 x 192 to 31528 x 120 x 472,
// forward, fp32 results and wgrads, each under every tile and split; the one
// it takes is 0.6% behind the fastest on average, at worst 1.12 times).
//   split kernel: 7000 to launch, set up and end and 1450 for a cluster's
//   barriers; per reduction block 350 to 640 (the operands' way from L2), per
//   tile an epilogue shared by the splits.  With u clusters to each place for
//   one that has its SMs to itself, blocks overlap and take 0.65 of that, but
//   all of a cluster's part 1 + 1.1 (u - 1) + 1.5 (ceil(u) - 1) times as long.
//   pair kernel: 10400, and per wave of tiles 770 a block (690, 560 for 192 and
//   128 columns), or the epilogue's 6200 (5000, 4300) where that is more.
//   Narrower tiles fill the pairs better: 4096 x 2048 -> 768 took 20.1 us with
//   256 columns and 19.0 with 192, 4096 x 4096 -> 1152 48 and 41 with 128.
struct DensePlan {
  bool pair;
  int bn, splits;
};
DensePlan plan_dense(const DenseCall& c) {
  struct Tile { int bn; double block, end, most; };  // most: CTAs per SM that were measured
  static const Tile kTiles[] = {{16, 350, 50, 2.6}, {32, 365, 100, 2.6}, {64, 500, 50, 2.6}, {128, 640, 4800, 4.6}};
  const double sms = sm_count();
  const int kb = static_cast<int>(cdiv(c.Kred, kBlockK));
  DensePlan best{false, 128, 1};
  double least = 1e300;
  for (const Tile& t : kTiles) {
    // 16 and 32 wide only swapped (their B is K-major); a wgrad has no rows
    // to swap, its 64 wide tile is a plain one
    const bool swap = t.bn < 128 && !c.a_mn;
    if (t.bn < 64 && !swap) continue;
    const double tiles = static_cast<double>(swap ? cdiv(c.N, kTileM) * cdiv(c.M, t.bn)
                                                  : cdiv(c.M, kTileM) * cdiv(c.N, t.bn));
    for (int s = 1; s <= 8; ++s) {
      if (s > 1 && kb < 2 * s) break;  // a split gets two blocks at least
      if (tiles * s > t.most * sms && (t.bn < 128 || s > 1)) break;
      const double u = tiles / static_cast<double>(lone_clusters(s));
      const double load = u <= 1 ? 1 : 1 + 1.1 * (u - 1) + 1.5 * (std::ceil(u) - 1);
      const double est = 7000 + (cdiv(kb, s) * t.block * (u <= 1 ? 1 : 0.65) + t.end / s) * load +
                         (s > 1 ? 1450 : 0);
      if (est < least) {
        least = est;
        best = DensePlan{false, t.bn, s};
      }
    }
  }
  if (c.out_type != MOE_FP32) {
    struct PairTile { int bn; double block, end; };
    static const PairTile kPairTiles[] = {{256, 770, 6200}, {192, 690, 5000}, {128, 560, 4300}};
    for (const PairTile& t : kPairTiles) {
      const int64_t pairs = sm_count() / 2;
      const double waves = static_cast<double>(cdiv(cdiv(c.M, 256) * cdiv(c.N, t.bn), pairs));
      const double est = 10400 + waves * std::max(kb * t.block, t.end);
      if (est < least) {
        least = est;
        best = DensePlan{true, t.bn, 1};
      }
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_dense(const DenseCall& c, cudaStream_t s) {
  const DensePlan plan = plan_dense(c);
  if (plan.pair)
    return c.type == MOE_BF16 ? launch_pair_type<__nv_bfloat16>(c, plan.bn, s)
                              : launch_pair_type<__half>(c, plan.bn, s);
  if (c.a_mn) {
    if (plan.bn == 64) return launch_split<SplitShape<64, true, true, false>>(c, plan.splits, s);
    return launch_split<SplitShape<128, true, true, false>>(c, plan.splits, s);
  }
  switch (plan.bn) {
    case 16:
      return c.b_mn ? launch_split<SplitShape<16, true, false, true>>(c, plan.splits, s)
                    : launch_split<SplitShape<16, false, false, true>>(c, plan.splits, s);
    case 32:
      return c.b_mn ? launch_split<SplitShape<32, true, false, true>>(c, plan.splits, s)
                    : launch_split<SplitShape<32, false, false, true>>(c, plan.splits, s);
    case 64:
      return c.b_mn ? launch_split<SplitShape<64, true, false, true>>(c, plan.splits, s)
                    : launch_split<SplitShape<64, false, false, true>>(c, plan.splits, s);
    default:
      return c.b_mn ? launch_split<SplitShape<128, false, true, false>>(c, plan.splits, s)
                    : launch_split<SplitShape<128, false, false, false>>(c, plan.splits, s);
  }
}

}  // namespace moe
