// Tiles of 16-bit operands on the fifth-generation tensor cores: descriptors of
// 64-deep operand blocks in 128-byte-swizzled shared memory, the products of
// one block, and the driver's tensor-map encoder.
#pragma once

#include <cuda.h>

#include <mutex>

#include "common.cuh"

namespace moe {

constexpr int kBlockK = 64;
constexpr int kMmaK = 16;
constexpr int kChunk = 64 * kBlockK * 2;  // 64 columns x 64 reduction rows: 8 KB

// Instruction descriptor, kind::f16: as instr_desc_bf16, with the operand
// type as an argument (0: f16, 1: bf16; both operands the same).
__host__ __device__ constexpr uint32_t dense_idesc(int M, int N, bool a_mn, bool b_mn, uint32_t ty) {
  return (1u << 4) | (ty << 7) | (ty << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

// One lane of a converged warp, known to the compiler as such: what it issues
// alone needs no loop over lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The matrix descriptor of an operand's block at shared address 0, and the
// step from one MMA's 16 reduction elements to the next (in units of 16 bytes).
struct Operand {
  uint64_t desc;
  uint32_t step;
};
template <bool MN>
__device__ __forceinline__ Operand operand128() {
  return MN ? Operand{smem_desc_sw128(0, kChunk, 1024), 128} : Operand{smem_desc_sw128(0, 16, 1024), 2};
}
// The products of one reduction block: operands at shared addresses a and b.
template <int CG>
__device__ __forceinline__ void issue_block(uint32_t d, uint32_t a, uint32_t b, const Operand& oa,
                                            const Operand& ob, uint32_t idesc, uint32_t add) {
  const uint64_t ad = oa.desc | ((a >> 4) & 0x3FFFu), bd = ob.desc | ((b >> 4) & 0x3FFFu);
#pragma unroll
  for (int kk = 0; kk < kBlockK / kMmaK; ++kk)
    umma_bf16<CG>(d, ad + kk * oa.step, bd + kk * ob.step, idesc, kk > 0 ? 1u : add);
}

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

// Barriers of four epilogue warps (named barrier 1); the second tells whether all had `ok`.
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// A wait of the whole warp, polled by one lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& c) {
  bool ok = true;
  if (elect_one()) ok = mbar_wait(bar, parity, c);
  return __all_sync(0xffffffffu, ok);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// 16-bit rows for four-row gathers: a box is 64 columns of one row.
inline bool map_rows(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t ld) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {inner, rows}, strides[1] = {ld * 2};
  const cuuint32_t box[2] = {64, 1}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
