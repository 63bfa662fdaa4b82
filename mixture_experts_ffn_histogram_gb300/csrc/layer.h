// Internal launchers of the operators around the expert block (host side):
// layer norm, expert selection, linear layer.  Arguments were validated by
// the C entry points in layer_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// Rows of fp32 partial sums that a weight-gradient reduction keeps in its
// workspace at most: a few per SM on any device.
constexpr int64_t kPartialRows = 1024;

// The launch attribute of a kernel that starts with wait_for_previous, behind
// a kernel of the same call.
inline cudaLaunchAttribute overlap_attribute() {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

struct NormCall {
  const void *x, *res, *gamma, *beta;  // backward: x = dy, res = dres
  const void* r_in;                    // backward: the stored rows
  void *r, *y;                         // backward: y = dx
  float *mean, *rstd;                  // backward: read
  void *dgamma, *dbeta;
  float* partials;
  int64_t ldx, ldres, ldr, ldy;
  float eps;
  int64_t rows;
  int32_t D;
  moe_dtype type, wtype;
};
cudaError_t launch_layer_norm(const NormCall& c, cudaStream_t s);
cudaError_t launch_layer_norm_bwd(const NormCall& c, cudaStream_t s);

// out0[c] (c < split) and out1[c - split] = sum over P rows of partials
// [P][C], in a fixed order.  type: of out0 and out1.  The launch before it on
// the stream is the one that writes the partials.
cudaError_t launch_join_partials(const float* partials, int P, int64_t C, int64_t split, void* out0,
                                 void* out1, moe_dtype type, cudaStream_t s);

// The selection kernel gives every group of experts its own lanes of a warp:
// the largest power of two of lanes that divides the group, or all that there
// are when that leaves more than kTopkPerLane experts to a lane.
constexpr int kTopkPerLane = 32;
inline int topk_group_lanes(const moe_topk_dims& d) {
  const int gs = d.E / d.groups, most = 32 / d.groups;
  int lanes = 1;
  while (lanes * 2 <= most && gs % (lanes * 2) == 0) lanes *= 2;
  return (gs + lanes - 1) / lanes <= kTopkPerLane ? lanes : most;
}
cudaError_t launch_route_topk(const float* logits, const float* bias, int32_t* ids, float* w,
                              const moe_topk_dims& d, cudaStream_t s);
cudaError_t launch_route_topk_bwd(const float* logits, const int32_t* ids, const float* dw,
                                  float* dlogits, const moe_topk_dims& d, cudaStream_t s);

// One dense product C [M, N] = A B with the linear layer's epilogue
//   z = A B + bias,  C = act(z) + res.
// a_mn: A is stored [Kred, M] (its M axis contiguous) instead of [M, Kred];
// b_mn: B is stored [Kred, N] instead of [N, Kred].  16-bit operands of `type`.
struct DenseCall {
  const void* a;
  const void* b;
  int64_t lda, ldb;
  bool a_mn, b_mn;
  int64_t M, N, Kred;
  const float* bias;
  const void* res;
  int64_t ldres;
  void* c;
  int64_t ldc;
  void* z;
  int64_t ldz;
  moe_dtype type, out_type;
  int act;
  int32_t* dev_status;
  bool follows;  // the launch before it on the stream is one of the same call
};
cudaError_t launch_dense(const DenseCall& c, cudaStream_t s);

// dz = dy * act'(z) in `type` (dz NULL: not written) and its column sums
// (db NULL: none) through `partials` [kPartialRows][N].
struct ActGradCall {
  const void* dy;
  int64_t lddy;
  const void* z;
  int64_t ldz;
  void* dz;  // [M, N] contiguous
  float* db;
  float* partials;
  int64_t M, N;
  moe_dtype type, dy_type;
  int act;
};
cudaError_t launch_act_grad(const ActGradCall& c, cudaStream_t s);

}  // namespace moe
