// C entry points of the operators around the expert block: argument checks,
// workspace layout, launches.  The operations are documented in include/moe.h.
#include <cstdint>

#include "kernels.h"
#include "layer.h"
#include "moe.h"

namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool is_dtype(int t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_FP32; }
size_t size_of(int t) { return t == MOE_FP32 ? 4 : 2; }
moe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 257;

// A matrix of `cols` columns whose elements only need their own alignment.
bool element_mat(const moe_mat& m, int64_t cols, int type) {
  return m.p != nullptr && aligned(m.p, size_of(type)) && m.ld >= cols;
}
// A matrix moved in 16-byte pieces.
bool vector_mat(const moe_mat& m, int64_t cols, int type) {
  return m.p != nullptr && aligned(m.p, 16) && m.ld >= cols && m.ld < (int64_t{1} << 36) &&
         m.ld % (16 / static_cast<int64_t>(size_of(type))) == 0;
}

size_t round256(size_t n) { return (n + 255u) & ~static_cast<size_t>(255u); }

moe_status check_norm(int64_t rows, int32_t D, moe_dtype type, moe_dtype wtype) {
  if (!is_dtype(type) || !is_dtype(wtype)) return MOE_ERR_INVALID_ARG;
  if (wtype != type && wtype != MOE_FP32) return MOE_ERR_UNSUPPORTED;
  if (D < 1 || D > 8192 || rows < 0 || rows >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_topk(const moe_topk_dims& d) {
  if (d.gate != MOE_GATE_SIGMOID && d.gate != MOE_GATE_SOFTMAX) return MOE_ERR_INVALID_ARG;
  if (d.group_top != 1 && d.group_top != 2) return MOE_ERR_INVALID_ARG;
  if (d.T < 0 || d.E < 1 || d.E > 1024 || d.K < 1 || d.K > 32) return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d.T) * d.K >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED;
  if (d.groups < 1 || d.groups > 32 || d.E % d.groups != 0) return MOE_ERR_UNSUPPORTED;
  if (d.top_groups < 1 || d.top_groups > d.groups) return MOE_ERR_UNSUPPORTED;
  if (d.K > d.top_groups * (d.E / d.groups)) return MOE_ERR_UNSUPPORTED;
  const int lanes = moe::topk_group_lanes(d);
  if (d.top_groups < d.groups && (d.E / d.groups + lanes - 1) / lanes > moe::kTopkPerLane)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_linear(const moe_linear_dims& d) {
  if (!is_dtype(d.type) || !is_dtype(d.out_type)) return MOE_ERR_INVALID_ARG;
  if (d.act < MOE_ACT_NONE || d.act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  if (d.type == MOE_FP32) return MOE_ERR_UNSUPPORTED;
  if (d.out_type != d.type && d.out_type != MOE_FP32) return MOE_ERR_UNSUPPORTED;
  if (d.M < 0 || d.M > kMaxRows || d.K < 8 || d.N < 8 || d.K % 8 != 0 || d.N % 8 != 0)
    return MOE_ERR_UNSUPPORTED;
  if (d.K > (1 << 22) || d.N > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace of the linear backward: dz [M, N], then the partial column sums.
size_t dz_bytes(const moe_linear_dims& d) {
  const bool own = d.act != MOE_ACT_NONE || d.out_type != d.type;
  return own ? round256(static_cast<size_t>(d.M) * d.N * size_of(d.type)) : 0;
}

}  // namespace

extern "C" {

moe_status moe_layer_norm(moe_mat x, moe_mat res, const void* gamma, const void* beta, moe_mat r,
                          moe_mat y, float* mean, float* rstd, float eps, int64_t rows, int32_t D,
                          moe_dtype type, moe_dtype wtype, cudaStream_t stream) {
  const moe_status st = check_norm(rows, D, type, wtype);
  if (st != MOE_OK) return st;
  if ((mean == nullptr) != (rstd == nullptr)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!element_mat(x, D, type) || !element_mat(y, D, type)) return MOE_ERR_INVALID_ARG;
  if (res.p != nullptr && (!element_mat(res, D, type) || !element_mat(r, D, type)))
    return MOE_ERR_INVALID_ARG;
  if (gamma == nullptr || beta == nullptr || !aligned(gamma, size_of(wtype)) ||
      !aligned(beta, size_of(wtype)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  moe::NormCall c{};
  c.x = x.p;
  c.ldx = x.ld;
  c.gamma = gamma;
  c.beta = beta;
  if (res.p != nullptr) {
    c.res = res.p;
    c.ldres = res.ld;
    c.r = r.p;
    c.ldr = r.ld;
  }
  c.y = y.p;
  c.ldy = y.ld;
  c.mean = mean;
  c.rstd = rstd;
  c.eps = eps;
  c.rows = rows;
  c.D = D;
  c.type = type;
  c.wtype = wtype;
  return from_cuda(moe::launch_layer_norm(c, stream));
}

size_t moe_layer_norm_workspace_bytes(int64_t rows, int32_t D) {
  if (check_norm(rows, D, MOE_FP32, MOE_FP32) != MOE_OK) return 0;
  const int64_t parts = rows < moe::kPartialRows ? rows : moe::kPartialRows;
  return round256(static_cast<size_t>(parts) * 2 * static_cast<size_t>(D) * sizeof(float));
}

moe_status moe_layer_norm_bwd(moe_mat dy, moe_mat r, const void* gamma, const float* mean,
                              const float* rstd, moe_mat dres, moe_mat dx, void* dgamma,
                              void* dbeta, void* ws, int64_t rows, int32_t D, moe_dtype type,
                              moe_dtype wtype, cudaStream_t stream) {
  const moe_status st = check_norm(rows, D, type, wtype);
  if (st != MOE_OK) return st;
  if ((dgamma == nullptr) != (dbeta == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(dgamma, size_of(wtype)) || !aligned(dbeta, size_of(wtype))) return MOE_ERR_INVALID_ARG;
  if (rows == 0) {
    if (dgamma == nullptr) return MOE_OK;
    const size_t n = static_cast<size_t>(D) * size_of(wtype);
    const cudaError_t err = cudaMemsetAsync(dgamma, 0, n, stream);
    return from_cuda(err != cudaSuccess ? err : cudaMemsetAsync(dbeta, 0, n, stream));
  }
  if (!element_mat(dy, D, type) || !element_mat(r, D, type) || !element_mat(dx, D, type))
    return MOE_ERR_INVALID_ARG;
  if (dres.p != nullptr && !element_mat(dres, D, type)) return MOE_ERR_INVALID_ARG;
  if (gamma == nullptr || mean == nullptr || rstd == nullptr || !aligned(gamma, size_of(wtype)) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  if (dgamma != nullptr && (ws == nullptr || !aligned(ws, 16))) return MOE_ERR_INVALID_ARG;
  moe::NormCall c{};
  c.x = dy.p;
  c.ldx = dy.ld;
  c.r_in = r.p;
  c.ldr = r.ld;
  c.gamma = gamma;
  c.mean = const_cast<float*>(mean);
  c.rstd = const_cast<float*>(rstd);
  c.res = dres.p;
  c.ldres = dres.p != nullptr ? dres.ld : 0;
  c.y = dx.p;
  c.ldy = dx.ld;
  c.dgamma = dgamma;
  c.dbeta = dbeta;
  c.partials = dgamma != nullptr ? static_cast<float*>(ws) : nullptr;
  c.rows = rows;
  c.D = D;
  c.type = type;
  c.wtype = wtype;
  return from_cuda(moe::launch_layer_norm_bwd(c, stream));
}

moe_status moe_route_topk(const float* logits, const float* bias, int32_t* ids, float* w,
                          moe_topk_dims d, cudaStream_t stream) {
  const moe_status st = check_topk(d);
  if (st != MOE_OK) return st;
  if (d.T == 0) return MOE_OK;
  if (logits == nullptr || !aligned(logits, 16) || ids == nullptr || !aligned(ids, 16) ||
      w == nullptr || !aligned(w, 16) || !aligned(bias, 16))
    return MOE_ERR_INVALID_ARG;
  return from_cuda(moe::launch_route_topk(logits, bias, ids, w, d, stream));
}

moe_status moe_route_topk_bwd(const float* logits, const int32_t* ids, const float* dw,
                              float* dlogits, moe_topk_dims d, cudaStream_t stream) {
  d.groups = d.top_groups = d.group_top = 1;  // not read
  if (d.K > d.E) return MOE_ERR_UNSUPPORTED;
  const moe_status st = check_topk(d);
  if (st != MOE_OK) return st;
  if (d.T == 0) return MOE_OK;
  if (logits == nullptr || !aligned(logits, 16) || ids == nullptr || !aligned(ids, 16) ||
      dw == nullptr || !aligned(dw, 16) || dlogits == nullptr || !aligned(dlogits, 16))
    return MOE_ERR_INVALID_ARG;
  return from_cuda(moe::launch_route_topk_bwd(logits, ids, dw, dlogits, d, stream));
}

moe_status moe_linear(moe_mat x, moe_mat w, const float* bias, moe_mat res, moe_mat y, moe_mat z,
                      int32_t* dev_status, moe_linear_dims d, cudaStream_t stream) {
  const moe_status st = check_linear(d);
  if (st != MOE_OK) return st;
  if (!aligned(dev_status, 16)) return MOE_ERR_INVALID_ARG;
  if (d.M == 0) return MOE_OK;
  if (!vector_mat(x, d.K, d.type) || !vector_mat(w, d.N, d.type) || !vector_mat(y, d.N, d.out_type))
    return MOE_ERR_INVALID_ARG;
  if (res.p != nullptr && !vector_mat(res, d.N, d.out_type)) return MOE_ERR_INVALID_ARG;
  if (z.p != nullptr && !vector_mat(z, d.N, d.type)) return MOE_ERR_INVALID_ARG;
  if (!aligned(bias, 16)) return MOE_ERR_INVALID_ARG;
  moe::DenseCall c{};
  c.a = x.p;
  c.lda = x.ld;
  c.b = w.p;
  c.ldb = w.ld;
  c.b_mn = true;
  c.M = d.M;
  c.N = d.N;
  c.Kred = d.K;
  c.bias = bias;
  c.res = res.p;
  c.ldres = res.ld;
  c.c = y.p;
  c.ldc = y.ld;
  c.z = z.p;
  c.ldz = z.ld;
  c.type = static_cast<moe_dtype>(d.type);
  c.out_type = static_cast<moe_dtype>(d.out_type);
  c.act = d.act;
  c.dev_status = dev_status;
  return from_cuda(moe::launch_dense(c, stream));
}

size_t moe_linear_workspace_bytes(moe_linear_dims d) {
  if (check_linear(d) != MOE_OK) return 0;
  return dz_bytes(d) + round256(static_cast<size_t>(moe::kPartialRows) * d.N * sizeof(float));
}

moe_status moe_linear_bwd(moe_mat dy, moe_mat z, moe_mat x, moe_mat w, moe_mat dx_add, moe_mat dx,
                          moe_mat dw, float* db, int32_t* dev_status, void* ws, moe_linear_dims d,
                          cudaStream_t stream) {
  const moe_status st = check_linear(d);
  if (st != MOE_OK) return st;
  if (!aligned(dev_status, 16)) return MOE_ERR_INVALID_ARG;
  if (dx.p == nullptr && dw.p == nullptr && db == nullptr) return MOE_ERR_INVALID_ARG;
  if (dw.p != nullptr && !vector_mat(dw, d.N, d.type)) return MOE_ERR_INVALID_ARG;
  if (!aligned(db, 16)) return MOE_ERR_INVALID_ARG;
  if (d.M == 0) {
    cudaError_t err = cudaSuccess;
    if (dw.p != nullptr)
      err = cudaMemset2DAsync(dw.p, static_cast<size_t>(dw.ld) * 2, 0, static_cast<size_t>(d.N) * 2,
                              static_cast<size_t>(d.K), stream);
    if (err == cudaSuccess && db != nullptr)
      err = cudaMemsetAsync(db, 0, static_cast<size_t>(d.N) * sizeof(float), stream);
    return from_cuda(err);
  }
  const bool products = dx.p != nullptr || dw.p != nullptr;
  if (!vector_mat(dy, d.N, d.out_type)) return MOE_ERR_INVALID_ARG;
  if (d.act != MOE_ACT_NONE && !vector_mat(z, d.N, d.type)) return MOE_ERR_INVALID_ARG;
  if (dx.p != nullptr && (!vector_mat(dx, d.K, d.type) || !vector_mat(w, d.N, d.type)))
    return MOE_ERR_INVALID_ARG;
  if (dx_add.p != nullptr && dx.p != nullptr && !vector_mat(dx_add, d.K, d.type))
    return MOE_ERR_INVALID_ARG;
  if (dw.p != nullptr && !vector_mat(x, d.K, d.type)) return MOE_ERR_INVALID_ARG;
  const bool own_dz = products && dz_bytes(d) > 0;  // dz is not dy itself
  if ((own_dz || db != nullptr) && (ws == nullptr || !aligned(ws, 16))) return MOE_ERR_INVALID_ARG;

  const moe_dtype type = static_cast<moe_dtype>(d.type);
  const void* dz = own_dz ? ws : dy.p;
  const int64_t lddz = own_dz ? d.N : dy.ld;
  if (own_dz || db != nullptr) {
    moe::ActGradCall a{};
    a.dy = dy.p;
    a.lddy = dy.ld;
    a.z = d.act != MOE_ACT_NONE ? z.p : nullptr;
    a.ldz = z.ld;
    a.dz = own_dz ? ws : nullptr;
    a.db = db;
    a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + dz_bytes(d));
    a.M = d.M;
    a.N = d.N;
    a.type = type;
    a.dy_type = static_cast<moe_dtype>(d.out_type);
    a.act = d.act;
    const cudaError_t err = moe::launch_act_grad(a, stream);
    if (err != cudaSuccess) return from_cuda(err);
  }
  moe::DenseCall c{};
  c.type = c.out_type = type;
  c.act = MOE_ACT_NONE;
  c.dev_status = dev_status;
  if (dx.p != nullptr) {
    c.a = dz;
    c.lda = lddz;
    c.b = w.p;  // [K, N]: its rows are dx's columns, N the reduction
    c.ldb = w.ld;
    c.M = d.M;
    c.N = d.K;
    c.Kred = d.N;
    c.res = dx_add.p;
    c.ldres = dx_add.ld;
    c.c = dx.p;
    c.ldc = dx.ld;
    c.follows = own_dz || db != nullptr;
    const cudaError_t err = moe::launch_dense(c, stream);
    if (err != cudaSuccess) return from_cuda(err);
  }
  if (dw.p != nullptr) {
    c.follows = own_dz || db != nullptr || dx.p != nullptr;
    c.a = x.p;
    c.lda = x.ld;
    c.a_mn = true;
    c.b = dz;
    c.ldb = lddz;
    c.b_mn = true;
    c.M = d.K;
    c.N = d.N;
    c.Kred = d.M;
    c.res = nullptr;
    c.c = dw.p;
    c.ldc = dw.ld;
    const cudaError_t err = moe::launch_dense(c, stream);
    if (err != cudaSuccess) return from_cuda(err);
  }
  return MOE_OK;
}

}  // extern "C"
