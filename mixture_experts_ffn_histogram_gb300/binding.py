"""ctypes binding of libmoe.so: one Python function per C entry point, with the
same name, that only marshals arguments (torch tensors -> device pointers,
dims -> ``moe_dims``, stream -> ``cudaStream_t``) and raises on a non-OK
status.  Every step of the block runs in the library's CUDA kernels; there is
no other implementation behind these functions, and they fail loudly when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from ._build import LIB

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CUDA = 3
MOE_ERR_DEVICE = 4
MOE_ERR_TIMEOUT = 5

SCORE_SOFTMAX_TOPK = 0
SCORE_SIGMOID_NORM = 1
SCORE_GIVEN = 2

ENTRY_POINTS = (
    "moe_workspace_bytes", "moe_status_string", "moe_abi_version", "moe_route_histogram",
    "moe_permute", "moe_permute_bwd", "moe_grouped_gemm_fc1_swiglu",
    "moe_grouped_gemm_fc1_swiglu_bwd", "moe_grouped_gemm_fc2", "moe_grouped_gemm_fc2_bwd",
    "moe_combine", "moe_combine_bwd", "moe_selftest_bounded_wait", "moe_route_histogram_noalloc",
    "moe_mx_bytes", "moe_mx_quantize_wi", "moe_mx_quantize_wo", "moe_mx_permute_quantize",
    "moe_mx_grouped_gemm_fc1_swiglu", "moe_mx_grouped_gemm_fc2",
    "moe_grouped_gemm_fc1_swiglu_experts", "moe_grouped_gemm_fc1_bwd_experts",
    "moe_fused_forward", "moe_mx_combine_bwd", "moe_mx_quantize_rows", "moe_mx_quantize_tokens", "moe_mx_grouped_gemm_fc2_bwd",
    "moe_mx_grouped_gemm_fc1_bwd",
    "moe_layer_norm", "moe_layer_norm_bwd", "moe_layer_norm_workspace_bytes", "moe_route_topk",
    "moe_route_topk_bwd", "moe_linear", "moe_linear_bwd", "moe_linear_workspace_bytes",
    "moe_decode", "moe_decode_workspace_bytes", "moe_block_norm", "moe_block_norm_bwd",
    "moe_block_norm_workspace_bytes", "moe_adapter_plan", "moe_adapter_plan_bytes", "moe_adapters",
    "moe_adapters_workspace_bytes",
)

# moe_dtype
BF16, FP16, FP32 = range(3)
DTYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
# moe_gate, moe_act: names -> values
GATES = {"sigmoid": 0, "softmax": 1}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

# moe_mx_buffer
(MX_XQ, MX_XSC, MX_WIQ, MX_WISC, MX_WOQ, MX_WOSC, MX_HQ, MX_HSC, MX_DYQ, MX_DYSC, MX_DZQ,
 MX_DZSC, MX_WIQ_BWD, MX_WISC_BWD, MX_WOQ_BWD, MX_WOSC_BWD, MX_XT, MX_XTSC, MX_HT, MX_HTSC,
 MX_DYT, MX_DYTSC, MX_DZT, MX_DZTSC) = range(24)

# int32 capacity of the fixed scratch behind moe_route_histogram_noalloc
NOALLOC_ROUTE_SCRATCH_INTS = 262144


class MoeDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("D", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("F", ctypes.c_int32)]

    def __repr__(self):
        return f"MoeDims(T={self.T}, D={self.D}, E={self.E}, K={self.K}, F={self.F})"


class MoeMat(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("ld", ctypes.c_int64)]


class MoeTopkDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("K", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class MoeLinearDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
                ("type", ctypes.c_int32), ("out_type", ctypes.c_int32), ("act", ctypes.c_int32)]


class MoeBlockNormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("D", ctypes.c_int32), ("type", ctypes.c_int32),
                ("wtype", ctypes.c_int32), ("eps", ctypes.c_float), ("scale", ctypes.c_float),
                ("offset", ctypes.c_float)]


class MoeAdapterDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "K", "N", "slots", "rank", "type")]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str | None = None):
        super().__init__(f"{fn}: {detail or status_string(status)} (status {status})")
        self.status = status


_lock = threading.Lock()
_lib = None


def dims(T, D, E, K, F) -> MoeDims:
    return MoeDims(T, D, E, K, F)


def topk_dims(T, E, K, gate="sigmoid", groups=1, top_groups=1, group_top=1, renorm=True,
              scale=1.0) -> MoeTopkDims:
    return MoeTopkDims(T, E, K, GATES[gate], groups, top_groups, group_top, int(renorm), scale)


def linear_dims(M, K, N, dtype=torch.bfloat16, out_dtype=None, act="none") -> MoeLinearDims:
    return MoeLinearDims(M, K, N, DTYPES[dtype], DTYPES[out_dtype or dtype], ACTS[act])


def block_norm_dims(rows, D, dtype=torch.bfloat16, weight_dtype=torch.float32, eps=1e-6, scale=1.0,
                    offset=0.0) -> MoeBlockNormDims:
    return MoeBlockNormDims(rows, D, DTYPES[dtype], DTYPES[weight_dtype], eps, scale, offset)


def adapter_dims(T, K, N, slots, rank, dtype=torch.bfloat16) -> MoeAdapterDims:
    return MoeAdapterDims(T, K, N, slots, rank, DTYPES[dtype])


def library_path() -> str:
    return LIB


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so.  Raises if it has not been built: there is no
    fallback implementation."""
    global _lib
    if _lib is not None:  # set once, complete
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB):
            raise RuntimeError(
                f"libmoe.so not found at {LIB}; build it first "
                "(mixture_experts_ffn_histogram_gb300._build.build())")
        L = ctypes.CDLL(LIB)
        P, I, D_ = ctypes.c_void_p, ctypes.c_int, MoeDims
        sig = {
            "moe_workspace_bytes": ([D_], ctypes.c_size_t),
            "moe_status_string": ([I], ctypes.c_char_p),
            "moe_abi_version": ([], I),
            "moe_route_histogram": ([P, P, I, P, P, P, P, P, P, P, P, D_, P], I),
            "moe_permute": ([P, P, P, D_, P], I),
            "moe_permute_bwd": ([P, P, P, D_, P], I),
            "moe_grouped_gemm_fc1_swiglu": ([P, P, P, P, P, P, P, D_, P], I),
            "moe_grouped_gemm_fc1_swiglu_bwd": ([P, P, P, P, P, P, P, P, P, D_, P], I),
            "moe_grouped_gemm_fc2": ([P, P, P, P, P, P, D_, P], I),
            "moe_grouped_gemm_fc2_bwd": ([P, P, P, P, P, P, P, P, P, D_, P], I),
            "moe_combine": ([P, P, P, P, D_, P], I),
            "moe_fused_forward": ([P, P, P, P, P, P, P, P, P, P, P, D_, P], I),
            "moe_combine_bwd": ([P, P, P, P, P, P, D_, P], I),
            "moe_selftest_bounded_wait": ([P, ctypes.c_uint64, P], I),
            "moe_route_histogram_noalloc": ([P, P, I, P, P, P, P, P, P, P, D_, P], I),
            "moe_mx_bytes": ([D_, I], ctypes.c_size_t),
            "moe_grouped_gemm_fc1_swiglu_experts": ([P, P, P, I, I, P, P, P, P, D_, P], I),
            "moe_grouped_gemm_fc1_bwd_experts": ([P, P, P, P, I, I, P, P, P, P, D_, P], I),
            "moe_mx_quantize_wi": ([P, P, P, P, P, D_, P], I),
            "moe_mx_quantize_wo": ([P, P, P, P, P, D_, P], I),
            "moe_mx_permute_quantize": ([P, P, P, P, P, D_, P], I),
            "moe_mx_grouped_gemm_fc1_swiglu": ([P, P, P, P, P, P, P, P, P, P, D_, P], I),
            "moe_mx_grouped_gemm_fc2": ([P, P, P, P, P, P, P, D_, P], I),
            "moe_mx_combine_bwd": ([P] * 9 + [D_, P], I),
            "moe_mx_quantize_rows": ([P, I, P, P, P, D_, P], I),
            "moe_mx_quantize_tokens": ([P, P, I, P, P, P, D_, P], I),
            "moe_mx_grouped_gemm_fc2_bwd": ([P] * 13 + [D_, P], I),
            "moe_mx_grouped_gemm_fc1_bwd": ([P] * 12 + [D_, P], I),
        }
        M, L64, F = MoeMat, ctypes.c_int64, ctypes.c_float
        sig.update({
            "moe_layer_norm": ([M, M, P, P, M, M, P, P, F, L64, ctypes.c_int32, I, I, P], I),
            "moe_layer_norm_bwd": ([M, M, P, P, P, M, M, P, P, P, L64, ctypes.c_int32, I, I, P],
                                   I),
            "moe_layer_norm_workspace_bytes": ([L64, ctypes.c_int32], ctypes.c_size_t),
            "moe_route_topk": ([P, P, P, P, MoeTopkDims, P], I),
            "moe_route_topk_bwd": ([P, P, P, P, MoeTopkDims, P], I),
            "moe_linear": ([M, M, P, M, M, M, P, MoeLinearDims, P], I),
            "moe_linear_bwd": ([M] * 7 + [P, P, P, MoeLinearDims, P], I),
            "moe_linear_workspace_bytes": ([MoeLinearDims], ctypes.c_size_t),
            "moe_decode": ([M, P, P, P, P, I, P, P, M, M, P, P, ctypes.c_int32, D_, I, P], I),
            "moe_decode_workspace_bytes": ([D_], ctypes.c_size_t),
            "moe_block_norm": ([M, M, P, P, P, P, M, M, P, P, MoeBlockNormDims, P], I),
            "moe_block_norm_bwd": ([M] * 4 + [P] * 6 + [M, M] + [P] * 5 + [MoeBlockNormDims, P], I),
            "moe_block_norm_workspace_bytes": ([MoeBlockNormDims], ctypes.c_size_t),
            "moe_adapter_plan": ([P] + [ctypes.c_int32] * 3 + [P, P, P], I),
            "moe_adapter_plan_bytes": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_size_t),
            "moe_adapters": ([M, P, P, P, M, M, P, P, P, ctypes.c_int32, MoeAdapterDims, P], I),
            "moe_adapters_workspace_bytes": ([MoeAdapterDims], ctypes.c_size_t),
        })
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


# the current stream of a device as an integer, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _s(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def stream_of(stream, device) -> int:
    """The stream of a call on `device`: the given one (a Stream or its
    integer), or the device's current one.  A launch goes to the thread's
    current device whatever its pointers are, so that has to be `device`."""
    if device.type == "cuda" and _current_device() != device.index:
        raise RuntimeError(f"the call's tensors are on {device}, which is not the current device "
                           f"(cuda:{_current_device()}): make it so with torch.cuda.device")
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ok(name, st):
    if st != MOE_OK:
        raise MoeError(name, st)


def moe_workspace_bytes(d: MoeDims) -> int:
    return int(lib().moe_workspace_bytes(d))


def moe_abi_version() -> int:
    return int(lib().moe_abi_version())


def moe_route_histogram(logits, bias, mode, ids, w, group_sizes, group_offsets, pos, row_src,
                        dev_status, ws, d: MoeDims, stream=None):
    _ok("moe_route_histogram", lib().moe_route_histogram(
        _p(logits), _p(bias), int(mode), _p(ids), _p(w), _p(group_sizes), _p(group_offsets),
        _p(pos), _p(row_src), _p(dev_status), _p(ws), d, _s(stream)))


def moe_route_histogram_noalloc(logits, bias, mode, ids, w, group_sizes, group_offsets, pos,
                                row_src, dev_status, d: MoeDims, stream=None):
    """moe_route_histogram with no workspace: for callers that cannot allocate
    device memory.  Its scratch is a fixed 1 MiB array inside the library,
    shared by every call (calls that overlap on the GPU race on it)."""
    st = lib().moe_route_histogram_noalloc(
        _p(logits), _p(bias), int(mode), _p(ids), _p(w), _p(group_sizes), _p(group_offsets),
        _p(pos), _p(row_src), _p(dev_status), d, _s(stream))
    if st == MOE_ERR_UNSUPPORTED:
        need = 2 * ((d.T + 255) // 256) * d.E
        if need > NOALLOC_ROUTE_SCRATCH_INTS:
            raise MoeError("moe_route_histogram_noalloc", st,
                           f"needs {need} int32 of fixed scratch (2*ceil(T/256)*E) but the "
                           f"library holds {NOALLOC_ROUTE_SCRATCH_INTS}")
    _ok("moe_route_histogram_noalloc", st)


def moe_permute(x, pos, xs, d: MoeDims, stream=None):
    _ok("moe_permute", lib().moe_permute(_p(x), _p(pos), _p(xs), d, _s(stream)))


def moe_permute_bwd(dxs, pos, dx, d: MoeDims, stream=None):
    _ok("moe_permute_bwd", lib().moe_permute_bwd(_p(dxs), _p(pos), _p(dx), d, _s(stream)))


def moe_grouped_gemm_fc1_swiglu(xs, wi, group_offsets, h, z, dev_status, ws, d: MoeDims,
                                stream=None):
    _ok("moe_grouped_gemm_fc1_swiglu", lib().moe_grouped_gemm_fc1_swiglu(
        _p(xs), _p(wi), _p(group_offsets), _p(h), _p(z), _p(dev_status), _p(ws), d, _s(stream)))


def moe_grouped_gemm_fc1_swiglu_bwd(grad, z, xs, wi, group_offsets, dxs, dwi, dev_status, ws,
                                    d: MoeDims, stream=None):
    _ok("moe_grouped_gemm_fc1_swiglu_bwd", lib().moe_grouped_gemm_fc1_swiglu_bwd(
        _p(grad), _p(z), _p(xs), _p(wi), _p(group_offsets), _p(dxs), _p(dwi), _p(dev_status),
        _p(ws), d, _s(stream)))


def moe_grouped_gemm_fc2(h, wo, group_offsets, ys, dev_status, ws, d: MoeDims, stream=None):
    _ok("moe_grouped_gemm_fc2", lib().moe_grouped_gemm_fc2(
        _p(h), _p(wo), _p(group_offsets), _p(ys), _p(dev_status), _p(ws), d, _s(stream)))


def moe_grouped_gemm_fc2_bwd(dys, h, wo, z, group_offsets, dh_or_dz, dwo, dev_status, ws,
                             d: MoeDims, stream=None):
    _ok("moe_grouped_gemm_fc2_bwd", lib().moe_grouped_gemm_fc2_bwd(
        _p(dys), _p(h), _p(wo), _p(z), _p(group_offsets), _p(dh_or_dz), _p(dwo),
        _p(dev_status), _p(ws), d, _s(stream)))


def moe_combine(ys, w, pos, out, d: MoeDims, stream=None):
    _ok("moe_combine", lib().moe_combine(_p(ys), _p(w), _p(pos), _p(out), d, _s(stream)))


def moe_fused_forward(x, w, row_src, group_offsets, wi, wo, h, acc, out, dev_status, ws,
                      d: MoeDims, stream=None):
    _ok("moe_fused_forward", lib().moe_fused_forward(
        _p(x), _p(w), _p(row_src), _p(group_offsets), _p(wi), _p(wo), _p(h), _p(acc), _p(out),
        _p(dev_status), _p(ws), d, _s(stream)))


def moe_combine_bwd(dout, ys, w, pos, dys, dw, d: MoeDims, stream=None):
    _ok("moe_combine_bwd", lib().moe_combine_bwd(
        _p(dout), _p(ys), _p(w), _p(pos), _p(dys), _p(dw), d, _s(stream)))


def moe_selftest_bounded_wait(dev_status, limit_ns: int, stream=None):
    _ok("moe_selftest_bounded_wait",
        lib().moe_selftest_bounded_wait(_p(dev_status), int(limit_ns), _s(stream)))


def moe_grouped_gemm_fc1_swiglu_experts(xs, wi_part, group_offsets, e_begin, e_end, h, z,
                                        dev_status, ws, d: MoeDims, stream=None):
    _ok("moe_grouped_gemm_fc1_swiglu_experts", lib().moe_grouped_gemm_fc1_swiglu_experts(
        _p(xs), _p(wi_part), _p(group_offsets), int(e_begin), int(e_end), _p(h), _p(z),
        _p(dev_status), _p(ws), d, _s(stream)))


def moe_grouped_gemm_fc1_bwd_experts(dz, xs, wi_part, group_offsets, e_begin, e_end, dxs,
                                     dwi_part, dev_status, ws, d: MoeDims, stream=None):
    _ok("moe_grouped_gemm_fc1_bwd_experts", lib().moe_grouped_gemm_fc1_bwd_experts(
        _p(dz), _p(xs), _p(wi_part), _p(group_offsets), int(e_begin), int(e_end), _p(dxs),
        _p(dwi_part), _p(dev_status), _p(ws), d, _s(stream)))


# ------------------------------------------------------------------ MXFP8
def moe_mx_bytes(d: MoeDims, which: int) -> int:
    return int(lib().moe_mx_bytes(d, int(which)))


def moe_mx_quantize_wi(wi, wq, wsc, d: MoeDims, stream=None, wq_bwd=None, wsc_bwd=None):
    _ok("moe_mx_quantize_wi", lib().moe_mx_quantize_wi(_p(wi), _p(wq), _p(wsc), _p(wq_bwd),
                                                       _p(wsc_bwd), d, _s(stream)))


def moe_mx_quantize_wo(wo, wq, wsc, d: MoeDims, stream=None, wq_bwd=None, wsc_bwd=None):
    _ok("moe_mx_quantize_wo", lib().moe_mx_quantize_wo(_p(wo), _p(wq), _p(wsc), _p(wq_bwd),
                                                       _p(wsc_bwd), d, _s(stream)))


def moe_mx_permute_quantize(x, pos, group_offsets, xq, xsc, d: MoeDims, stream=None):
    _ok("moe_mx_permute_quantize", lib().moe_mx_permute_quantize(
        _p(x), _p(pos), _p(group_offsets), _p(xq), _p(xsc), d, _s(stream)))


def moe_mx_grouped_gemm_fc1_swiglu(xq, xsc, wq, wsc, group_offsets, hq, hsc, h, dev_status,
                                   d: MoeDims, stream=None, z=None):
    _ok("moe_mx_grouped_gemm_fc1_swiglu", lib().moe_mx_grouped_gemm_fc1_swiglu(
        _p(xq), _p(xsc), _p(wq), _p(wsc), _p(group_offsets), _p(hq), _p(hsc), _p(h), _p(z),
        _p(dev_status), d, _s(stream)))


def moe_mx_grouped_gemm_fc2(hq, hsc, wq, wsc, group_offsets, ys, dev_status, d: MoeDims,
                            stream=None):
    _ok("moe_mx_grouped_gemm_fc2", lib().moe_mx_grouped_gemm_fc2(
        _p(hq), _p(hsc), _p(wq), _p(wsc), _p(group_offsets), _p(ys), _p(dev_status), d,
        _s(stream)))


def moe_mx_combine_bwd(dout, ys, w, pos, group_offsets, dys, dyq, dysc, dw, d: MoeDims,
                       stream=None):
    _ok("moe_mx_combine_bwd", lib().moe_mx_combine_bwd(
        _p(dout), _p(ys), _p(w), _p(pos), _p(group_offsets), _p(dys), _p(dyq), _p(dysc), _p(dw),
        d, _s(stream)))


def moe_mx_quantize_rows(src, C, group_offsets, q, sc, d: MoeDims, stream=None):
    _ok("moe_mx_quantize_rows", lib().moe_mx_quantize_rows(
        _p(src), int(C), _p(group_offsets), _p(q), _p(sc), d, _s(stream)))


def moe_mx_quantize_tokens(src, row_src, C, group_offsets, qt, sct, d: MoeDims, stream=None):
    _ok("moe_mx_quantize_tokens", lib().moe_mx_quantize_tokens(
        _p(src), _p(row_src), int(C), _p(group_offsets), _p(qt), _p(sct), d, _s(stream)))


def moe_mx_grouped_gemm_fc2_bwd(dyq, dysc, woq, wosc, z, ht, htsc, dyt, dytsc, group_offsets,
                                dz, dwo, dev_status, d: MoeDims, stream=None):
    _ok("moe_mx_grouped_gemm_fc2_bwd", lib().moe_mx_grouped_gemm_fc2_bwd(
        _p(dyq), _p(dysc), _p(woq), _p(wosc), _p(z), _p(ht), _p(htsc), _p(dyt), _p(dytsc),
        _p(group_offsets), _p(dz), _p(dwo), _p(dev_status), d, _s(stream)))


def moe_mx_grouped_gemm_fc1_bwd(dzq, dzsc, wiq, wisc, xt, xtsc, dzt, dztsc, group_offsets, dxs,
                                dwi, dev_status, d: MoeDims, stream=None):
    _ok("moe_mx_grouped_gemm_fc1_bwd", lib().moe_mx_grouped_gemm_fc1_bwd(
        _p(dzq), _p(dzsc), _p(wiq), _p(wisc), _p(xt), _p(xtsc), _p(dzt), _p(dztsc),
        _p(group_offsets), _p(dxs), _p(dwi), _p(dev_status), d, _s(stream)))


# ------------------------------------------------------------ layer operators
_NO_MAT = MoeMat(None, 0)


def _m(t):
    """A 2-D tensor with contiguous columns (any row stride) as a moe_mat."""
    if t is None:
        return _NO_MAT
    (rows, cols), (ld, inner) = t.shape, t.stride()
    if inner != 1 and cols > 1:
        raise ValueError("matrices passed to libmoe need contiguous columns")
    if rows < 2:  # its row stride is never used, and torch leaves it arbitrary
        ld = (cols + 7) // 8 * 8
    return MoeMat(t.data_ptr(), ld)


def moe_layer_norm(x, res, gamma, beta, r, y, mean, rstd, eps: float, stream=None):
    rows, D = x.shape
    _ok("moe_layer_norm", lib().moe_layer_norm(
        _m(x), _m(res), _p(gamma), _p(beta), _m(r), _m(y), _p(mean), _p(rstd), eps, rows, D,
        DTYPES[x.dtype], DTYPES[gamma.dtype], _s(stream)))


def moe_layer_norm_workspace_bytes(rows: int, D: int) -> int:
    return int(lib().moe_layer_norm_workspace_bytes(rows, D))


def moe_layer_norm_bwd(dy, r, gamma, mean, rstd, dres, dx, dgamma, dbeta, ws, stream=None):
    rows, D = dy.shape
    _ok("moe_layer_norm_bwd", lib().moe_layer_norm_bwd(
        _m(dy), _m(r), _p(gamma), _p(mean), _p(rstd), _m(dres), _m(dx), _p(dgamma), _p(dbeta),
        _p(ws), rows, D, DTYPES[dy.dtype], DTYPES[gamma.dtype], _s(stream)))


def moe_route_topk(logits, bias, ids, w, d: MoeTopkDims, stream=None):
    _ok("moe_route_topk", lib().moe_route_topk(_p(logits), _p(bias), _p(ids), _p(w), d,
                                               _s(stream)))


def moe_route_topk_bwd(logits, ids, dw, dlogits, d: MoeTopkDims, stream=None):
    _ok("moe_route_topk_bwd", lib().moe_route_topk_bwd(_p(logits), _p(ids), _p(dw), _p(dlogits),
                                                       d, _s(stream)))


def moe_linear(x, w, bias, res, y, z, dev_status, d: MoeLinearDims, stream=None):
    _ok("moe_linear", lib().moe_linear(_m(x), _m(w), _p(bias), _m(res), _m(y), _m(z),
                                       _p(dev_status), d, _s(stream)))


def moe_linear_workspace_bytes(d: MoeLinearDims) -> int:
    return int(lib().moe_linear_workspace_bytes(d))


def moe_linear_bwd(dy, z, x, w, dx_add, dx, dw, db, dev_status, ws, d: MoeLinearDims,
                   stream=None):
    _ok("moe_linear_bwd", lib().moe_linear_bwd(
        _m(dy), _m(z), _m(x), _m(w), _m(dx_add), _m(dx), _m(dw), _p(db), _p(dev_status), _p(ws),
        d, _s(stream)))


def moe_decode_workspace_bytes(d: MoeDims) -> int:
    return int(lib().moe_decode_workspace_bytes(d))


def moe_decode(x, wi, wo, logits, bias, mode, ids, w, res, out, dev_status, ws, d: MoeDims,
               stream=None):
    _ok("moe_decode", lib().moe_decode(
        _m(x), _p(wi), _p(wo), _p(logits), _p(bias), int(mode), _p(ids), _p(w), _m(res), _m(out),
        _p(dev_status), _p(ws), x.shape[0], d, DTYPES[x.dtype], _s(stream)))


def moe_block_norm(y, res, post, pre, gate, token_gate, r, u, rstd_y, rstd_r, d: MoeBlockNormDims,
                   stream=None):
    _ok("moe_block_norm", lib().moe_block_norm(
        _m(y), _m(res), _p(post), _p(pre), _p(gate), _p(token_gate), _m(r), _m(u), _p(rstd_y),
        _p(rstd_r), d, _s(stream)))


def moe_block_norm_workspace_bytes(d: MoeBlockNormDims) -> int:
    return int(lib().moe_block_norm_workspace_bytes(d))


def moe_block_norm_bwd(du, dr, r, y, post, pre, gate, token_gate, rstd_y, rstd_r, dres, dy, dpost,
                       dpre, dgate, dtoken_gate, ws, d: MoeBlockNormDims, stream=None):
    _ok("moe_block_norm_bwd", lib().moe_block_norm_bwd(
        _m(du), _m(dr), _m(r), _m(y), _p(post), _p(pre), _p(gate), _p(token_gate), _p(rstd_y),
        _p(rstd_r), _m(dres), _m(dy), _p(dpost), _p(dpre), _p(dgate), _p(dtoken_gate), _p(ws), d,
        _s(stream)))


def moe_adapter_plan_bytes(T: int, slots: int) -> int:
    return int(lib().moe_adapter_plan_bytes(int(T), int(slots)))


def moe_adapter_plan(ids, T: int, slots: int, plan, dev_status, stream=None):
    _ok("moe_adapter_plan", lib().moe_adapter_plan(
        _p(ids), ids.shape[0], int(T), int(slots), _p(plan), _p(dev_status), _s(stream)))


def moe_adapters_workspace_bytes(d: MoeAdapterDims) -> int:
    return int(lib().moe_adapters_workspace_bytes(d))


def moe_adapters(x, a, b, scale, res, y, plan, dev_status, ws, d: MoeAdapterDims, stream=None):
    _ok("moe_adapters", lib().moe_adapters(
        _m(x), _p(a), _p(b), _p(scale), _m(res), _m(y), _p(plan), _p(dev_status), _p(ws), x.shape[0], d,
        _s(stream)))
