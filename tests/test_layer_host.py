"""Refusals of the operators around the block, made before anything is
launched: through the C entry points (with pointers that are never read) and
through the Python operators."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_histogram_gb300 import binding as B
from mixture_experts_ffn_histogram_gb300.layer import LayerNorm, Linear, MoELayer, TopKRouter

P = 1 << 20          # an aligned address that no refused call touches
BAD, UNSUP = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_ffn_histogram_gb300 import _build
    _build.build()


def mat(p=P, ld=64):
    return B.MoeMat(p, ld)


NO = B.MoeMat(None, 0)


def norm(x=mat(), res=NO, gamma=P, beta=P, r=NO, y=mat(), mean=P, rstd=P, rows=4, D=64, t=0, wt=2):
    return B.lib().moe_layer_norm(x, res, gamma, beta, r, y, mean, rstd, 1e-5, rows, D, t, wt, None)


def norm_bwd(dy=mat(), r=mat(), gamma=P, mean=P, rstd=P, dres=NO, dx=mat(), dg=P, db=P, ws=P, rows=4,
             D=64, t=0, wt=2):
    return B.lib().moe_layer_norm_bwd(dy, r, gamma, mean, rstd, dres, dx, dg, db, ws, rows, D, t, wt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(D=0), UNSUP), (dict(D=8193, x=mat(ld=9000), y=mat(ld=9000)), UNSUP), (dict(rows=-1), UNSUP),
    (dict(rows=1 << 31), UNSUP), (dict(t=3), BAD), (dict(t=-1), BAD), (dict(t=0, wt=1), UNSUP),
    (dict(t=2, wt=0), UNSUP), (dict(x=NO), BAD), (dict(y=NO), BAD), (dict(gamma=None), BAD),
    (dict(beta=None), BAD), (dict(mean=None), BAD), (dict(rstd=None), BAD), (dict(x=mat(ld=63)), BAD),
    (dict(x=mat(p=P + 1)), BAD), (dict(gamma=P + 2), BAD), (dict(res=mat()), BAD),
    (dict(res=mat(ld=0), r=mat()), BAD), (dict(mean=P + 2), BAD),
])
def test_norm_refusals(kw, want):
    assert norm(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dg=None), BAD), (dict(db=None), BAD), (dict(ws=None), BAD), (dict(ws=P + 4), BAD),
    (dict(dy=NO), BAD), (dict(r=NO), BAD), (dict(dx=NO), BAD), (dict(gamma=None), BAD),
    (dict(mean=None), BAD), (dict(dres=mat(ld=5)), BAD), (dict(D=10000), UNSUP), (dict(wt=1), UNSUP),
    (dict(dg=P + 2), BAD),
])
def test_norm_backward_refusals(kw, want):
    assert norm_bwd(**kw) == want


def topk(logits=P, bias=P, ids=P, w=P, bwd=False, **kw):
    d = dict(T=4, E=64, K=4, gate=0, groups=8, top_groups=4, group_top=2, renorm=1, scale=1.0)
    d.update(kw)
    dd = B.MoeTopkDims(*[d[n] for n, _ in B.MoeTopkDims._fields_])
    if bwd:
        return B.lib().moe_route_topk_bwd(logits, ids, w, bias, dd, None)
    return B.lib().moe_route_topk(logits, bias, ids, w, dd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(E=0), UNSUP), (dict(E=1025, groups=1, top_groups=1), UNSUP), (dict(K=0), UNSUP),
    (dict(K=33, top_groups=8), UNSUP), (dict(T=-1), UNSUP), (dict(groups=7), UNSUP),
    (dict(groups=0), UNSUP), (dict(groups=64), UNSUP), (dict(top_groups=9), UNSUP),
    (dict(top_groups=0), UNSUP), (dict(top_groups=1, K=9), UNSUP), (dict(gate=2), BAD),
    (dict(group_top=3), BAD), (dict(group_top=0), BAD), (dict(logits=None), BAD), (dict(ids=None), BAD),
    (dict(w=None), BAD), (dict(logits=P + 4), BAD), (dict(bias=P + 4), BAD),
    (dict(T=1 << 30, K=4), UNSUP), (dict(E=1023, groups=3, top_groups=2), UNSUP),
])
def test_topk_refusals(kw, want):
    assert topk(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(K=65, E=64), UNSUP), (dict(E=2000), UNSUP), (dict(gate=5), BAD), (dict(bias=None), BAD),
    (dict(ids=None), BAD), (dict(w=P + 8), BAD),
])
def test_topk_backward_refusals(kw, want):
    assert topk(bwd=True, **kw) == want


def linear(x=mat(), w=mat(), bias=P, res=NO, y=mat(), z=NO, M=4, K=64, N=64, t=0, o=0, act=4, st=P):
    d = B.MoeLinearDims(M, K, N, t, o, act)
    return B.lib().moe_linear(x, w, bias, res, y, z, st, d, None)


def linear_bwd(dy=mat(), z=mat(), x=mat(), w=mat(), add=NO, dx=mat(), dw=mat(), db=P, M=4, K=64, N=64, t=0,
               o=0, act=4, st=P, ws=P):
    d = B.MoeLinearDims(M, K, N, t, o, act)
    return B.lib().moe_linear_bwd(dy, z, x, w, add, dx, dw, db, st, ws, d, None)


SIZES = [
    (dict(K=63), UNSUP), (dict(N=12), UNSUP), (dict(K=0), UNSUP), (dict(N=-8), UNSUP), (dict(M=-1), UNSUP),
    (dict(M=(1 << 31) - 1), UNSUP), (dict(t=2), UNSUP), (dict(t=0, o=1), UNSUP), (dict(t=7), BAD),
    (dict(o=9), BAD), (dict(act=5), BAD), (dict(act=-1), BAD), (dict(st=P + 4), BAD),
]


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(x=NO), BAD), (dict(w=NO), BAD), (dict(y=NO), BAD), (dict(x=mat(ld=56)), BAD),
    (dict(x=mat(ld=68)), BAD), (dict(w=mat(p=P + 8)), BAD), (dict(y=mat(ld=66)), BAD),
    (dict(o=2, y=mat(ld=66)), BAD), (dict(res=mat(ld=60)), BAD), (dict(z=mat(ld=8)), BAD),
    (dict(bias=P + 4), BAD),
])
def test_linear_refusals(kw, want):
    assert linear(**kw) == want


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(dx=NO, dw=NO, db=None), BAD), (dict(dy=NO), BAD), (dict(z=NO), BAD), (dict(x=NO), BAD),
    (dict(w=NO), BAD), (dict(ws=None), BAD), (dict(ws=P + 4), BAD), (dict(add=mat(ld=60)), BAD),
    (dict(dx=mat(ld=4)), BAD), (dict(dw=mat(p=P + 4)), BAD), (dict(db=P + 4), BAD),
])
def test_linear_backward_refusals(kw, want):
    assert linear_bwd(**kw) == want


def test_workspace_sizes():
    assert B.moe_layer_norm_workspace_bytes(10, 64) >= 10 * 2 * 64 * 4
    assert B.moe_layer_norm_workspace_bytes(10, 0) == 0
    d = B.linear_dims(100, 64, 128, act="silu")
    assert B.moe_linear_workspace_bytes(d) >= 100 * 128 * 2 + 1024 * 128 * 4
    assert B.moe_linear_workspace_bytes(B.linear_dims(100, 63, 128)) == 0
    assert ctypes.sizeof(B.MoeMat) == 16 and ctypes.sizeof(B.MoeTopkDims) == 36
    assert ctypes.sizeof(B.MoeLinearDims) == 32


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


F32 = torch.float32


def test_norm_checks_its_tensors():
    op = LayerNorm(8, 64, device="cpu")
    g = t(64, dtype=F32)
    for args, kw in (((t(9, 64), g, g), {}), ((t(8, 63), g, g), {}), ((t(8, 64, dtype=F32), g, g), {}),
                     ((t(8, 64), t(64), g), {}), ((t(8, 64), g, t(65, dtype=F32)), {}),
                     ((t(8, 64), g, g), {"res": t(7, 64)}), ((t(8, 8, 8), g, g), {}),
                     ((t(8, 128)[:, ::2], g, g), {})):
        with pytest.raises(ValueError):
            op.forward(*args, **kw)
    with pytest.raises(RuntimeError):
        op.backward(t(8, 64), t(8, 64), g)                     # no forward yet
    st = t(8, dtype=F32)
    with pytest.raises(ValueError):
        op.backward(t(8, 64), t(8, 64), g, mean=st, rstd=st[:7])
    with pytest.raises(RuntimeError):
        LayerNorm(8, 64, train=False, device="cpu").backward(t(8, 64), t(8, 64), g, mean=st, rstd=st)
    with pytest.raises(ValueError):
        LayerNorm(8, 64, torch.float16, torch.bfloat16, device="cpu")
    with pytest.raises(RuntimeError):                               # no kernel for CPU tensors
        op.forward(t(8, 64), g, g)
    with pytest.raises(B.MoeError):                                 # rows on one another
        B.moe_layer_norm(t(1, 64).expand(8, 64), None, g, g, None, t(8, 64), None, None, 1e-5, stream=0)


def test_router_checks_its_tensors():
    op = TopKRouter(8, 16, 2, train=True, device="cpu")
    for a, b in ((t(9, 16, dtype=F32), None), (t(8, 15, dtype=F32), None), (t(8, 16), None),
                 (t(8, 16, dtype=F32), t(15, dtype=F32)), (t(16, 8, dtype=F32).t(), None)):
        with pytest.raises(ValueError):
            op.forward(a, b)
    with pytest.raises(RuntimeError):
        op.backward(t(8, 2, dtype=F32), t(8, 16, dtype=F32))
    with pytest.raises(ValueError):
        op.backward(t(8, 3, dtype=F32), t(8, 16, dtype=F32), ids=t(8, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        TopKRouter(8, 16, 2, score="tanh", device="cpu")
    with pytest.raises(B.MoeError):
        B.moe_route_topk(t(8, 16, dtype=F32), None, t(8, 20), t(8, 20), B.topk_dims(8, 16, 20), stream=0)


def test_linear_checks_its_tensors():
    op = Linear(8, 64, 128, act="silu", train=True, device="cpu")
    w = t(64, 128)
    for args, kw in (((t(9, 64), w), {}), ((t(8, 72), w), {}), ((t(8, 64), t(128, 64)), {}),
                     ((t(8, 64), t(128, 64).t()), {}), ((t(8, 64, dtype=F32), w), {}),
                     ((t(8, 64), w), {"bias": t(128)}), ((t(8, 64), w), {"res": t(8, 64)}),
                     ((t(8, 64), w), {"res": t(8, 128, dtype=F32)})):
        with pytest.raises(ValueError):
            op.forward(*args, **kw)
    with pytest.raises(RuntimeError):
        op.backward(t(8, 128), t(8, 64), w)
    with pytest.raises(ValueError):
        op.backward(t(8, 128), t(8, 64), w, z=t(8, 120))
    with pytest.raises(RuntimeError):
        Linear(8, 64, 128, device="cpu").backward(t(8, 128), t(8, 64), w)
    for bad in (dict(K=60), dict(N=100), dict(dtype=F32), dict(act="tanh"),
                dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            Linear(**{**dict(M=8, K=64, N=128, device="cpu"), **bad})


def test_layer_checks_its_rows():
    lay = MoELayer(8, 64, 8, 2, 64, shared=64, device="cpu", score="sigmoid")
    with pytest.raises(ValueError):
        lay.forward(t(7, 64), {})
    with pytest.raises(RuntimeError):
        lay.backward(None, t(8, 64), {})
