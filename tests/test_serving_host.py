"""Refusals of the operators that serve and wrap the expert block, made before
anything is launched: through the C entry points (with pointers that are never
read) and through the Python operators; and what a call does on the host."""
import pytest
import torch

from mixture_experts_ffn_histogram_gb300 import binding as B
from mixture_experts_ffn_histogram_gb300.layer import (AdapterBatch, BlockNorm, DecodeLayer, LowRankAdapters,
                                                       MoEDecode)

P = 1 << 20          # an aligned address that no refused call touches
BAD, UNSUP = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_ffn_histogram_gb300 import _build
    _build.build()


def mat(p=P, ld=64):
    return B.MoeMat(p, ld)


NO = B.MoeMat(None, 0)


# ------------------------------------------------------------- the C entry points
def decode(x=mat(ld=128), wi=P, wo=P, logits=P, bias=None, mode=0, ids=P, w=P, res=NO, out=mat(ld=128), status=P,
           ws=P, n=4, t=0, **dims):
    d = dict(T=8, D=128, E=16, K=2, F=64)
    d.update(dims)
    return B.lib().moe_decode(x, wi, wo, logits, bias, mode, ids, w, res, out, status, ws, n,
                              B.dims(**d), t, None)


@pytest.mark.parametrize("kw,want", [
    (dict(D=96), UNSUP), (dict(D=0), UNSUP), (dict(D=16448), UNSUP), (dict(F=100), UNSUP), (dict(F=16448), UNSUP),
    (dict(E=0), UNSUP), (dict(E=1025), UNSUP), (dict(K=0), UNSUP), (dict(K=17), UNSUP), (dict(E=64, K=33), UNSUP),
    (dict(T=257), UNSUP), (dict(T=-1), UNSUP), (dict(T=256, K=9), UNSUP), (dict(t=2), UNSUP), (dict(t=3), BAD),
    (dict(mode=3), BAD), (dict(mode=-1), BAD), (dict(n=9), BAD), (dict(n=-1), BAD), (dict(x=NO), BAD),
    (dict(x=mat(ld=120)), BAD), (dict(x=mat(ld=132)), BAD), (dict(x=mat(P + 8, 128)), BAD), (dict(out=NO), BAD),
    (dict(out=mat(ld=64)), BAD), (dict(wi=None), BAD), (dict(wo=None), BAD), (dict(wi=P + 8), BAD),
    (dict(ws=None), BAD), (dict(ws=P + 4), BAD), (dict(logits=None), BAD), (dict(logits=P + 2), BAD),
    (dict(bias=P + 1), BAD), (dict(mode=2, ids=None), BAD), (dict(mode=2, w=None), BAD), (dict(ids=P + 2), BAD),
    (dict(res=mat(ld=100)), BAD), (dict(status=P + 1), BAD),
])
def test_decode_refusals(kw, want):
    assert decode(**kw) == want


def test_decode_of_no_token_does_nothing():
    assert decode(n=0, x=NO, out=NO) == B.MOE_OK


def test_decode_workspace():
    assert B.moe_decode_workspace_bytes(B.dims(8, 100, 16, 2, 64)) == 0
    small = B.moe_decode_workspace_bytes(B.dims(1, 2816, 128, 8, 704))
    large = B.moe_decode_workspace_bytes(B.dims(256, 2816, 128, 8, 704))
    assert 0 < small < large and small % 256 == 0


def norm(y=mat(), res=mat(), post=P, pre=P, gate=None, tg=None, r=mat(), u=mat(), sy=P, sr=P, rows=4, D=64, t=0,
         wt=2):
    d = B.MoeBlockNormDims(rows, D, t, wt, 1e-6, 1.0, 0.0)
    return B.lib().moe_block_norm(y, res, post, pre, gate, tg, r, u, sy, sr, d, None)


@pytest.mark.parametrize("kw,want", [
    (dict(D=0), UNSUP), (dict(D=8193), UNSUP), (dict(rows=-1), UNSUP), (dict(rows=1 << 31), UNSUP), (dict(t=3), BAD),
    (dict(wt=1), UNSUP), (dict(t=2, wt=0), UNSUP), (dict(res=NO), BAD), (dict(r=NO), BAD), (dict(u=NO), BAD),
    (dict(y=mat(ld=63)), BAD), (dict(res=mat(P + 1)), BAD), (dict(u=mat(ld=10)), BAD), (dict(post=P + 2), BAD),
    (dict(gate=P + 2), BAD), (dict(tg=P + 2), BAD), (dict(sy=P + 2), BAD), (dict(y=NO), BAD),
    (dict(y=NO, post=None, pre=None), BAD), (dict(y=NO, post=None, gate=P), BAD), (dict(y=NO, post=None, tg=P), BAD),
])
def test_block_norm_refusals(kw, want):
    assert norm(**kw) == want


def norm_bwd(du=mat(), dr=mat(), r=mat(), y=mat(), post=P, pre=P, gate=P, tg=P, sy=P, sr=P, dres=mat(), dy=mat(),
             dpost=P, dpre=P, dgate=P, dtg=P, ws=P, rows=4, D=64, t=0, wt=2):
    d = B.MoeBlockNormDims(rows, D, t, wt, 1e-6, 1.0, 0.0)
    return B.lib().moe_block_norm_bwd(du, dr, r, y, post, pre, gate, tg, sy, sr, dres, dy, dpost, dpre, dgate, dtg,
                                      ws, d, None)


@pytest.mark.parametrize("kw,want", [
    (dict(D=9000), UNSUP), (dict(du=NO), BAD), (dict(r=NO), BAD), (dict(sr=None), BAD), (dict(sy=None), BAD),
    (dict(dres=NO), BAD), (dict(y=NO), BAD), (dict(post=None), BAD), (dict(pre=None), BAD), (dict(gate=None), BAD),
    (dict(tg=None), BAD), (dict(ws=None), BAD), (dict(ws=P + 8), BAD), (dict(dr=mat(ld=3)), BAD),
    (dict(dy=mat(ld=3)), BAD), (dict(pre=None, dpre=None), BAD), (dict(pre=None, dpre=None, du=NO, dr=NO), BAD),
    (dict(dpost=P + 2), BAD), (dict(dtg=P + 1), BAD),
])
def test_block_norm_backward_refusals(kw, want):
    assert norm_bwd(**kw) == want


def adapters(x=mat(ld=128), a=P, b=P, scale=P, res=NO, y=mat(ld=64), plan=P, status=P, ws=P, n=4, **dims):
    d = dict(T=8, K=128, N=64, slots=2, rank=8, type=0)
    d.update(dims)
    return B.lib().moe_adapters(x, a, b, scale, res, y, plan, status, ws, n, B.MoeAdapterDims(**d), None)


@pytest.mark.parametrize("kw,want", [
    (dict(K=100), UNSUP), (dict(N=60), UNSUP), (dict(K=0), UNSUP), (dict(rank=12), UNSUP), (dict(rank=136), UNSUP),
    (dict(rank=0), UNSUP), (dict(slots=0), UNSUP), (dict(slots=1025), UNSUP), (dict(T=(1 << 20) + 1), UNSUP),
    (dict(type=2), UNSUP), (dict(type=7), BAD), (dict(n=9), BAD), (dict(n=-1), BAD), (dict(x=NO), BAD),
    (dict(x=mat(ld=127)), BAD), (dict(y=NO), BAD), (dict(y=mat(P + 8)), BAD), (dict(res=mat(ld=68)), BAD),
    (dict(a=None), BAD), (dict(b=P + 8), BAD), (dict(scale=None), BAD), (dict(scale=P + 2), BAD),
    (dict(plan=None), BAD), (dict(ws=None), BAD), (dict(status=P + 2), BAD),
])
def test_adapter_refusals(kw, want):
    assert adapters(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(slots=0), UNSUP), (dict(slots=1025), UNSUP), (dict(T=-1), UNSUP), (dict(T=1 << 21), UNSUP), (dict(n=9), BAD),
    (dict(n=-1), BAD), (dict(ids=None), BAD), (dict(ids=P + 2), BAD), (dict(plan=None), BAD), (dict(plan=P + 8), BAD),
])
def test_plan_refusals(kw, want):
    k = dict(ids=P, n=4, T=8, slots=3, plan=P, status=P)
    k.update(kw)
    assert B.lib().moe_adapter_plan(*k.values(), None) == want


# ---------------------------------------------------------- the Python operators
def test_constructors_refuse():
    for args in ((8, 100, 16, 2, 64), (300, 128, 16, 2, 64), (8, 128, 4, 8, 64), (256, 128, 64, 16, 64)):
        with pytest.raises(ValueError, match="unsupported sizes"):
            MoEDecode(*args, device="cpu")
    with pytest.raises(ValueError, match="not supported"):
        MoEDecode(8, 128, 16, 2, 64, dtype=F32, device="cpu")
    with pytest.raises(ValueError, match="score mode"):
        MoEDecode(8, 128, 16, 2, 64, score_mode=5, device="cpu")
    with pytest.raises(ValueError, match="not supported"):
        BlockNorm(8, 64, dtype=BF, weight_dtype=torch.float16, device="cpu")
    with pytest.raises(ValueError, match="unsupported sizes"):
        AdapterBatch(8, 0, device="cpu")
    with pytest.raises(ValueError, match="unsupported sizes"):
        LowRankAdapters(8, 64, 64, 2, 20, device="cpu")
    with pytest.raises(ValueError, match="not supported"):
        LowRankAdapters(8, 64, 64, 2, 8, dtype=F32, device="cpu")


def t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def _stand_in(op, launched):
    """`op` (built for the CPU) with kernels that only note that they were called."""
    def kernel(*args):
        launched.append(args)
        return 0
    op._fwd = op._bwd = kernel
    return op


def _calls():
    """(operator, a good call with arguments to change) for each operator and direction."""
    given = MoEDecode(8, 128, 16, 2, 64, B.SCORE_GIVEN, device="cpu")
    own = MoEDecode(8, 128, 16, 2, 64, device="cpu")
    x, wi, wo = t(8, 128), t(16, 128, 128), t(16, 64, 128)
    ids, w, l, b = t(8, 2, dtype=I32), t(8, 2, dtype=F32), t(8, 16, dtype=F32), t(16, dtype=F32)
    n = BlockNorm(8, 64, device="cpu")
    y, g, tg = t(8, 64), t(64, dtype=F32), t(8, dtype=F32)
    batch, ad = AdapterBatch(8, 3, device="cpu"), LowRankAdapters(8, 128, 64, 3, 16, device="cpu")
    _stand_in(batch, [])
    batch.group(t(8, dtype=I32), stream=0)
    one = t(8, dtype=I32)
    a, bb, sc = t(3, 16, 128), t(3, 64, 16), t(3, dtype=F32)
    return [
        (given, lambda **k: given.forward(**{**dict(x=x, wi=wi, wo=wo, ids=ids, w=w, res=x), **k})),
        (own, lambda **k: own.forward(**{**dict(x=x, wi=wi, wo=wo, logits=l, bias=b), **k})),
        (n, lambda **k: n.forward(**{**dict(res=y, y=y, post=g, pre=g, gate=g, token_gate=tg), **k})),
        (n, lambda **k: n.backward(**{**dict(du=y, dr=y, r=y, y=y, post=g, pre=g, gate=g, token_gate=tg, rstd_y=tg,
                                             rstd_r=tg), **k})),
        (batch, lambda **k: batch.group(**{**dict(ids=one), **k})),
        (ad, lambda **k: ad.forward(**{**dict(batch=batch, x=x, a=a, b=bb, scale=sc, res=y), **k})),
    ]


WRONG = [
    (0, dict(x=t(9, 128)), "x must"), (0, dict(x=t(8, 64)), "x must"), (0, dict(x=t(8, 128, dtype=F32)), "x must"),
    (0, dict(x=t(128, 8).t()), "x must"), (0, dict(wi=t(16, 128, 64)), "wi must"), (0, dict(wo=t(16, 128, 64)), "wo must"),
    (0, dict(wi=t(16, 128, 256)[:, :, ::2]), "wi must"), (0, dict(ids=None), "needs ids"), (0, dict(w=None), "needs ids"),
    (0, dict(ids=t(8, 2)), "ids must"), (0, dict(ids=t(7, 2, dtype=I32)), "ids must"), (0, dict(res=t(7, 128)), "res must"),
    (1, dict(logits=None), "needs logits"), (1, dict(logits=t(8, 15, dtype=F32)), "logits must"),
    (1, dict(bias=t(15, dtype=F32)), "bias must"), (1, dict(logits=t(8, 16)), "logits must"),
    (2, dict(res=t(9, 64)), "res must"), (2, dict(y=t(7, 64)), "y must"), (2, dict(post=t(64)), "post must"),
    (2, dict(pre=t(63, dtype=F32)), "pre must"), (2, dict(token_gate=t(7, dtype=F32)), "token_gate must"),
    (2, dict(y=None), "without y"), (3, dict(du=None), "du is"), (3, dict(pre=None), "du is"),
    (3, dict(du=None, pre=None, dr=None), "without pre"), (3, dict(y=t(8, 63)), "y must"),
    (3, dict(rstd_y=t(7, dtype=F32)), "rstd_y must"), (3, dict(rstd_r=t(8)), "rstd_r must"), (3, dict(dr=t(7, 64)), "dr must"),
    (4, dict(ids=t(9, dtype=I32)), "ids must"), (4, dict(ids=t(8)), "ids must"), (4, dict(ids=t(8, 1, dtype=I32)), "ids must"),
    (4, dict(ids=t(16, dtype=I32)[::2]), "ids must"),
    (5, dict(x=t(7, 128)), "grouped for 8"), (5, dict(x=t(8, 64)), "x must"), (5, dict(a=t(3, 128, 16)), "a must"),
    (5, dict(b=t(3, 16, 64)), "b must"), (5, dict(scale=t(2, dtype=F32)), "scale must"), (5, dict(res=t(8, 60)), "res must"),
]


@pytest.mark.parametrize("which,kw,message", WRONG)
def test_wrong_arguments_launch_nothing(which, kw, message):
    op, call = _calls()[which]
    launched = []
    _stand_in(op, launched)
    with pytest.raises(ValueError, match=message):
        call(stream=0, **kw)
    assert not launched
    call(stream=0)
    assert len(launched) == 1


def test_a_batch_of_other_sizes_is_refused():
    op, call = _calls()[5]
    launched = []
    _stand_in(op, launched)
    for other in (AdapterBatch(9, 3, device="cpu"), AdapterBatch(8, 2, device="cpu"), AdapterBatch(8, 3, device="cpu")):
        with pytest.raises(ValueError, match="batch"):
            call(stream=0, batch=other)     # the last was never grouped
    assert not launched


def test_backward_needs_a_forward_or_its_values():
    n = _stand_in(BlockNorm(8, 64, device="cpu"), [])
    y, g = t(8, 64), t(64, dtype=F32)
    with pytest.raises(RuntimeError, match="forward first"):
        n.backward(y, y, y=y, pre=g, stream=0)
    with pytest.raises(RuntimeError, match="forward first"):
        n.backward(None, y, y=y, post=g, stream=0)
    with pytest.raises(RuntimeError, match="train=True"):
        BlockNorm(8, 64, train=False, device="cpu").backward(None, y, y=y)


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("stream", [{}, {"stream": 0}])
def test_another_current_device_is_refused(monkeypatch, which, stream):
    op, call = _calls()[which]
    launched = []
    _stand_in(op, launched).device = torch.device("cuda", 0)
    monkeypatch.setattr(B, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(B, "_current_device", lambda: 1, raising=False)
    # (the adapters' batch stays on the CPU: that is refused first)
    with pytest.raises((RuntimeError, ValueError), match="current device" if which != 5 else "batch is for"):
        call(**stream)
    assert not launched


@pytest.mark.parametrize("which", range(6))
def test_calls_allocate_no_memory(monkeypatch, which):
    op, call = _calls()[which]
    _stand_in(op, [])

    def no(*a, **kw):
        raise AssertionError("an allocation in a call")

    for name in ("empty", "empty_like", "zeros", "zeros_like", "full"):
        monkeypatch.setattr(torch, name, no)
    call(stream=0)


def test_the_kernels_need_a_device():
    for op, call in _calls():
        if isinstance(op, AdapterBatch):
            continue
        with pytest.raises(RuntimeError, match="CUDA device"):
            call(stream=0)


def test_the_layer_refuses_a_batch_without_adapters():
    lay = DecodeLayer(4, 64, 8, 2, 64, 64, device="cpu")
    with pytest.raises(ValueError, match="without adapters"):
        lay.forward(t(4, 64), t(4, 64), {}, batch=AdapterBatch(4, 2, device="cpu"))
