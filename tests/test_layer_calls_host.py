"""What the operators around the block do at a call before anything is
launched, with stand-ins for the kernels and for the current device."""
import pytest
import torch

from mixture_experts_ffn_histogram_gb300 import binding as B
from mixture_experts_ffn_histogram_gb300.layer import LayerNorm, Linear, TopKRouter

F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_ffn_histogram_gb300 import _build
    _build.build()


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _stand_in(op, launched):
    """`op` (built for the CPU) with kernels that only note that they were called."""
    def kernel(*args):
        launched.append(args)
        return 0
    op._fwd = op._bwd = kernel
    return op


def _calls():
    """(operator, a call of it) for each operator and direction."""
    g, st, l = t(64, dtype=F32), t(8, dtype=F32), t(8, 16, dtype=F32)
    x, y, w = t(8, 64), t(8, 128), t(64, 128)
    dw, ids = t(8, 2, dtype=F32), t(8, 2, dtype=torch.int32)
    norm, router = LayerNorm(8, 64, device="cpu"), TopKRouter(8, 16, 2, train=True, device="cpu")
    lin = Linear(8, 64, 128, train=True, device="cpu")
    return [
        (norm, lambda **k: norm.forward(x, g, g, res=x, **k)),
        (norm, lambda **k: norm.backward(x, x, g, mean=st, rstd=st, **k)),
        (router, lambda **k: router.forward(l, **k)),
        (router, lambda **k: router.backward(dw, l, ids=ids, **k)),
        (lin, lambda **k: lin.forward(x, w, **k)),
        (lin, lambda **k: lin.backward(y, x, w, **k)),
    ]


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("stream", [{}, {"stream": 0}])
def test_another_current_device_is_refused(monkeypatch, which, stream):
    op, call = _calls()[which]
    launched = []
    _stand_in(op, launched).device = torch.device("cuda", 0)
    monkeypatch.setattr(B, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(B, "_current_device", lambda: 1, raising=False)
    with pytest.raises(RuntimeError, match="current device"):
        call(**stream)
    assert not launched
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    call(**stream)
    assert len(launched) == 1


@pytest.mark.parametrize("which", range(6))
def test_calls_allocate_no_memory(monkeypatch, which):
    """A buffer allocated in a call would come from the current stream's
    memory, which that stream may still use, and be written on the call's."""
    op, call = _calls()[which]
    _stand_in(op, [])

    def no(*args, **kw):
        raise AssertionError("an allocation in a call")

    for name in ("empty", "empty_like", "zeros", "zeros_like", "full"):
        monkeypatch.setattr(torch, name, no)
    call(stream=0)
