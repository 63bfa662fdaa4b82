"""The whole layer (norm, gate, routing, experts, shared expert) forward and
backward against 64-bit autograd of the same mathematics, and captured into a
graph."""
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import act, topk_weights

pytestmark = pytest.mark.gpu


def _make(T, D, E, F, S, seed):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).bfloat16().cuda()

    w = {"gamma": (1 + 0.1 * torch.randn(D, generator=g)).cuda(),
         "beta": (0.1 * torch.randn(D, generator=g)).cuda(),
         "wr": r(D, E, scale=D ** -0.5), "wi": r(E, D, 2 * F, scale=D ** -0.5),
         "wo": r(E, F, D, scale=F ** -0.5), "w1": r(D, S, scale=D ** -0.5),
         "b1": (0.1 * torch.randn(S, generator=g)).cuda(), "w2": r(S, D, scale=S ** -0.5),
         "b2": (0.1 * torch.randn(D, generator=g)).cuda()}
    return w, r(T, D), r(T, D), r(T, D), r(T, D), (0.05 * torch.randn(E, generator=g)).cuda()


def _reference(x, res, w, ids, gate, renorm, scale, name, eps):
    r = x + res
    mean = r.mean(1, keepdim=True)
    xh = (r - mean) / ((r - mean).square().mean(1, keepdim=True) + eps).sqrt()
    u = xh * w["gamma"] + w["beta"]
    p = topk_weights(u @ w["wr"], ids, gate, renorm, scale)
    m = torch.zeros_like(u)
    F = w["wo"].shape[1]
    for e in range(w["wi"].shape[0]):
        a = u @ w["wi"][e]
        y = (act(a[:, :F], "silu") * a[:, F:]) @ w["wo"][e]
        m = m + y * (p * (ids == e)).sum(1, keepdim=True)
    return r, act(u @ w["w1"] + w["b1"], name) @ w["w2"] + w["b2"] + m


# At most ten bf16 roundings lie on any path from an input to an output (the
# stored rows between the kernels), each of relative size 2^-8 at most.
LIMIT = 10 * 2.0 ** -8


def _near(name, got, want):
    off = (got.double() - want).norm() / want.norm()
    assert off <= LIMIT, f"{name}: relative error {float(off):.3g}"


@pytest.mark.parametrize("T,gate,renorm,name", [(200, "sigmoid", True, "silu"),
                                                 (1, "sigmoid", True, "gelu"),
                                                 (700, "softmax", False, "gelu")])
def test_layer_forward_and_backward(T, gate, renorm, name):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import MoELayer
    D, E, K, F, S = 256, 16, 4, 128, 192
    w, x, res, dr, df, bias = _make(T, D, E, F, S, T)
    lay = MoELayer(T, D, E, K, F, S, act=name, score=gate, groups=4, top_groups=2, group_top=2,
                   renorm=renorm, scale=2.0)
    r, f = lay.forward(x, w, res=res, bias=bias)
    dx = lay.backward(dr, df, w)
    torch.cuda.synchronize()
    for op in (lay.gate, lay.up, lay.down, lay.block):
        assert int(op.status.item()) == 0
    leaf = {k: v.double().requires_grad_(True) for k, v in w.items()}
    x64, res64 = x.double().requires_grad_(True), res.double()
    rr, ff = _reference(x64, res64, leaf, lay.router.ids, gate, renorm, 2.0, name, 1e-5)
    _near("r", r, rr.detach())
    _near("f", f, ff.detach())
    keys = list(leaf)
    grads = torch.autograd.grad([rr, ff], [x64] + [leaf[k] for k in keys], [dr.double(), df.double()])
    _near("dx", dx, grads[0])
    got = {"gamma": lay.norm.dgamma, "beta": lay.norm.dbeta, "wr": lay.gate.dw, "wi": lay.block.dwi,
           "wo": lay.block.dwo, "w1": lay.up.dw, "b1": lay.up.db, "w2": lay.down.dw, "b2": lay.down.db}
    for k, want in zip(keys, grads[1:]):
        _near(k, got[k], want)


def test_layer_in_a_graph_and_on_a_stream():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import MoELayer
    T, D, E, K, F, S = 256, 256, 16, 4, 128, 256
    w, x, res, dr, df, bias = _make(T, D, E, F, S, 3)
    lay = MoELayer(T, D, E, K, F, S, score="sigmoid")

    def step(stream=None):
        r, f = lay.forward(x, w, res=res, bias=bias, stream=stream)
        return [r, f, lay.backward(dr, df, w, stream=stream), lay.gate.dw, lay.norm.dgamma]

    ref = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for t in out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
