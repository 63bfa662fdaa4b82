"""The served layer's routing modes: what it takes and refuses (CPU), and the
modes beside the default one against 64-bit mathematics (GPU)."""
import pytest
import torch

from mixture_experts_ffn_histogram_gb300 import binding as B
from mixture_experts_ffn_histogram_gb300.layer import BlockNorm, DecodeLayer, TopKRouter
from tests.gpu_common import need_gpu
from tests.layer_refs import act, half_step
from tests.serving_refs import experts, select

BF, F32 = torch.bfloat16, torch.float32


def _weights(D, E, F, S, seed, device):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0, t=BF):
        return (scale * torch.randn(*shape, generator=g)).to(t).to(device)

    return {"wr": r(D, E, scale=D ** -0.5), "wi": r(E, D, 2 * F, scale=D ** -0.5), "wo": r(E, F, D, scale=F ** -0.5),
            "w1": r(D, S, scale=D ** -0.5), "b1": r(S, scale=0.1, t=F32), "w2": r(S, D, scale=S ** -0.5),
            "b2": r(D, scale=0.1, t=F32), "post": r(D, scale=0.1, t=F32), "pre": r(D, scale=0.1, t=F32)}


def _stand_ins(lay, called):
    """The layer's operators (built for the CPU) with kernels that only note their calls."""
    for name in ("gate", "up", "down", "experts", "norm"):
        op = getattr(lay, name)
        if op is not None:
            def kernel(*args, name=name):
                called.append(name)
                return 0
            op._fwd = kernel
    return lay


def test_a_given_selection_is_handed_on():
    T, D, E, K, F, S = 4, 64, 5, 2, 64, 64
    called = []
    lay = _stand_ins(DecodeLayer(T, D, E, K, F, S, B.SCORE_GIVEN, device="cpu"), called)
    w = _weights(D, E, F, S, 1, "cpu")
    del w["wr"]
    x = torch.zeros(T, D, dtype=BF)
    ids, p = torch.zeros(T, K, dtype=torch.int32), torch.ones(T, K)
    lay.forward(x, x, w, ids=ids, w=p, stream=0)
    assert called == ["up", "down", "experts", "norm"]
    assert lay.experts.ids is ids and lay.experts.w is p


def test_arguments_by_place_are_as_before():
    T, D, E, K, F, S = 4, 64, 8, 2, 64, 64
    called = []
    lay = _stand_ins(DecodeLayer(T, D, E, K, F, S, device="cpu"), called)
    x = torch.zeros(T, D, dtype=BF)
    lay.forward(x, x, _weights(D, E, F, S, 1, "cpu"), None, None, 0)    # bias, batch, stream
    assert called == ["gate", "up", "down", "experts", "norm"]


@pytest.mark.parametrize("mode,given,bias,message", [
    (B.SCORE_GIVEN, (), False, "needs ids and w"), (B.SCORE_GIVEN, ("ids",), False, "needs ids and w"),
    (B.SCORE_GIVEN, ("w",), False, "needs ids and w"), (B.SCORE_GIVEN, ("ids", "w"), True, "no bias"),
    (B.SCORE_SOFTMAX_TOPK, ("ids", "w"), False, "selects the experts itself"),
    (B.SCORE_SIGMOID_NORM, ("w",), False, "selects the experts itself"),
])
def test_a_selection_of_the_other_kind_launches_nothing(mode, given, bias, message):
    T, D, E, K, F, S = 4, 64, 8, 2, 64, 64
    called = []
    lay = _stand_ins(DecodeLayer(T, D, E, K, F, S, mode, device="cpu"), called)
    x = torch.zeros(T, D, dtype=BF)
    have = {"ids": torch.zeros(T, K, dtype=torch.int32), "w": torch.ones(T, K)}
    with pytest.raises(ValueError, match=message):
        lay.forward(x, x, _weights(D, E, F, S, 1, "cpu"), bias=torch.zeros(E) if bias else None,
                    **{k: have[k] for k in given}, stream=0)
    assert not called


# At most seven roundings to 16 bits lie on any path from an input to an output
# (h twice, the results of the products and norms), each of relative size eps / 2
# at most.
def _near(name, got, want):
    off, limit = (got.double() - want).norm() / want.norm(), 7 * half_step(got.dtype)
    assert off <= limit, f"{name}: relative error {float(off):.3g}, limit {limit:.3g}"


@pytest.mark.gpu
@pytest.mark.parametrize("mode,T,E", [("sigmoid", 1, 16), ("sigmoid", 40, 24), ("given", 1, 60), ("given", 33, 60)])
def test_the_layer(mode, T, E):
    need_gpu()
    D, K, F, S, eps, branch, offset = 320, 4, 128, 192, 1e-6, 0.5, 1.0
    w = _weights(D, E, F, S, T, "cuda")
    g = torch.Generator().manual_seed(T)
    r = torch.randn(T, D, generator=g).to(BF).cuda()
    bias = (0.3 * torch.randn(E, generator=g)).cuda()
    front = BlockNorm(T, D, eps=eps, offset=offset, train=False)
    u = front.forward(r, pre=w["pre"])
    code = {"sigmoid": B.SCORE_SIGMOID_NORM, "given": B.SCORE_GIVEN}[mode]
    lay = DecodeLayer(T, D, E, K, F, S, code, eps=eps, branch=branch, offset=offset)
    if mode == "given":     # groups of experts, a bias that stays out of the weights, any number of experts
        logits = (u.float() @ w.pop("wr").float()).contiguous()
        chosen, p = TopKRouter(T, E, K, groups=6, top_groups=3, scale=2.5).forward(logits, bias)
        r1, u1 = lay.forward(r, u, w, ids=chosen, w=p)
    else:
        r1, u1 = lay.forward(r, u, w, bias=bias)
        chosen, p = select(lay.gate._y[:T], bias, K, mode)
        assert torch.equal(lay.experts.ids, chosen)
    torch.cuda.synchronize()
    assert int(lay.experts.status.item()) == 0
    d = {k: v.double() for k, v in w.items()}
    x = u.double()
    m = act(x @ d["w1"] + d["b1"], "silu") @ d["w2"] + d["b2"]
    m = m + experts(x, d["wi"], d["wo"], chosen, p, None, False)[0]
    n = m / (m.square().mean(1, keepdim=True) + eps).sqrt() * (d["post"] + offset)
    want = r.double() + branch * n
    _near("r", r1, want)
    _near("u", u1, want / (want.square().mean(1, keepdim=True) + eps).sqrt() * (d["pre"] + offset))
