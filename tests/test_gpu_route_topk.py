"""Expert selection with balance bias and groups against its definition in 64
bits (ids exactly), near ties, masked experts, and the weights' backward."""
import numpy as np
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import U32, assert_within, topk, topk_weights

pytestmark = pytest.mark.gpu

# T, E, K, gate, bias, groups, top_groups, group_top, renorm, scale
CASES = [
    (1, 1, 1, "sigmoid", True, 1, 1, 1, True, 1.0),
    (5, 8, 2, "softmax", False, 1, 1, 1, True, 1.0),
    (64, 8, 8, "sigmoid", True, 4, 4, 2, True, 2.5),
    (300, 128, 8, "softmax", False, 1, 1, 1, False, 1.0),
    (300, 128, 8, "softmax", True, 1, 1, 1, False, 1.0),
    (300, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (300, 256, 8, "sigmoid", False, 8, 4, 2, True, 2.5),
    (300, 256, 6, "softmax", False, 8, 3, 1, False, 16.0),
    (200, 160, 6, "softmax", True, 8, 3, 1, False, 16.0),   # groups that split a lane's experts
    (200, 48, 5, "sigmoid", True, 8, 3, 2, False, 1.0),
    (200, 50, 7, "sigmoid", True, 2, 1, 2, True, 1.0),
    (200, 33, 32, "sigmoid", True, 1, 1, 1, True, 1.0),
    (200, 33, 32, "softmax", False, 3, 3, 2, True, 1.0),
    (60, 384, 16, "sigmoid", True, 32, 9, 2, True, 1.0),
    (60, 1024, 32, "sigmoid", True, 16, 4, 2, True, 1.0),
    (60, 1000, 9, "softmax", True, 1, 1, 1, True, 1.0),
    (20, 32, 4, "sigmoid", True, 32, 7, 2, True, 1.0),        # groups of one expert
    (40, 1022, 8, "sigmoid", True, 2, 1, 2, True, 1.0),       # a group's size no power of two divides
    (40, 960, 8, "softmax", True, 3, 2, 2, False, 1.0),
    (40, 693, 8, "sigmoid", False, 7, 3, 2, True, 1.0),
]


def _run(l, b, K, gate, groups, top_groups, group_top, renorm, scale):
    from mixture_experts_ffn_histogram_gb300.layer import TopKRouter
    T, E = l.shape
    op = TopKRouter(T, E, K, gate, groups, top_groups, group_top, renorm, scale, train=True)
    ids, w = op.forward(torch.from_numpy(l).cuda(),
                        None if b is None else torch.from_numpy(b).cuda())
    torch.cuda.synchronize()
    return op, ids.cpu().numpy(), w


def _check(l, b, K, gate, groups, top_groups, group_top, renorm, scale):
    op, ids, w = _run(l, b, K, gate, groups, top_groups, group_top, renorm, scale)
    want, ww = topk(l, b, K, gate, groups, top_groups, group_top, renorm, scale)
    assert np.array_equal(ids, want), np.argwhere(ids != want)[:5]
    # sigmoid: exp, add, divide (8 roundings) and K terms of the sum; softmax
    # over all experts: the hardware exponential's (2 + 1.17 |l - m|) ulp in
    # the sum, which stays below 40 for logits a few units apart
    ww = torch.from_numpy(ww).cuda()
    assert_within("w", w, ww, (40 + K) * U32 * ww)
    return op


@pytest.mark.parametrize("T,E,K,gate,bias,groups,top_groups,group_top,renorm,scale", CASES)
def test_selection_and_weights(T, E, K, gate, bias, groups, top_groups, group_top, renorm, scale):
    need_gpu()
    rng = np.random.default_rng(T * 1000 + E)
    l = rng.standard_normal((T, E)).astype(np.float32)
    b = (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None
    _check(l, b, K, gate, groups, top_groups, group_top, renorm, scale)


# enough tokens that they go four to a warp (and a last warp that is not full)
MANY = [
    (5003, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (5001, 256, 8, "sigmoid", False, 8, 4, 2, False, 1.0),
    (5002, 256, 8, "softmax", True, 1, 1, 1, False, 1.0),
    (5003, 128, 8, "softmax", False, 1, 1, 1, True, 1.0),
    (5003, 160, 6, "softmax", True, 8, 3, 1, False, 16.0),
    (5003, 48, 5, "sigmoid", True, 3, 2, 2, True, 1.0),
    (5003, 50, 4, "sigmoid", True, 2, 1, 2, True, 1.0),
    (5003, 35, 2, "softmax", True, 7, 1, 2, False, 1.0),
    (5003, 8, 8, "sigmoid", True, 1, 1, 1, True, 1.0),
    (5003, 64, 1, "sigmoid", True, 4, 2, 1, True, 1.0),
    (5003, 250, 7, "softmax", True, 5, 4, 2, True, 1.0),
    (5003, 256, 16, "sigmoid", True, 8, 4, 2, True, 1.0),
    (5003, 96, 11, "softmax", True, 12, 5, 2, False, 1.0),
    (5003, 130, 13, "softmax", False, 1, 1, 1, False, 1.0),
    (5003, 512, 8, "sigmoid", True, 8, 4, 2, True, 1.0),
    (5003, 512, 16, "softmax", True, 8, 3, 2, False, 1.0),
    (5003, 384, 6, "sigmoid", True, 1, 1, 1, True, 1.0),
    (5003, 255, 12, "sigmoid", True, 3, 2, 2, True, 1.0),
    (5003, 96, 16, "softmax", False, 8, 2, 2, False, 1.0),   # all of the groups' experts are candidates
    (5003, 160, 16, "sigmoid", True, 8, 2, 1, True, 1.0),
    (5003, 16, 5, "softmax", True, 1, 1, 1, True, 1.0),
    (5003, 32, 4, "sigmoid", True, 2, 1, 1, True, 1.0),
    (5003, 20, 16, "sigmoid", True, 1, 1, 1, False, 1.0),
    (1003, 20, 7, "sigmoid", True, 1, 1, 1, False, 1.0),
    (1003, 64, 9, "softmax", True, 8, 3, 2, True, 1.0),
]


@pytest.mark.parametrize("T,E,K,gate,bias,groups,top_groups,group_top,renorm,scale", MANY)
def test_many_tokens(T, E, K, gate, bias, groups, top_groups, group_top, renorm, scale):
    """As above; some tokens with masked experts, few or none left, with equal
    logits, and with logits a few units in the last place apart."""
    need_gpu()
    rng = np.random.default_rng(T + E)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[:400][rng.random((400, E)) < 0.6] = -np.inf
    l[400] = -np.inf
    l[401] = np.nan
    l[402:440] = 0.25
    l[440:800] = np.float32(0.7) + rng.integers(-4, 5, (360, E)).astype(np.float32) * np.float32(2.0 ** -24)
    l[800:900] = np.round(l[800:900], 1)
    l[900, E // 2] = np.inf
    b = (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None
    if bias:
        b[: E // 2] = (rng.integers(-3, 4, E // 2) * 2.0 ** -26).astype(np.float32)
    _check(l, b, K, gate, groups, top_groups, group_top, renorm, scale)


@pytest.mark.parametrize("gate", ["sigmoid", "softmax"])
def test_scores_next_to_one_another(gate):
    """Logits a few units in the last place apart, under biases that differ as
    little: fp32 scores tie or swap, the ids are still those of 64 bits."""
    need_gpu()
    rng = np.random.default_rng(5)
    T, E = 400, 64
    l = np.float32(0.7) + rng.integers(-4, 5, (T, E)).astype(np.float32) * np.float32(2.0 ** -24)
    b = (rng.integers(-3, 4, E) * 2.0 ** -26).astype(np.float32)
    _check(l.astype(np.float32), b, 8, gate, 4, 2, 2, True, 1.0)


def test_exact_ties_go_to_the_lowest():
    need_gpu()
    l = np.zeros((9, 128), dtype=np.float32)
    for b in (None, np.zeros(128, dtype=np.float32)):
        _, ids, _ = _run(l, b, 8, "sigmoid", 8, 4, 2, True, 1.0)
        assert (ids == np.arange(8)).all()
    l[:, 1::2] = -0.0
    _, ids, _ = _run(l, None, 8, "softmax", 1, 1, 1, True, 1.0)
    assert (ids == np.arange(8)).all()


@pytest.mark.parametrize("gate", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_masked_experts(gate, bias, groups, top_groups, group_top):
    """Experts masked with -inf or NaN; a row with fewer experts left than K,
    with one, with none; saturated and infinite logits."""
    need_gpu()
    rng = np.random.default_rng(11)
    T, E, K = 60, 64, 6
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[rng.random((T, E)) < 0.5] = -np.inf
    l[3, ::3] = np.nan
    l[4] = -np.inf
    l[5] = -np.inf
    l[5, 41] = 0.5
    l[6] = -np.inf
    l[6, 10:13] = [1.0, 2.0, 2.0]
    l[7] *= 30
    l[8, 7] = np.inf
    l[9] = np.nan
    b = (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None
    _check(l, b, K, gate, groups, top_groups, group_top, True, 1.0)


@pytest.mark.parametrize("gate", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (70, 128, 8), (40, 50, 7), (30, 300, 32)])
def test_backward(gate, renorm, T, E, K):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import TopKRouter
    g = torch.Generator().manual_seed(E)
    l = torch.randn(T, E, generator=g)
    dw = torch.randn(T, K, generator=g).cuda()
    op = TopKRouter(T, E, K, gate, renorm=renorm, scale=2.0, group_top=1, train=True)
    ids, _ = op.forward(l.cuda())
    got = op.backward(dw, l.cuda())
    l64 = l.double().cuda().requires_grad_(True)
    w = topk_weights(l64, ids, gate, renorm, 2.0)
    (want,) = torch.autograd.grad(w, l64, dw.double())
    # 2 sum |dw| bounds every term that cancels; sums of K and E terms
    s = torch.sigmoid(l64) if gate == "sigmoid" else torch.softmax(l64, 1)
    q = s.detach().gather(1, ids.long())
    total = q.sum(1, keepdim=True) if renorm else 1.0
    mag = 4.0 * dw.double().abs().sum(1, keepdim=True) * torch.ones_like(want) / total
    mag = mag * (s.detach() if gate == "softmax" else 1.0) + 4.0 * dw.double().abs().sum(1, keepdim=True) * U32
    assert_within("dlogits", got, want, (48 + K) * U32 * mag)
    # against differences of the 64-bit weights (the selection held fixed)
    if T * E <= 2000:
        h, l0 = 1e-5, l.double().cuda()
        for e in range(0, E, max(1, E // 5)):
            step = torch.zeros(T, E, dtype=torch.float64, device="cuda")
            step[:, e] = h
            d = (topk_weights(l0 + step, ids, gate, renorm, 2.0)
                 - topk_weights(l0 - step, ids, gate, renorm, 2.0)) / (2 * h)
            assert ((d * dw.double()).sum(1) - got[:, e].double()).abs().max() < 1e-5


def test_dropped_ids_carry_no_gradient():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import TopKRouter
    for gate, renorm in (("sigmoid", True), ("sigmoid", False), ("softmax", True)):
        op = TopKRouter(4, 16, 3, gate, renorm=renorm, group_top=1, train=True)
        l = torch.randn(4, 16, generator=torch.Generator().manual_seed(1)).cuda()
        dw = torch.ones(4, 3, device="cuda")
        ids = torch.tensor([[0, 1, 2], [-1, 5, 16], [-1, -7, 99], [3, 2, 1]],
                           dtype=torch.int32, device="cuda")
        got = op.backward(dw, l, ids=ids)
        assert not got[2].any()
        assert not got[1][[0, 1, 2, 3, 4, 6, 15]].any()
        if not renorm:
            s = torch.sigmoid(l[1, 5].double())
            assert abs(float(got[1, 5]) - float(s * (1 - s))) < 1e-6


def test_the_block_takes_the_selection():
    """ids and w of the router go through the block's histogram unchanged."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    from mixture_experts_ffn_histogram_gb300.block import MoEBlock
    from mixture_experts_ffn_histogram_gb300.layer import TopKRouter
    T, D, E, K, F = 96, 64, 16, 4, 64
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).cuda()
    l[5] = -float("inf")
    op = TopKRouter(T, E, K, "sigmoid", 4, 2, 2)
    ids, w = op.forward(l, torch.zeros(E, device="cuda"))
    blk = MoEBlock(T, D, E, K, F, B.SCORE_GIVEN, train=False)
    x = torch.randn(T, D, device="cuda").bfloat16()
    wi = (0.1 * torch.randn(E, D, 2 * F, device="cuda")).bfloat16()
    wo = (0.1 * torch.randn(E, F, D, device="cuda")).bfloat16()
    out = blk.forward(x, wi, wo, ids=ids, w=w)
    assert int(blk.status.item()) == 0
    assert torch.equal(blk.group_sizes.long(), torch.bincount(ids.flatten().long(), minlength=E))
    assert not out[5].any()


def test_empty_batch_and_graph():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import TopKRouter
    op = TopKRouter(500, 64, 4, "sigmoid", 8, 4, 2, train=True)
    l = torch.randn(500, 64, device="cuda")
    b = 0.05 * torch.randn(64, device="cuda")
    assert op.forward(l[:0], b)[0].shape == (0, 4)
    assert op.backward(torch.empty(0, 4, device="cuda"), l[:0]).shape == (0, 64)
    ids, w = op.forward(l, b)
    dl = op.backward(w, l).clone()
    ids, w = ids.clone(), w.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        i2, w2 = op.forward(l, b)
        d2 = op.backward(w2, l)
    i2.zero_(), w2.zero_(), d2.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(i2, ids) and torch.equal(w2, w) and torch.equal(d2, dl)
