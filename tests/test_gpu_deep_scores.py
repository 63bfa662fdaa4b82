"""Sigmoid routing weights where the chosen scores are smaller than fp32 holds,
of the block's routing and of the expert layer for a few tokens: they are
shares, which do not depend on that."""
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import U32, assert_within
from tests.deep_scores import deep_logits, sigmoid_shares

pytestmark = pytest.mark.gpu


def _check(l, ids, w, K):
    order = torch.argsort(-l.double(), dim=1, stable=True)[:, :K]
    assert torch.equal(ids.long(), order)
    want = sigmoid_shares(torch.take_along_dim(l, order, dim=1))
    # the exponential, its rounded argument (differences of at most ten), the
    # quotient, K terms of the sum, the division; a score that is a subnormal
    # number beside ordinary ones is off by two of their steps, and the sum it
    # is divided by is a quarter at least where one score is about 0
    assert_within("w", w, want, (40 + K) * U32 * want + 8 * 2.0 ** -149)


@pytest.mark.parametrize("T,E,K", [(30, 40, 6), (700, 64, 8), (6000, 130, 3)])
def test_the_blocks_routing(T, E, K):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    l = deep_logits(T, E, T).cuda()
    d = B.dims(T, 64, E, K, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.empty(T, K, **i32), torch.empty(T, K, device="cuda")
    ws = torch.zeros(B.moe_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    B.moe_route_histogram(l, None, B.SCORE_SIGMOID_NORM, ids, w, torch.empty(E, **i32), torch.empty(E + 1, **i32),
                          torch.empty(T, K, **i32), torch.empty(T * K, **i32), torch.zeros(1, **i32), ws, d)
    torch.cuda.synchronize()
    _check(l, ids, w, K)


@pytest.mark.parametrize("T,E,K", [(8, 40, 6), (64, 70, 8)])   # selected by every block, and exchanged
def test_the_layer_for_a_few_tokens(T, E, K):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    from mixture_experts_ffn_histogram_gb300.layer import MoEDecode
    D = F = 64
    g = torch.Generator().manual_seed(T)
    bf = torch.bfloat16
    x, wi, wo = (torch.randn(*s, generator=g).to(bf).cuda() for s in ((T, D), (E, D, 2 * F), (E, F, D)))
    l = deep_logits(T, E, T).cuda()
    op = MoEDecode(T, D, E, K, F, B.SCORE_SIGMOID_NORM)
    out = op.forward(x, wi, wo, logits=l)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0 and bool(torch.isfinite(out).all())
    _check(l, op.ids, op.w, K)
