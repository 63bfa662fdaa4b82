"""Routing weights and their gradient where the chosen scores are smaller than
fp32 holds: the shares of a token do not depend on that."""
import numpy as np
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import U32, assert_within, topk, topk_weights
from tests.test_gpu_route_topk import _run

pytestmark = pytest.mark.gpu

# one token a warp, eight lanes a token, sixteen
SIZES = [(301, 64, 6), (5003, 64, 6), (5003, 256, 12)]


def _deep(gate, T, E, rng):
    """Logits of tokens whose best lie below -50, -90, -100, -200 and -500; for
    the softmax, of tokens with one expert as far above all others (which its
    bias keeps out).  Some tokens are ordinary, some masked in part or whole."""
    l = rng.standard_normal((T, E)).astype(np.float32)
    for i, off in enumerate((50, 90, 100, 200, 500)):
        if gate == "sigmoid":
            l[i::7] -= off
        else:
            l[i::7, 3] += off
    l[10::11, ::2] = -np.inf
    l[7] = -np.inf
    b = np.zeros(E, dtype=np.float32)
    b[3] = -2.0
    return l, b


@pytest.mark.parametrize("gate", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_shares(gate, T, E, K):
    need_gpu()
    l, b = _deep(gate, T, E, np.random.default_rng(T + E))
    _, ids, w = _run(l, b, K, gate, 1, 1, 1, True, 2.0)
    want, ww = topk(l, b, K, gate, 1, 1, 1, True, 2.0)
    assert np.array_equal(ids, want)
    # as for ordinary tokens: the exponential, its rounded argument (differences
    # of at most ten), K terms of the sum, the division
    ww = torch.from_numpy(ww).cuda()
    assert_within("w", w, ww, (40 + K) * U32 * ww)
    assert bool((w.sum(1)[8:] > 1.9).all())


@pytest.mark.parametrize("T,E,K", SIZES)
def test_small_sigmoids(T, E, K):
    """Without renormalisation the weight is the score, a subnormal number too."""
    need_gpu()
    rng = np.random.default_rng(T)
    l = rng.uniform(-104, -86, (T, E)).astype(np.float32)
    _, ids, w = _run(l, None, K, "sigmoid", 1, 1, 1, False, 1.0)
    want, ww = topk(l, None, K, "sigmoid", 1, 1, 1, False, 1.0)
    assert np.array_equal(ids, want)
    # the exponential's two steps and one more, of the subnormals' spacing where
    # the number is one
    ww = torch.from_numpy(ww).cuda()
    assert_within("w", w, ww, 4 * (2 * U32 * ww + 2.0 ** -149))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,K", [(300, 64, 6), (40, 50, 1)])
def test_backward(renorm, T, E, K):
    """dl_k = q_k (g_k - sum g q) (1 - s_k) with renorm, g_k s_k (1 - s_k)
    without, from the chosen logits."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import TopKRouter
    l, b = _deep("sigmoid", T, E, np.random.default_rng(K))
    if not renorm:
        l = np.maximum(l, np.float32(-104))
    l = torch.from_numpy(l).cuda()
    l = torch.where(torch.isinf(l), torch.full_like(l, -70.0), l)
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).cuda()
    op = TopKRouter(T, E, K, "sigmoid", renorm=renorm, scale=2.0, group_top=1, train=True)
    ids, _ = op.forward(l, torch.from_numpy(b).cuda())
    got = op.backward(dw, l)
    l64 = l.double().requires_grad_(True)
    w = topk_weights(l64, ids, "sigmoid", renorm, 2.0)
    (want,) = torch.autograd.grad(w, l64, dw.double())
    g = 2.0 * dw.double().abs()
    s = torch.sigmoid(l64.detach()).gather(1, ids.long())
    mag = s * g
    if renorm:
        q = s / s.sum(1, keepdim=True)
        mag = q * (g + (g * q).sum(1, keepdim=True))
    lim = torch.zeros_like(want).scatter_(1, ids.long(), (48 + K) * U32 * mag + 4 * (1 + g) * 2.0 ** -149)
    assert_within("dlogits", got, want, lim)
