"""Expert selection where fp32 cannot tell who is in: the ids are still those
of 64-bit arithmetic."""
import numpy as np
import pytest

from tests.gpu_common import need_gpu
from tests.test_gpu_route_topk import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,K,groups,top_groups", [
    (300, 1024, 4, 8, 4),       # a token a warp
    (300, 960, 3, 3, 2),        # ... and groups of no power of two
    (5003, 512, 9, 8, 4),       # sixteen lanes a token
    (5003, 256, 4, 8, 4),       # eight
])
@pytest.mark.parametrize("size", [0.5, 6.0, 300.0])
def test_groups_under_biases_of_opposite_sign(gate, T, E, K, groups, top_groups, size):
    """A group's two best have biases +size and -size: their sum is small, and
    what the sums with the biases lose to rounding is not."""
    need_gpu()
    rng = np.random.default_rng(E + T)
    # logits so near that the groups' sums lie within those roundings
    near = size * 2.0 ** -24 * (E if gate == "softmax" else 4) * 8
    l = (0.3 + near * rng.standard_normal((T, E))).astype(np.float32)
    b = np.full(E, -size, dtype=np.float32)
    b[rng.integers(0, E // groups, groups) + np.arange(groups) * (E // groups)] = size
    _check(l, b, K, gate, groups, top_groups, 2, True, 1.0)


@pytest.mark.parametrize("T", [300, 5003])
def test_groups_under_the_lowest_bias(T):
    """Experts switched off by the lowest finite bias stay ahead of masked
    ones, and their group (whose sum is past the lowest number) ahead of a
    masked group."""
    need_gpu()
    rng = np.random.default_rng(T)
    E, low = 64, np.finfo(np.float32).min
    b = (0.1 * rng.standard_normal(E)).astype(np.float32)
    b[8:16] = low                            # group 1: all off
    b[17:24] = low                           # group 2: one left
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[:, :8] = -np.inf                       # group 0: masked
    l[:, 27:] = -np.inf                      # ... and all but three of the rest
    for top_groups in (2, 3, 4):
        _check(l, b, 8, "sigmoid", 8, top_groups, 2, True, 1.0)


def _border_tokens(gate, T, E, K, crowd, rng):
    """Tokens whose K-th and (K+1)-th experts have small scores, no bias and
    values that fp32 tells apart, while an expert with a large score and a bias
    that almost cancels it (so with a far larger error) lies about there too.
    crowd: how many more lie a little below."""
    n = K + 1 + crowd                    # experts with small scores: ids 2 ..
    b = np.zeros(E, dtype=np.float32)
    b[0] = -0.9
    # just above a value that the large score, a multiple of 2^-24, can give
    mid = np.round((1e-5 + 0.9) * 2 ** 24) / 2 ** 24 + float(b[0]) + 5e-9
    gap = 1e-9 if gate == "softmax" else 2e-10
    t = np.full((T, E), 1e-8)
    t[:, 2:2 + K - 1] = 1e-4 * (1 + np.arange(K - 1))
    t[:, 1 + K], t[:, 2 + K] = mid + gap / 2, mid - gap / 2
    t[:, 3 + K:2 + n] = mid - 1e-6 - 1e-9 * np.arange(crowd)
    if gate == "softmax":
        b[1] = -1.0                      # takes what the others leave of the sum
    large = mid - float(b[0]) + rng.uniform(-6e-8, 6e-8, T)
    if gate == "sigmoid":
        l = np.log(t) - np.log1p(-t)
        l[:, 0] = np.log(large / (1 - large))
    else:
        t[:, 0] = large
        t[:, 1] = 1 - large - t[:, 2:].sum(1)
        l = np.log(t)
    # the small ones in any places
    order = np.concatenate([[0, 1], 2 + rng.permutation(E - 2)])
    return np.ascontiguousarray(l[:, order]).astype(np.float32), b


@pytest.mark.parametrize("gate", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,K,crowd", [
    (1500, 64, 3, 0),           # a token a warp, candidates one a lane
    (1500, 128, 4, 60),         # ... more candidates than lanes
    (1500, 512, 20, 60),
    (5003, 64, 3, 0),           # eight lanes a token
    (5003, 512, 12, 0),         # sixteen
    (5003, 256, 6, 60),         # ... left to the whole warp
])
def test_an_expert_left_out_further_down(gate, T, E, K, crowd):
    need_gpu()
    l, b = _border_tokens(gate, T, E, K, crowd, np.random.default_rng(E + K))
    _check(l, b, K, gate, 1, 1, 1, False, 1.0)


def test_many_equal_experts():
    """All scores equal, and all but one: ties by id, whatever lies near."""
    need_gpu()
    for T in (300, 5003):
        l = np.zeros((T, 128), dtype=np.float32)
        b = np.zeros(128, dtype=np.float32)
        _check(l, b, 8, "sigmoid", 1, 1, 1, True, 1.0)
        l[::2, 100] = np.float32(2.0 ** -23)
        l[1::3, 3] = np.float32(-2.0 ** -23)
        _check(l, b, 8, "sigmoid", 1, 1, 1, True, 1.0)
        _check(l, b, 8, "softmax", 1, 1, 1, True, 1.0)


@pytest.mark.parametrize("gate", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [300, 5003])
def test_scores_that_fp32_flushes(gate, T):
    """A score just below 2^-126 beside one just above, under biases as small."""
    need_gpu()
    rng = np.random.default_rng(T)
    l = np.full((T, 16), -120.0, dtype=np.float32)
    b = np.zeros(16, dtype=np.float32)
    l[:, 2] = rng.uniform(-87.6, -87.4, T)
    l[:, 7] = rng.uniform(-87.2, -87.1, T)
    b[2] = 8e-39
    if gate == "softmax":
        l[:, 5], b[5] = 0.0, -3.0
    _check(l, b, 1, gate, 1, 1, 1, False, 1e30)
