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
