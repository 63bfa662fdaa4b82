"""Sigmoid routing weights of the oracle where the chosen scores are smaller
than fp32 holds: they are shares, which do not depend on that."""
import numpy as np
import torch

import oracle
from tests.deep_scores import deep_logits, sigmoid_shares


def test_shares_of_deep_scores():
    oracle.build()
    T, E, K = 120, 40, 6
    l = deep_logits(T, E, 1)
    ids, w = oracle.route(l.numpy(), None, oracle.SIGMOID_NORM, T, E, K)
    want = sigmoid_shares(torch.take_along_dim(l, torch.from_numpy(ids).long(), dim=1))
    # as on the device (tests/test_gpu_deep_scores.py)
    off = np.abs(w - want.numpy())
    assert np.all(off <= (40 + K) * 2.0 ** -24 * want.numpy() + 8 * 2.0 ** -149)
    assert np.all(np.abs(w.astype(np.float64).sum(1) - 1) <= (K + 1) * 2.0 ** -24)
