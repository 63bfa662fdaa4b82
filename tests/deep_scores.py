"""Sigmoid scores that are smaller than fp32 holds, and their shares."""
import torch


def deep_logits(T, E, seed):
    """fp32 logits of tokens whose best lie around 0, -50, -90, -100, -200 and
    -500, some of them masked in part; of tokens with a few experts far above
    the others; of tokens whose experts all lie at the type's lowest value."""
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g)
    for i, off in enumerate((0, 50, 90, 100, 200, 500)):
        l[i::8] -= off
    l[6::8, 2:] -= 95
    l[7::8] = torch.finfo(torch.float32).min
    l[11::12, ::2] = float("-inf")
    return l


def sigmoid_shares(scores):
    """Shares of the sigmoids of each row's scores, in 64 bits, by their logarithms."""
    return torch.softmax(torch.nn.functional.logsigmoid(scores.double()), dim=1)
