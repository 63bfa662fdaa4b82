"""Plain 64-bit implementations of the operators around the block, and the
error bounds their GPU results are held to.

Every bound is  half a step of the output's type, relative to the value
(``torch.finfo(t).eps / 2``), plus the arithmetic's own error: a count of
rounded fp32 operations (2^-24 each) times the magnitudes that enter, which
the reference computes next to the value.
"""
import math

import numpy as np
import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the type's subnormals: the absolute part of a rounding."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def assert_within(name, got, want, arith):
    """|got - want| <= half a step of got's type + arith (a tensor or number)."""
    assert got.shape == want.shape, f"{name}: shape {tuple(got.shape)} vs {tuple(want.shape)}"
    u = half_step(got.dtype)
    g = got.detach().double()
    lim = u * want.abs() * (1 + 2.0 ** -8) + tiny(got.dtype) + arith
    bad = ~((g - want).abs() <= lim)
    if bad.any():
        i = bad.flatten().nonzero()[:5, 0]
        raise AssertionError(
            f"{name}: {int(bad.sum())} of {bad.numel()} outside their bound; at flat {i.tolist()}: "
            f"got {g.flatten()[i].tolist()} want {want.flatten()[i].tolist()} "
            f"bound {lim.expand_as(want).flatten()[i].tolist()}")


# ------------------------------------------------------------------ layer norm
def norm_fwd(r, gamma, beta, eps):
    """(y, mean, rstd, the bound's magnitudes for y) in 64 bits."""
    r, g, b = r.double(), gamma.double(), beta.double()
    mean = r.mean(1, keepdim=True)
    rstd = 1 / ((r - mean).square().mean(1, keepdim=True) + eps).sqrt()
    y = (r - mean) * rstd * g + b
    mag = g.abs() * rstd * (r.abs() + r.abs().mean(1, keepdim=True)) + b.abs()
    return y, mean[:, 0], rstd[:, 0], mag


def norm_bwd(dy, r, gamma, mean, rstd, dres):
    """(dx, dgamma, dbeta) and the bounds' magnitudes of each."""
    dy, r, g = dy.double(), r.double(), gamma.double()
    m, rs = mean.double()[:, None], rstd.double()[:, None]
    xh, xm = (r - m) * rs, (r.abs() + m.abs()) * rs
    a = dy * g
    dx = rs * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    mag = rs * (a.abs() + a.abs().mean(1, keepdim=True) + xm * (a.abs() * xm).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        mag = mag + dres.double().abs()
    return ((dx, (dy * xh).sum(0), dy.sum(0)),
            (mag, (dy.abs() * xm).sum(0), dy.abs().sum(0)))


# --------------------------------------------------------------------- routing
def scores(l, gate):
    """Scores of fp64 logits; masked (-inf or NaN) experts score 0."""
    l = np.where(np.isnan(l), -np.inf, l)
    dead = np.isneginf(l)
    with np.errstate(over="ignore", invalid="ignore"):
        if gate == "sigmoid":
            return np.where(dead, 0.0, 1 / (1 + np.exp(-l)))
        m = l.max(1, keepdims=True)
        e = np.where(dead, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
        tot = e.sum(1, keepdims=True)
        return np.where(tot > 0, e / np.where(tot > 0, tot, 1.0), 0.0)


def topk(logits, bias, K, gate, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """(ids, w) by their definition, one token at a time."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    T, E = l.shape
    s = scores(l, gate)
    dead = np.isneginf(l)
    sel = l if bias is None else np.where(dead, -np.inf, s + np.asarray(bias, dtype=np.float64))
    by = np.where(dead, -np.inf, s) if bias is None and group_top == 2 else sel
    ids = np.zeros((T, K), dtype=np.int32)
    gs = E // groups
    for t in range(T):
        cand = np.arange(E)
        if groups > 1:
            score = []
            for g in range(groups):
                v = np.sort(by[t, g * gs:(g + 1) * gs])[::-1][:group_top]
                alive = v[v > -np.inf]
                score.append(alive.sum() if alive.size else -np.inf)
            best = sorted(range(groups), key=lambda g: (-score[g], g))[:top_groups]
            cand = np.concatenate([np.arange(g * gs, (g + 1) * gs) for g in sorted(best)])
        ids[t] = sorted(cand, key=lambda e: (-sel[t, e], e))[:K]
    w = np.take_along_axis(s, ids.astype(np.int64), axis=1)
    if renorm:
        tot = w.sum(1, keepdims=True)
        w = np.where(tot > 0, w / np.where(tot > 0, tot, 1.0), 0.0)
    return ids, w * scale


def topk_weights(l, ids, gate, renorm, scale):
    """The weights as a differentiable function of fp64 torch logits."""
    s = torch.sigmoid(l) if gate == "sigmoid" else torch.softmax(l, dim=1)
    w = s.gather(1, ids.long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return w * scale


# ---------------------------------------------------------------------- linear
def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    z = z.detach().clone().requires_grad_(True)
    (g,) = torch.autograd.grad(act(z, name).sum() + 0 * z.sum(), z)
    if name == "relu":
        g = (z > 0).to(g.dtype)
    return g.detach()


# An activation's own error: of its value, 2^-20 (1 + |z|) covers the hardware
# exponential (2 + 1.17 |z| ulp) and the 1.5e-7 of the erfc approximation; of
# its slope the same with z^2 (the derivative multiplies sigmoid (1 - sigmoid) by z).
ACT_ERR = 2.0 ** -20
# Largest slope of the activations (gelu: 1.129, gelu_tanh: 1.130, silu: 1.100).
MAX_SLOPE = 1.13


def sum_error(K, fp32):
    """Error of a K-term product sum, relative to the sum of magnitudes: the
    tensor core adds 16 products at a time to an fp32 accumulator, truncating
    (2^-23 each); an fp32 result restarts the chain every 512 products and
    adds the pieces in fp32; a split of the reduction only shortens chains."""
    steps = min(K, 512) / 16 + K / 512 if fp32 else K / 16
    return (steps + 16) * 2.0 ** -23
