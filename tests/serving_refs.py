"""Plain 64-bit implementations of the operators that serve and wrap the
expert block, and the error bounds their GPU results are held to (made up as
in ``layer_refs``: half a step of the output's type, plus counted rounded
operations times the magnitudes that enter)."""
import torch

from tests.layer_refs import ACT_ERR, MAX_SLOPE, U32, half_step, sum_error


# ------------------------------------------------------- expert layer, few tokens
def select(logits, bias, K, mode):
    """(ids, w) of the block's routing: scores are fp32 sums, the lower expert
    first among equal ones; w in 64 bits."""
    s = (logits if bias is None else logits + bias).double()
    ids = torch.argsort(-s, dim=1, stable=True)[:, :K]
    best = torch.take_along_dim(s, ids, dim=1)
    p = torch.exp(best - best[:, :1]) if mode == "softmax" else torch.sigmoid(best)
    return ids.int(), p / p.sum(1, keepdim=True)


def experts(x, wi, wo, ids, w, res, own_weights):
    """(out, its bound's arithmetic part).  own_weights: the routing weights
    were computed by the kernel too, in fp32."""
    T, D = x.shape
    E, F = wi.shape[0], wo.shape[1]
    out = torch.zeros(T, D, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    e1, e2 = sum_error(D, False), sum_error(F, False)
    u = half_step(x.dtype)
    sub = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps  # h below the normal numbers
    # a score's exponential (its argument's rounding and the function's 2 ulp),
    # the K-term sum and the division, and the given weight's product
    ew = ((w.shape[1] + 12) if own_weights else 0) * U32
    for e in sorted(set(ids.flatten().tolist())):
        if not 0 <= e < E:
            continue
        t, k = torch.nonzero(ids == e, as_tuple=True)
        a, b = x[t].double(), wi[e].double()
        z, za = a @ b, a.abs() @ b.abs()
        g, up = z[:, :F], z[:, F:]
        silu = g * torch.sigmoid(g)
        h = silu * up
        dh = (MAX_SLOPE * e1 * za[:, :F] * up.abs() + silu.abs() * e1 * za[:, F:]
              + ACT_ERR * (1 + g.abs()) * h.abs() + u * h.abs() + sub)
        c = wo[e].double()
        y = h @ c
        ey = dh @ c.abs() + e2 * (h.abs() @ c.abs())
        wk = w[t, k].double()[:, None]
        out.index_add_(0, t, wk * y)
        err.index_add_(0, t, wk.abs() * (ey * (1 + 2.0 ** -6) + (ew + w.shape[1] * U32) * y.abs()))
    if res is not None:
        out = out + res.double()
        err = err + 2 * U32 * out.abs()
    return out, err
