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


# ----------------------------------------------------------- norms around a block
def block_norm(res, y, post, pre, gate, token_gate, scale, offset, eps, r=None):
    """dict of r, u, rstd_y, rstd_r in 64 bits (u from the given stored r), and
    the bounds' magnitudes of r and u."""
    out, f = {}, res.double()
    D = f.shape[1]
    out["r"], out["r_mag"] = f, f.abs()
    if y is not None:
        n = y.double()
        if post is not None:
            out["rstd_y"] = 1 / (n.square().mean(1) + eps).sqrt()
            n = n * out["rstd_y"][:, None] * (post.double() + offset)
        c = scale * torch.ones(D, dtype=torch.float64, device=f.device) if gate is None else scale * gate.double()
        branch = n * c
        if token_gate is not None:
            branch = branch * token_gate.double()[:, None]
        out["r"], out["r_mag"] = f + branch, f.abs() + branch.abs()
        if post is not None and offset:
            out["r_mag"] = out["r_mag"] + branch.abs() * ((post.double().abs() + abs(offset))
                                                          / (post.double() + offset).abs().clamp(min=1e-30))
    if pre is not None:
        s = out["r"] if r is None else r.double()
        out["rstd_r"] = 1 / (s.square().mean(1) + eps).sqrt()
        out["u"] = s * out["rstd_r"][:, None] * (pre.double() + offset)
        out["u_mag"] = s.abs() * out["rstd_r"][:, None] * (pre.double().abs() + abs(offset))
    return out


def block_norm_bwd(du, dr, r, y, post, pre, gate, token_gate, rstd_y, rstd_r, scale, offset):
    """dict of name -> (gradient, magnitude of what enters it), in 64 bits from
    the stored rows and statistics."""
    shape = (dr if dr is not None else du).shape
    n, D = shape
    dev = (dr if dr is not None else du).device
    zero, one = torch.zeros(shape, dtype=torch.float64, device=dev), torch.ones(D, dtype=torch.float64, device=dev)
    d, dm, out = zero, zero, {}
    if dr is not None:
        d, dm = dr.double(), dr.double().abs()
    if pre is not None:
        rs, q, qm = rstd_r.double()[:, None], pre.double() + offset, pre.double().abs() + abs(offset)
        rh, u = r.double() * rs, du.double()
        a, am = u * q, u.abs() * qm
        m, mm = (a * rh).mean(1, keepdim=True), (am * rh.abs()).mean(1, keepdim=True)
        d, dm = d + rs * (a - m * rh), dm + rs * (am + mm * rh.abs())
        out["dpre"] = ((u * rh).sum(0), (u * rh).abs().sum(0))
    out["dres"] = (d, dm)
    if y is None:
        return out
    yh, ry = y.double(), 1.0
    if post is not None:
        ry = rstd_y.double()[:, None]
        yh = yh * ry
    p = one if post is None else post.double() + offset
    pm = one if post is None else post.double().abs() + abs(offset)
    g0 = one if gate is None else gate.double()
    g, gm = scale * g0 * p, abs(scale) * g0.abs() * pm
    t = 1.0 if token_gate is None else token_gate.double()[:, None]
    ta = abs(t) if token_gate is None else t.abs()
    b, bm = (g * yh * d).sum(1, keepdim=True), (gm * yh.abs() * dm).sum(1, keepdim=True)
    dy, dym = t * g * d, ta * gm * dm
    if post is not None:
        dy, dym = ry * (dy - t * b * yh / D), ry * (dym + ta * bm * yh.abs() / D)
    out["dy"] = (dy, dym)
    e, em = (t * d * yh).sum(0), (ta * dm * yh.abs()).sum(0)
    if post is not None:
        out["dpost"] = (scale * g0 * e, abs(scale) * g0.abs() * em)
    if gate is not None:
        out["dgate"] = (scale * p * e, abs(scale) * pm * em)
    if token_gate is not None:
        out["dtoken_gate"] = (b[:, 0], bm[:, 0])
    return out


# ------------------------------------------------------------- low-rank adapters
def adapters(x, a, b, scale, ids, res):
    """(y, its bound's arithmetic part)."""
    T, K = x.shape
    S, r = a.shape[:2]
    y = torch.zeros(T, b.shape[1], dtype=torch.float64, device=x.device)
    err = torch.zeros_like(y)
    u = half_step(x.dtype)
    sub = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps  # v below the normal numbers
    for s in range(S):
        t = torch.nonzero(ids == s)[:, 0]
        c = float(scale[s])
        p, q, w = x[t].double(), a[s].double(), b[s].double()
        v, vm = c * (p @ q.t()), abs(c) * (p.abs() @ q.abs().t())
        # the sum over K (cut in up to 32 parts), the scale, the rounding
        dv = (sum_error(K, False) + 34 * U32) * vm + u * v.abs() * (1 + 2.0 ** -6) + sub
        y[t] = v @ w.t()
        err[t] = dv @ w.abs().t() + (r / 16 + 18) * 2 * U32 * (v.abs() @ w.abs().t())
    if res is not None:
        y = y + res.double()
        err = err + 2 * U32 * y.abs()
    return y, err
