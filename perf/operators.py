"""Cases of the operators around the expert block: layer norm (with the residual
add in front of it), routing with a balance bias and expert groups, and the
linear layer with bias, activation and residual in its epilogue; forward and
backward.

Each operator is written here in its plain form (``own`` false: elementary
torch operations in 32 bits, the routing's scores in 64 because the selection
compares values next to one another) and called through the framework
(``own`` true).  ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # one token of a served request, the widest layer: latency
        dict(name="norm_one_token", op="norm", direction="fwd", rows=1, D=7168, dtype="bf16",
             weights="bf16", res=True, stats=False),
        # the long-sequence training batch: residual add, norm, statistics kept
        dict(name="norm_train_fwd", op="norm", direction="fwd", rows=32768, D=2816, dtype="bf16",
             weights="fp32", res=True, stats=True),
        # ... and its backward, with the residual stream's gradient added
        dict(name="norm_train_bwd", op="norm", direction="bwd", rows=32768, D=2816, dtype="bf16",
             weights="fp32", res=True, stats=True),
        # fp32 rows of an odd width (a ragged batch in a full-precision run)
        dict(name="norm_odd_bwd", op="norm", direction="bwd", rows=4099, D=1001, dtype="fp32",
             weights="fp32", res=False, stats=True),
        # a small decode batch through the group-limited router
        dict(name="route_decode", op="route", direction="fwd", T=16, E=256, K=8, score="sigmoid",
             bias=True, groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5),
        # the same router over a training batch
        dict(name="route_train_fwd", op="route", direction="fwd", T=32768, E=256, K=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2, renorm=True,
             scale=2.5),
        # backward of a softmax router whose weights are not renormalised (dense gradient)
        dict(name="route_softmax_bwd", op="route", direction="bwd", T=32768, E=128, K=8,
             score="softmax", bias=False, groups=1, top_groups=1, group_top=1, renorm=False,
             scale=1.0),
        # the shared expert's first product for a handful of decoded tokens
        dict(name="linear_decode", op="linear", direction="fwd", M=4, K=7168, N=2048,
             dtype="bf16", out="bf16", act="silu", bias=True, res=False, keep_z=False),
        # router logits in fp32, a ragged number of tokens
        dict(name="linear_logits", op="linear", direction="fwd", M=8191, K=7168, N=256,
             dtype="bf16", out="fp32", act="none", bias=False, res=False, keep_z=False),
        # the shared expert's first product in training: gelu, pre-activation kept
        dict(name="linear_gelu", op="linear", direction="fwd", M=4096, K=2048, N=768,
             dtype="fp16", out="fp16", act="gelu", bias=True, res=False, keep_z=True),
        # the shared expert's second product over the long-sequence batch, the routed
        # experts' output as its residual
        dict(name="linear_residual", op="linear", direction="fwd", M=32768, K=704, N=2816,
             dtype="bf16", out="bf16", act="none", bias=True, res=True, keep_z=False),
        # training backward of a wide first product: dx added to another branch's, dw, db
        dict(name="linear_bwd", op="linear", direction="bwd", M=8192, K=7168, N=2048,
             dtype="bf16", out="bf16", act="silu", bias=True, res=True, keep_z=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "route", "linear"))
    if op == "norm":
        direction = rng.choice(("fwd", "bwd"))
        rows, D = _log(rng, 1, 32768), _log(rng, 16, 8192)
        if rng.random() < 0.6:
            D = D // 16 * 16 + 8        # whole 16-byte vectors, odd in number
        dtype = rng.choice(("bf16", "fp16", "fp32"))
        rows = max(1, min(rows, 32768 * 2816 * 2 // (D * SIZE[dtype])))
        return dict(op=op, direction=direction, rows=rows, D=D, dtype=dtype,
                    weights=rng.choice(("fp32", dtype)), res=rng.random() < 0.5,
                    stats=direction == "bwd" or rng.random() < 0.5)
    if op == "route":
        E = rng.choice((8, 16, 32, 48, 64, 96, 128, 160, 256, 384, 512))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 4])
        top_groups = rng.randint(1, groups)
        K = rng.randint(1, min(16, top_groups * (E // groups)))
        T = min(_log(rng, 1, 32768), 32768 * 256 // E)
        return dict(op=op, direction=rng.choice(("fwd", "fwd", "bwd")), T=T, E=E, K=K,
                    score=rng.choice(("sigmoid", "softmax")), bias=rng.random() < 0.6,
                    groups=groups, top_groups=top_groups, group_top=rng.choice((1, 2)),
                    renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)))
    direction = rng.choice(("fwd", "fwd", "bwd"))
    M = _log(rng, 1, 32768)
    K, N = _width(rng), _width(rng)
    most = 8192 * 7168 * 2048 if direction == "bwd" else 32768 * 704 * 2816
    M = max(1, min(M, most // (K * N), 32768 * 6336 // (K + 2 * N)))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
    out = "fp32" if direction == "fwd" and N <= 512 and rng.random() < 0.3 else dtype
    return dict(op=op, direction=direction, M=M, K=K, N=N, dtype=dtype, out=out, act=act,
                bias=rng.random() < 0.6, res=rng.random() < 0.5,
                keep_z=act != "none" and (direction == "bwd" or rng.random() < 0.5))


def _width(rng):
    """A width of the linear layer: an odd multiple of 8 or of 64."""
    if rng.random() < 0.5:
        return 64 * (2 * _log(rng, 1, 56) - 1)
    return 8 * (2 * _log(rng, 4, 448) - 1)


# --------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "norm":
        n, D, dt = c["rows"], c["D"], DTYPES[c["dtype"]]
        # a residual stream: channels of different spread, some far wider, an offset of its own
        spread = torch.exp(0.5 * _randn(g, D))
        spread[:: max(1, D // 16)] *= 8
        x = (_randn(g, n, D) * spread + 0.3 * _randn(g, D)).to(dt)
        wt = DTYPES[c["weights"]]
        s["gamma"] = (1 + 0.2 * _randn(g, D)).to(wt)
        s["beta"] = (0.1 * _randn(g, D)).to(wt)
        if c["direction"] == "fwd":
            s["x"] = x
            s["res"] = _randn(g, n, D).to(dt) if c["res"] else None
        else:
            s["r"] = x
            s["dy"] = _randn(g, n, D).to(dt)
            s["dres"] = _randn(g, n, D).to(dt) if c["res"] else None
            f = x.float()
            s["mean"] = f.mean(1)
            s["rstd"] = torch.rsqrt((f - s["mean"][:, None]).square().mean(1) + EPS)
    elif c["op"] == "route":
        T, E, K = c["T"], c["E"], c["K"]
        s["logits"] = _randn(g, T, E)
        # a balance bias moves by small steps: small next to the scores' spread
        s["bias"] = 0.05 * _randn(g, E) if c["bias"] else None
        if c["direction"] == "bwd":
            s["ids"] = torch.sort(s["logits"], dim=1, descending=True,
                                  stable=True).indices[:, :K].to(torch.int32).contiguous()
            s["dw"] = _randn(g, T, K)
    else:
        M, K, N, dt = c["M"], c["K"], c["N"], DTYPES[c["dtype"]]
        s["x"] = _randn(g, M, K).to(dt)
        s["w"] = (_randn(g, K, N) / math.sqrt(K)).to(dt)
        s["bias"] = 0.5 * _randn(g, N) if c["bias"] else None
        if c["direction"] == "fwd":
            s["res"] = _randn(g, M, N).to(DTYPES[c["out"]]) if c["res"] else None
        else:
            z = s["x"] @ s["w"]
            s["z"] = (z + s["bias"].to(dt) if c["bias"] else z) if c["act"] != "none" else None
            s["dy"] = _randn(g, M, N).to(dt)
            s["dx_add"] = _randn(g, M, K).to(dt) if c["res"] else None
    if own:
        s["op"] = _handle(c)
    return s


def _handle(c):
    """The framework's operator with its output buffers and workspace, as a program keeps it."""
    from mixture_experts_ffn_histogram_gb300 import layer
    train = c["direction"] == "bwd"
    if c["op"] == "norm":
        return layer.LayerNorm(c["rows"], c["D"], dtype=DTYPES[c["dtype"]],
                               weight_dtype=DTYPES[c["weights"]], eps=EPS,
                               train=train or c["stats"])
    if c["op"] == "route":
        return layer.TopKRouter(c["T"], c["E"], c["K"], score=c["score"], groups=c["groups"],
                                top_groups=c["top_groups"], group_top=c["group_top"],
                                renorm=c["renorm"], scale=c["scale"], train=train)
    return layer.Linear(c["M"], c["K"], c["N"], dtype=DTYPES[c["dtype"]],
                        out_dtype=DTYPES[c["out"]], act=c["act"], train=train or c["keep_z"])


# ----------------------------------------------------------------- the passes
def run(state):
    c = state["case"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "linear": _own_linear}[c["op"]](state, c)
    return {"norm": _plain_norm, "route": _plain_route, "linear": _plain_linear}[c["op"]](state, c)


def _own_norm(s, c):
    op = s["op"]
    if c["direction"] == "fwd":
        y = op.forward(s["x"], s["gamma"], s["beta"], res=s["res"])
        out = [y]
        if c["res"]:
            out.append(op.r)
        if c["stats"]:
            out += [op.mean, op.rstd]
        return out
    dx = op.backward(s["dy"], s["r"], s["gamma"], mean=s["mean"], rstd=s["rstd"], dres=s["dres"])
    return [dx, op.dgamma, op.dbeta]


def _own_route(s, c):
    op = s["op"]
    if c["direction"] == "fwd":
        return list(op.forward(s["logits"], bias=s["bias"]))
    return [op.backward(s["dw"], s["logits"], ids=s["ids"])]


def _own_linear(s, c):
    op = s["op"]
    if c["direction"] == "fwd":
        y = op.forward(s["x"], s["w"], bias=s["bias"], res=s["res"])
        return [y, op.z] if c["keep_z"] else [y]
    dx = op.backward(s["dy"], s["x"], s["w"], z=s["z"], dx_add=s["dx_add"], need_db=c["bias"])
    return [dx, op.dw, op.db] if c["bias"] else [dx, op.dw]


def _plain_norm(s, c):
    dt, wt = DTYPES[c["dtype"]], DTYPES[c["weights"]]
    gamma, beta = s["gamma"].float(), s["beta"].float()
    if c["direction"] == "fwd":
        r = s["x"]
        if c["res"]:
            r = (r.float() + s["res"].float()).to(dt)
        f = r.float()
        mean = f.mean(1, keepdim=True)
        d = f - mean
        rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
        y = (d * rstd * gamma + beta).to(dt)
        out = [y]
        if c["res"]:
            out.append(r)
        if c["stats"]:
            out += [mean[:, 0], rstd[:, 0]]
        return out
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["r"].float() - s["mean"][:, None]) * rstd
    a = dy * gamma
    dx = rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    if c["res"]:
        dx = dx + s["dres"].float()
    return [dx.to(dt), (dy * xh).sum(0).to(wt), dy.sum(0).to(wt)]


def _plain_scores(logits, score):
    """Scores of the experts in the logits' type; the experts in their selection order's values."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _plain_route(s, c):
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    if c["direction"] == "fwd":
        # 64 bits: the selection compares scores that lie next to one another
        l64 = s["logits"].double()
        p = _plain_scores(l64, c["score"])
        sel = p + s["bias"].double() if c["bias"] else l64
        if G > 1:
            by = p if not c["bias"] and c["group_top"] == 2 else sel
            best = torch.sort(by.view(T, G, E // G), dim=2, descending=True).values
            of_group = best[:, :, : c["group_top"]].sum(2)
            order = torch.sort(of_group, dim=1, descending=True, stable=True).indices
            keep = torch.zeros(T, G, dtype=torch.bool, device=sel.device)
            keep.scatter_(1, order[:, : c["top_groups"]], True)
            keep = keep[:, :, None].expand(T, G, E // G).reshape(T, E)
            sel = torch.where(keep, sel, -math.inf)
        ids = torch.sort(sel, dim=1, descending=True, stable=True).indices[:, :K]
        w = p.gather(1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return [ids.to(torch.int32), (w * c["scale"]).float()]
    ids, dw = s["ids"].long(), s["dw"]
    p = _plain_scores(s["logits"], c["score"])
    sel = p.gather(1, ids)
    d = dw * c["scale"]
    if c["renorm"]:
        total = sel.sum(1, keepdim=True)
        d = (d - (d * sel).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_(1, ids, d)
    if c["score"] == "sigmoid":
        return [dp * p * (1 - p)]
    return [p * (dp - (dp * p).sum(1, keepdim=True))]


def _plain_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _plain_act_grad(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _plain_linear(s, c):
    dt = DTYPES[c["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    if c["direction"] == "fwd":
        z = x @ w
        if c["bias"]:
            z = z + s["bias"]
        y = _plain_act(z, c["act"])
        if c["res"]:
            y = y + s["res"].float()
        y = y.to(DTYPES[c["out"]])
        return [y, z.to(dt)] if c["keep_z"] else [y]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _plain_act_grad(s["z"].float(), c["act"])
    dx = dz @ w.t()
    if c["res"]:
        dx = dx + s["dx_add"].float()
    out = [dx.to(dt), (x.t() @ dz).to(dt)]
    return out + [dz.sum(0)] if c["bias"] else out


# ----------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "norm":
        n, s = c["rows"] * c["D"], SIZE[c["dtype"]]
        if c["direction"] == "fwd":
            b = n * s * (4 if c["res"] else 2) + (8 * c["rows"] if c["stats"] else 0)
            return {"bytes": b + 2 * c["D"] * SIZE[c["weights"]], "flops": 8 * n}
        b = n * s * (4 if c["res"] else 3) + 8 * c["rows"]
        return {"bytes": b + 3 * c["D"] * SIZE[c["weights"]], "flops": 14 * n}
    if c["op"] == "route":
        n, k = c["T"] * c["E"], c["T"] * c["K"]
        if c["direction"] == "fwd":
            return {"bytes": 4 * n + 8 * k + (4 * c["E"] if c["bias"] else 0), "flops": 8 * n}
        dense = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": 4 * n + (4 * n if dense else 4 * k) + 8 * k, "flops": 8 * n}
    M, K, N, s = c["M"], c["K"], c["N"], SIZE[c["dtype"]]
    if c["direction"] == "fwd":
        o = SIZE[c["out"]]
        b = s * (M * K + K * N) + o * M * N + (4 * N if c["bias"] else 0)
        b += (o * M * N if c["res"] else 0) + (s * M * N if c["keep_z"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    b = s * (2 * M * K + 2 * K * N + M * N) + (4 * N if c["bias"] else 0)
    b += (s * M * K if c["res"] else 0) + (s * M * N if c["act"] != "none" else 0)
    return {"bytes": b, "flops": 4 * M * N * K}


# -------------------------------------------------------------- in 64 bits
def exact(case, seed):
    global own
    was, own = own, False       # the inputs alone: nothing of the framework
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = s["case"]
    t = {k: v.to(torch.float64) for k, v in s.items()
         if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if c["op"] == "norm":
        return _exact_norm(s, t, c)
    if c["op"] == "route":
        return _exact_route(s, c)
    return _exact_linear(t, c)


def _exact_norm(s, t, c):
    D = c["D"]
    if c["direction"] == "fwd":
        # the norm is of the residual stream as it is stored, in the rows' type
        total = t["x"] + t["res"] if c["res"] else t["x"]
        r = total.to(DTYPES[c["dtype"]]).double()
        mean = r.sum(1) / D
        var = ((r - mean[:, None]) ** 2).sum(1) / D
        rstd = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(t["beta"], (r - mean[:, None]) * rstd[:, None], t["gamma"])
        out = [y]
        if c["res"]:
            out.append(total)
        if c["stats"]:
            out += [mean, rstd]
        return out
    xh = (t["r"] - t["mean"][:, None]) * t["rstd"][:, None]
    u = t["dy"] * t["gamma"]
    m1 = u.sum(1) / D
    m2 = torch.einsum("ij,ij->i", u, xh) / D
    dx = (u - m1[:, None] - xh * m2[:, None]) * t["rstd"][:, None]
    if c["res"]:
        dx += t["dres"]
    ones = torch.ones(c["rows"], dtype=torch.float64, device=dx.device)
    return [dx, torch.einsum("ij,ij->j", t["dy"], xh), ones @ t["dy"]]


def _exact_route(s, c):
    l = s["logits"].cpu().numpy().astype(np.float64)
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    if c["score"] == "sigmoid":
        p = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    else:
        p = np.exp(l - np.logaddexp.reduce(l, axis=1, keepdims=True))
    if c["direction"] == "fwd":
        b = s["bias"].cpu().numpy().astype(np.float64) if c["bias"] else None
        key = l if b is None else p + b
        if G > 1:
            v = (p if b is None and c["group_top"] == 2 else key).reshape(T, G, E // G)
            first = v.max(axis=2)
            if c["group_top"] == 2:
                first = first + np.partition(v, -2, axis=2)[:, :, -2]
            rank = np.argsort(np.argsort(-first, axis=1, kind="stable"), axis=1, kind="stable")
            key = np.where(np.repeat(rank < c["top_groups"], E // G, axis=1), key, -np.inf)
        ids = np.argsort(-key, axis=1, kind="stable")[:, :K]
        w = np.take_along_axis(p, ids, axis=1)
        if c["renorm"]:
            w = w / w.sum(axis=1, keepdims=True)
        return [ids.astype(np.int32), w * c["scale"]]
    ids = s["ids"].cpu().numpy().astype(np.int64)
    dw = s["dw"].cpu().numpy().astype(np.float64) * c["scale"]
    sel = np.take_along_axis(p, ids, axis=1)
    if c["renorm"]:
        total = sel.sum(axis=1, keepdims=True)
        dsel = dw / total - (dw * sel).sum(axis=1, keepdims=True) / total ** 2
    else:
        dsel = dw
    if c["score"] == "sigmoid":
        d = np.zeros((T, E))
        np.put_along_axis(d, ids, dsel * sel * (1 - sel), axis=1)
        return [d]
    d = -p * (dsel * sel).sum(axis=1, keepdims=True)
    np.put_along_axis(d, ids, np.take_along_axis(d, ids, axis=1) + dsel * sel, axis=1)
    return [d]


def _exact_act(z, act):
    """(act(z), act'(z)) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        # 1/2 (1 + tanh u) = sigmoid(2 u)
        k = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(k * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * k * (1 + 0.134145 * z ** 2)
    p = torch.sigmoid(z)
    return z * p, p + z * p * (1 - p)


def _exact_linear(t, c):
    if c["direction"] == "fwd":
        z = torch.matmul(t["x"], t["w"])
        if c["bias"]:
            z += t["bias"]
        y = _exact_act(z, c["act"])[0]
        if c["res"]:
            y = y + t["res"]
        return [y, z] if c["keep_z"] else [y]
    dz = t["dy"] * _exact_act(t["z"], c["act"])[1] if c["act"] != "none" else t["dy"]
    dx = torch.matmul(dz, t["w"].T)
    if c["res"]:
        dx += t["dx_add"]
    out = [dx, torch.matmul(t["x"].T, dz)]
    return out + [dz.sum(0)] if c["bias"] else out
