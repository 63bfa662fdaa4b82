"""Cases of the operators that serve and wrap the expert block: the whole
expert layer for a few tokens, RMS norms after and before a block with its
gate and residual scale (forward and backward), and low-rank adapters of many
requests beside a shared projection.

Each operator is written here in its plain form (``own`` false: elementary
torch operations in 32 bits) and called through the framework (``own`` true).
``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # one request decoding: eight experts' weights, latency next to bandwidth
        dict(name="experts_one_token", op="experts", T=1, D=2816, E=128, K=8, F=704, dtype="bf16",
             route="softmax", bias=False, res=False),
        # a small batch of requests, the shared expert's output as the residual
        dict(name="experts_decode", op="experts", T=16, D=2048, E=128, K=8, F=768, dtype="bf16",
             route="softmax", bias=False, res=True),
        # the widest experts for a handful of tokens, routed by a router of its own
        dict(name="experts_wide", op="experts", T=4, D=7168, E=256, K=8, F=2048, dtype="bf16",
             route="given", bias=False, res=True),
        # the largest batch, unevenly routed: some experts see dozens of the tokens
        dict(name="experts_batch", op="experts", T=128, D=2816, E=128, K=8, F=704, dtype="fp16",
             route="sigmoid", bias=True, res=False),
        # one token's norms around its block, the widest rows: latency
        dict(name="norm_one_token", op="norm", direction="fwd", rows=1, D=7168, dtype="bf16",
             weights="bf16", post=True, pre=True, gate=False, token_gate=False, scale=1.0),
        # the long-sequence training batch: both norms, a gate for each channel
        dict(name="norm_train_fwd", op="norm", direction="fwd", rows=32768, D=2816, dtype="bf16",
             weights="fp32", post=True, pre=True, gate=True, token_gate=False, scale=0.5),
        # ... and its backward
        dict(name="norm_train_bwd", op="norm", direction="bwd", rows=32768, D=2816, dtype="bf16",
             weights="fp32", post=True, pre=True, gate=True, token_gate=False, scale=0.5),
        # a full-precision run with odd rows, gated by token
        dict(name="norm_odd_bwd", op="norm", direction="bwd", rows=4099, D=1001, dtype="fp32",
             weights="fp32", post=True, pre=True, gate=False, token_gate=True, scale=1.0),
        # one token of one request with an adapter
        dict(name="adapters_one_token", op="adapters", T=1, K=7168, N=2048, rank=16, slots=8,
             dtype="bf16", mix="tokens", none=0.0, res=True),
        # a decode batch: nearly every token has an adapter of its own, a few have none
        dict(name="adapters_decode", op="adapters", T=61, K=2816, N=2816, rank=16, slots=64,
             dtype="fp16", mix="tokens", none=0.1, res=True),
        # prompts of several requests, each with its adapter
        dict(name="adapters_prompt", op="adapters", T=8191, K=7168, N=2048, rank=64, slots=8,
             dtype="bf16", mix="runs", none=0.1, res=True),
        # a long batch in which the requests' tokens lie mixed
        dict(name="adapters_mixed", op="adapters", T=32768, K=2048, N=1536, rank=32, slots=16,
             dtype="bf16", mix="tokens", none=0.05, res=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("experts", "norm", "adapters"))
    if op == "experts":
        while True:
            c = dict(op=op, T=_log(rng, 1, 128), D=64 * _log(rng, 2, 112),
                     E=rng.choice((4, 8, 16, 60, 64, 128, 160, 256)), K=rng.randint(1, 8),
                     F=64 * _log(rng, 1, 32), dtype=rng.choice(("bf16", "bf16", "fp16")),
                     route=rng.choice(("softmax", "sigmoid", "given")), bias=rng.random() < 0.4,
                     res=rng.random() < 0.5)
            c["K"] = min(c["K"], c["E"])
            if c["route"] == "given":
                c["bias"] = False
            if 6 * c["E"] * c["D"] * c["F"] <= 2.0e9:
                return c
    if op == "norm":
        direction = rng.choice(("fwd", "bwd"))
        D = _log(rng, 16, 8192)
        if rng.random() < 0.7:
            D = max(16, D // 8 * 8)
        dtype = rng.choice(("bf16", "fp16", "fp32"))
        rows = min(_log(rng, 1, 32768), max(1, 32768 * 2816 * 2 // (D * SIZE[dtype])))
        post, pre = rng.choice(((True, True), (True, True), (True, False), (False, True)))
        return dict(op=op, direction=direction, rows=rows, D=D, dtype=dtype,
                    weights=rng.choice(("fp32", dtype)), post=post, pre=pre,
                    gate=rng.random() < 0.4, token_gate=rng.random() < 0.3,
                    scale=rng.choice((1.0, 0.5, 0.22)))
    K, N, rank = 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 896), rng.choice((8, 16, 16, 24, 32, 64, 128))
    T = min(_log(rng, 1, 32768), max(1, 8191 * 7168 // (K + 2 * N)))
    slots = rng.choice((1, 2, 4, 8, 16, 64))
    return dict(op=op, T=T, K=K, N=N, rank=rank, slots=slots, dtype=rng.choice(("bf16", "fp16")),
                mix=rng.choice(("tokens", "runs")), none=rng.choice((0.0, 0.1)),
                res=rng.random() < 0.8)


# --------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "experts":
        T, D, E, K, F, dt = c["T"], c["D"], c["E"], c["K"], c["F"], DTYPES[c["dtype"]]
        s["x"] = _randn(g, T, D, dtype=dt)
        s["wi"] = _randn(g, E, D, 2 * F, dtype=dt).mul_(D ** -0.5)
        s["wo"] = _randn(g, E, F, D, dtype=dt).mul_(F ** -0.5)
        s["res"] = _randn(g, T, D, dtype=dt) if c["res"] else None
        logits = _randn(g, T, E)
        if c["route"] == "given":   # what a router of its own hands over
            top = torch.sort(logits, dim=1, descending=True, stable=True)
            s["ids"] = top.indices[:, :K].to(torch.int32).contiguous()
            p = torch.sigmoid(top.values[:, :K])
            s["w"] = (2.5 * p / p.sum(1, keepdim=True)).contiguous()
        else:
            s["logits"] = logits
            s["bias"] = 0.5 * _randn(g, E) if c["bias"] else None
    elif c["op"] == "norm":
        n, D, dt, wt = c["rows"], c["D"], DTYPES[c["dtype"]], DTYPES[c["weights"]]
        # a residual stream: channels of different spread, some far wider
        spread = torch.exp(0.5 * _randn(g, D))
        spread[:: max(1, D // 16)] *= 8
        s["y"] = _randn(g, n, D).to(dt)
        stream = (_randn(g, n, D) * spread).to(dt)
        s["post"] = (1 + 0.2 * _randn(g, D)).to(wt) if c["post"] else None
        s["pre"] = (1 + 0.2 * _randn(g, D)).to(wt) if c["pre"] else None
        s["gate"] = (0.5 + 0.2 * _randn(g, D)).to(wt) if c["gate"] else None
        s["token_gate"] = torch.sigmoid(_randn(g, n)) if c["token_gate"] else None
        if c["direction"] == "fwd":
            s["res"] = stream
        else:
            s["r"] = stream
            s["du"] = _randn(g, n, D).to(dt) if c["pre"] else None
            s["dr"] = _randn(g, n, D).to(dt)
            s["rstd_y"] = torch.rsqrt(s["y"].float().square().mean(1) + EPS) if c["post"] else None
            s["rstd_r"] = torch.rsqrt(stream.float().square().mean(1) + EPS) if c["pre"] else None
    else:
        T, K, N, r, S, dt = c["T"], c["K"], c["N"], c["rank"], c["slots"], DTYPES[c["dtype"]]
        s["x"] = _randn(g, T, K, dtype=dt)
        s["a"] = _randn(g, S, r, K, dtype=dt).mul_(K ** -0.5)
        s["b"] = _randn(g, S, N, r, dtype=dt).mul_(0.2 * r ** -0.5)
        s["scale"] = 0.5 + torch.rand(S, generator=g, device="cuda")
        s["res"] = _randn(g, T, N, dtype=dt) if c["res"] else None
        h = torch.Generator()
        h.manual_seed(int(seed))
        if c["mix"] == "tokens":
            ids = torch.randint(S, (T,), generator=h)
            ids[torch.rand(T, generator=h) < c["none"]] = -1
        else:   # one adapter (or none) for each run of tokens, of ragged lengths
            runs = max(1, min(T, 2 * S))
            cuts = torch.sort(torch.randint(T, (runs,), generator=h)).values
            of_run = torch.randint(S, (runs + 1,), generator=h)
            of_run[torch.rand(runs + 1, generator=h) < c["none"]] = -1
            ids = of_run[torch.searchsorted(cuts, torch.arange(T), right=True)]
        s["ids"] = ids.to(torch.int32).cuda()
        # the plain form's plan: the rows of each adapter that the batch names
        s["rows"] = [(int(a), torch.nonzero(ids == a)[:, 0].cuda()) for a in torch.unique(ids) if a >= 0]
    if own:
        _handle(s, c)
    return s


def _handle(s, c):
    """The framework's operator with its output buffers and workspace, as a program keeps it
    (for the adapters with the batch's grouping, which all of a step's projections share)."""
    from mixture_experts_ffn_histogram_gb300 import binding, layer
    if c["op"] == "experts":
        mode = {"softmax": binding.SCORE_SOFTMAX_TOPK, "sigmoid": binding.SCORE_SIGMOID_NORM,
                "given": binding.SCORE_GIVEN}[c["route"]]
        s["op"] = layer.MoEDecode(c["T"], c["D"], c["E"], c["K"], c["F"], mode, dtype=DTYPES[c["dtype"]])
    elif c["op"] == "norm":
        s["op"] = layer.BlockNorm(c["rows"], c["D"], dtype=DTYPES[c["dtype"]],
                                  weight_dtype=DTYPES[c["weights"]], eps=EPS, scale=c["scale"],
                                  train=c["direction"] == "bwd")
    else:
        s["batch"] = layer.AdapterBatch(c["T"], c["slots"])
        s["batch"].group(s["ids"])
        s["op"] = layer.LowRankAdapters(c["T"], c["K"], c["N"], c["slots"], c["rank"],
                                        dtype=DTYPES[c["dtype"]])


# ----------------------------------------------------------------- the passes
def run(state):
    c = state["case"]
    if own:
        return {"experts": _own_experts, "norm": _own_norm, "adapters": _own_adapters}[c["op"]](state, c)
    return {"experts": _plain_experts, "norm": _plain_norm, "adapters": _plain_adapters}[c["op"]](state, c)


def _own_experts(s, c):
    if c["route"] == "given":
        return [s["op"].forward(s["x"], s["wi"], s["wo"], ids=s["ids"], w=s["w"], res=s["res"])]
    return [s["op"].forward(s["x"], s["wi"], s["wo"], logits=s["logits"], bias=s["bias"], res=s["res"])]


def _own_norm(s, c):
    op = s["op"]
    if c["direction"] == "fwd":
        u = op.forward(s["res"], s["y"], s["post"], s["pre"], gate=s["gate"], token_gate=s["token_gate"])
        return [op.r, u] if c["pre"] else [op.r]
    dres = op.backward(s["du"], s["dr"], s["r"], s["y"], s["post"], s["pre"], gate=s["gate"],
                       token_gate=s["token_gate"], rstd_y=s["rstd_y"], rstd_r=s["rstd_r"])
    out = [dres, op.dy]
    for given, grad in ((c["post"], op.dpost), (c["pre"], op.dpre), (c["gate"], op.dgate),
                        (c["token_gate"], op.dtoken_gate)):
        if given:
            out.append(grad)
    return out


def _own_adapters(s, c):
    return [s["op"].forward(s["batch"], s["x"], s["a"], s["b"], s["scale"], res=s["res"])]


def _plain_experts(s, c):
    T, K, F = c["T"], c["K"], c["F"]
    if c["route"] == "given":
        ids, w = s["ids"].long(), s["w"]
    else:
        score = s["logits"] + s["bias"] if c["bias"] else s["logits"]
        top = torch.sort(score, dim=1, descending=True, stable=True)
        ids, best = top.indices[:, :K], top.values[:, :K]
        p = torch.exp(best - best[:, :1]) if c["route"] == "softmax" else 1 / (1 + torch.exp(-best))
        w = p / p.sum(1, keepdim=True)
    x = s["x"].float()
    rows = []
    for t in range(T):
        z = torch.matmul(x[t], s["wi"][ids[t]].float())             # [K, 2F]
        h = z[:, :F] / (1 + torch.exp(-z[:, :F])) * z[:, F:]
        y = torch.matmul(h[:, None], s["wo"][ids[t]].float())[:, 0]  # [K, D]
        rows.append((w[t][:, None] * y).sum(0))
    out = torch.stack(rows)
    if c["res"]:
        out = out + s["res"].float()
    return [out.to(DTYPES[c["dtype"]])]


def _plain_norm(s, c):
    dt, wt, scale = DTYPES[c["dtype"]], DTYPES[c["weights"]], c["scale"]
    y = s["y"].float()
    g = scale * (s["gate"].float() if c["gate"] else torch.ones_like(y[0]))
    tg = s["token_gate"][:, None] if c["token_gate"] else 1.0
    post = s["post"].float() if c["post"] else 1.0
    if c["direction"] == "fwd":
        n = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * post if c["post"] else y
        r = (s["res"].float() + tg * g * n).to(dt)
        if not c["pre"]:
            return [r]
        f = r.float()
        return [r, (f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * s["pre"].float()).to(dt)]
    dr = s["dr"].float()
    if c["pre"]:
        rs = s["rstd_r"][:, None]
        xh = s["r"].float() * rs
        du = s["du"].float()
        a = du * s["pre"].float()
        dpre = (du * xh).sum(0)
        dr = dr + rs * (a - xh * (a * xh).mean(1, keepdim=True))
    yh = y * s["rstd_y"][:, None] if c["post"] else y
    dn = tg * g * post * dr
    dy = dn
    if c["post"]:
        dy = s["rstd_y"][:, None] * (dn - yh * (dn * yh).mean(1, keepdim=True))
    out = [dr.to(dt), dy.to(dt)]
    along = (tg * dr * yh).sum(0)
    if c["post"]:
        out.append((g * along).to(wt))
    if c["pre"]:
        out.append(dpre.to(wt))
    if c["gate"]:
        out.append((scale * post * along).to(wt))
    if c["token_gate"]:
        out.append((g * post * dr * yh).sum(1))
    return out


def _plain_adapters(s, c):
    dt = DTYPES[c["dtype"]]
    out = s["res"].float() if c["res"] else torch.zeros(c["T"], c["N"], device="cuda")
    for a, rows in s["rows"]:
        v = s["x"][rows].float() @ s["a"][a].float().t()
        out[rows] += s["scale"][a] * (v @ s["b"][a].float().t())
    return [out.to(dt)]


# ----------------------------------------------------------------------- work
def work(case):
    c = case
    s = SIZE[c["dtype"]]
    if c["op"] == "experts":
        T, D, E, K, F = c["T"], c["D"], c["E"], c["K"], c["F"]
        # the experts that T tokens name, on average
        live = E * (1 - (1 - K / E) ** T)
        b = s * (live * 3 * D * F + T * D * (3 if c["res"] else 2))
        b += 8 * T * K if c["route"] == "given" else 4 * T * E + (4 * E if c["bias"] else 0)
        return {"bytes": int(b), "flops": 6 * T * K * D * F}
    if c["op"] == "norm":
        n, wb, D = c["rows"] * c["D"], SIZE[c["weights"]], c["D"]
        weights = c["post"] + c["pre"] + c["gate"]
        per_row = 4 * c["rows"] * (c["token_gate"] * (1 if c["direction"] == "fwd" else 2))
        if c["direction"] == "fwd":
            return {"bytes": n * s * (4 if c["pre"] else 3) + weights * D * wb + per_row, "flops": 10 * n}
        # read y, dr (r, du with the norm before the block), write dres, dy
        per_row += 4 * c["rows"] * (c["post"] + c["pre"])
        needs_y = c["post"] or c["gate"] or c["token_gate"]
        arrays = 3 + (1 if needs_y else 0) + (2 if c["pre"] else 0)
        return {"bytes": n * s * arrays + 2 * weights * D * wb + per_row, "flops": 20 * n}
    T, K, N, r, S = c["T"], c["K"], c["N"], c["rank"], c["slots"]
    tokens = T * (1 - c["none"])
    live = S * (1 - (1 - 1 / S) ** (tokens if c["mix"] == "tokens" else min(tokens, 2 * S)))
    b = s * (tokens * K + T * N * (2 if c["res"] else 1) + live * r * (K + N)) + 4 * (T + S)
    return {"bytes": int(b), "flops": int(2 * tokens * r * (K + N))}


# -------------------------------------------------------------- in 64 bits
def exact(case, seed):
    global own
    was, own = own, False       # the inputs alone: nothing of the framework
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"experts": _exact_experts, "norm": _exact_norm, "adapters": _exact_adapters}[case["op"]](s, s["case"])


def _exact_experts(s, c):
    K, F = c["K"], c["F"]
    if c["route"] == "given":
        ids, w = s["ids"].long(), s["w"].double()
    else:
        # the definition compares the sums as fp32 holds them; equal ones by their number
        score = (s["logits"] + s["bias"] if c["bias"] else s["logits"]).double()
        ids = torch.argsort(-score, dim=1, stable=True)[:, :K]
        best = torch.take_along_dim(score, ids, dim=1)
        w = torch.softmax(best, dim=1)
        if c["route"] == "sigmoid":
            p = torch.sigmoid(best)
            w = p / p.sum(dim=1, keepdim=True)
    out = s["res"].double() if c["res"] else torch.zeros(c["T"], c["D"], dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():
        t, k = torch.nonzero(ids == e, as_tuple=True)
        up = s["x"][t].double() @ s["wi"][e].double()
        gate, up = up.split(F, dim=1)
        y = (gate * torch.sigmoid(gate) * up) @ s["wo"][e].double()
        out.index_add_(0, t, y * w[t, k][:, None])
    return [out]


def _exact_norm(s, c):
    """Forward from the formulas; gradients by automatic differentiation of them."""
    D, bwd = c["D"], c["direction"] == "bwd"
    leaf = {}
    for k in ("y", "post", "pre", "gate", "token_gate", "res"):
        v = s.get(k)
        leaf[k] = v.double().requires_grad_(bwd) if v is not None else None
    if bwd:     # r is given: a stream that yields it, moved along with the branch
        leaf["res"] = torch.zeros_like(s["r"], dtype=torch.float64).requires_grad_(True)
    branch = leaf["y"]
    if c["post"]:
        rstd = 1 / torch.sqrt((leaf["y"] ** 2).sum(1) / D + EPS)
        branch = torch.einsum("ij,i,j->ij", branch, rstd, leaf["post"])
    if c["gate"]:
        branch = branch * leaf["gate"]
    if c["token_gate"]:
        branch = branch * leaf["token_gate"].unsqueeze(1)
    r = leaf["res"] + c["scale"] * branch
    if not bwd:
        # the norm before the next block is of the stream as it is stored
        r_next = r.to(DTYPES[c["dtype"]]).double()
        if not c["pre"]:
            return [r]
        rstd = 1 / torch.sqrt((r_next ** 2).sum(1) / D + EPS)
        return [r, torch.einsum("ij,i,j->ij", r_next, rstd, leaf["pre"])]
    r = r + (s["r"].double() - r.detach())
    target = (r * s["dr"].double()).sum()
    if c["pre"]:
        u = r * leaf["pre"] / torch.sqrt((r ** 2).sum(1, keepdim=True) / D + EPS)
        target = target + (u * s["du"].double()).sum()
    wanted = ["res", "y"] + [k for k in ("post", "pre", "gate", "token_gate") if c[k]]
    return list(torch.autograd.grad(target, [leaf[k] for k in wanted]))


def _exact_adapters(s, c):
    out = s["res"].double() if c["res"] else torch.zeros(c["T"], c["N"], dtype=torch.float64, device="cuda")
    ids = s["ids"].long()
    for a in range(c["slots"]):
        rows = torch.nonzero(ids == a).squeeze(1)
        delta = torch.einsum("tr,nr->tn", torch.einsum("tk,rk->tr", s["x"][rows].double(), s["a"][a].double()),
                             s["b"][a].double())
        out.index_add_(0, rows, delta * s["scale"][a].double())
    return [out]
