"""Norms after and before a block, with its gate and residual scale, against
their definition in 64 bits, against automatic differentiation and against
differences."""
import itertools

import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import assert_within
from tests.serving_refs import block_norm, block_norm_bwd

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def _data(rows, D, dt, wt, parts, seed):
    """res, y, du, dr and the weights and gates whose first letters are in parts."""
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0, base=0.0, t=dt):
        return (base + scale * torch.randn(*shape, generator=g)).to(t).cuda()

    spread = torch.exp(torch.randn(D, generator=g)).to(dt).cuda()
    d = dict(res=r(rows, D) * spread, y=r(rows, D), du=r(rows, D), dr=r(rows, D))
    w = dict(post=r(D, scale=0.3, base=1, t=wt), pre=r(D, scale=0.3, base=1, t=wt),
             gate=r(D, scale=0.4, t=wt), token_gate=r(rows, t=F32))
    return d, {k: w[k] if k[:2] in parts else None for k in w}


def _arith(D):
    """Roundings that a row's value sees: its products and sums (a dozen), a sum
    over D by threads of up to 16 elements, warps and blocks, the root."""
    return (12 + 16 + 5 + 5 + 4) * U * 4


def _check_forward(op, d, w, scale, offset, eps):
    dt, D = d["res"].dtype, d["res"].shape[1]
    got = op.forward(d["res"], d["y"], w["post"], w["pre"], gate=w["gate"], token_gate=w["token_gate"])
    torch.cuda.synchronize()
    ref = block_norm(d["res"], d["y"], **w, scale=scale, offset=offset, eps=eps, r=op.r)
    if d["y"] is not None:
        assert_within("r", op.r, ref["r"], _arith(D) * ref["r_mag"])
    else:
        assert op.r is d["res"]
    if w["pre"] is None:
        assert got is op.r and op.u is None
    else:
        assert_within("u", got, ref["u"], _arith(D) * ref["u_mag"])
    if op.train:
        for k, part in (("rstd_y", "post"), ("rstd_r", "pre")):
            if w[part] is None:
                assert getattr(op, k) is None
            else:
                assert_within(k, getattr(op, k), ref[k], _arith(D) * ref[k])


def _check_backward(op, d, w, scale, offset, du=True, dr=True):
    rows, D = d["res"].shape
    gu = d["du"] if w["pre"] is not None else None
    gr = d["dr"] if dr else None
    got = {"dres": op.backward(gu, gr, op.r, d["y"], **w)}
    torch.cuda.synchronize()
    for k in ("dy", "dpost", "dpre", "dgate", "dtoken_gate"):
        got[k] = getattr(op, k)
    ref = block_norm_bwd(gu, gr, op.r, d["y"], **w, rstd_y=op.rstd_y, rstd_r=op.rstd_r, scale=scale,
                         offset=offset)
    for k, v in got.items():
        assert (v is None) == (k not in ref), k
        if v is None:
            continue
        want, mag = ref[k]
        # sums over the rows: walked by a block (rows / blocks of them in one
        # chain), then 64 threads and a warp
        count = 0 if k in ("dres", "dy", "dtoken_gate") else rows / 64 + 64
        assert_within(k, v, want, (_arith(D) + (count + 8) * U) * mag)


PARTS = [("po", "pr"), ("po", "pr", "ga"), ("po", "pr", "to"), ("po", "pr", "ga", "to"), ("po",), ("pr",),
         ("po", "ga"), ("po", "to"), ("pr", "ga"), ("pr", "to"), ("pr", "ga", "to"), ("ga",), ("to",), ()]


@pytest.mark.parametrize("rows,D,dt,wt", [
    (1, 7168, BF, BF), (1, 1, F32, F32), (3, 17, HF, F32), (2, 8192, BF, F32), (5, 8192, F32, F32),
    (700, 256, BF, F32), (2500, 129, BF, BF), (2500, 1001, F32, F32), (2600, 255, HF, HF),
    (2500, 4097, BF, F32), (1300, 2816, HF, F32), (33, 1000, BF, F32), (9, 63, F32, F32),
])
def test_forward_and_backward(rows, D, dt, wt):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import BlockNorm
    scale, eps = 0.5, 1e-6
    op = BlockNorm(rows, D, dtype=dt, weight_dtype=wt, eps=eps, scale=scale)
    for i, parts in enumerate(PARTS[:4] if rows * D > 500000 else PARTS):
        d, w = _data(rows, D, dt, wt, parts, rows + D + i)
        _check_forward(op, d, w, scale, 0.0, eps)
        _check_backward(op, d, w, scale, 0.0)


@pytest.mark.parametrize("rows,D,dt", [(2500, 513, BF), (40, 512, F32)])
def test_without_y_and_without_dr(rows, D, dt):
    """u = norm(res), in front of the first block; nothing else flowing into r."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import BlockNorm
    op = BlockNorm(rows, D, dtype=dt, eps=1e-5, scale=2.0, offset=1.0)
    d, w = _data(rows, D, dt, F32, ("pr",), 3)
    for y, dr in itertools.product((None, d["y"]), (True, False)):
        _check_forward(op, dict(d, y=y), w, 2.0, 1.0, 1e-5)
        _check_backward(op, dict(d, y=y), w, 2.0, 1.0, dr=dr)
        assert (op.dy is None) == (y is None)


def test_gradients_against_automatic_differentiation():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import BlockNorm
    rows, D, eps, scale, offset = 50, 200, 1e-6, 0.7, 1.0
    d, w = _data(rows, D, F32, F32, ("po", "pr", "ga", "to"), 8)
    op = BlockNorm(rows, D, dtype=F32, eps=eps, scale=scale, offset=offset)
    op.forward(d["res"], d["y"], **w)
    dres = op.backward(d["du"], d["dr"], y=d["y"], **w)
    leaf = {k: v.double().requires_grad_(True) for k, v in dict(w, res=d["res"], y=d["y"]).items()}

    def total(v):
        yh = v["y"] / (v["y"].square().mean(1, keepdim=True) + eps).sqrt()
        r = v["res"] + scale * v["token_gate"][:, None] * v["gate"] * (v["post"] + offset) * yh
        u = (v["pre"] + offset) * r / (r.square().mean(1, keepdim=True) + eps).sqrt()
        return (u * d["du"].double()).sum() + (r * d["dr"].double()).sum()

    total(leaf).backward()
    got = dict(res=dres, y=op.dy, post=op.dpost, pre=op.dpre, gate=op.dgate, token_gate=op.dtoken_gate)
    # fp32 throughout: 2^-15 covers some hundred roundings of terms of the gradient's own size
    for k, v in got.items():
        off = (v.double() - leaf[k].grad).norm() / leaf[k].grad.norm()
        assert off < 2.0 ** -15, f"{k}: {float(off):.2e}"
    # and by differences, along one direction for each argument
    g = torch.Generator().manual_seed(4)
    for k, v in got.items():
        way = torch.randn(v.shape, generator=g, dtype=torch.float64).cuda()
        h = 1e-5
        with torch.no_grad():
            up, down = (total({**leaf, k: leaf[k] + s * h * way}) for s in (1, -1))
        diff, along = float((up - down) / (2 * h)), float((v.double() * way).sum())
        # the difference's own error: h^2 of the third derivative, and 2^-52 / h of the sums
        assert abs(diff - along) <= 1e-4 * float((v.double() * way).abs().sum()), k


def test_strides_places_and_fewer_rows():
    """Rows that lie in wider ones, at odd places; rows behind the call's last
    are left as they were; results repeat bit for bit."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import BlockNorm
    rows, D = 3000, 300
    for dt, shift, extra in ((BF, 3, 5), (F32, 1, 3), (HF, 8, 12), (BF, 0, 1)):
        d, w = _data(rows, D, dt, F32, ("po", "pr", "ga"), shift)
        lie = {}
        for k, v in d.items():
            wide = torch.zeros(rows, D + extra + shift, dtype=dt, device="cuda")
            wide[:, shift:shift + D] = v
            lie[k] = wide[:, shift:shift + D]
        op = BlockNorm(rows, D, dtype=dt, scale=1.5)
        _check_forward(op, lie, w, 1.5, 0.0, 1e-6)
        _check_backward(op, lie, w, 1.5, 0.0)
        first = [op.r.clone(), op.u.clone(), op._dres.clone(), op.dy.clone(), op._dw.clone()]
        op.forward(lie["res"], lie["y"], **w)
        op.backward(lie["du"], lie["dr"], y=lie["y"], **w)
        for a, b in zip(first, (op.r, op.u, op._dres, op.dy, op._dw)):
            assert torch.equal(a, b)
        for n in (0, 1, 77):
            for t in (op._r, op._u, op._dres, op._dy_out):
                t.fill_(3.0)
            part = {k: v[:n] for k, v in lie.items()}
            _check_forward(op, part, w, 1.5, 0.0, 1e-6)
            _check_backward(op, part, w, 1.5, 0.0)
            for t in (op._r, op._u, op._dres, op._dy_out):
                assert bool((t[n:] == 3.0).all())


def test_bad_and_empty_rows():
    """A NaN or infinity stays in its row; a row of zeros gives zeros."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import BlockNorm
    rows, D = 40, 264
    d, w = _data(rows, D, BF, F32, ("po", "pr"), 2)
    op = BlockNorm(rows, D, scale=1.0)
    d["res"][7], d["y"][7] = 0.0, 0.0
    u0 = op.forward(d["res"], d["y"], **w).clone()
    assert torch.equal(u0[7], torch.zeros_like(u0[7])) and bool(torch.isfinite(u0).all())
    assert bool(torch.isfinite(op.backward(d["du"], d["dr"], y=d["y"], **w)).all())
    y = d["y"].clone()
    y[3, 5], y[9, 0] = float("nan"), float("inf")
    u = op.forward(d["res"], y, **w)
    keep = [t for t in range(rows) if t not in (3, 9)]
    assert torch.equal(u[keep], u0[keep]) and bool(torch.isnan(u[3]).all())


def test_the_largest_batch():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import BlockNorm
    rows, D = 32768, 2816
    d, w = _data(64, D, BF, F32, ("po", "pr", "ga"), 1)
    d = {k: v.repeat(rows // 64, 1) for k, v in d.items()}
    op = BlockNorm(rows, D, scale=0.5)
    op.forward(d["res"], d["y"], **w)
    op.backward(d["du"], d["dr"], y=d["y"], **w)
    r, u, dy, dres = op.r, op.u, op.dy, op._dres
    for t in (r, u, dy, dres):  # every repetition of the rows gives the same
        assert torch.equal(t.view(rows // 64, 64, D), t[:64].expand(rows // 64, 64, D))
    few = BlockNorm(64, D, scale=0.5)
    _check_forward(few, {k: v[:64] for k, v in d.items()}, w, 0.5, 0.0, 1e-6)
    assert torch.equal(few.r, r[:64]) and torch.equal(few.u, u[:64])
    few.backward(d["du"][:64], d["dr"][:64], y=d["y"][:64], **w)
    for name in ("dpost", "dpre", "dgate"):
        a, b = getattr(op, name).double(), getattr(few, name).double() * (rows // 64)
        # 512 times the same 64 rows, summed in two orders: 2^-24 for each addition of a chain
        assert float((a - b).abs().max()) <= (rows / 152 + 200) * U * float(b.abs().max() * 8)


def test_another_stream_and_a_graph():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import BlockNorm
    rows, D = 500, 768
    d, w = _data(rows, D, BF, F32, ("po", "pr", "to"), 6)
    op = BlockNorm(rows, D)
    want = [op.forward(d["res"], d["y"], **w).clone(), op.backward(d["du"], d["dr"], y=d["y"], **w).clone(),
            op.dpost.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.forward(d["res"], d["y"], **w, stream=side)
    op.backward(d["du"], d["dr"], y=d["y"], **w, stream=side)
    side.synchronize()
    for a, b in zip(want, (op.u, op._dres, op.dpost)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(d["res"], d["y"], **w)
        op.backward(d["du"], d["dr"], y=d["y"], **w)
    for t in (op._u, op._dres, op._dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (op.u, op._dres, op.dpost)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,D,dt", [(300, 256, BF), (2500, 301, BF), (40, 33, F32), (3, 7168, HF)])
def test_norms_on_their_own_results(rows, D, dt):
    """The stream and the normalised rows of a call are res and y of the next;
    backward, dres and dy are dr and du of the one before."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import BlockNorm
    for parts in (("po", "pr", "ga", "to"), ("pr",)):
        d, w = _data(rows, D, dt, F32, parts, rows)
        op = BlockNorm(rows, D, dtype=dt, scale=0.5)
        op.forward(d["res"], d["y"], **w)
        r, u = op.r.clone(), op.u.clone()
        op.forward(r, u, **w)
        want = [op.r.clone(), op.u.clone()]
        ry, rr = op.rstd_y, op.rstd_r
        saved = dict(r=want[0], y=u, **w, rstd_y=None if ry is None else ry.clone(), rstd_r=rr.clone())
        op.forward(d["res"], d["y"], **w)
        op.forward(op.r, op.u, **w)
        assert torch.equal(op.r, want[0]) and torch.equal(op.u, want[1])
        op.backward(d["du"], d["dr"], **saved)
        dr, du = op._dres.clone(), op.dy.clone()
        want = [op.backward(du, dr, **saved).clone(), op.dy.clone(), op.dpre.clone()]
        op.backward(d["du"], d["dr"], **saved)
        got = op.backward(op.dy, op._dres, **saved)
        for a, b in zip((got, op.dy, op.dpre), want):
            assert torch.equal(a, b)
