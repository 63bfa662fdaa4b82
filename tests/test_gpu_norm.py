"""Layer norm forward and backward against 64 bits: widths from one column to
the widest, odd ones, row strides, offsets of the rows, each type, in-place
use, no rows, and captured graphs."""
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import U32, assert_within, norm_bwd, norm_fwd

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

# rows, D, type, weights' type, residual, padding of the row stride
CASES = [
    (1, 7168, BF, BF, True, 0),
    (1, 1, F32, F32, False, 0),
    (3, 17, BF, F32, True, 0),
    (5, 1001, F32, F32, True, 0),
    (7, 1001, HF, HF, True, 3),
    (33, 256, BF, F32, True, 0),
    (700, 64, HF, F32, False, 0),
    (700, 504, BF, BF, True, 8),
    (640, 2816, BF, F32, True, 0),
    (640, 2816, BF, F32, False, 1),      # rows off the 16-byte boundary
    (130, 4100, F32, F32, True, 4),
    (9, 8192, F32, F32, True, 0),
    (9, 8191, F32, F32, True, 0),
    (20, 8191, BF, BF, False, 0),
    (650, 8192, HF, HF, True, 0),
    (1300, 8, F32, F32, True, 0),
]


def _rand(g, n, D, dt, pad):
    base = torch.randn(n, D + pad, generator=g).to(dt).cuda()
    return base[:, :D]


def _inputs(rows, D, dt, wt, res, pad, offset=0.0):
    g = torch.Generator().manual_seed(rows * 10007 + D)
    x = _rand(g, rows, D, dt, pad)
    if offset:
        x.add_(offset)
    return {
        "x": x, "res": _rand(g, rows, D, dt, pad) if res else None,
        "gamma": (1 + 0.3 * torch.randn(D, generator=g)).to(wt).cuda(),
        "beta": (0.3 * torch.randn(D, generator=g)).to(wt).cuda(),
        "dy": _rand(g, rows, D, dt, pad), "dres": _rand(g, rows, D, dt, pad) if res else None,
    }


@pytest.mark.parametrize("rows,D,dt,wt,res,pad", CASES)
def test_forward_and_backward(rows, D, dt, wt, res, pad):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import LayerNorm
    i = _inputs(rows, D, dt, wt, res, pad, offset=4.0 if rows % 2 else 0.0)
    op = LayerNorm(rows, D, dt, wt, EPS)
    y = op.forward(i["x"], i["gamma"], i["beta"], res=i["res"])
    r = i["x"]
    if res:
        r = (i["x"].float() + i["res"].float()).to(dt)
        assert torch.equal(op.r, r)
    yr, mean, rstd, mag = norm_fwd(r, i["gamma"], i["beta"], EPS)
    # sums of D terms in trees at most 32 deep, then some ten operations
    assert_within("y", y, yr, 64 * U32 * mag)
    assert_within("mean", op.mean, mean, 64 * U32 * r.double().abs().mean(1))
    # the variance's error, from the mean's, is relative: 2 (mean |r|)^2 / var
    spread = (r.double().abs().mean(1) * rstd) ** 2
    assert_within("rstd", op.rstd, rstd, rstd * U32 * (64 + 64 * 64 * U32 * spread))
    dx = op.backward(i["dy"], r, i["gamma"], dres=i["dres"])
    want, mags = norm_bwd(i["dy"], r, i["gamma"], op.mean, op.rstd, i["dres"])
    assert_within("dx", dx, want[0], 64 * U32 * mags[0])
    # at most rows / (blocks) terms in a row, then 32-way trees
    assert_within("dgamma", op.dgamma, want[1], (128 + rows / 64) * U32 * mags[1])
    assert_within("dbeta", op.dbeta, want[2], (128 + rows / 64) * U32 * mags[2])


def test_gradient_against_differences():
    """dx, dgamma, dbeta of a scalar loss against central differences of the
    64-bit forward (step 1e-5: truncation 1e-10, far below fp32's rounding)."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import LayerNorm
    i = _inputs(6, 40, F32, F32, False, 0)
    op = LayerNorm(6, 40, F32, F32, EPS)
    op.forward(i["x"], i["gamma"], i["beta"])
    dx = op.backward(i["dy"], i["x"], i["gamma"])

    def loss(x, g, b):
        return (norm_fwd(x, g, b, EPS)[0] * i["dy"].double()).sum()

    args = [i["x"].double(), i["gamma"].double(), i["beta"].double()]
    h = 1e-5
    for k, got in ((0, dx), (1, op.dgamma), (2, op.dbeta)):
        flat = args[k].flatten()
        num = torch.zeros_like(flat)
        for j in range(flat.numel()):
            hi, lo = [a.clone() for a in args], [a.clone() for a in args]
            hi[k].view(-1)[j] += h
            lo[k].view(-1)[j] -= h
            num[j] = (loss(*hi) - loss(*lo)) / (2 * h)
        assert (got.double().flatten() - num).abs().max() < 1e-5 * max(1.0, float(num.abs().max()))


def test_fewer_rows_none_and_one():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import LayerNorm
    i = _inputs(64, 96, BF, F32, True, 0)
    op = LayerNorm(64, 96, BF, F32, EPS)
    full = op.forward(i["x"], i["gamma"], i["beta"], res=i["res"]).clone()
    assert torch.equal(op.forward(i["x"][:1], i["gamma"], i["beta"], res=i["res"][:1]), full[:1])
    y = op.forward(i["x"][:0], i["gamma"], i["beta"], res=i["res"][:0])
    assert y.shape == (0, 96)
    op.dgamma.fill_(7.0)
    op.dbeta.fill_(7.0)
    op.backward(i["dy"][:0], op.r, i["gamma"], dres=i["dres"][:0])
    assert not op.dgamma.any() and not op.dbeta.any()


def test_in_place_and_a_constant_row():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    i = _inputs(40, 2816, BF, F32, True, 0)
    i["x"][3] = 2.0
    i["res"][3] = -2.0
    y, r = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    st = torch.empty(2, 40, device="cuda")
    B.moe_layer_norm(i["x"], i["res"], i["gamma"], i["beta"], r, y, st[0], st[1], EPS)
    # a constant row has variance 0: y = beta
    assert torch.equal(y[3], i["beta"].to(BF))
    x2, s2 = i["x"].clone(), i["res"].clone()
    B.moe_layer_norm(x2, s2, i["gamma"], i["beta"], s2, x2, st[0], st[1], EPS)
    assert torch.equal(x2, y) and torch.equal(s2, r)
    ws = torch.empty(B.moe_layer_norm_workspace_bytes(40, 2816), dtype=torch.uint8, device="cuda")
    dg, db = torch.empty(2816, device="cuda"), torch.empty(2816, device="cuda")
    dx = torch.empty_like(y)
    B.moe_layer_norm_bwd(i["dy"], r, i["gamma"], st[0], st[1], i["dres"], dx, dg, db, ws)
    d2 = i["dres"].clone()
    B.moe_layer_norm_bwd(i["dy"], r, i["gamma"], st[0], st[1], d2, d2, None, None, None)
    assert torch.equal(d2, dx)


def test_a_bad_row_stays_alone():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import LayerNorm
    i = _inputs(50, 264, BF, F32, False, 0)
    i["x"][7, 5] = float("inf")
    i["x"][8, 0] = float("nan")
    op = LayerNorm(50, 264, BF, F32, EPS, train=False)
    y = op.forward(i["x"], i["gamma"], i["beta"])
    bad = ~torch.isfinite(y.float()).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 8]


def test_reproducible_other_stream_and_graph():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import LayerNorm
    i = _inputs(2000, 1408, BF, BF, True, 0)
    op = LayerNorm(2000, 1408, BF, BF, EPS)

    def step(stream=None):
        y = op.forward(i["x"], i["gamma"], i["beta"], res=i["res"], stream=stream)
        dx = op.backward(i["dy"], op.r, i["gamma"], dres=i["dres"], stream=stream)
        return [y, dx, op.dgamma, op.dbeta]

    ref = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for t in out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


# many rows (each block walks several, some past 32) whose arrays start at
# offsets of their own within a 16-byte unit; rows, D, type, weights' type,
# residual, offsets and row strides' padding of x, res, dy, dres
MANY = [
    (40000, 21, BF, F32, True, (0, 1, 2, 3), (0, 3, 1, 0)),
    (6000, 125, F32, F32, True, (1, 0, 3, 2), (0, 1, 0, 2)),
    (13000, 333, HF, HF, True, (0, 7, 5, 3), (0, 0, 1, 3)),
    (7000, 1001, BF, BF, False, (5, 0, 2, 0), (0, 0, 7, 0)),
    (1300, 2047, F32, F32, True, (3, 3, 3, 3), (1, 1, 1, 1)),
    (900, 4095, BF, F32, True, (1, 2, 3, 4), (0, 1, 2, 3)),
    (12000, 264, BF, F32, True, (0, 0, 0, 0), (0, 0, 0, 0)),
    # alike: odd widths, one after the other
    (9000, 129, BF, F32, True, (0, 0, 0, 0), (0, 0, 0, 0)),
    (13000, 251, F32, F32, True, (0, 0, 0, 0), (0, 0, 0, 0)),
    (3000, 333, HF, HF, False, (0, 0, 0, 0), (0, 0, 0, 0)),
    (2750, 1001, BF, BF, True, (0, 0, 0, 0), (0, 0, 0, 0)),
    (5200, 1406, F32, F32, False, (0, 0, 0, 0), (0, 0, 0, 0)),
    (2500, 4097, BF, F32, True, (0, 0, 0, 0), (0, 0, 0, 0)),
    (2500, 8177, HF, F32, True, (0, 0, 0, 0), (0, 0, 0, 0)),
    (2437, 8185, F32, F32, True, (0, 0, 0, 0), (0, 0, 0, 0)),
    (2500, 8191, BF, BF, True, (0, 0, 0, 0), (0, 0, 0, 0)),
    (6000, 1408, HF, F32, False, (0, 0, 0, 0), (8, 8, 8, 8)),
]


@pytest.mark.parametrize("rows,D,dt,wt,res,offs,pads", MANY)
def test_many_rows_at_any_offset(rows, D, dt, wt, res, offs, pads):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import LayerNorm
    g = torch.Generator(device="cuda").manual_seed(rows + D)

    def mat(i):
        ld = D + pads[i]
        flat = torch.randn(offs[i] + rows * ld, generator=g, device="cuda").to(dt)
        return flat[offs[i]:].view(rows, ld)[:, :D]

    x, s, dy, dres = (mat(i) for i in range(4))
    gamma = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wt)
    beta = (0.3 * torch.randn(D, generator=g, device="cuda")).to(wt)
    op = LayerNorm(rows, D, dt, wt, EPS)
    y = op.forward(x, gamma, beta, res=s if res else None)
    r = (x.float() + s.float()).to(dt) if res else x
    if res:
        assert torch.equal(op.r, r)
    yr, mean, rstd, mag = norm_fwd(r, gamma, beta, EPS)
    assert_within("y", y, yr, 64 * U32 * mag)
    dx = op.backward(dy, r, gamma, dres=dres if res else None)
    want, mags = norm_bwd(dy, r, gamma, op.mean, op.rstd, dres if res else None)
    assert_within("dx", dx, want[0], 64 * U32 * mags[0])
    # a thread's sum over its rows (152 blocks at least), then at most 160 terms
    assert_within("dgamma", op.dgamma, want[1], (160 + rows / 152) * U32 * mags[1])
    assert_within("dbeta", op.dbeta, want[2], (160 + rows / 152) * U32 * mags[2])


def test_neighbours_of_ragged_rows_stay():
    """Rows inside a wider matrix: what lies between them is not written."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    g = torch.Generator(device="cuda").manual_seed(5)
    for dt in (BF, F32):
        wide = torch.randn(60, 45, generator=g, device="cuda").to(dt)
        x = wide[:, 3:40]
        y = torch.full((60, 51), 7.0, dtype=dt, device="cuda")
        r = torch.full((60, 47), 9.0, dtype=dt, device="cuda")
        w = torch.ones(37, device="cuda")
        b = torch.zeros(37, device="cuda")
        B.moe_layer_norm(x, x, w, b, r[:, 1:38], y[:, 5:42], None, None, EPS)
        assert torch.equal(r[:, 1:38], (2 * x.float()).to(dt))
        assert bool((r[:, :1] == 9).all()) and bool((r[:, 38:] == 9).all())
        assert bool((y[:, :5] == 7).all()) and bool((y[:, 42:] == 7).all())
        assert bool((y[:, 5:42] != 7).all())
        st = torch.rand(2, 60, device="cuda")
        dx = torch.full((60, 41), 3.0, dtype=dt, device="cuda")
        B.moe_layer_norm_bwd(x, x, w, st[0], st[1], x, dx[:, 2:39], None, None, None)
        assert bool((dx[:, :2] == 3).all()) and bool((dx[:, 39:] == 3).all())


@pytest.mark.parametrize("dt,D,off,pad", [(BF, 333, 0, 0), (BF, 264, 3, 5), (F32, 1001, 1, 2), (HF, 150, 7, 0)])
def test_shifted_rows_and_their_neighbours(dt, D, off, pad):
    """All arrays with the same odd offset and stride: what lies between the
    rows is not written, and neither it nor a bad row reaches another row."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    rows, ld = 2600, D + pad
    g = torch.Generator(device="cuda").manual_seed(D)

    def mat(fill):
        flat = torch.full((off + rows * ld + 8,), fill, dtype=dt, device="cuda")
        return flat, flat[off:off + rows * ld].view(rows, ld)[:, :D]

    bad = {100: (0, float("nan")), 200: (D - 1, float("nan")), 300: (D - 1, float("inf"))}
    (_, x), (_, s), (_, dy), (_, dres) = (mat(float("nan")) for _ in range(4))
    for m in (x, s, dy, dres):
        m.copy_(torch.randn(rows, D, generator=g, device="cuda"))
    w, b = torch.rand(D, generator=g, device="cuda"), torch.rand(D, generator=g, device="cuda")
    (yf, y), (rf, r), (df, dx) = (mat(7.0) for _ in range(3))
    clean = x.clone()
    for row, (col, v) in bad.items():
        x[row, col] = v
    st = torch.empty(2, rows, device="cuda")
    B.moe_layer_norm(x, s, w, b, r, y, st[0], st[1], EPS)
    assert (~torch.isfinite(y.float())).any(1).nonzero().flatten().tolist() == sorted(bad)
    x.copy_(clean)
    B.moe_layer_norm(x, s, w, b, r, y, st[0], st[1], EPS)
    want = (x.float() + s.float()).to(dt)
    assert torch.equal(r, want)
    yr, mean, rstd, mag = norm_fwd(want, w, b, EPS)
    assert_within("y", y, yr, 64 * U32 * mag)
    ws = torch.empty(B.moe_layer_norm_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    dg, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    B.moe_layer_norm_bwd(dy, r, w, st[0], st[1], dres, dx, dg, db, ws)
    ref, mags = norm_bwd(dy, r, w, st[0], st[1], dres)
    assert_within("dx", dx, ref[0], 64 * U32 * mags[0])
    assert_within("dgamma", dg, ref[1], (160 + rows / 152) * U32 * mags[1])
    assert_within("dbeta", db, ref[2], (160 + rows / 152) * U32 * mags[2])
    for flat in (yf, rf, df):  # only the rows were written
        keep = torch.ones_like(flat, dtype=torch.bool)
        keep[off:off + rows * ld].view(rows, ld)[:, :D] = False
        assert bool((flat[keep] == 7).all())
    dy[400, D - 1] = float("nan")
    B.moe_layer_norm_bwd(dy, r, w, st[0], st[1], dres, dx, dg, db, ws)
    assert (~torch.isfinite(dx.float())).any(1).nonzero().flatten().tolist() == [400]
    assert (~torch.isfinite(dg)).nonzero().flatten().tolist() == [D - 1]
