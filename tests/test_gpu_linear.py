"""The linear layer forward and backward against 64 bits: rows from one to
many, ragged sizes, row strides, each type, activation and epilogue, in-place
residual, no rows, bad rows, graphs."""
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import ACT_ERR, MAX_SLOPE, U32, act, act_slope, assert_within, half_step, sum_error

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

# M, K, N, type, out, act, bias, res, pad of every row stride
CASES = [
    (1, 8, 8, BF, BF, "none", False, False, 0),
    (1, 2048, 768, BF, BF, "silu", True, True, 0),
    (4, 7168, 256, HF, HF, "gelu", True, False, 0),
    (16, 72, 200, BF, BF, "relu", True, True, 8),
    (17, 520, 136, BF, BF, "gelu_tanh", True, True, 0),
    (33, 1000, 1000, HF, HF, "silu", False, True, 16),
    (64, 256, 2816, BF, BF, "none", True, False, 0),
    (65, 64, 64, BF, BF, "gelu", True, True, 0),
    (127, 200, 328, HF, HF, "none", False, True, 8),
    (129, 704, 392, BF, BF, "silu", True, True, 0),
    (300, 2048, 768, BF, BF, "gelu", True, False, 0),
    (1, 2816, 128, BF, F32, "none", False, False, 0),
    (40, 1536, 64, HF, F32, "gelu", True, True, 0),
    (333, 7168, 256, BF, F32, "silu", True, True, 8),
    (200, 4104, 72, BF, F32, "gelu_tanh", True, True, 0),
    (1030, 520, 1032, BF, BF, "silu", True, True, 0),
    (2100, 328, 1544, HF, HF, "gelu", True, True, 8),
    (4100, 704, 2816, BF, BF, "none", True, True, 0),
    # shapes of the pair kernel's narrower tiles, in one of the three products each
    (4096, 1096, 760, BF, BF, "gelu", True, False, 0),
    (4096, 1032, 1160, HF, HF, "none", True, True, 8),
    (1100, 4224, 760, BF, BF, "silu", True, True, 0),
    (700, 4096, 1152, BF, BF, "none", False, True, 0),
    (4096, 520, 1096, BF, BF, "relu", True, True, 8),
]


def _rand(g, n, m, dt, pad, scale=1.0):
    return (scale * torch.randn(n, m + pad, generator=g)).to(dt).cuda()[:, :m]


def _inputs(M, K, N, dt, out, bias, res, pad):
    g = torch.Generator().manual_seed(M * 31 + K * 7 + N)
    return {
        "x": _rand(g, M, K, dt, pad), "w": _rand(g, K, N, dt, pad, K ** -0.5),
        "bias": torch.randn(N, generator=g).cuda() if bias else None,
        "res": _rand(g, M, N, out, pad) if res else None,
        "dy": _rand(g, M, N, out, pad), "dx_add": _rand(g, M, K, dt, pad) if res else None,
    }


def check_forward(i, y, z, name, dt, out):
    x, w = i["x"].double(), i["w"].double()
    K = x.shape[1]
    zr, mag = x @ w, x.abs() @ w.abs()
    if i["bias"] is not None:
        zr = zr + i["bias"].double()
        mag = mag + i["bias"].double().abs()
    err = sum_error(K, out == F32) * mag
    if z is not None:
        assert_within("z", z, zr, err)
    yr = act(zr, name)
    # fp32 results use the accurate functions: a few ulp of the value
    own = 0.0 if name == "none" else (16 * U32 if out == F32 else ACT_ERR) * (1 + zr.abs())
    if i["res"] is not None:
        yr = yr + i["res"].double()
        own = own + 2 * U32 * i["res"].double().abs()
    assert_within("y", y, yr, MAX_SLOPE * err + own + U32 * yr.abs())


def check_backward(i, z, dx, dw, db, name, dt):
    x, w, dy = i["x"].double(), i["w"].double(), i["dy"].double()
    dz, dze = dy, torch.zeros_like(dy)
    if name != "none":
        zd = z.double()
        dz = dy * act_slope(zd, name)
        dze = dy.abs() * ACT_ERR * (1 + zd.square())
    u = half_step(dt) * (1 + 2.0 ** -8)
    rounded = dze + (u * dz.abs() + 2.0 ** -25 if dt == HF else u * dz.abs())
    if name == "none" and i["dy"].dtype == dt:
        rounded = dze
    if dx is not None:
        want = dz @ w.t()
        lim = rounded @ w.t().abs() + sum_error(w.shape[1], False) * (dz.abs() @ w.t().abs())
        if i["dx_add"] is not None:
            want = want + i["dx_add"].double()
            lim = lim + 2 * U32 * want.abs()
        assert_within("dx", dx, want, lim)
    if dw is not None:
        lim = x.t().abs() @ rounded + sum_error(x.shape[0], False) * (x.t().abs() @ dz.abs())
        assert_within("dw", dw, x.t() @ dz, lim)
    if db is not None:
        # sums of at most rows / 64 terms in a row, then trees
        lim = dze.sum(0) + (64 + dz.shape[0] / 64) * U32 * dz.abs().sum(0)
        assert_within("db", db, dz.sum(0), lim)


@pytest.mark.parametrize("M,K,N,dt,out,name,bias,res,pad", CASES)
def test_forward(M, K, N, dt, out, name, bias, res, pad):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    i = _inputs(M, K, N, dt, out, bias, res, pad)
    y = torch.full((M, N + pad), 7.0, dtype=out, device="cuda")
    z = torch.full((M, N + pad), 7.0, dtype=dt, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = B.linear_dims(M, K, N, dt, out, name)
    B.moe_linear(i["x"], i["w"], i["bias"], i["res"], y[:, :N], z[:, :N], st, d)
    assert int(st.item()) == 0
    check_forward(i, y[:, :N], z[:, :N], name, dt, out)
    assert (y[:, N:] == 7).all() and (z[:, N:] == 7).all()  # nothing beside the rows
    y2 = torch.empty((M, N), dtype=out, device="cuda")
    B.moe_linear(i["x"], i["w"], i["bias"], i["res"], y2, None, st, d)
    assert torch.equal(y2, y[:, :N])
    if res:  # in place over the residual
        r = i["res"]
        B.moe_linear(i["x"], i["w"], i["bias"], r, r, None, st, d)
        assert torch.equal(r, y2)


@pytest.mark.parametrize("M,K,N,dt,out,name,bias,res,pad", CASES)
def test_backward(M, K, N, dt, out, name, bias, res, pad):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    i = _inputs(M, K, N, dt, out, bias, res, pad)
    z = (i["x"].float() @ i["w"].float()).to(dt) if name != "none" else None
    d = B.linear_dims(M, K, N, dt, out, name)
    ws = torch.empty(B.moe_linear_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    dx = torch.full((M, K + pad), 7.0, dtype=dt, device="cuda")
    dw = torch.full((K, N + pad), 7.0, dtype=dt, device="cuda")
    db = torch.empty(N, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_linear_bwd(i["dy"], z, i["x"], i["w"], i["dx_add"], dx[:, :K], dw[:, :N], db, st, ws, d)
    assert int(st.item()) == 0
    check_backward(i, z, dx[:, :K], dw[:, :N], db, name, dt)
    assert (dx[:, K:] == 7).all() and (dw[:, N:] == 7).all()
    # each gradient alone is the same
    dx2, dw2, db2 = (torch.empty((M, K), dtype=dt, device="cuda"),
                     torch.empty((K, N), dtype=dt, device="cuda"), torch.empty(N, device="cuda"))
    B.moe_linear_bwd(i["dy"], z, None, i["w"], i["dx_add"], dx2, None, None, st, ws, d)
    B.moe_linear_bwd(i["dy"], z, i["x"], None, None, None, dw2, None, st, ws, d)
    B.moe_linear_bwd(i["dy"], z, None, None, None, None, None, db2, st, ws, d)
    assert torch.equal(dx2, dx[:, :K]) and torch.equal(dw2, dw[:, :N]) and torch.equal(db2, db)


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", [BF, HF])
def test_activations_over_their_range(name, dt):
    """Pre-activations from -60 to 60 through the value (an identity weight)
    and the slope."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import Linear
    n = 64
    v = torch.cat([torch.linspace(-60, 60, 4096), torch.linspace(-6, 6, 4096),
                   torch.tensor([0.0, -0.0, 1e-6, -1e-6] * 16)])
    x = v.to(dt).view(-1, n).cuda()
    w = torch.eye(n).to(dt).cuda()
    op = Linear(x.shape[0], n, n, dt, act=name, train=True)
    y = op.forward(x, w)
    check_forward({"x": x, "w": w, "bias": None, "res": None}, y, op.z, name, dt, dt)
    dy = torch.ones_like(x)
    dx = op.backward(dy, x, w)
    check_backward({"x": x, "w": w, "dy": dy, "dx_add": None}, op.z, dx, op.dw, op.db, name, dt)


def test_gradient_against_differences():
    """The backward's formula (64 bits) against central differences of the
    forward's; the kernels are held to the formula above."""
    g = torch.Generator().manual_seed(0)
    z = 3 * torch.randn(400, generator=g, dtype=torch.float64)
    for name in ("gelu", "gelu_tanh", "silu"):
        h = 1e-5
        num = (act(z + h, name) - act(z - h, name)) / (2 * h)
        assert (num - act_slope(z, name)).abs().max() < 1e-9


def test_no_rows():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import Linear
    op = Linear(16, 64, 128, act="silu", train=True)
    x, w = torch.empty(0, 64, device="cuda").bfloat16(), torch.ones(64, 128, device="cuda").bfloat16()
    assert op.forward(x, w).shape == (0, 128)
    op.dw.fill_(3.0)
    op.db.fill_(3.0)
    dx = op.backward(torch.empty(0, 128, device="cuda").bfloat16(), x, w)
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and not op.dw.any() and not op.db.any()


@pytest.mark.parametrize("M", [3, 40, 300, 1100])
def test_a_bad_row_stays_alone(M):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import Linear
    i = _inputs(M, 328, 1032, BF, BF, True, True, 0)
    i["x"][1, 3] = float("nan")
    i["res"][2, 7] = float("inf")
    op = Linear(M, 328, 1032, act="none")
    y = op.forward(i["x"], i["w"], i["bias"], i["res"])
    bad = ~torch.isfinite(y.float())
    assert bad[1].all() and bad[2].nonzero().flatten().tolist() == [7]
    assert int(bad.sum()) == 1032 + 1


@pytest.mark.parametrize("M", [5, 700])
def test_reproducible_other_stream_and_graph(M):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import Linear
    i = _inputs(M, 1032, 520, BF, BF, True, True, 0)
    op = Linear(M, 1032, 520, act="gelu", train=True)

    def step(stream=None):
        y = op.forward(i["x"], i["w"], i["bias"], i["res"], stream=stream)
        dx = op.backward(i["dy"], i["x"], i["w"], dx_add=i["dx_add"], stream=stream)
        return [y, op.z, dx, op.dw, op.db]

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
