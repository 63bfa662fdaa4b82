"""The linear layer's activations where they could hide or lose something:
NaN rows, far tails, the largest numbers."""
import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,dt,out", [(3, BF, BF), (40, HF, HF), (300, BF, F32), (1100, BF, BF)])
def test_a_nan_row_stays_nan(name, M, dt, out):
    """A NaN in a row of x reaches that row of y, z and dx, and no other."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import Linear
    K, N = 328, 1032
    g = torch.Generator().manual_seed(M)
    x, w = torch.randn(M, K, generator=g).to(dt).cuda(), (K ** -0.5 * torch.randn(K, N, generator=g)).to(dt).cuda()
    x[1, 3] = float("nan")
    op = Linear(M, K, N, dt, out, act=name, train=True)
    y = op.forward(x, w)
    rows = torch.arange(M, device="cuda") == 1
    assert torch.equal(torch.isnan(y), rows[:, None].expand(M, N))
    if name == "none":
        return
    assert torch.equal(torch.isnan(op.z), rows[:, None].expand(M, N))
    dx = op.backward(torch.randn(M, N, generator=g).to(out).cuda(), x, w)
    assert torch.equal(torch.isnan(dx), rows[:, None].expand(M, K))
    assert bool(torch.isnan(op.db).all())


@pytest.mark.parametrize("dt,low", [(BF, -13.0), (HF, -5.8)])
def test_the_tail_of_gelu(dt, low):
    """Value and slope far below zero, where both are tiny: to half a step of
    the result.  (About the slope's zero at -0.75 an absolute bound holds.)"""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import Linear
    n = 64
    x = torch.linspace(low, -1.5, 64 * n).to(dt).view(-1, n).cuda()
    w = torch.eye(n).to(dt).cuda()
    op = Linear(x.shape[0], n, n, dt, act="gelu", train=True)
    y = op.forward(x, w)
    assert torch.equal(op.z, x)
    dx = op.backward(torch.ones_like(x), x, w)
    z = x.double()
    cdf = 0.5 * torch.erfc(-z / 2 ** 0.5)
    pdf = torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    # the tail's polynomial, some ten roundings, the exponential's argument
    # (z^2/2 log2 e, 1.5 roundings of it), and the result's own rounding
    own = 2.0 ** -17 + 10 * 2.0 ** -24 + 1.5 * z * z * 2.0 ** -24
    half = torch.finfo(dt).eps / 2 * (1 + 2.0 ** -8)
    sub = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    for name, got, want, mag in (("gelu", y, z * cdf, z.abs() * cdf),
                                 ("slope", dx, cdf + z * pdf, cdf + z.abs() * pdf)):
        off = (got.double() - want).abs() - (half * want.abs() + sub + own * mag)
        assert float(off.max()) <= 0, f"{name}: at z = {float(z.flatten()[off.flatten().argmax()])}"


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", [BF, HF])
def test_the_largest_numbers(name, dt):
    """act(z) = z and act'(z) = 1 far above zero, 0 and 0 far below, up to the
    type's largest and lowest number."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import Linear
    n, most = 64, torch.finfo(dt).max
    x = torch.logspace(2.4, torch.tensor(most).double().log10().item(), 4 * n, dtype=torch.float64).clamp(max=most)
    x = torch.cat([x, -x]).to(dt).view(-1, n).cuda()
    w = torch.eye(n).to(dt).cuda()
    op = Linear(x.shape[0], n, n, dt, act=name, train=True)
    y = op.forward(x, w)
    up = x > 0 if name != "none" else torch.ones_like(x, dtype=torch.bool)
    assert torch.equal(y, torch.where(up, x, torch.zeros_like(x)))
    if name == "none":
        return
    assert torch.equal(op.z, x)
    dx = op.backward(torch.ones_like(x), x, w, need_dw=False)
    assert torch.equal(dx, up.to(dt))
    assert torch.equal(op.db, up.float().sum(0))
