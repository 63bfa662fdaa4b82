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
