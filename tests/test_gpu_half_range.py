"""What is held in 16 bits between the two products, at the border of fp16's
range: right up to it, infinite past it in that token's result alone; bf16 has
fp32's range."""
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import assert_within
from tests.serving_refs import adapters, experts

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def _hold(out, want, err, over):
    """Finite and right but for the rows `over`, of which nothing is."""
    keep = [t for t in range(out.shape[0]) if t not in over]
    assert_within("out", out[keep], want[keep], err[keep])
    assert not bool(torch.isfinite(out[over]).any())


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("T", [3, 20])
def test_the_expert_layer(T, dt):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import MoEDecode
    D, E, K, F = 128, 4, 2, 192
    g = torch.Generator().manual_seed(T)
    x = torch.zeros(T, D)
    x[:, 0] = 200.0 * torch.rand(T, generator=g)
    x[0, 0], x[1, 0], x[2, 0] = 255.0, 1.0, 257.0      # h is about their squares: 65025, ..., 66049
    wi, wo = torch.zeros(E, D, 2 * F), 2.0 ** -12 * torch.rand(E, F, D, generator=g) + 2.0 ** -12
    wi[:, 0] = 1.0
    x, wi, wo = x.to(dt).cuda(), wi.to(dt).cuda(), wo.to(dt).cuda()
    l = torch.randn(T, E, generator=g).cuda()
    op = MoEDecode(T, D, E, K, F, dtype=dt)
    out = op.forward(x, wi, wo, logits=l)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    want, err = experts(x, wi, wo, op.ids, op.w, None, True)
    _hold(out, want, err, [2] if dt is HF else [])


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("T", [6, 400])
def test_the_adapters(T, dt):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import AdapterBatch, LowRankAdapters
    K, N, slots, rank = 64, 136, 2, 8
    g = torch.Generator().manual_seed(T)
    x = torch.zeros(T, K)
    x[:, 0] = 200.0 * torch.rand(T, generator=g)
    x[0, 0], x[1, 0], x[2, 0] = 255.0, 257.0, 128.0
    a, b = torch.zeros(slots, rank, K), 2.0 ** -12 * torch.rand(slots, N, rank, generator=g) + 2.0 ** -12
    a[:, :, 0] = 256.0
    scale = torch.tensor([1.0, 2.0]).cuda()
    ids = torch.zeros(T, dtype=torch.int32)
    ids[2], ids[3] = 1, -1                  # 65280, 65792, twice 32768
    x, a, b, ids = x.to(dt).cuda(), a.to(dt).cuda(), b.to(dt).cuda(), ids.cuda()
    op = LowRankAdapters(T, K, N, slots, rank, dtype=dt)
    y = op.forward(AdapterBatch(T, slots).group(ids), x, a, b, scale)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    want, err = adapters(x, a, b, scale, ids, None)
    _hold(y, want, err, [1, 2] if dt is HF else [])
