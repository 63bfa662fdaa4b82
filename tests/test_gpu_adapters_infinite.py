"""Low-rank adapters of tokens with an infinity, at ranks that are no whole
sixteens: the ranks that fill up the last sixteen take no part."""
import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rank", [8, 24, 40, 72])
@pytest.mark.parametrize("T,slots", [(9, 4), (400, 1)])     # rows gathered, and copied
def test_an_infinity_stays_one(T, slots, rank):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import AdapterBatch, LowRankAdapters
    K, N = 640, 72
    g = torch.Generator().manual_seed(rank)

    def positive(*shape):
        return (0.1 + torch.rand(*shape, generator=g)).to(torch.bfloat16).cuda()

    x, a, b = positive(T, K), positive(slots, rank, K), positive(slots, N, rank)
    x[5, 1], x[T - 1, K - 1] = float("inf"), float("-inf")
    ids = (torch.arange(T) % slots).int().cuda()
    op = LowRankAdapters(T, K, N, slots, rank)
    y = op.forward(AdapterBatch(T, slots).group(ids), x, a, b, torch.ones(slots, device="cuda"))
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    assert bool((y[5] == float("inf")).all()) and bool((y[T - 1] == float("-inf")).all())
    rest = [t for t in range(T) if t not in (5, T - 1)]
    assert bool(torch.isfinite(y[rest]).all())
