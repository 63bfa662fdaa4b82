"""What the operators that keep counters in their workspaces leave there, and
that no call reads what an earlier one left: each call's tokens, weights and
routing differ from those of the calls before, and its result is that of an
operator just built, bit for bit."""
import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _decode_flags(op):
    """The counters, the blocks' flags and the tiles' flags of a MoEDecode: by the
    capacity, as the kernel's host side lays them out."""
    slots = op.T * op.K
    tiles = min(slots, op.E + slots // 64) * (op.F // 64)
    return op.ws[:1024 + 4 * tiles]


# runs of blocks that meet inside tiles; whole tiles; claimed tiles; one tile to an expert and several
@pytest.mark.parametrize("T,D,E,K,F", [(1, 704, 40, 8, 320), (6, 1024, 40, 4, 512), (24, 1088, 96, 6, 192),
                                       (200, 256, 5, 2, 128)])
@pytest.mark.parametrize("mode", [0, 2])
def test_the_expert_layer(T, D, E, K, F, mode):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import MoEDecode
    g = torch.Generator().manual_seed(T + mode)
    op = MoEDecode(T, D, E, K, F, mode)
    for n in (T, T, max(1, T // 2), T, 1, T):
        x, wi, wo = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((n, D), (E, D, 2 * F), (E, F, D)))
        if mode == 2:
            how = dict(ids=torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(n)]).int().cuda(),
                       w=torch.rand(n, K, generator=g).cuda())
        else:
            how = dict(logits=torch.randn(n, E, generator=g).cuda())
        out = op.forward(x, wi, wo, **how)
        fresh = MoEDecode(T, D, E, K, F, mode)
        assert torch.equal(out, fresh.forward(x, wi, wo, **how))
        torch.cuda.synchronize()
        assert not bool(_decode_flags(op).any())
        assert int(op.status.item()) == 0


# the reduction cut, its parts joined by the last to arrive; by a kernel of their own; not cut
@pytest.mark.parametrize("T,K,N,slots,rank", [(61, 2816, 264, 30, 16), (900, 2048, 264, 400, 24),
                                              (130, 2048, 264, 1, 24), (256, 1024, 264, 7, 8),
                                              (1500, 2048, 136, 3, 64), (5000, 192, 136, 2, 32)])
def test_the_adapters(T, K, N, slots, rank):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import AdapterBatch, LowRankAdapters
    g = torch.Generator().manual_seed(T)
    batch, op = AdapterBatch(T, slots), LowRankAdapters(T, K, N, slots, rank)
    counters = op.ws[:4 * (T // 128 + min(slots + 1, T))]
    for n in (T, T, max(1, T // 3), T, 1, T):
        x, a, b, res = (torch.randn(*s, generator=g).to(BF).cuda()
                        for s in ((n, K), (slots, rank, K), (slots, N, rank), (n, N)))
        ids = torch.randint(-1, slots, (n,), generator=g).int().cuda()
        scale = torch.rand(slots, generator=g).cuda()
        y = op.forward(batch.group(ids), x, a, b, scale, res=res)
        fresh = LowRankAdapters(T, K, N, slots, rank)
        own = AdapterBatch(T, slots).group(ids)
        assert torch.equal(y, fresh.forward(own, x, a, b, scale, res=res))
        torch.cuda.synchronize()
        assert not bool(counters.any())
        assert int(op.status.item()) == 0 and int(batch.status.item()) == 0
