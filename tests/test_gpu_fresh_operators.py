"""Operators whose workspace holds counters, called on another stream than the
one they were built on as soon as they are built: the buffers that have to be
zero are, whatever the memory held and whatever the building stream still has
to do."""
import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _decode():
    from mixture_experts_ffn_histogram_gb300.layer import MoEDecode
    T, D, E, K, F = 24, 512, 32, 4, 256
    g = torch.Generator().manual_seed(1)
    x, wi, wo = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((T, D), (E, D, 2 * F), (E, F, D)))
    l = torch.randn(T, E, generator=g).cuda()

    def run(stream=None):
        op = MoEDecode(T, D, E, K, F)
        return [op], op.forward(x, wi, wo, logits=l, stream=stream)

    return run


def _adapters():
    from mixture_experts_ffn_histogram_gb300.layer import AdapterBatch, LowRankAdapters
    T, K, N, slots, rank = 200, 1024, 256, 60, 16
    g = torch.Generator().manual_seed(2)
    x, a, b, res = (torch.randn(*s, generator=g).to(BF).cuda()
                    for s in ((T, K), (slots, rank, K), (slots, N, rank), (T, N)))
    ids, scale = torch.randint(-1, slots, (T,), generator=g).int().cuda(), torch.ones(slots, device="cuda")

    def run(stream=None):
        batch, op = AdapterBatch(T, slots), LowRankAdapters(T, K, N, slots, rank)
        return [batch, op], op.forward(batch.group(ids, stream=stream), x, a, b, scale, res=res, stream=stream)

    return run


@pytest.mark.parametrize("make", [_decode, _adapters])
def test_called_at_once_on_another_stream(make):
    need_gpu()
    run = make()
    ops, out = run()
    torch.cuda.synchronize()
    want = out.clone()
    for op in ops:      # the memory that the next ones are built in
        for name in ("ws", "plan", "status"):
            t = getattr(op, name, None)
            if t is not None:
                t.view(torch.uint8).fill_(255)
    del ops, op, t, out
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)       # some 25 ms of work of the building stream
    ops, out = run(side)
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert [int(op.status.item()) for op in ops] == [0] * len(ops)
