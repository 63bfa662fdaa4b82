"""Low-rank adapters of many requests beside a shared projection, and the plan
that groups a batch by adapter, against their definition in 64 bits."""
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import assert_within
from tests.serving_refs import adapters

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def _data(T, K, N, slots, rank, dt, seed, none=0.2, ids=None):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).to(dt).cuda()

    if ids is None:
        ids = torch.randint(slots, (T,), generator=g)
        ids[torch.rand(T, generator=g) < none] = -1
    return dict(x=r(T, K), a=r(slots, rank, K, scale=K ** -0.5), b=r(slots, N, rank, scale=rank ** -0.5),
                scale=(0.5 + torch.rand(slots, generator=g)).cuda(), res=r(T, N), ids=ids.int().cuda())


def _ops(T, K, N, slots, rank, dt=BF):
    from mixture_experts_ffn_histogram_gb300.layer import AdapterBatch, LowRankAdapters
    return AdapterBatch(T, slots), LowRankAdapters(T, K, N, slots, rank, dtype=dt)


def _check(batch, op, d, res, group=True):
    if group:
        batch.group(d["ids"])
    y = op.forward(batch, d["x"], d["a"], d["b"], d["scale"], res=res)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    want, err = adapters(d["x"], d["a"], d["b"], d["scale"], d["ids"], res)
    assert_within("y", y, want, err)
    none = (d["ids"] < 0) | (d["ids"] >= op.slots)
    assert torch.equal(y[none], res[none] if res is not None else torch.zeros_like(y[none]))
    return y


@pytest.mark.parametrize("T,slots", [(1, 1), (1, 1024), (31, 3), (128, 1), (129, 2), (1000, 7), (5000, 1024),
                                     (32769, 64), (200, 200)])
def test_the_plan(T, slots):
    """Tokens sorted by adapter, stable; tiles of one adapter, up to 128 tokens."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import AdapterBatch
    g = torch.Generator().manual_seed(T + slots)
    batch = AdapterBatch(T, slots)
    for n in (T, T // 2, 0):
        ids = torch.randint(-1, slots, (n,), generator=g)
        if n > 40:
            ids[5:30] = 0
        batch.group(ids.int().cuda())
        torch.cuda.synchronize()
        plan = batch.plan.cpu()
        head = plan[:32].view(torch.int32).tolist()
        most = T // 128 + min(slots + 1, T)
        tiles = plan[32:32 + 16 * most].view(torch.int32).view(-1, 4)[:head[2] + head[3]].tolist()
        order = plan[32 + 16 * most:].view(torch.int32)[:n].long()
        key = torch.where(ids < 0, slots, ids)
        assert head[:2] == [n, slots] and head[4] == int((ids >= 0).sum())
        assert torch.equal(order, torch.argsort(key, stable=True))
        want = []
        at = 0
        for s in range(slots + 1):
            c = int((key == s).sum())
            want += [[s, at + i, min(128, c - i)] for i in range(0, c, 128)]
            at += c
        assert [t[:3] for t in tiles] == want
    assert int(batch.status.item()) == 0


@pytest.mark.parametrize("T,K,N,slots,rank,dt", [
    (1, 64, 64, 1, 8, BF), (1, 7168, 2048, 8, 16, BF), (2, 72, 40, 3, 24, HF), (61, 2816, 2816, 64, 16, HF),
    (17, 512, 1000, 4, 128, BF), (300, 200, 136, 2, 40, BF), (128, 1024, 512, 1, 64, HF), (129, 8, 8, 1, 8, BF),
    (4097, 704, 2816, 5, 32, BF), (2000, 2048, 8, 300, 16, BF), (9000, 320, 520, 2, 64, BF),
    (257, 1600, 96, 3, 24, HF), (300, 1992, 72, 40, 128, BF), (2000, 264, 136, 1024, 8, BF),
])
@pytest.mark.parametrize("with_res", [False, True])
def test_the_adapters(T, K, N, slots, rank, dt, with_res):
    need_gpu()
    d = _data(T, K, N, slots, rank, dt, T + K)
    batch, op = _ops(T, K, N, slots, rank, dt)
    _check(batch, op, d, d["res"] if with_res else None)


def test_all_of_one_adapter_and_none_at_all():
    need_gpu()
    T, K, N, slots, rank = 700, 256, 264, 9, 16
    batch, op = _ops(T, K, N, slots, rank)
    for s in (8, 0, -1):
        d = _data(T, K, N, slots, rank, BF, 5, ids=torch.full((T,), s))
        _check(batch, op, d, d["res"])
    ids = torch.arange(T) // 100 - 1       # runs: the first without an adapter
    d = _data(T, K, N, slots, rank, BF, 6, ids=ids)
    _check(batch, op, d, d["res"])


def test_ids_outside_the_pool_are_reported():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    T, K, N, slots, rank = 50, 128, 128, 4, 8
    ids = torch.arange(T) % 7 - 2          # -2 .. 4
    d = _data(T, K, N, slots, rank, BF, 1, ids=ids)
    batch, op = _ops(T, K, N, slots, rank)
    _check(batch, op, d, d["res"])
    assert int(batch.status.item()) == B.MOE_ERR_DEVICE


def test_in_place_strides_and_fewer_tokens():
    """Rows of wider matrices, y in res's place, calls of different lengths;
    the rows behind the last stay, and results repeat bit for bit."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    T, K, N, slots, rank = 200, 320, 256, 6, 32
    d = _data(T, K, N, slots, rank, BF, 2)
    wide = torch.zeros(T, K + 64, dtype=BF, device="cuda")
    wide[:, 8:K + 8] = d["x"]
    d["x"] = wide[:, 8:K + 8]
    batch, op = _ops(T, K, N, slots, rank)
    first = _check(batch, op, d, d["res"]).clone()
    for _ in range(3):
        assert torch.equal(op.forward(batch, d["x"], d["a"], d["b"], d["scale"], res=d["res"]), first)
    own = d["res"].clone()
    B.moe_adapters(d["x"], d["a"], d["b"], d["scale"], own, own, batch.plan, op.status, op.ws, op.d)
    assert torch.equal(own, first)
    for n in (0, 1, 37, 150):
        op._y.fill_(5.0)
        part = dict(d, x=d["x"][:n], res=d["res"][:n], ids=d["ids"][:n].contiguous())
        y = _check(batch, op, part, part["res"])
        assert y.shape == (n, N) and bool((op._y[n:] == 5.0).all())


def test_a_plan_of_other_tokens_is_reported():
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    T, K, N, slots, rank = 40, 64, 64, 2, 8
    d = _data(T, K, N, slots, rank, BF, 3)
    batch, op = _ops(T, K, N, slots, rank)
    batch.group(d["ids"][:20].contiguous())
    op._y.fill_(5.0)
    B.moe_adapters(d["x"], d["a"], d["b"], d["scale"], d["res"], op._y, batch.plan, op.status, op.ws, op.d)
    torch.cuda.synchronize()
    assert int(op.status.item()) == B.MOE_ERR_DEVICE and bool((op._y == 5.0).all())


def test_another_stream_and_a_graph():
    need_gpu()
    T, K, N, slots, rank = 96, 512, 384, 5, 16
    d = _data(T, K, N, slots, rank, BF, 4)
    batch, op = _ops(T, K, N, slots, rank)
    want = _check(batch, op, d, d["res"]).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    batch.group(d["ids"], stream=side)
    y = op.forward(batch, d["x"], d["a"], d["b"], d["scale"], res=d["res"], stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    ids, x = d["ids"].clone(), d["x"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        batch.group(ids)
        y = op.forward(batch, x, d["a"], d["b"], d["scale"], res=d["res"])
    for seed in (7, 8):
        other = _data(T, K, N, slots, rank, BF, seed)
        ids.copy_(other["ids"])
        x.copy_(other["x"])
        graph.replay()
        torch.cuda.synchronize()
        ref, err = adapters(x, d["a"], d["b"], d["scale"], ids, d["res"])
        assert_within("y", y, ref, err)


def test_one_bad_token_leaves_the_others():
    need_gpu()
    T, K, N, slots, rank = 64, 256, 128, 3, 16
    d = _data(T, K, N, slots, rank, BF, 9, none=0.0)
    batch, op = _ops(T, K, N, slots, rank)
    want = _check(batch, op, d, d["res"]).clone()
    x = d["x"].clone()
    x[5, 1], x[40, 200] = float("nan"), float("inf")
    got = op.forward(batch, x, d["a"], d["b"], d["scale"], res=d["res"])
    keep = [t for t in range(T) if t not in (5, 40)]
    assert torch.equal(got[keep], want[keep])
    assert bool(torch.isnan(got[5]).all()) and not bool(torch.isfinite(got[40]).any())


@pytest.mark.parametrize("T,slots", [(30, 4), (700, 9), (900, 300)])
def test_a_layer_on_its_own_result_and_in_a_graph(T, slots):
    """The result of a call is the rows, and the residual, of the next; one by
    one and captured, with the plan of other ids for each replay."""
    need_gpu()
    K, rank = 328, 24
    d = _data(T, K, K, slots, rank, HF, T)
    batch, op = _ops(T, K, K, slots, rank, HF)
    ids, x = d["ids"].clone(), d["x"].clone()

    def step(a, res):
        return op.forward(batch, a, d["a"], d["b"], d["scale"], res=res)

    def chain():
        batch.group(ids)
        y = step(x, d["res"])
        return step(y, y)

    want = []
    cases = [d["ids"], d["ids"].flip(0).contiguous(), torch.full_like(ids, slots - 1)]
    for i in cases:
        batch.group(i)
        y = step(x, d["res"]).clone()
        want.append(step(y, y).clone())
        ids.copy_(i)
        assert torch.equal(chain(), want[-1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = chain()
    for i, ref in zip(cases, want):
        ids.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    assert int(op.status.item()) == 0
