"""A served layer (gate, shared expert with adapters, routed experts, norms
around them) as a run of its operators: against 64-bit mathematics, for few and
single tokens, and captured into a graph over several layers."""
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import act
from tests.serving_refs import adapters, experts, select

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def _weights(D, E, F, S, slots, rank, dt, seed):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0, t=dt, base=0.0):
        return (base + scale * torch.randn(*shape, generator=g)).to(t).cuda()

    f = torch.float32
    return {"wr": r(D, E, scale=D ** -0.5), "wi": r(E, D, 2 * F, scale=D ** -0.5), "wo": r(E, F, D, scale=F ** -0.5),
            "w1": r(D, S, scale=D ** -0.5), "b1": r(S, scale=0.1, t=f), "w2": r(S, D, scale=S ** -0.5),
            "b2": r(D, scale=0.1, t=f), "post": r(D, scale=0.1, t=f), "pre": r(D, scale=0.1, t=f),
            "a": r(slots, rank, S, scale=S ** -0.5), "b": r(slots, D, rank, scale=rank ** -0.5),
            "scale": r(slots, base=1.0, scale=0.1, t=f)}


def _reference(r, u, w, K, ids, logits, name, eps, branch, offset):
    """The layer in 64 bits, the experts chosen by the given logits."""
    d = {k: v.double() for k, v in w.items()}
    h = act(u @ d["w1"] + d["b1"], name)
    s = h @ d["w2"] + d["b2"] + adapters(h, d["a"], d["b"], d["scale"], ids, None)[0]
    chosen, p = select(logits, None, K, "softmax")
    m = experts(u, d["wi"], d["wo"], chosen, p, None, False)[0] + s
    n = m / (m.square().mean(1, keepdim=True) + eps).sqrt() * (d["post"] + offset)
    r = r + branch * n
    return r, r / (r.square().mean(1, keepdim=True) + eps).sqrt() * (d["pre"] + offset)


# At most eight roundings to 16 bits lie on any path from an input to an output
# (h twice, the adapters' v, the results of the products and norms), each of
# relative size eps / 2 at most.
def _near(name, got, want):
    off, limit = (got.double() - want).norm() / want.norm(), 8 * torch.finfo(got.dtype).eps / 2
    assert off <= limit, f"{name}: relative error {float(off):.3g}, limit {limit:.3g}"


@pytest.mark.parametrize("T,dt,slots", [(1, BF, 3), (13, BF, 5), (100, HF, 4), (256, BF, 2)])
def test_the_layer(T, dt, slots):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import AdapterBatch, BlockNorm, DecodeLayer
    D, E, K, F, S, rank, eps, branch, offset = 320, 16, 4, 128, 192, 16, 1e-6, 0.5, 1.0
    lay = DecodeLayer(T, D, E, K, F, S, dtype=dt, eps=eps, branch=branch, offset=offset, slots=slots, rank=rank)
    w = _weights(D, E, F, S, slots, rank, dt, T)
    g = torch.Generator().manual_seed(T)
    r = torch.randn(T, D, generator=g).to(dt).cuda()
    ids = torch.randint(-1, slots, (T,), generator=g).int().cuda()
    batch = AdapterBatch(T, slots)
    batch.group(ids)
    front = BlockNorm(T, D, dtype=dt, eps=eps, offset=offset, train=False)
    u = front.forward(r, pre=w["pre"])
    r1, u1 = lay.forward(r, u, w, batch=batch)
    torch.cuda.synchronize()
    for op in (lay.gate, lay.up, lay.down, lay.adapters, lay.experts, batch):
        assert int(op.status.item()) == 0
    want_r, want_u = _reference(r.double(), u.double(), w, K, ids, lay.gate._y[:T], "silu", eps, branch, offset)
    _near("r", r1, want_r)
    _near("u", u1, want_u)


def test_layers_in_a_graph():
    """Two layers and the front norm captured once; replays on other tokens and
    adapters equal the same calls made one by one."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import AdapterBatch, BlockNorm, DecodeLayer
    T, D, E, K, F, S, slots, rank = 6, 256, 8, 2, 64, 128, 3, 8
    lays = [DecodeLayer(T, D, E, K, F, S, slots=slots, rank=rank) for _ in range(2)]
    ws = [_weights(D, E, F, S, slots, rank, BF, i) for i in range(2)]
    front, batch = BlockNorm(T, D, train=False), AdapterBatch(T, slots)
    r, ids = torch.zeros(T, D, dtype=BF, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")

    def step():
        batch.group(ids)
        a, u = r, front.forward(r, pre=ws[0]["pre"])
        for lay, w in zip(lays, ws):
            a, u = lay.forward(a, u, w, batch=batch)
        return a, u

    g = torch.Generator().manual_seed(3)
    cases = [(torch.randn(T, D, generator=g).to(BF).cuda(), torch.randint(-1, slots, (T,), generator=g).int().cuda())
             for _ in range(3)]
    want = []
    for x, i in cases:
        r.copy_(x)
        ids.copy_(i)
        want.append([v.clone() for v in step()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for (x, i), (a, u) in zip(cases, want):
        r.copy_(x)
        ids.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], a) and torch.equal(out[1], u)
