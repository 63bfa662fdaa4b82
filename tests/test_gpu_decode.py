"""The expert layer for a few tokens against its definition in 64
bits: sizes, types, routings, and how it is called."""
import pytest
import torch

from tests.gpu_common import need_gpu
from tests.layer_refs import assert_within
from tests.serving_refs import experts, select

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
MODES = {"softmax": 0, "sigmoid": 1, "given": 2}


def _op(T, D, E, K, F, mode, dt=BF):
    from mixture_experts_ffn_histogram_gb300.layer import MoEDecode
    return MoEDecode(T, D, E, K, F, MODES[mode], dtype=dt)


def _data(T, D, E, K, F, dt, seed):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).to(dt).cuda()

    return dict(x=r(T, D), wi=r(E, D, 2 * F, scale=D ** -0.5), wo=r(E, F, D, scale=F ** -0.5), res=r(T, D),
                logits=torch.randn(T, E, generator=g).cuda(), bias=(0.5 * torch.randn(E, generator=g)).cuda(),
                w=torch.rand(T, K, generator=g).cuda(),
                ids=torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int().cuda())


def _check(op, d, ids, w, res, out, own):
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    want, err = experts(d["x"], d["wi"], d["wo"], ids, w, res, own)
    assert_within("out", out, want, err)
    assert not bool(op.ws[:1024].any())


@pytest.mark.parametrize("T,D,E,K,F,dt,mode", [
    (1, 64, 1, 1, 64, BF, "softmax"),            # one tile, one block
    (1, 256, 8, 2, 512, BF, "softmax"),
    (1, 2816, 128, 8, 704, BF, "softmax"),       # D no whole number of tiles
    (3, 448, 16, 4, 192, HF, "sigmoid"),
    (16, 2048, 128, 8, 768, BF, "sigmoid"),
    (17, 512, 60, 5, 320, BF, "given"),          # tiles of 32 tokens
    (33, 320, 4, 4, 128, HF, "given"),           # tiles of 64: every expert has all tokens
    (100, 256, 256, 8, 192, BF, "softmax"),
    (200, 192, 3, 2, 64, BF, "sigmoid"),         # more than 64 tokens to an expert
    (256, 128, 1000, 8, 64, BF, "softmax"),      # many experts
    (64, 128, 64, 32, 64, HF, "sigmoid"),        # the most slots to a token
    (5, 7168, 16, 3, 2048, BF, "given"),
])
@pytest.mark.parametrize("res", [False, True])
def test_the_layer(T, D, E, K, F, dt, mode, res):
    need_gpu()
    d = _data(T, D, E, K, F, dt, T + D)
    op = _op(T, D, E, K, F, mode, dt)
    r = d["res"] if res else None
    if mode == "given":
        out = op.forward(d["x"], d["wi"], d["wo"], ids=d["ids"], w=d["w"], res=r)
        return _check(op, d, d["ids"], d["w"], r, out, False)
    bias = d["bias"] if res else None
    out = op.forward(d["x"], d["wi"], d["wo"], logits=d["logits"], bias=bias, res=r)
    ids, w = select(d["logits"], bias, K, mode)
    assert torch.equal(op.ids, ids)
    assert_within("w", op.w, w, (K + 12) * 2.0 ** -24 * w)
    _check(op, d, ids, w, r, out, True)


def test_equal_scores_and_masked_experts():
    """Equal scores take the lower expert; experts at -inf are taken last, with
    weight 0, and their rows are still finite."""
    need_gpu()
    T, D, E, K, F = 6, 128, 40, 6, 64
    d = _data(T, D, E, K, F, BF, 5)
    l = torch.zeros(T, E, device="cuda")
    l[1] = -0.0
    l[1, 20:] = 0.0
    l[2, 3:] = float("-inf")
    l[3, ::2] = torch.finfo(torch.float32).min
    l[4, 30:] = 2.0
    l[5] = torch.arange(E, device="cuda").flip(0) // 3
    op = _op(T, D, E, K, F, "softmax")
    out = op.forward(d["x"], d["wi"], d["wo"], logits=l)
    ids, w = select(l, None, K, "softmax")
    assert torch.equal(op.ids, ids)
    _check(op, d, ids, w, None, out, True)
    assert float(op.w[2, 3:].abs().max()) == 0.0


def test_an_expert_named_more_than_once_by_a_token():
    need_gpu()
    T, D, E, K, F = 40, 256, 6, 5, 128
    d = _data(T, D, E, K, F, BF, 9)
    ids = torch.randint(E, (T, K), generator=torch.Generator().manual_seed(1)).int().cuda()
    ids[3] = 2
    op = _op(T, D, E, K, F, "given")
    out = op.forward(d["x"], d["wi"], d["wo"], ids=ids, w=d["w"])
    _check(op, d, ids, d["w"], None, out, False)


@pytest.mark.parametrize("res", [False, True])
def test_ids_outside_the_experts_are_reported_and_dropped(res):
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    T, D, E, K, F = 9, 192, 8, 3, 64
    d = _data(T, D, E, K, F, BF, 3)
    ids = d["ids"].clone()
    ids[0, 1], ids[4], ids[8, 0] = -1, E, 2 ** 30
    r = d["res"] if res else None
    op = _op(T, D, E, K, F, "given")
    out = op.forward(d["x"], d["wi"], d["wo"], ids=ids, w=d["w"], res=r)
    torch.cuda.synchronize()
    assert int(op.status.item()) == B.MOE_ERR_DEVICE
    want, err = experts(d["x"], d["wi"], d["wo"], ids, d["w"], r, False)
    assert_within("out", out, want, err)
    assert torch.equal(out[4], r[4] if res else torch.zeros_like(out[4]))
    # none at all
    op.status.zero_()
    out = op.forward(d["x"], d["wi"], d["wo"], ids=torch.full_like(ids, -1), w=d["w"], res=r)
    torch.cuda.synchronize()
    assert torch.equal(out, r if res else torch.zeros_like(out))


def test_fewer_tokens_strides_and_reproducible_results():
    """Calls of different lengths through one operator, from columns of wider
    rows: the rows behind the last stay, results repeat bit for bit, and the
    counters are left for the next call."""
    need_gpu()
    T, D, E, K, F = 48, 640, 32, 4, 256
    d = _data(T, D, E, K, F, BF, 11)
    wide = torch.randn(T, D + 64, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    x, res = wide[:, 32:D + 32], torch.cat([d["res"], d["res"]], 1)[:, D:]
    d["x"] = x
    op = _op(T, D, E, K, F, "softmax")
    first = op.forward(x, d["wi"], d["wo"], logits=d["logits"], res=res).clone()
    ids, w = select(d["logits"], None, K, "softmax")
    _check(op, d, ids, w, res, first, True)
    for n in (1, 7, 0, 48, 31):
        op._out.fill_(7.0)
        out = op.forward(x[:n], d["wi"], d["wo"], logits=d["logits"][:n], res=res[:n])
        assert out.shape == (n, D) and torch.equal(out[:n], op._out[:n])
        assert bool((op._out[n:] == 7.0).all())
        want, err = experts(x[:n], d["wi"], d["wo"], ids[:n], w[:n], res[:n], True)
        assert_within("out", out, want, err)
    for _ in range(5):
        assert torch.equal(op.forward(x, d["wi"], d["wo"], logits=d["logits"], res=res), first)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0


def test_claimed_tiles_repeat_bit_for_bit():
    """Enough tiles that CTAs claim them one by one: whoever takes one, the
    result is the same; shorter calls through the same operator in between."""
    need_gpu()
    T, D, E, K, F = 24, 1088, 96, 6, 192
    d = _data(T, D, E, K, F, BF, 31)
    op = _op(T, D, E, K, F, "sigmoid")
    first = op.forward(d["x"], d["wi"], d["wo"], logits=d["logits"], res=d["res"]).clone()
    ids, w = select(d["logits"], None, K, "sigmoid")
    assert len(set(ids.flatten().tolist())) * ((D + 127) // 128) >= 4 * 152
    _check(op, d, ids, w, d["res"], first, True)
    for n in (24, 1, 24, 12, 24):
        out = op.forward(d["x"][:n], d["wi"], d["wo"], logits=d["logits"][:n], res=d["res"][:n])
        if n == T:
            assert torch.equal(out, first)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0 and not bool(op.ws[:1024].any())


def test_another_stream_and_a_graph():
    need_gpu()
    T, D, E, K, F = 8, 512, 16, 4, 256
    d = _data(T, D, E, K, F, BF, 21)
    op = _op(T, D, E, K, F, "softmax")
    want = op.forward(d["x"], d["wi"], d["wo"], logits=d["logits"]).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = op.forward(d["x"], d["wi"], d["wo"], logits=d["logits"], stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    x, l = d["x"].clone(), d["logits"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = op.forward(x, d["wi"], d["wo"], logits=l)
    for seed in (1, 2):
        other = _data(T, D, E, K, F, BF, seed)
        x.copy_(other["x"])
        l.copy_(other["logits"])
        graph.replay()
        torch.cuda.synchronize()
        ids, w = select(l, None, K, "softmax")
        ref, err = experts(x, d["wi"], d["wo"], ids, w, None, True)
        assert_within("out", out, ref, err)
    assert int(op.status.item()) == 0


def test_one_bad_token_leaves_the_others():
    """A NaN or infinity in one token reaches that token's row alone."""
    need_gpu()
    T, D, E, K, F = 20, 256, 4, 2, 128
    d = _data(T, D, E, K, F, BF, 8)
    op = _op(T, D, E, K, F, "given")
    want = op.forward(d["x"], d["wi"], d["wo"], ids=d["ids"], w=d["w"]).clone()
    x = d["x"].clone()
    x[3, 7], x[11, 0] = float("nan"), float("inf")
    got = op.forward(x, d["wi"], d["wo"], ids=d["ids"], w=d["w"])
    keep = [t for t in range(T) if t not in (3, 11)]
    assert torch.equal(got[keep], want[keep])
    assert bool(torch.isnan(got[3]).all()) and not bool(torch.isfinite(got[11]).any())


def test_two_layers_at_once_and_among_other_kernels():
    """Layers on streams of their own, each of which wants all SMs at once, with
    products and copies in between: every result as when alone, no wait given
    up."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300.layer import Linear
    T, D, E, K, F = 12, 512, 32, 4, 256
    cases = [_data(T, D, E, K, F, BF, i) for i in range(3)]
    ops = [_op(T, D, E, K, F, "softmax") for _ in cases]
    lins = [Linear(300, D, 1024) for _ in cases]
    wide = [torch.randn(300, D, device="cuda").to(BF) for _ in cases]
    w = torch.randn(D, 1024, device="cuda").to(BF)
    want = [op.forward(d["x"], d["wi"], d["wo"], logits=d["logits"]).clone() for op, d in zip(ops, cases)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    for i in range(60):
        for op, d, lin, x, ref, s in zip(ops, cases, lins, wide, want, streams):
            with torch.cuda.stream(s):
                if i % 3 == 0:
                    lin.forward(x, w)
                out = op.forward(d["x"], d["wi"], d["wo"], logits=d["logits"])
                if i % 20 == 19:
                    wrong.add_((out != ref).sum())
    torch.cuda.synchronize()
    assert [int(op.status.item()) for op in ops] == [0, 0, 0]
    assert int(wrong.item()) == 0


@pytest.mark.parametrize("T", [9, 40])   # selected by every block, and exchanged between them
@pytest.mark.parametrize("mode", ["softmax", "sigmoid"])
def test_odd_scores_select_as_the_block_does(T, mode):
    """Rows with NaN and infinities, all masked or all equal: the ids and weights
    of the block's routing."""
    need_gpu()
    from mixture_experts_ffn_histogram_gb300 import binding as B
    D, E, K, F = 64, 70, 6, 64
    d = _data(T, D, E, K, F, BF, 13)
    l, inf = d["logits"], float("inf")
    l[0], l[1, 3], l[2, 5], l[3] = -inf, float("nan"), inf, float("nan")
    l[4, 4:], l[5], l[6, :10], l[7, 66:] = -inf, torch.finfo(torch.float32).min, inf, float("nan")
    l[8] = 200.0 * l[8]
    op = _op(T, D, E, K, F, mode)
    dims = B.dims(T, D, E, K, F)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.empty(T, K, **i32), torch.empty(T, K, device="cuda")
    ws = torch.zeros(B.moe_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    for bias in (d["bias"], None):
        op.forward(d["x"], d["wi"], d["wo"], logits=l, bias=bias)
        B.moe_route_histogram(l, bias, MODES[mode], ids, w, torch.empty(E, **i32), torch.empty(E + 1, **i32),
                              torch.empty(T, K, **i32), torch.empty(T * K, **i32), torch.zeros(1, **i32), ws, dims)
        torch.cuda.synchronize()
        assert torch.equal(op.ids, ids) and int(op.status.item()) == 0
        # each is within its own bound of the exact weight
        assert torch.allclose(op.w, w, rtol=2 * (K + 12) * 2.0 ** -24, atol=2.0 ** -126, equal_nan=True)


def test_the_layer_on_its_own_result():
    """The result of a call is the rows, and the residual, of the next."""
    need_gpu()
    for T in (1, 7, 90):
        d = _data(T, 192, 12, 3, 128, BF, T)
        op = _op(T, 192, 12, 3, 128, "softmax")

        def step(x, res):
            return op.forward(x, d["wi"], d["wo"], logits=d["logits"], res=res)

        first = step(d["x"], None).clone()
        want = step(first, first).clone()
        assert torch.equal(step(step(d["x"], None), op._out), want)
