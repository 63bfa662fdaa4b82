"""The operators around the expert block, and a whole layer of them.

``LayerNorm`` (with the residual add in front of it), ``TopKRouter`` (expert
selection with a balance bias and expert groups) and ``Linear`` (bias,
activation and residual in the product's epilogue) each own their output
buffers and workspace, like ``MoEBlock``: allocated once for a largest number
of rows, written by every call (a call's outputs are views of them and hold
until the next one).  Calls run on the current stream, or the one given.

``MoELayer`` runs them together with the expert block as one pre-norm
feed-forward layer, forward and backward.
"""
from __future__ import annotations

import torch

from . import binding as B
from .block import MoEBlock


def _check(name, t, shape, dtype, device):
    """A tensor of another shape, type or device would be read (or written)
    out of bounds or misread: reject it before any launch."""
    if t.dtype != dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on {device}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} needs contiguous columns, got strides {list(t.stride())}")


def _launchable(device):
    if device.type != "cuda":
        raise RuntimeError(f"the operator's buffers are on {device}: its kernels need a CUDA device")


def _rows(name, t, cap, width):
    if t.dim() != 2 or t.shape[1] != width or t.shape[0] > cap:
        raise ValueError(f"{name} must be [rows <= {cap}, {width}], got {list(t.shape)}")
    return t.shape[0]


class LayerNorm:
    """y = norm(x + res) * gamma + beta over rows of D, up to ``rows`` of them.

    ``forward`` leaves r = x + res (rounded to the rows' type) in ``r`` when
    res is given, and with ``train`` the rows' ``mean`` and ``rstd``.
    ``backward`` takes the normalised rows (r, or x without a residual) and
    returns dx, the gradient of x and res alike; ``dgamma`` and ``dbeta`` hold
    the weights' gradients."""

    def __init__(self, rows, D, dtype=torch.bfloat16, weight_dtype=torch.float32, eps=1e-5,
                 train=True, device="cuda"):
        if dtype not in B.DTYPES or weight_dtype not in (dtype, torch.float32):
            raise ValueError(f"rows of {dtype} with weights of {weight_dtype} are not supported")
        self.rows, self.D, self.dtype, self.weight_dtype = rows, D, dtype, weight_dtype
        self.eps, self.train = eps, train
        dev = torch.device(device)
        self._y = torch.empty((rows, D), dtype=dtype, device=dev)
        self._r = None
        self.device = self._y.device
        self.r = self.mean = self.rstd = None
        if train:
            self._stats = torch.empty((2, rows), dtype=torch.float32, device=dev)
            self._dx = torch.empty((rows, D), dtype=dtype, device=dev)
            self.dgamma = torch.empty(D, dtype=weight_dtype, device=dev)
            self.dbeta = torch.empty(D, dtype=weight_dtype, device=dev)
            self.ws = torch.empty(max(B.moe_layer_norm_workspace_bytes(rows, D), 256),
                                  dtype=torch.uint8, device=dev)

    def forward(self, x, gamma, beta, res=None, stream=None):
        n = _rows("x", x, self.rows, self.D)
        dev = self.device
        _check("x", x, x.shape, self.dtype, dev)
        _check("gamma", gamma, (self.D,), self.weight_dtype, dev)
        _check("beta", beta, (self.D,), self.weight_dtype, dev)
        r = None
        if res is not None:
            _check("res", res, x.shape, self.dtype, dev)
            if self._r is None:
                self._r = torch.empty_like(self._y)
            r = self._r[:n]
        y = self._y[:n]
        if self.train:
            self.mean, self.rstd = self._stats[0, :n], self._stats[1, :n]
        _launchable(dev)
        B.moe_layer_norm(x, res, gamma, beta, r, y, self.mean, self.rstd, self.eps, stream)
        self.r = x if r is None else r
        return y

    def backward(self, dy, r, gamma, mean=None, rstd=None, dres=None, stream=None):
        if not self.train:
            raise RuntimeError("the norm was built without train=True")
        mean = self.mean if mean is None else mean
        rstd = self.rstd if rstd is None else rstd
        if mean is None or rstd is None:
            raise RuntimeError("backward needs a forward first, or its mean and rstd")
        n = _rows("dy", dy, self.rows, self.D)
        dev = self.device
        _check("dy", dy, dy.shape, self.dtype, dev)
        _check("r", r, dy.shape, self.dtype, dev)
        _check("gamma", gamma, (self.D,), self.weight_dtype, dev)
        _check("mean", mean, (n,), torch.float32, dev)
        _check("rstd", rstd, (n,), torch.float32, dev)
        if dres is not None:
            _check("dres", dres, dy.shape, self.dtype, dev)
        dx = self._dx[:n]
        _launchable(dev)
        B.moe_layer_norm_bwd(dy, r, gamma, mean, rstd, dres, dx, self.dgamma, self.dbeta, self.ws,
                             stream)
        return dx


class TopKRouter:
    """Selection of K of E experts for up to T tokens: scores sigmoid(l) or
    softmax(l), a balance bias that steers the selection only, choice limited
    to the ``top_groups`` best of ``groups`` groups of experts (a group's score
    is the sum of its ``group_top`` best), weights renormalised and scaled.

    ``forward`` returns (ids int32 [T, K], w fp32 [T, K]), which
    ``MoEBlock(score_mode=SCORE_GIVEN)`` takes; ``backward`` turns dw into
    dlogits [T, E]."""

    def __init__(self, T, E, K, score="sigmoid", groups=1, top_groups=1, group_top=2, renorm=True,
                 scale=1.0, train=False, device="cuda"):
        if score not in B.GATES:
            raise ValueError(f"score must be one of {sorted(B.GATES)}, got {score!r}")
        self.T, self.E, self.K, self.train = T, E, K, train
        self.d = B.topk_dims(T, E, K, score, groups, top_groups, group_top, renorm, scale)
        dev = torch.device(device)
        self._ids = torch.empty((T, K), dtype=torch.int32, device=dev)
        self._w = torch.empty((T, K), dtype=torch.float32, device=dev)
        self.device = self._w.device
        self.ids = self.w = None
        if train:
            self._dlogits = torch.empty((T, E), dtype=torch.float32, device=dev)

    def forward(self, logits, bias=None, stream=None):
        n = _rows("logits", logits, self.T, self.E)
        _check("logits", logits, logits.shape, torch.float32, self.device)
        if bias is not None:
            _check("bias", bias, (self.E,), torch.float32, self.device)
        self.d.T = n
        self.ids, self.w = self._ids[:n], self._w[:n]
        _launchable(self.device)
        B.moe_route_topk(logits, bias, self.ids, self.w, self.d, stream)
        return self.ids, self.w

    def backward(self, dw, logits, ids=None, stream=None):
        if not self.train:
            raise RuntimeError("the router was built without train=True")
        ids = self.ids if ids is None else ids
        if ids is None:
            raise RuntimeError("backward needs a forward first, or its ids")
        n = _rows("logits", logits, self.T, self.E)
        _check("logits", logits, logits.shape, torch.float32, self.device)
        _check("dw", dw, (n, self.K), torch.float32, self.device)
        _check("ids", ids, (n, self.K), torch.int32, self.device)
        self.d.T = n
        out = self._dlogits[:n]
        _launchable(self.device)
        B.moe_route_topk_bwd(logits, ids, dw, out, self.d, stream)
        return out


class Linear:
    """y = act(x w + bias) + res for up to M rows, w [K, N].

    ``dtype`` (bf16 or fp16) is that of x and w; ``out_dtype`` that of y and
    res (the same, or fp32).  With ``train`` and an activation the forward
    keeps the pre-activation in ``z``.  ``backward`` returns dx (plus
    ``dx_add``, another branch's gradient of x) and leaves ``dw`` and ``db``;
    the residual's gradient is dy itself."""

    def __init__(self, M, K, N, dtype=torch.bfloat16, out_dtype=None, act="none", train=False,
                 device="cuda"):
        out_dtype = out_dtype or dtype
        if act not in B.ACTS:
            raise ValueError(f"act must be one of {sorted(B.ACTS)}, got {act!r}")
        if dtype not in (torch.bfloat16, torch.float16) or out_dtype not in (dtype, torch.float32):
            raise ValueError(f"a linear layer of {dtype} with {out_dtype} results is not supported")
        if K % 8 or N % 8:
            raise ValueError(f"K and N must be multiples of 8, got K={K}, N={N}")
        self.M, self.K, self.N, self.act, self.train = M, K, N, act, train
        self.dtype, self.out_dtype = dtype, out_dtype
        self.d = B.linear_dims(M, K, N, dtype, out_dtype, act)
        dev = torch.device(device)
        self._y = torch.empty((M, N), dtype=out_dtype, device=dev)
        self.device = self._y.device
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.z = None
        self._z = None
        if train:
            if act != "none":
                self._z = torch.empty((M, N), dtype=dtype, device=dev)
            self._dx = torch.empty((M, K), dtype=dtype, device=dev)
            self.dw = torch.empty((K, N), dtype=dtype, device=dev)
            self.db = torch.empty(N, dtype=torch.float32, device=dev)
            self.ws = torch.empty(B.moe_linear_workspace_bytes(self.d), dtype=torch.uint8,
                                  device=dev)

    def forward(self, x, w, bias=None, res=None, stream=None):
        n = _rows("x", x, self.M, self.K)
        dev = self.device
        _check("x", x, x.shape, self.dtype, dev)
        _check("w", w, (self.K, self.N), self.dtype, dev)
        if bias is not None:
            _check("bias", bias, (self.N,), torch.float32, dev)
        if res is not None:
            _check("res", res, (n, self.N), self.out_dtype, dev)
        self.d.M = n
        y = self._y[:n]
        if self._z is not None:
            self.z = self._z[:n]
        _launchable(dev)
        B.moe_linear(x, w, bias, res, y, self.z, self.status, self.d, stream)
        return y

    def backward(self, dy, x, w, z=None, dx_add=None, need_dx=True, need_dw=True, need_db=True,
                 stream=None):
        if not self.train:
            raise RuntimeError("the linear layer was built without train=True")
        n = _rows("x", x, self.M, self.K)
        dev = self.device
        _check("dy", dy, (n, self.N), self.out_dtype, dev)
        _check("x", x, x.shape, self.dtype, dev)
        _check("w", w, (self.K, self.N), self.dtype, dev)
        if self.act != "none":
            z = self.z if z is None else z
            if z is None:
                raise RuntimeError("backward needs a forward first, or its z")
            _check("z", z, (n, self.N), self.dtype, dev)
        else:
            z = None
        if dx_add is not None:
            _check("dx_add", dx_add, x.shape, self.dtype, dev)
        self.d.M = n
        dx = self._dx[:n] if need_dx else None
        _launchable(dev)
        B.moe_linear_bwd(dy, z, x, w, dx_add, dx, self.dw if need_dw else None,
                         self.db if need_db else None, self.status, self.ws, self.d, stream)
        return dx


class MoELayer:
    """A pre-norm feed-forward layer: routed experts beside a shared dense one.

        r      = x + res                          (LayerNorm's residual add)
        u      = norm(r) gamma + beta
        l      = u wr                              (Linear, fp32)
        ids, p = route(l, bias)                    (TopKRouter)
        m      = experts(u; ids, p; wi, wo)        (MoEBlock, SwiGLU)
        f      = act(u w1 + b1) w2 + b2 + m        (two Linears; m is the residual)

    ``forward`` returns (r, f); the next layer's norm adds them.  ``backward``
    takes the gradients of both and returns dx (= dres); the weights'
    gradients are ``norm.dgamma/dbeta``, ``gate.dw`` (wr), ``block.dwi/dwo``,
    ``up.dw/db`` (w1, b1) and ``down.dw/db`` (w2, b2)."""

    WEIGHTS = ("gamma", "beta", "wr", "wi", "wo", "w1", "b1", "w2", "b2")

    def __init__(self, T, D, E, K, F, shared, act="silu", eps=1e-5, train=True, device="cuda",
                 **router):
        bf = torch.bfloat16
        self.train = train
        self.norm = LayerNorm(T, D, bf, torch.float32, eps, train, device)
        self.gate = Linear(T, D, E, bf, torch.float32, "none", train, device)
        self.router = TopKRouter(T, E, K, train=train, device=device, **router)
        self.block = MoEBlock(T, D, E, K, F, B.SCORE_GIVEN, train=train, device=device)
        self.up = Linear(T, D, shared, bf, None, act, train, device)
        self.down = Linear(T, shared, D, bf, None, "none", train, device)
        self.saved = None

    def forward(self, x, weights, res=None, bias=None, stream=None):
        g = weights
        if x.shape[0] != self.block.T:
            raise ValueError(f"x must have {self.block.T} rows, got {x.shape[0]}")
        u = self.norm.forward(x, g["gamma"], g["beta"], res=res, stream=stream)
        logits = self.gate.forward(u, g["wr"], stream=stream)
        ids, w = self.router.forward(logits, bias, stream=stream)
        m = self._experts(u, g["wi"], g["wo"], ids, w, stream)
        h = self.up.forward(u, g["w1"], g["b1"], stream=stream)
        f = self.down.forward(h, g["w2"], g["b2"], res=m, stream=stream)
        self.saved = (u, logits, h)
        return self.norm.r, f

    def _experts(self, u, wi, wo, ids, w, stream):
        # the block copies given ids and w with torch: on the launching stream
        if stream is None:
            return self.block.forward(u, wi, wo, ids=ids, w=w)
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream)
        with torch.cuda.stream(s):
            return self.block.forward(u, wi, wo, ids=ids, w=w)

    def backward(self, dr, df, weights, stream=None):
        """dr (may be None): what flows into r past this layer; df: into f."""
        if self.saved is None:
            raise RuntimeError("backward needs a forward first")
        g, (u, logits, h) = weights, self.saved
        dh = self.down.backward(df, h, g["w2"], stream=stream)
        du = self.block.backward(df, g["wi"], g["wo"], stream=stream)
        dlogits = self.router.backward(self.block.dw, logits, stream=stream)
        du = self.up.backward(dh, u, g["w1"], dx_add=du, stream=stream)
        du = self.gate.backward(dlogits, u, g["wr"], dx_add=du, need_db=False, stream=stream)
        return self.norm.backward(du, self.norm.r, g["gamma"], dres=dr, stream=stream)
