"""The operators around the expert block, and a whole layer of them.

``LayerNorm`` (with the residual add in front of it), ``TopKRouter`` (expert
selection with a balance bias and expert groups) and ``Linear`` (bias,
activation and residual in the product's epilogue) each own their output
buffers and workspace, like ``MoEBlock``: allocated once for a largest number
of rows, written by every call (a call's outputs are views of them and hold
until the next one).  Calls run on the current stream, or the one given, of
the device that the operator was built on, which has to be the current one.

``MoELayer`` runs them together with the expert block as one pre-norm
feed-forward layer, forward and backward.
"""
from __future__ import annotations

import torch

from . import binding as B
from .block import MoEBlock


class _Arg:
    """One tensor argument of an operator: its type, device and (where fixed)
    shape, checked on every call before anything is launched, since a tensor
    of another shape would be read or written out of bounds."""

    __slots__ = ("name", "dtype", "device", "index", "shape", "mat", "contiguous")

    def __init__(self, name, dtype, device, shape=None, contiguous=False):
        self.name, self.dtype, self.device, self.shape = name, dtype, device, shape
        self.index = device.index if device.type == "cuda" else -1
        self.mat = B.MoeMat(None, 0)
        self.contiguous = contiguous

    def refuse(self, t, shape):
        raise ValueError(f"{self.name} must be {self.dtype} {list(shape)} with contiguous "
                         f"{'elements' if self.contiguous else 'columns'} on {self.device}, got "
                         f"{t.dtype} {list(t.shape)}, strides {list(t.stride())} on {t.device}")

    def first(self, t, cap, width):
        """The number of rows of the call, from its first matrix, whose MoeMat
        this leaves in ``mat``."""
        shape = t.shape
        if (len(shape) != 2 or shape[1] != width or shape[0] > cap or t.dtype is not self.dtype
                or t.get_device() != self.index):
            self.refuse(t, (f"<= {cap}", width))
        ld, inner = t.stride()
        if inner != 1 and width > 1:
            self.refuse(t, shape)
        n = shape[0]
        m = self.mat
        m.p = t.data_ptr()
        m.ld = ld if n > 1 else (width + 7) // 8 * 8
        return n

    def rows(self, t, cap, width):
        """The number of rows of the call, from its first contiguous tensor."""
        shape = t.shape
        if len(shape) != 2 or shape[1] != width or shape[0] > cap:
            self.refuse(t, (f"<= {cap}", width))
        return shape[0]

    def matrix(self, t, shape):
        """A 2-D tensor as a MoeMat (of this argument: valid until its next call)."""
        if t.dtype is not self.dtype or t.shape != shape or t.get_device() != self.index:
            self.refuse(t, shape)
        ld, inner = t.stride()
        if inner != 1 and shape[1] > 1:
            self.refuse(t, shape)
        m = self.mat
        m.p = t.data_ptr()
        m.ld = ld if shape[0] > 1 else (shape[1] + 7) // 8 * 8
        return m

    def pointer(self, t, shape):
        """A contiguous tensor as its address."""
        if (t.dtype is not self.dtype or t.shape != shape or t.get_device() != self.index
                or not t.is_contiguous()):
            self.refuse(t, shape)
        return t.data_ptr()


def _own(t):
    """A buffer of the operator's own, as a MoeMat."""
    return B.MoeMat(t.data_ptr(), t.stride(0))


_NO = B.MoeMat(None, 0)     # a matrix that is not given


def _refused(fn, status):
    raise B.MoeError(fn, status)


def _entry(name, device):
    """A C entry point, for an operator whose buffers lie on `device`."""
    if device.type == "cuda":
        return getattr(B.lib(), name)

    def refuse(*args):
        raise RuntimeError(f"the operator's buffers are on {device}: its kernels need a CUDA device")
    return refuse


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
        self.eps, self.train = float(eps), train
        dev = torch.device(device)
        self._y = torch.empty((rows, D), dtype=dtype, device=dev)
        self.device = dev = self._y.device
        self._r = torch.empty_like(self._y)
        self.r = self.mean = self.rstd = None
        self._my, self._mr = _own(self._y), _own(self._r)
        self._p_mean = self._p_rstd = None
        self._width = (D,)
        if train:
            self._stats = torch.empty((2, rows), dtype=torch.float32, device=dev)
            self._mean, self._rstd = self._stats[0], self._stats[1]
            self._dx = torch.empty((rows, D), dtype=dtype, device=dev)
            self.dgamma = torch.empty(D, dtype=weight_dtype, device=dev)
            self.dbeta = torch.empty(D, dtype=weight_dtype, device=dev)
            self.ws = torch.empty(max(B.moe_layer_norm_workspace_bytes(rows, D), 256),
                                  dtype=torch.uint8, device=dev)
            self._mdx = _own(self._dx)
            self._p_mean, self._p_rstd = self._mean.data_ptr(), self._rstd.data_ptr()
            self._p_dgamma, self._p_dbeta = self.dgamma.data_ptr(), self.dbeta.data_ptr()
            self._p_ws = self.ws.data_ptr()
        self._x, self._res = _Arg("x", dtype, dev), _Arg("res", dtype, dev)
        self._dy, self._rin, self._dres = (_Arg(n, dtype, dev) for n in ("dy", "r", "dres"))
        self._gamma, self._beta = (_Arg(n, weight_dtype, dev, contiguous=True)
                                   for n in ("gamma", "beta"))
        self._amean, self._arstd = (_Arg(n, torch.float32, dev, contiguous=True)
                                    for n in ("mean", "rstd"))
        self._type, self._wtype = B.DTYPES[dtype], B.DTYPES[weight_dtype]
        self._fwd, self._bwd = _entry("moe_layer_norm", dev), _entry("moe_layer_norm_bwd", dev)

    def forward(self, x, gamma, beta, res=None, stream=None):
        D = self.D
        n = self._x.first(x, self.rows, D)
        pg, pb = self._gamma.pointer(gamma, self._width), self._beta.pointer(beta, self._width)
        whole = n == self.rows
        mres = mr = _NO
        r = x
        if res is not None:
            mres = self._res.matrix(res, (n, D))
            r, mr = self._r if whole else self._r[:n], self._mr
        st = self._fwd(self._x.mat, mres, pg, pb, mr, self._my, self._p_mean, self._p_rstd, self.eps,
                       n, D, self._type, self._wtype, B.stream_of(stream, self.device))
        if st:
            _refused("moe_layer_norm", st)
        self.r = r
        if self.train:
            self.mean, self.rstd = self._mean, self._rstd
            if not whole:
                self.mean, self.rstd = self._mean[:n], self._rstd[:n]
        return self._y if whole else self._y[:n]

    def backward(self, dy, r, gamma, mean=None, rstd=None, dres=None, stream=None):
        if not self.train:
            raise RuntimeError("the norm was built without train=True")
        mean = self.mean if mean is None else mean
        rstd = self.rstd if rstd is None else rstd
        if mean is None or rstd is None:
            raise RuntimeError("backward needs a forward first, or its mean and rstd")
        D = self.D
        n = self._dy.first(dy, self.rows, D)
        mrin = self._rin.matrix(r, (n, D))
        pg = self._gamma.pointer(gamma, self._width)
        pm, ps = self._amean.pointer(mean, (n,)), self._arstd.pointer(rstd, (n,))
        mres = _NO if dres is None else self._dres.matrix(dres, (n, D))
        st = self._bwd(self._dy.mat, mrin, pg, pm, ps, mres, self._mdx, self._p_dgamma, self._p_dbeta,
                       self._p_ws, n, D, self._type, self._wtype, B.stream_of(stream, self.device))
        if st:
            _refused("moe_layer_norm_bwd", st)
        return self._dx if n == self.rows else self._dx[:n]


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
        self.device = dev = self._w.device
        self._p_ids, self._p_w = self._ids.data_ptr(), self._w.data_ptr()
        self._experts = (E,)
        self.ids = self.w = None
        if train:
            self._dlogits = torch.empty((T, E), dtype=torch.float32, device=dev)
            self._p_dl = self._dlogits.data_ptr()
        f32 = torch.float32
        self._l = _Arg("logits", f32, dev, contiguous=True)
        self._b = _Arg("bias", f32, dev, contiguous=True)
        self._dw = _Arg("dw", f32, dev, contiguous=True)
        self._i = _Arg("ids", torch.int32, dev, contiguous=True)
        self._fwd, self._bwd = _entry("moe_route_topk", dev), _entry("moe_route_topk_bwd", dev)

    def forward(self, logits, bias=None, stream=None):
        n = self._l.rows(logits, self.T, self.E)
        pl = self._l.pointer(logits, (n, self.E))
        pb = None if bias is None else self._b.pointer(bias, self._experts)
        self.d.T = n
        st = self._fwd(pl, pb, self._p_ids, self._p_w, self.d, B.stream_of(stream, self.device))
        if st:
            _refused("moe_route_topk", st)
        if n == self.T:
            self.ids, self.w = self._ids, self._w
        else:
            self.ids, self.w = self._ids[:n], self._w[:n]
        return self.ids, self.w

    def backward(self, dw, logits, ids=None, stream=None):
        if not self.train:
            raise RuntimeError("the router was built without train=True")
        ids = self.ids if ids is None else ids
        if ids is None:
            raise RuntimeError("backward needs a forward first, or its ids")
        n = self._l.rows(logits, self.T, self.E)
        pl = self._l.pointer(logits, (n, self.E))
        pd, pi = self._dw.pointer(dw, (n, self.K)), self._i.pointer(ids, (n, self.K))
        self.d.T = n
        st = self._bwd(pl, pi, pd, self._p_dl, self.d, B.stream_of(stream, self.device))
        if st:
            _refused("moe_route_topk_bwd", st)
        return self._dlogits if n == self.T else self._dlogits[:n]


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
        self.device = dev = self._y.device
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.z = self._z = None
        self._mz = _NO
        self._my, self._p_status = _own(self._y), self.status.data_ptr()
        if train:
            if act != "none":
                self._z = torch.empty((M, N), dtype=dtype, device=dev)
                self._mz = _own(self._z)
            self._dx = torch.empty((M, K), dtype=dtype, device=dev)
            self.dw = torch.empty((K, N), dtype=dtype, device=dev)
            self.db = torch.empty(N, dtype=torch.float32, device=dev)
            self.ws = torch.empty(B.moe_linear_workspace_bytes(self.d), dtype=torch.uint8,
                                  device=dev)
            self._mdx, self._mdw = _own(self._dx), _own(self.dw)
            self._p_db, self._p_ws = self.db.data_ptr(), self.ws.data_ptr()
        self._x, self._w = _Arg("x", dtype, dev), _Arg("w", dtype, dev)
        self._b = _Arg("bias", torch.float32, dev, contiguous=True)
        self._res, self._dy = _Arg("res", out_dtype, dev), _Arg("dy", out_dtype, dev)
        self._zin, self._add = _Arg("z", dtype, dev), _Arg("dx_add", dtype, dev)
        self._fwd, self._bwd = _entry("moe_linear", dev), _entry("moe_linear_bwd", dev)
        self._wshape, self._bshape = (K, N), (N,)

    def forward(self, x, w, bias=None, res=None, stream=None):
        n = self._x.first(x, self.M, self.K)
        mw = self._w.matrix(w, self._wshape)
        pb = None if bias is None else self._b.pointer(bias, self._bshape)
        mres = _NO if res is None else self._res.matrix(res, (n, self.N))
        self.d.M = n
        st = self._fwd(self._x.mat, mw, pb, mres, self._my, self._mz, self._p_status, self.d,
                       B.stream_of(stream, self.device))
        if st:
            _refused("moe_linear", st)
        whole = n == self.M
        if self._z is not None:
            self.z = self._z if whole else self._z[:n]
        return self._y if whole else self._y[:n]

    def backward(self, dy, x, w, z=None, dx_add=None, need_dx=True, need_dw=True, need_db=True,
                 stream=None):
        if not self.train:
            raise RuntimeError("the linear layer was built without train=True")
        K, N = self.K, self.N
        n = self._x.first(x, self.M, K)
        mdy, mw = self._dy.matrix(dy, (n, N)), self._w.matrix(w, self._wshape)
        mz = _NO
        if self.act != "none":
            z = self.z if z is None else z
            if z is None:
                raise RuntimeError("backward needs a forward first, or its z")
            mz = self._zin.matrix(z, (n, N))
        madd = _NO if dx_add is None else self._add.matrix(dx_add, (n, K))
        self.d.M = n
        st = self._bwd(mdy, mz, self._x.mat, mw, madd, self._mdx if need_dx else _NO,
                       self._mdw if need_dw else _NO, self._p_db if need_db else None,
                       self._p_status, self._p_ws, self.d, B.stream_of(stream, self.device))
        if st:
            _refused("moe_linear_bwd", st)
        if not need_dx:
            return None
        return self._dx if n == self.M else self._dx[:n]


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
