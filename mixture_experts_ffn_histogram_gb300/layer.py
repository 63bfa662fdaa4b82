"""The operators around the expert block, and whole layers of them.

``LayerNorm`` (with the residual add in front of it), ``TopKRouter`` (expert
selection with a balance bias and expert groups) and ``Linear`` (bias,
activation and residual in the product's epilogue), and those that serve and
wrap the block, ``MoEDecode`` (the whole expert layer for a few tokens),
``BlockNorm`` (RMS norms after and before a block) and ``LowRankAdapters``
(beside a shared projection; grouped by an ``AdapterBatch``), each own their
output buffers and workspace, like ``MoEBlock``: allocated once for a largest number
of rows, written by every call (a call's outputs are views of them and hold
until the next one).  Calls run on the current stream, or the one given, of
the device that the operator was built on, which has to be the current one.

``MoELayer`` runs the first three together with the expert block as one
pre-norm feed-forward layer, forward and backward; ``DecodeLayer`` runs
``Linear`` and the others as one served layer.
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


def _zeros(size, dtype, dev):
    """A buffer that holds zeros for a call on whatever stream: the fill has
    ended.  (While a graph is captured it is part of that graph.)"""
    t = torch.zeros(size, dtype=dtype, device=dev)
    if t.is_cuda:
        with torch.cuda.device(t.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()
    return t


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


class BlockNorm:
    """RMS norms after and before a block, with its gate and residual scale:

        r = res + scale * token_gate * gate * norm(y) * (post + offset)
        u = norm(r) * (pre + offset)

    over rows of D, up to ``rows`` of them: y is what the block returned, res
    the residual stream, r the stream behind the block and u the next block's
    input.  Any of post, pre, gate (a weight for each channel) and token_gate
    (fp32, one for each row) may be None: no norm, no gate.  y None: u =
    norm(res), in front of the first block.

    ``forward`` returns u (r without pre) and leaves ``r``, ``u``, and with
    ``train`` the rows' ``rstd_y`` and ``rstd_r``.  ``backward`` takes the
    gradients of u and of r (what else flows into the stream; may be None with
    pre) and returns the gradient of res; ``dy``, ``dpost``, ``dpre``,
    ``dgate`` and ``dtoken_gate`` hold the others, None where the call gave no
    such argument."""

    def __init__(self, rows, D, dtype=torch.bfloat16, weight_dtype=torch.float32, eps=1e-6, scale=1.0,
                 offset=0.0, train=True, device="cuda"):
        if dtype not in B.DTYPES or weight_dtype not in (dtype, torch.float32):
            raise ValueError(f"rows of {dtype} with weights of {weight_dtype} are not supported")
        if not 1 <= D <= 8192:
            raise ValueError(f"unsupported sizes: D={D} (1 <= D <= 8192)")
        self.rows, self.D, self.dtype, self.weight_dtype, self.train = rows, D, dtype, weight_dtype, train
        self.d = B.block_norm_dims(rows, D, dtype, weight_dtype, eps, scale, offset)
        dev = torch.device(device)
        self._r = torch.empty((rows, D), dtype=dtype, device=dev)
        self.device = dev = self._r.device
        self._u = torch.empty_like(self._r)
        self.r = self.u = self.rstd_y = self.rstd_r = None
        self.dy = self.dpost = self.dpre = self.dgate = self.dtoken_gate = None
        self._mr, self._mu = _own(self._r), _own(self._u)
        self._p_stats = (None, None)
        if train:
            self._stats = torch.empty((2, rows), dtype=torch.float32, device=dev)
            self._dres, self._dy_out = torch.empty_like(self._r), torch.empty_like(self._r)
            self._dw = torch.empty((3, D), dtype=weight_dtype, device=dev)
            self._dtg = torch.empty(rows, dtype=torch.float32, device=dev)
            self.ws = torch.empty(max(B.moe_block_norm_workspace_bytes(self.d), 256), dtype=torch.uint8,
                                  device=dev)
            self._mdres, self._mdy = _own(self._dres), _own(self._dy_out)
            self._sy, self._sr = self._stats[0], self._stats[1]
            self._p_stats = (self._sy.data_ptr(), self._sr.data_ptr())
            self._grads = tuple(self._dw.unbind(0))     # of post, pre and gate
            self._p_dpost, self._p_dpre, self._p_dgate = (t.data_ptr() for t in self._grads)
            self._p_ws = self.ws.data_ptr()
            self._p_dtg = self._dtg.data_ptr()
        self._res, self._y, self._rin, self._du, self._dr = (
            _Arg(n, dtype, dev) for n in ("res", "y", "r", "du", "dr"))
        self._weights = tuple(_Arg(n, weight_dtype, dev, contiguous=True) for n in ("post", "pre", "gate"))
        self._rowwise = tuple(_Arg(n, torch.float32, dev, contiguous=True)
                              for n in ("token_gate", "rstd_y", "rstd_r"))
        self._width = (D,)
        self._fwd, self._bwd = _entry("moe_block_norm", dev), _entry("moe_block_norm_bwd", dev)

    def _given(self, n, y, post, pre, gate, token_gate):
        """The addresses of the weights and gates (None where not given)."""
        if y is None and (pre is None or post is not None or gate is not None or token_gate is not None):
            raise ValueError("without y there is only the norm before the block: pre, and no post or gates")
        w = self._width
        a, b, c = self._weights
        return (None if post is None else a.pointer(post, w), None if pre is None else b.pointer(pre, w),
                None if gate is None else c.pointer(gate, w),
                None if token_gate is None else self._rowwise[0].pointer(token_gate, (n,)))

    def forward(self, res, y=None, post=None, pre=None, gate=None, token_gate=None, stream=None):
        D = self.D
        n = self._res.first(res, self.rows, D)
        p = self._given(n, y, post, pre, gate, token_gate)
        my = _NO if y is None else self._y.matrix(y, (n, D))
        self.d.rows = n
        st = self._fwd(my, self._res.mat, *p, self._mr, self._mu, *self._p_stats, self.d,
                       B.stream_of(stream, self.device))
        if st:
            _refused("moe_block_norm", st)
        whole = n == self.rows
        self.r = res if y is None else (self._r if whole else self._r[:n])
        self.u = None if pre is None else (self._u if whole else self._u[:n])
        if self.train:
            self.rstd_y = None if post is None else (self._sy if whole else self._sy[:n])
            self.rstd_r = None if pre is None else (self._sr if whole else self._sr[:n])
        return self.r if pre is None else self.u

    def backward(self, du, dr, r=None, y=None, post=None, pre=None, gate=None, token_gate=None,
                 rstd_y=None, rstd_r=None, stream=None):
        if not self.train:
            raise RuntimeError("the norms were built without train=True")
        if (du is None) != (pre is None):
            raise ValueError("du is the gradient of the norm before the next block: given with pre, and only then")
        if dr is None and pre is None:
            raise ValueError("without pre the gradient of r has to be given")
        D = self.D
        first, arg = (du, self._du) if du is not None else (dr, self._dr)
        n = arg.first(first, self.rows, D)
        p = self._given(n, y, post, pre, gate, token_gate)
        mdu = mr = mdr = my = _NO
        py = pr = None
        if du is not None:
            mdu = self._du.mat
            r = self.r if r is None else r
            rstd_r = self.rstd_r if rstd_r is None else rstd_r
            if r is None or rstd_r is None:
                raise RuntimeError("backward needs a forward first, or its r and rstd_r")
            mr, pr = self._rin.matrix(r, (n, D)), self._rowwise[2].pointer(rstd_r, (n,))
        if dr is not None:
            mdr = self._dr.matrix(dr, (n, D))
        if y is not None:
            my = self._y.matrix(y, (n, D))
            if post is not None:
                rstd_y = self.rstd_y if rstd_y is None else rstd_y
                if rstd_y is None:
                    raise RuntimeError("backward needs a forward first, or its rstd_y")
                py = self._rowwise[1].pointer(rstd_y, (n,))
        self.d.rows = n
        st = self._bwd(mdu, mdr, mr, my, *p, py, pr, self._mdres, _NO if y is None else self._mdy,
                       None if post is None else self._p_dpost, None if pre is None else self._p_dpre,
                       None if gate is None else self._p_dgate, None if token_gate is None else self._p_dtg,
                       self._p_ws, self.d, B.stream_of(stream, self.device))
        if st:
            _refused("moe_block_norm_bwd", st)
        whole = n == self.rows
        self.dy = None if y is None else (self._dy_out if whole else self._dy_out[:n])
        dpost, dpre, dgate = self._grads
        self.dpost = None if post is None else dpost
        self.dpre = None if pre is None else dpre
        self.dgate = None if gate is None else dgate
        self.dtoken_gate = None if token_gate is None else (self._dtg if whole else self._dtg[:n])
        return self._dres if whole else self._dres[:n]


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
        self.status = _zeros(1, torch.int32, dev)
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


class AdapterBatch:
    """Which adapter each token of a batch uses: up to T tokens, ``slots``
    adapters in the pool.  ``group`` takes ids (int32, one a token: a slot, or
    -1 for none) and sorts the tokens by adapter on the device; every
    ``LowRankAdapters`` of the batch's step takes it so.  An id outside
    [-1, slots) is reported in ``status`` and taken as -1."""

    def __init__(self, T, slots, device="cuda"):
        need = B.moe_adapter_plan_bytes(T, slots)
        if need == 0:
            raise ValueError(f"unsupported sizes: T={T}, slots={slots} (T <= 2^20, 1 <= slots <= 1024)")
        self.T, self.slots, self.n = T, slots, None
        dev = torch.device(device)
        self.plan = _zeros(need, torch.uint8, dev)
        self.device = dev = self.plan.device
        self.status = _zeros(1, torch.int32, dev)
        self._ids = _Arg("ids", torch.int32, dev, contiguous=True)
        self._p_plan, self._p_status = self.plan.data_ptr(), self.status.data_ptr()
        self._fwd = _entry("moe_adapter_plan", dev)

    def group(self, ids, stream=None):
        n = ids.shape[0] if ids.dim() == 1 else -1
        if not 0 <= n <= self.T:
            self._ids.refuse(ids, (f"<= {self.T}",))
        p = self._ids.pointer(ids, (n,))
        st = self._fwd(p, n, self.T, self.slots, self._p_plan, self._p_status, B.stream_of(stream, self.device))
        if st:
            _refused("moe_adapter_plan", st)
        self.n = n
        return self


class LowRankAdapters:
    """y = res + scale[s] (x a[s]^T) b[s]^T for up to T tokens, each with the
    adapter s that the batch names for it (none: y = res), beside a shared
    projection whose result is res (None: zeros).

    A pool of ``slots`` adapters of one ``rank`` (a multiple of 8 up to 128;
    narrower ones padded with zeros): a [slots, rank, K], b [slots, N, rank]
    in bf16 or fp16 like the rows, scale fp32 [slots].  ``batch`` is an
    ``AdapterBatch`` of the same T and slots, grouped for these tokens on the
    same stream or before.  ``status`` is the kernels' error word.  In fp16 a
    scale[s] x a[s]^T of 65520 or more is infinite; bf16 has fp32's range."""

    def __init__(self, T, K, N, slots, rank, dtype=torch.bfloat16, device="cuda"):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"adapters of {dtype} are not supported")
        self.T, self.K, self.N, self.slots, self.rank, self.dtype = T, K, N, slots, rank, dtype
        self.d = B.adapter_dims(T, K, N, slots, rank, dtype)
        need = B.moe_adapters_workspace_bytes(self.d)
        if need == 0:
            raise ValueError(f"unsupported sizes: T={T}, K={K}, N={N}, slots={slots}, rank={rank} (K, N and rank "
                             "multiples of 8, rank <= 128, T <= 2^20, 1 <= slots <= 1024)")
        dev = torch.device(device)
        self._y = torch.empty((T, N), dtype=dtype, device=dev)
        self.device = dev = self._y.device
        self.status = _zeros(1, torch.int32, dev)
        self.ws = _zeros(need, torch.uint8, dev)
        self._my, self._p_status, self._p_ws = _own(self._y), self.status.data_ptr(), self.ws.data_ptr()
        self._x, self._res = _Arg("x", dtype, dev), _Arg("res", dtype, dev)
        self._a, self._b = (_Arg(n, dtype, dev, contiguous=True) for n in ("a", "b"))
        self._scale = _Arg("scale", torch.float32, dev, contiguous=True)
        self._ashape, self._bshape, self._sshape = (slots, rank, K), (slots, N, rank), (slots,)
        self._fwd = _entry("moe_adapters", dev)

    def forward(self, batch, x, a, b, scale, res=None, stream=None):
        n = self._x.first(x, self.T, self.K)
        if batch.T != self.T or batch.slots != self.slots or batch.device != self.device:
            raise ValueError(f"the batch is for {batch.T} tokens and {batch.slots} slots on {batch.device}, the "
                             f"adapters for {self.T} and {self.slots} on {self.device}")
        if batch.n != n:
            raise ValueError(f"the batch was grouped for {batch.n} tokens, the call has {n}")
        pa, pb = self._a.pointer(a, self._ashape), self._b.pointer(b, self._bshape)
        ps = self._scale.pointer(scale, self._sshape)
        mres = _NO if res is None else self._res.matrix(res, (n, self.N))
        st = self._fwd(self._x.mat, pa, pb, ps, mres, self._my, batch._p_plan, self._p_status, self._p_ws, n,
                       self.d, B.stream_of(stream, self.device))
        if st:
            _refused("moe_adapters", st)
        return self._y if n == self.T else self._y[:n]


class MoEDecode:
    """The whole expert layer for up to T tokens, a few (T <= 256): routing,
    both expert products with SwiGLU and the weighted combine, in two kernels
    that read the weights of the experts named, once.

    ``score_mode`` and the routing arguments are ``MoEBlock``'s: logits (and
    bias), or ids and w of a router's own (``SCORE_GIVEN``).  ``forward``
    returns out = experts(x) + res for bf16 or fp16 rows; ``ids`` and ``w``
    hold the selection.  ``status`` is MoEBlock's: an id outside [0, E) is
    reported there and its slot dropped.  In fp16 an inner value (silu of the
    gate times up) of 65520 or more is infinite; bf16 has fp32's range.  Longer
    batches and training: ``MoEBlock``."""

    def __init__(self, T, D, E, K, F, score_mode=B.SCORE_SOFTMAX_TOPK, dtype=torch.bfloat16,
                 device="cuda"):
        if score_mode not in (B.SCORE_SOFTMAX_TOPK, B.SCORE_SIGMOID_NORM, B.SCORE_GIVEN):
            raise ValueError(f"unknown score mode {score_mode!r}")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"an expert layer of {dtype} is not supported")
        self.T, self.D, self.E, self.K, self.F = T, D, E, K, F
        self.mode, self.dtype = score_mode, dtype
        self.d = B.dims(T, D, E, K, F)
        need = B.moe_decode_workspace_bytes(self.d)
        if need == 0:
            raise ValueError(f"unsupported sizes: {self.d} (T <= 256, T * K <= 2048, K <= min(E, 32), "
                             "E <= 1024, D and F multiples of 64 up to 16384)")
        dev = torch.device(device)
        self._out = torch.empty((T, D), dtype=dtype, device=dev)
        self.device = dev = self._out.device
        self.status = _zeros(1, torch.int32, dev)
        self.ws = _zeros(need, torch.uint8, dev)
        self._given = score_mode == B.SCORE_GIVEN
        self.ids = self.w = None
        if not self._given:
            self._ids = torch.empty((T, K), dtype=torch.int32, device=dev)
            self._w = torch.empty((T, K), dtype=torch.float32, device=dev)
            self._p_ids, self._p_w = self._ids.data_ptr(), self._w.data_ptr()
        self._mout, self._p_status, self._p_ws = _own(self._out), self.status.data_ptr(), self.ws.data_ptr()
        f32 = torch.float32
        self._x, self._res = _Arg("x", dtype, dev), _Arg("res", dtype, dev)
        self._wi, self._wo = (_Arg(n, dtype, dev, contiguous=True) for n in ("wi", "wo"))
        self._l, self._b = (_Arg(n, f32, dev, contiguous=True) for n in ("logits", "bias"))
        self._i, self._win = _Arg("ids", torch.int32, dev, contiguous=True), _Arg("w", f32, dev, contiguous=True)
        self._wishape, self._woshape, self._experts = (E, D, 2 * F), (E, F, D), (E,)
        self._type, self._fwd = B.DTYPES[dtype], _entry("moe_decode", dev)

    def forward(self, x, wi, wo, logits=None, bias=None, ids=None, w=None, res=None, stream=None):
        n = self._x.first(x, self.T, self.D)
        pwi, pwo = self._wi.pointer(wi, self._wishape), self._wo.pointer(wo, self._woshape)
        pl = pb = None
        slots = (n, self.K)
        if self._given:
            if ids is None or w is None:
                raise ValueError("the layer was built for a given selection: it needs ids and w")
            pi, pw = self._i.pointer(ids, slots), self._win.pointer(w, slots)
        else:
            if logits is None:
                raise ValueError("the layer selects the experts itself: it needs logits")
            pl = self._l.pointer(logits, (n, self.E))
            pb = None if bias is None else self._b.pointer(bias, self._experts)
            ids, w = (self._ids, self._w) if n == self.T else (self._ids[:n], self._w[:n])
            pi, pw = self._p_ids, self._p_w
        mres = _NO if res is None else self._res.matrix(res, (n, self.D))
        st = self._fwd(self._x.mat, pwi, pwo, pl, pb, self.mode, pi, pw, mres, self._mout, self._p_status,
                       self._p_ws, n, self.d, self._type, B.stream_of(stream, self.device))
        if st:
            _refused("moe_decode", st)
        self.ids, self.w = ids, w
        return self._out if n == self.T else self._out[:n]


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


class DecodeLayer:
    """A feed-forward layer that serves up to T tokens, a few: routed experts
    beside a shared dense one with the requests' adapters on its second
    product, and the norms around them.

        l  = u wr                                        (Linear, fp32)
        h  = act(u w1 + b1),  s = h w2 + b2              (two Linears)
        s += scale[a] (h a_a^T) b_a^T                    (LowRankAdapters, with a batch)
        m  = experts(u; l, bias) + s                     (MoEDecode)
        r' = r + branch * norm(m) (post + offset)        (BlockNorm)
        u' = norm(r') (pre + offset)

    With ``SCORE_GIVEN`` a router of its own selects (``TopKRouter``, say, on
    logits of any number of experts): ``forward`` takes its ids and w, there is
    no gate and no wr.

    ``forward`` takes the residual stream r and u, its norm, and returns both
    behind the layer (views of the norm's buffers, ``norm.r`` and ``norm.u``).
    D is ``BlockNorm``'s, up to 8192."""

    WEIGHTS = ("wr", "wi", "wo", "w1", "b1", "w2", "b2", "post", "pre")
    ADAPTERS = ("a", "b", "scale")

    def __init__(self, T, D, E, K, F, shared, score_mode=B.SCORE_SOFTMAX_TOPK, act="silu",
                 dtype=torch.bfloat16, eps=1e-6, branch=1.0, offset=0.0, slots=0, rank=8, device="cuda"):
        self.gate = None if score_mode == B.SCORE_GIVEN else Linear(T, D, E, dtype, torch.float32, device=device)
        self.up = Linear(T, D, shared, dtype, act=act, device=device)
        self.down = Linear(T, shared, D, dtype, device=device)
        self.adapters = LowRankAdapters(T, shared, D, slots, rank, dtype, device) if slots else None
        self.experts = MoEDecode(T, D, E, K, F, score_mode, dtype, device)
        self.norm = BlockNorm(T, D, dtype, torch.float32, eps, branch, offset, train=False, device=device)

    def forward(self, r, u, weights, bias=None, batch=None, stream=None, ids=None, w=None):
        g = weights
        if batch is not None and self.adapters is None:
            raise ValueError("the layer was built without adapters (slots=0)")
        if self.gate is None:
            if ids is None or w is None or bias is not None:
                raise ValueError("the layer was built for a given selection: it needs ids and w, and no bias")
            logits = None
        elif ids is not None or w is not None:
            raise ValueError("the layer selects the experts itself: no ids or w")
        else:
            logits = self.gate.forward(u, g["wr"], stream=stream)
        h = self.up.forward(u, g["w1"], g["b1"], stream=stream)
        s = self.down.forward(h, g["w2"], g["b2"], stream=stream)
        if batch is not None:
            s = self.adapters.forward(batch, h, g["a"], g["b"], g["scale"], res=s, stream=stream)
        m = self.experts.forward(u, g["wi"], g["wo"], logits=logits, bias=bias, ids=ids, w=w, res=s,
                                 stream=stream)
        u = self.norm.forward(r, m, g["post"], g["pre"], stream=stream)
        return self.norm.r, u
