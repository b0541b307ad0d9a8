"""A block's operators between its matrix products, with torch tensors in place of raw pointers.

``FusedDropout`` is dropout whose mask is computed from a counter, with the add of the
residual stream.  ``FusedRouter`` routes tokens to experts, steps the bias that balances
them, and moves the rows there and back.  ``FusedGroupNorm`` is group norm with an
activation, channels last.  Each has its backward pass.  As in ``operators.py`` they hold
the device that was current when they were made (and a plan of the library there), check
their arguments and launch on the current stream or ``stream``; outputs that are not given
are allocated for the stream of the launch, and inputs stay the caller's.
"""

from __future__ import annotations

import torch

from . import _capi, _stream
from .operators import _DTYPES, _F32, _elsewhere, _empty, _on, _Plan, _rows, _vector

_I32 = torch.int32
_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}
_ACTIVATIONS = {"none": 0, "silu": 1}


def _choice(name, value, table):
    if value not in table:
        raise ValueError(f"{name} must be one of {', '.join(table)}, got {value!r}")
    return table[value]


def _dtype(t):
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def _grid(name, t, shape, dtype, device):
    """Address of a contiguous CUDA matrix of that shape and type."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        _elsewhere(name, t, device, f"contiguous CUDA tensor of shape {tuple(shape)}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of shape {tuple(shape)}")
    return t.data_ptr()


class FusedDropout:
    """Dropout of elements with probability ``p``; its mask is never stored.

    The mask depends on ``seed``, ``site`` (which tells the dropouts of a model apart), the
    step counter that a call is given (int32 [1] on the device, as ``FusedAdamW.step`` takes
    it; None: 0) and an element's place in its dense matrix, and on nothing else.  Tensors of
    any shape whose last axis is contiguous, float32, float16 or bfloat16.
    """

    def __init__(self, p: float, seed: int = 0, site: int = 0):
        self.p = float(p)
        if not 0.0 <= self.p <= 1.0:
            raise ValueError("p must lie in [0, 1]")
        self.seed, self.site = int(seed) % (1 << 64), int(site)
        if not 0 <= self.site < 1 << 32:
            raise ValueError("site must fit 32 bits")
        self.device = torch.cuda.current_device()

    def _matrix(self, name, t, like):
        """(address, row stride) of t, of like's shape and type, as a matrix of rows."""
        if t.get_device() != self.device:
            _elsewhere(name, t, self.device, "CUDA tensor")
        if t.dtype != like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if t.shape != like.shape:
            raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
        if t.is_contiguous():
            return t.data_ptr(), t.shape[-1] if t.dim() else 1
        if t.dim() != 2:
            try:
                t = t.view(-1, t.shape[-1])
            except RuntimeError:
                raise ValueError(f"{name} must be a matrix of rows at one stride") from None
        return t.data_ptr(), _rows(name, t, None, None, self.device)

    def _call(self, names, x, step, residual, y):
        if torch.cuda.current_device() != self.device:
            raise RuntimeError(f"the dropout was made on device {self.device}, which is not the current one")
        dtype = _dtype(x)
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        at, stride = self._matrix(names[0], x, x)
        out, out_stride = self._matrix(names[1], y, x)
        extra, extra_stride = (None, 0) if residual is None else self._matrix("residual", residual, x)
        width = x.shape[-1] if x.dim() else 1
        rows = x.numel() // width if width else 0
        _capi.adamw_dropout(dtype, rows, width, at, stride, extra, extra_stride, out, out_stride, self.p, self.seed,
                            _vector("step", step, 1, self.device, _I32), self.site, _stream(None))
        return y

    def forward(self, x, step=None, residual=None, *, y=None, stream=None):
        """y = residual + dropout(x); y may be x or the residual."""
        if stream is not None:
            with _on(stream):
                return self.forward(x, step, residual, y=y)
        return self._call(("x", "y"), x, step, residual, y)

    def backward(self, dy, step=None, *, dx=None, stream=None):
        """The gradient of x from that of y, with the step of the forward pass; dx may be dy.  The
        residual's gradient is dy itself."""
        if stream is not None:
            with _on(stream):
                return self.backward(dy, step, dx=dx)
        return self._call(("dy", "dx"), dy, step, None, dx)


class FusedRouter(_Plan):
    """Routing of up to ``max_tokens`` tokens to ``top_k`` of ``experts`` experts each.

    score "softmax" or "sigmoid"; with ``groups`` a token's experts are those of its
    ``top_groups`` best groups, by their largest score (group_score "max") or the sum of
    their two largest ("top2"; where one expert of a group is there, that one's);
    ``renormalise``: a token's weights sum to ``scale``.
    """

    _destroy = staticmethod(_capi.adamw_router_plan_destroy)

    def __init__(self, max_tokens: int, experts: int, top_k: int, *, score="softmax", groups=1, top_groups=None,
                 group_score="max", renormalise=True, scale=1.0):
        router = _capi.adamw_router(int(experts), int(top_k), int(groups), int(groups if top_groups is None else top_groups),
                                    _choice("score", score, _SCORES), _choice("group_score", group_score, _GROUP_SCORES),
                                    bool(renormalise), float(scale))
        self.plan = _capi.adamw_router_plan_create(router, int(max_tokens))
        self.device = torch.cuda.current_device()
        self.experts, self.top_k = int(experts), int(top_k)

    def _logits(self, name, t, dtype=None, shape=None):
        stride = _rows(name, t, dtype, shape, self.device)
        if t.shape[1] != self.experts:
            raise ValueError(f"{name} must have {self.experts} columns, got {t.shape[1]}")
        return stride

    def _slots(self, slots, tokens):
        return _grid("slots", slots, (tokens, self.top_k), _I32, self.device)

    def route(self, logits, bias=None, *, weights=None, ids=None, slots=None, starts=None, stream=None):
        """(weights, ids, slots, starts): a token's experts, best first, their weights, each
        assignment's place when all are ordered by expert, and where each expert's begin."""
        if stream is not None:
            with _on(stream):
                return self.route(logits, bias, weights=weights, ids=ids, slots=slots, starts=starts)
        dtype, stride = _dtype(logits), self._logits("logits", logits)
        dev, tokens = self.device, logits.shape[0]
        shape = (tokens, self.top_k)
        if weights is None:
            weights = _empty(shape, logits)
        if ids is None:
            ids = _empty(shape, logits, _I32)
        if slots is None:
            slots = _empty(shape, logits, _I32)
        if starts is None:
            starts = _empty(self.experts + 1, logits, _I32)
        _capi.adamw_route(self.plan, dtype, tokens, logits.data_ptr(), stride, _vector("bias", bias, self.experts, dev),
                          _grid("weights", weights, shape, _F32, dev), _grid("ids", ids, shape, _I32, dev),
                          _grid("slots", slots, shape, _I32, dev), _vector("starts", starts, self.experts + 1, dev, _I32),
                          _stream(None))
        return weights, ids, slots, starts

    def backward(self, dweights, logits, ids, *, dlogits=None, stream=None):
        """The gradient of the logits from that of the weights; dlogits may be the logits."""
        if stream is not None:
            with _on(stream):
                return self.backward(dweights, logits, ids, dlogits=dlogits)
        dtype, stride = _dtype(logits), self._logits("logits", logits)
        tokens = logits.shape[0]
        shape = (tokens, self.top_k)
        if dlogits is None:
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        out = self._logits("dlogits", dlogits, logits.dtype, logits.shape)
        _capi.adamw_route_backward(self.plan, dtype, tokens, logits.data_ptr(), stride,
                                   _grid("ids", ids, shape, _I32, self.device),
                                   _grid("dweights", dweights, shape, _F32, self.device), dlogits.data_ptr(), out,
                                   _stream(None))
        return dlogits

    def balance(self, bias, starts, rate, *, stream=None):
        """Steps the bias in place: up by ``rate`` for experts with less than the mean load, down for
        those with more.  ``starts`` may be the sum of several calls'."""
        if stream is not None:
            with _on(stream):
                return self.balance(bias, starts, rate)
        if bias is None or starts is None:
            raise ValueError("bias and starts must be given")
        _capi.adamw_route_balance(self.plan, _vector("starts", starts, self.experts + 1, self.device, _I32), rate,
                                  _vector("bias", bias, self.experts, self.device), _stream(None))
        return bias

    def dispatch(self, x, slots, *, xs=None, stream=None):
        """xs[slots[t, j]] = x[t]: rows ordered by expert, for the experts' products.  Rows of xs that no
        slot names (behind the last assignment, where a token has fewer than top_k) are left as they
        were, and are 0 in an xs that is made here, which costs a pass over it."""
        if stream is not None:
            with _on(stream):
                return self.dispatch(x, slots, xs=xs)
        dtype, stride = _dtype(x), _rows("x", x, None, None, self.device)
        tokens, width = x.shape
        at = self._slots(slots, tokens)
        if xs is None:
            xs = torch.zeros((tokens * self.top_k, width), dtype=x.dtype, device=x.device)
        out = _rows("xs", xs, x.dtype, (xs.shape[0], width), self.device)
        _capi.adamw_route_dispatch(self.plan, dtype, tokens, width, x.data_ptr(), stride, at, xs.data_ptr(), xs.shape[0],
                                   out, _stream(None))
        return xs

    def combine(self, ys, slots, weights=None, *, y=None, stream=None):
        """y[t] = sum over j of weights[t, j] ys[slots[t, j]].  Without weights it is the backward pass of
        ``dispatch``."""
        if stream is not None:
            with _on(stream):
                return self.combine(ys, slots, weights, y=y)
        dtype, stride = _dtype(ys), _rows("ys", ys, None, None, self.device)
        tokens, width = slots.shape[0], ys.shape[1]
        at = self._slots(slots, tokens)
        if weights is not None:
            weights = _grid("weights", weights, (tokens, self.top_k), _F32, self.device)
        if y is None:
            y = torch.empty((tokens, width), dtype=ys.dtype, device=ys.device)
        out = _rows("y", y, ys.dtype, (tokens, width), self.device)
        _capi.adamw_route_combine(self.plan, dtype, tokens, width, ys.data_ptr(), ys.shape[0], stride, at, weights,
                                  y.data_ptr(), out, _stream(None))
        return y

    def combine_backward(self, dy, ys, slots, weights, *, dys=None, dweights=None, stream=None):
        """(dys, dweights): dys[slots[t, j]] = weights[t, j] dy[t], dweights[t, j] = <dy[t], ys[slots[t, j]]>.
        dys may be ys.  Rows of ys that no slot names have no gradient: those of a given dys are left as
        they were, and are 0 in one that is made here, which costs a pass over it."""
        if stream is not None:
            with _on(stream):
                return self.combine_backward(dy, ys, slots, weights, dys=dys, dweights=dweights)
        dtype, stride = _dtype(ys), _rows("ys", ys, None, None, self.device)
        tokens, width = slots.shape[0], ys.shape[1]
        shape = (tokens, self.top_k)
        dy_stride = _rows("dy", dy, ys.dtype, (tokens, width), self.device)
        at = self._slots(slots, tokens)
        if dys is None:
            dys = torch.zeros(ys.shape, dtype=ys.dtype, device=ys.device)
        if dweights is None:
            dweights = _empty(shape, ys)
        out = _rows("dys", dys, ys.dtype, ys.shape, self.device)
        _capi.adamw_route_combine_backward(
            self.plan, dtype, tokens, width, dy.data_ptr(), dy_stride, ys.data_ptr(), ys.shape[0], stride, at,
            _grid("weights", weights, shape, _F32, self.device), dys.data_ptr(), out,
            _grid("dweights", dweights, shape, _F32, self.device), _stream(None))
        return dys, dweights


class FusedGroupNorm(_Plan):
    """Group norm with an activation ("none" or "silu") over channels-last tensors.

    [samples, positions, channels], float32, float16 or bfloat16, the channels contiguous and any
    other strides; weight and bias float32 or of the elements' dtype, or None; mean and rstd
    float32 [samples, groups].  ``max_samples`` samples per call at most.  A group whose squared
    distances from the mean add up to more than float32 holds has rstd 0.
    """

    _destroy = staticmethod(_capi.adamw_group_norm_plan_destroy)

    def __init__(self, channels: int, groups: int, max_samples: int, eps: float = 1e-5, activation: str = "none"):
        self.plan = _capi.adamw_group_norm_plan_create(int(channels), int(groups), int(max_samples), float(eps),
                                                       _choice("activation", activation, _ACTIVATIONS))
        self.device = torch.cuda.current_device()
        self.channels, self.groups = int(channels), int(groups)
        # the argument records, filled anew by every call
        self._views = {name: _capi.adamw_channels_last() for name in ("x", "y", "dy", "dx")}

    def status(self) -> int:
        """Device-side fault bits (0 = healthy); raises AdamWError if a bounded wait gave up."""
        return _capi.adamw_group_norm_plan_status(self.plan)

    def _view(self, name, t, like=None):
        if t.get_device() != self.device:
            _elsewhere(name, t, self.device, "CUDA tensor")
        if t.dim() != 3 or t.shape[2] != self.channels:
            raise ValueError(f"{name} must be [samples, positions, {self.channels}], got {tuple(t.shape)}")
        if like is not None:
            if t.dtype != like.dtype:
                raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
            if t.shape != like.shape:
                raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
        sample, position, step = t.stride()
        if step != 1 and self.channels > 1:
            raise ValueError(f"{name} must be contiguous along its last axis")
        v = self._views[name]
        v.data = t.data_ptr()
        # a lone position's or sample's stride says nothing
        v.position_stride = position if t.shape[1] > 1 else self.channels
        v.sample_stride = sample if t.shape[0] > 1 else 0
        return v

    def _weights(self, x, weight, bias, given=None):
        for t in (weight, bias, given):
            if t is not None:
                if t.dtype not in (_F32, x.dtype):
                    raise TypeError(f"the weight must be float32 or {x.dtype}, got {t.dtype}")
                return t.dtype
        return x.dtype

    def forward(self, x, weight=None, bias=None, *, y=None, mean=None, rstd=None, stream=None):
        """(y, mean, rstd); y may be x."""
        if stream is not None:
            with _on(stream):
                return self.forward(x, weight, bias, y=y, mean=mean, rstd=rstd)
        dtype, view = _dtype(x), self._view("x", x)
        kind, dev = self._weights(x, weight, bias), self.device
        samples, positions, channels = x.shape
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if mean is None:
            mean = _empty((samples, self.groups), x)
        if rstd is None:
            rstd = _empty((samples, self.groups), x)
        _capi.adamw_group_norm_forward(
            self.plan, dtype, _DTYPES[kind], samples, positions, view, _vector("weight", weight, channels, dev, kind),
            _vector("bias", bias, channels, dev, kind), self._view("y", y, x),
            _grid("mean", mean, (samples, self.groups), _F32, dev), _grid("rstd", rstd, (samples, self.groups), _F32, dev),
            _stream(None))
        return y, mean, rstd

    def backward(self, dy, x, weight, bias, mean, rstd, *, dx=None, dweight=None, dbias=None, stream=None):
        """(dx, dweight, dbias) from the forward pass's x, weight, bias, mean and rstd; the weight's and
        bias's gradients in the weight's dtype (the elements' when both are None).  dx may be dy or x."""
        if stream is not None:
            with _on(stream):
                return self.backward(dy, x, weight, bias, mean, rstd, dx=dx, dweight=dweight, dbias=dbias)
        dtype, view = _dtype(x), self._view("x", x)
        kind, dev = self._weights(x, weight, bias, dweight if dweight is not None else dbias), self.device
        samples, positions, channels = x.shape
        if dx is None:
            dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if dweight is None:
            dweight = _empty(channels, x, kind)
        if dbias is None:
            dbias = _empty(channels, x, kind)
        _capi.adamw_group_norm_backward(
            self.plan, dtype, _DTYPES[kind], samples, positions, self._view("dy", dy, x), view,
            _vector("weight", weight, channels, dev, kind), _vector("bias", bias, channels, dev, kind),
            _grid("mean", mean, (samples, self.groups), _F32, dev), _grid("rstd", rstd, (samples, self.groups), _F32, dev),
            self._view("dx", dx, x), _vector("dweight", dweight, channels, dev, kind),
            _vector("dbias", dbias, channels, dev, kind), _stream(None))
        return dx, dweight, dbias
