"""Losses on token log-probabilities, and layer norm, with torch tensors in place of raw pointers.

``FusedTokenLoss`` scores tokens, and gives the clipped policy loss and the
preference loss with the gradient of the logits.  ``FusedLayerNorm`` is layer
norm forward and backward with the gradients of its weight and bias.  Both hold
a plan of the library (its workspace) on the current device, check their
arguments and launch on the current stream or ``stream``; all arithmetic runs in
the library's CUDA kernels.  Outputs that are not given are allocated for the stream
of the launch.  Inputs stay the caller's: one that was made on another stream has to
be ready on this one, and to be kept until the work is done.
"""

from __future__ import annotations

import torch

from . import _capi, _stream

_DTYPES = {torch.float32: _capi.F32, torch.float16: _capi.F16, torch.bfloat16: _capi.BF16}
_LABEL_BYTES = {torch.int32: 4, torch.int64: 8}
_F32 = torch.float32


def _elsewhere(name, t, device, what):
    """Raises unless no device in particular is asked for and t is on a GPU."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a {what}")
    if device is not None:
        raise ValueError(f"{name} is on device {t.get_device()}, the plan on device {device}")


def _rows(name, t, dtype=None, shape=None, device=None):
    """Checks a matrix of rows (the last axis contiguous) and returns its row stride."""
    if t.get_device() != device:
        _elsewhere(name, t, device, "CUDA matrix")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a CUDA matrix")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    rows, width = here = t.shape
    if shape is not None and here != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(here)}")
    stride, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    if rows < 2:
        return width
    if stride < width:
        raise ValueError(f"{name} has overlapping rows")
    return stride


def _vector(name, t, n, device=None, dtype=_F32):
    """Address of a contiguous CUDA vector of n elements; None stays None."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        _elsewhere(name, t, device, f"contiguous CUDA tensor of {n} elements")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} elements")
    return t.data_ptr()


def _empty(n, like, dtype=_F32):
    return torch.empty(n, dtype=dtype, device=like.device)


def _on(stream):
    """A context with ``stream`` (a stream or its handle) as the current one."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))    # 0 and 1: the default one
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


class _Plan:
    """A plan of the library on the device that was current when it was made."""

    _destroy = None

    def close(self) -> None:
        if getattr(self, "plan", None):
            self._destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class FusedTokenLoss(_Plan):
    """Losses on the log-probability of one token per row of logits.

    ``max_rows`` rows per call at most; ``max_pairs`` pairs for ``preference``.
    logits [rows, vocab] float32, float16 or bfloat16, any row stride; labels
    int32 or int64 [rows], a label outside [0, vocab) (such as -100) marks a row
    that counts for nothing; per-row inputs and outputs float32 [rows].
    """

    _destroy = staticmethod(_capi.adamw_loss_plan_destroy)

    def __init__(self, max_rows: int, max_pairs: int = 0):
        self.plan = _capi.adamw_loss_plan_create(int(max_rows), int(max_pairs))
        self.device = torch.cuda.current_device()
        # the argument records, filled anew by every call
        self._z = _capi.adamw_logits()
        self._policy = _capi.adamw_policy()
        self._preference = _capi.adamw_preference()

    def status(self) -> int:
        """Device-side fault bits (0 = healthy); raises AdamWError if a bounded wait gave up."""
        return _capi.adamw_loss_plan_status(self.plan)

    def _logits(self, logits, labels, temperature):
        if logits.dtype not in _DTYPES:
            raise TypeError(f"unsupported logits dtype {logits.dtype}")
        if labels.dtype not in _LABEL_BYTES:
            raise TypeError(f"labels must be int32 or int64, got {labels.dtype}")
        z, dev = self._z, self.device
        z.row_stride = _rows("logits", logits, None, None, dev)
        z.rows, z.vocab = logits.shape
        z.labels = _vector("labels", labels, logits.shape[0], dev, labels.dtype)
        z.logits = logits.data_ptr()
        z.label_bytes = _LABEL_BYTES[labels.dtype]
        z.dtype = _DTYPES[logits.dtype]
        z.temperature = temperature
        return z

    def _gradient(self, logits, dlogits, backward):
        if not backward:
            return None, None, 0
        if dlogits is None:
            dlogits = torch.empty_like(logits)
        return dlogits, dlogits.data_ptr(), _rows("dlogits", dlogits, logits.dtype, logits.shape, self.device)

    def logps(self, logits, labels, *, temperature=1.0, logps=None, lse=None, stream=None):
        """(logps, lse) of every row: the log-probability of its token and the log of its sum of
        exponentials, 0 where the row has no token."""
        if stream is not None:
            with _on(stream):
                return self.logps(logits, labels, temperature=temperature, logps=logps, lse=lse)
        z = self._logits(logits, labels, temperature)
        n, dev = logits.shape[0], self.device
        if logps is None:
            logps = _empty(n, logits)
        if lse is None:
            lse = _empty(n, logits)
        _capi.adamw_token_logps(self.plan, z, _vector("logps", logps, n, dev), _vector("lse", lse, n, dev),
                                _stream(None))
        return logps, lse

    def policy(self, logits, labels, weights, advantages, old_logps=None, ref_logps=None, *,
               clip=(0.2, 0.2), kl_coef=0.0, temperature=1.0, grad_scale=None, backward=True,
               stats=None, logps=None, dlogits=None, stream=None):
        """Clipped policy loss with a KL term: (stats, logps, dlogits).

        stats float32 [4]: the loss (sum of weights times rows' terms), its policy part, the KL
        sum, the weight of the clipped rows.  ``weights`` is the mask already divided by whatever
        the mean runs over.  dlogits (None when ``backward`` is false) is the gradient of
        stats[0], times ``grad_scale``; it may be given, also as the logits themselves.
        """
        if stream is not None:
            with _on(stream):
                return self.policy(logits, labels, weights, advantages, old_logps, ref_logps, clip=clip,
                                   kl_coef=kl_coef, temperature=temperature, grad_scale=grad_scale,
                                   backward=backward, stats=stats, logps=logps, dlogits=dlogits)
        z = self._logits(logits, labels, temperature)
        n, dev = logits.shape[0], self.device
        p = self._policy
        p.weights = _vector("weights", weights, n, dev)
        p.advantages = _vector("advantages", advantages, n, dev)
        p.old_logps = _vector("old_logps", old_logps, n, dev)
        p.ref_logps = _vector("ref_logps", ref_logps, n, dev)
        p.clip_low, p.clip_high = clip
        p.kl_coef = kl_coef
        p.grad_scale_dev = _vector("grad_scale", grad_scale, 1, dev)
        if stats is None:
            stats = _empty(4, logits)
        if logps is None:
            logps = _empty(n, logits)
        dlogits, at, stride = self._gradient(logits, dlogits, backward)
        _capi.adamw_policy_loss(self.plan, z, p, _vector("stats", stats, 4, dev),
                                _vector("logps", logps, n, dev), at, stride, _stream(None))
        return stats, logps, dlogits

    def preference(self, logits, labels, weights, ref_logps, seq_starts, *, beta=0.1,
                   label_smoothing=0.0, temperature=1.0, grad_scale=None, backward=True, stats=None,
                   rewards=None, logps=None, dlogits=None, stream=None):
        """Preference loss over pairs of sequences: (stats, rewards, logps, dlogits).

        seq_starts int32 [2 pairs + 1] (on the device): sequence s is rows seq_starts[s] to
        seq_starts[s + 1] - 1; the chosen ones first, then the rejected ones in the same order.
        ``weights`` (or None) weighs a row in its sequence's sum.  stats float32 [4]: the loss,
        the share of pairs with the chosen one ahead, mean chosen and mean rejected reward;
        rewards float32 [2 pairs].
        """
        if stream is not None:
            with _on(stream):
                return self.preference(logits, labels, weights, ref_logps, seq_starts, beta=beta,
                                       label_smoothing=label_smoothing, temperature=temperature,
                                       grad_scale=grad_scale, backward=backward, stats=stats, rewards=rewards,
                                       logps=logps, dlogits=dlogits)
        z = self._logits(logits, labels, temperature)
        n, dev = logits.shape[0], self.device
        pairs = (seq_starts.numel() - 1) // 2
        p = self._preference
        p.weights = _vector("weights", weights, n, dev)
        p.ref_logps = _vector("ref_logps", ref_logps, n, dev)
        p.seq_starts = _vector("seq_starts", seq_starts, 2 * pairs + 1, dev, torch.int32)
        p.n_pairs = pairs
        p.beta = beta
        p.label_smoothing = label_smoothing
        p.grad_scale_dev = _vector("grad_scale", grad_scale, 1, dev)
        if stats is None:
            stats = _empty(4, logits)
        if rewards is None:
            rewards = _empty(2 * pairs, logits)
        if logps is None:
            logps = _empty(n, logits)
        dlogits, at, stride = self._gradient(logits, dlogits, backward)
        _capi.adamw_preference_loss(self.plan, z, p, _vector("stats", stats, 4, dev),
                                    _vector("rewards", rewards, 2 * pairs, dev),
                                    _vector("logps", logps, n, dev), at, stride, _stream(None))
        return stats, rewards, logps, dlogits


class FusedLayerNorm(_Plan):
    """Layer norm over rows of ``width`` elements.

    Rows [rows, width] float32, float16 or bfloat16, any row stride; weight and bias
    float32 or of the rows' dtype, or None; mean and rstd float32 [rows].
    """

    _destroy = staticmethod(_capi.adamw_layer_norm_plan_destroy)

    def __init__(self, width: int, eps: float = 1e-5):
        self.plan = _capi.adamw_layer_norm_plan_create(int(width), float(eps))
        self.device = torch.cuda.current_device()
        self.width = int(width)

    def status(self) -> int:
        """Device-side fault bits (0 = healthy); raises AdamWError if a bounded wait gave up."""
        return _capi.adamw_layer_norm_plan_status(self.plan)

    def _check(self, x, weight):
        if x.dtype not in _DTYPES:
            raise TypeError(f"unsupported dtype {x.dtype}")
        if weight is not None and weight.dtype not in (torch.float32, x.dtype):
            raise TypeError(f"the weight must be float32 or {x.dtype}, got {weight.dtype}")
        stride = _rows("x", x, None, None, self.device)
        if x.shape[1] != self.width:
            raise ValueError(f"x must have {self.width} columns, got {x.shape[1]}")
        return stride, (x.dtype if weight is None else weight.dtype)

    def forward(self, x, weight=None, bias=None, *, y=None, mean=None, rstd=None, stream=None):
        """(y, mean, rstd)"""
        if stream is not None:
            with _on(stream):
                return self.forward(x, weight, bias, y=y, mean=mean, rstd=rstd)
        stride, wdt = self._check(x, weight if weight is not None else bias)
        n, dev = x.shape[0], self.device
        if y is None:
            y = torch.empty_like(x)
        if mean is None:
            mean = _empty(n, x)
        if rstd is None:
            rstd = _empty(n, x)
        _capi.adamw_layer_norm_forward(
            self.plan, _DTYPES[x.dtype], _DTYPES[wdt], n, x.data_ptr(), stride,
            _vector("weight", weight, self.width, dev, wdt), _vector("bias", bias, self.width, dev, wdt),
            y.data_ptr(), _rows("y", y, x.dtype, x.shape, dev), _vector("mean", mean, n, dev),
            _vector("rstd", rstd, n, dev), _stream(None))
        return y, mean, rstd

    def backward(self, dy, x, weight, mean, rstd, *, dx=None, dweight=None, dbias=None, stream=None):
        """(dx, dweight, dbias) from the forward pass's x, mean and rstd; the weight's and bias's
        gradients in the weight's dtype (the rows' when the weight is None)."""
        if stream is not None:
            with _on(stream):
                return self.backward(dy, x, weight, mean, rstd, dx=dx, dweight=dweight, dbias=dbias)
        stride, wdt = self._check(x, weight)
        n, dev = x.shape[0], self.device
        if dx is None:
            dx = torch.empty_like(x)
        if dweight is None:
            dweight = _empty(self.width, x, wdt)
        if dbias is None:
            dbias = _empty(self.width, x, wdt)
        _capi.adamw_layer_norm_backward(
            self.plan, _DTYPES[x.dtype], _DTYPES[wdt], n, dy.data_ptr(),
            _rows("dy", dy, x.dtype, x.shape, dev), x.data_ptr(), stride,
            _vector("weight", weight, self.width, dev, wdt), _vector("mean", mean, n, dev),
            _vector("rstd", rstd, n, dev), dx.data_ptr(), _rows("dx", dx, x.dtype, x.shape, dev),
            _vector("dweight", dweight, self.width, dev, wdt), _vector("dbias", dbias, self.width, dev, wdt),
            _stream(None))
        return dx, dweight, dbias
