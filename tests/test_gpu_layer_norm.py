"""GPU: layer norm forward and backward against the float64 definition.

Tolerances (u = 2^-24, all float32): the mean is off by at most a few u of the
row's mean magnitude (pairwise sums of 8 or more partial sums), xhat by a few u
of (|xhat| + |mean| rstd): with rows of |mean| rstd below 8 that is under
64 u = 4e-6 of (1 + |xhat|).  A column sum over R rows split over P partial
sums is off by at most (R / P + P) u of the sum of magnitudes: 2e-5 covers
R = 33,000 with P = 300.  Outputs of 16 bits add half an ulp (2^-9, 2^-12).
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import AdamWError, FusedLayerNorm, _capi
from oracle import layer_norm as LN

from _support import assert_guards_intact, dev, empty, guarded_empty

pytestmark = pytest.mark.gpu
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -24, torch.bfloat16: 0.0}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def wide(t):
    return t.detach().double().cpu().numpy()


def rows_of(a, dtype, pad=0, shift=0):
    """A guarded device matrix of a's values in dtype, `pad` elements between rows."""
    r, c = a.shape
    t = guarded_empty(r * (c + pad), dtype, shift).view(r, c + pad)
    t.fill_(7.0)
    t = t[:, :c]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def vec_of(a, dtype):
    t = empty(a.size, dtype)
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def close(got, want, size, dtype, rel):
    """|got - want| <= rel * size + the output type's half ulp of the result."""
    err = np.abs(wide(got) - want)
    bound = rel * size + (HALF_ULP[dtype] * (np.abs(want) + rel * size) + TINY[dtype])
    worst = np.max(err - bound) if err.size else -1.0
    assert worst <= 0, (float(worst), float(err.max()))


def check(rows, width, dtype, wdtype, pad=0, shift=0, offset=0.5, none=False, seed=0):
    rng = np.random.default_rng(seed + rows * 7 + width)
    x = rows_of(rng.normal(offset, 1.5, (rows, width)), dtype, pad, shift)
    dy = rows_of(rng.normal(0, 1, (rows, width)), dtype, pad, shift)
    w = None if none else vec_of(rng.normal(1, 0.2, width), wdtype)
    b = None if none else vec_of(rng.normal(0, 0.2, width), wdtype)
    y, dx = (rows_of(np.zeros((rows, width)), dtype, pad, shift) for _ in range(2))
    odt = dtype if none else wdtype
    dw, db = empty(width, odt), empty(width, odt)
    mean, rstd = empty(rows), empty(rows)
    ln = FusedLayerNorm(width)
    ln.forward(x, w, b, y=y, mean=mean, rstd=rstd)
    ln.backward(dy, x, w, mean, rstd, dx=dx, dweight=dw, dbias=db)
    torch.cuda.synchronize()
    assert_guards_intact()
    if pad:
        for t in (y, dx):
            assert (t.as_strided((rows, pad), t.stride(), t.storage_offset() + width) == 7.0).all()
    X, DY = wide(x), wide(dy)
    W, B = (None, None) if none else (wide(w), wide(b))
    wy, wm, wr = LN.forward(X, W, B)
    one = np.ones(width) if none else np.abs(W)
    xhat = (X - wm[:, None]) * wr[:, None]
    ratio = 1 + np.abs(wm * wr)[:, None]
    close(mean, wm, np.abs(X).mean(1) + 1e-30, torch.float32, 2e-6)
    close(rstd, wr, wr, torch.float32, 4e-6)
    close(y, wy, (np.abs(xhat) + ratio) * one, dtype, 4e-6)
    # the backward pass takes the library's own mean and rstd, as a user's program does
    gx, gw, gb = LN.backward(DY, X, W, wide(mean), wide(rstd))
    g = np.abs(DY) * one
    size = wide(rstd)[:, None] * (g + g.mean(1, keepdims=True)
                                  + np.abs(xhat) * (g * (np.abs(xhat) + ratio)).mean(1, keepdims=True))
    close(dx, gx, size * ratio, dtype, 4e-6)
    close(dw, gw, (np.abs(DY) * (np.abs(xhat) + ratio)).sum(0), odt, 2e-5)
    close(db, gb, np.abs(DY).sum(0), odt, 2e-5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [1, 2, 7, 8, 31, 64, 255, 256, 257, 768, 1000, 1601, 2048, 4096, 5001, 8192,
                                   12_288, 20_003, 40_960])
def test_widths(width, dtype):
    # one element: x - mean is 0, and rstd = 1 / sqrt(eps) magnifies nothing
    check(3 if width > 1 else 2, width, dtype, torch.float32, offset=0.0 if width == 1 else 0.5)


@pytest.mark.parametrize("rows", [1, 2, 151, 303, 305, 2000])
@pytest.mark.parametrize("width", [96, 1601, 4096])
def test_rows(rows, width):
    check(rows, width, torch.bfloat16, torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [8193, 10_001, 12_288, 36_864])
def test_wide_rows(width, dtype):
    check(700 if width < 20_000 else 310, width, dtype, dtype)
    check(5, width, dtype, torch.float32, pad=3, shift=1)


def test_many_rows():
    check(33_000, 65, torch.float32, torch.float32)
    check(33_000, 128, torch.float16, torch.float16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [64, 1000, 1601, 4096])
@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 0), (0, 1), (5, 3)])
def test_strides_and_alignment(width, dtype, pad, shift):
    check(9, width, dtype, dtype, pad, shift)


def compare(x, dy, y, dx):
    """Both passes without parameters, on matrices given, with the bounds above."""
    X, DY, dtype = wide(x), wide(dy), x.dtype
    ln = FusedLayerNorm(x.shape[1])
    _, mean, rstd = ln.forward(x, y=y)
    _, dw, db = ln.backward(dy, x, None, mean, rstd, dx=dx)
    torch.cuda.synchronize()
    assert_guards_intact()
    wy, wm, wr = LN.forward(X)
    gx, gw, gb = LN.backward(DY, X, None, wide(mean), wide(rstd))
    xhat = np.abs((X - wm[:, None]) * wr[:, None])
    ratio = 1 + np.abs(wm * wr)[:, None]
    g = np.abs(DY)
    close(y, wy, xhat + ratio, dtype, 4e-6)
    size = wide(rstd)[:, None] * (g + g.mean(1, keepdims=True)
                                  + xhat * (g * (xhat + ratio)).mean(1, keepdims=True))
    close(dx, gx, size * ratio, dtype, 4e-6)
    close(dw, gw, (g * (xhat + ratio)).sum(0), dtype, 2e-5)
    close(db, gb, g.sum(0), dtype, 2e-5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 7, 40, 700])
@pytest.mark.parametrize("width", [3, 8, 17, 505, 509, 1021, 2045, 8190])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 2), (2, 7), (4, 3)])
def test_what_lies_beside_a_row_is_not_used(rows, width, dtype, pad, shift):
    """NaN between the rows, which share 16-byte words with it; rows of few elements in one word."""
    rng = np.random.default_rng(rows + 31 * width + pad)
    make = lambda a: rows_of(a, dtype, pad, shift)
    x, dy = make(rng.normal(0.5, 1.5, (rows, width))), make(rng.normal(0, 1, (rows, width)))
    y, dx = make(np.zeros((rows, width))), make(np.zeros((rows, width)))
    for t in (x, dy):
        t.as_strided((rows, pad), t.stride(), t.storage_offset() + width).fill_(float("nan"))
    compare(x, dy, y, dx)
    for t in (y, dx):
        assert (t.as_strided((rows, pad), t.stride(), t.storage_offset() + width) == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [5, 64, 1000, 1601, 4100, 9001, 20_003])
@pytest.mark.parametrize("rows", [1, 40, 700])
def test_matrices_that_lie_each_in_its_own_way(rows, width, dtype):
    rng = np.random.default_rng(rows + 31 * width)
    x = rows_of(rng.normal(0.5, 1.5, (rows, width)), dtype, 3, 1)
    dy = rows_of(rng.normal(0, 1, (rows, width)), dtype, 0, 2)
    y, dx = rows_of(np.zeros((rows, width)), dtype), rows_of(np.zeros((rows, width)), dtype, 1, 5)
    compare(x, dy, y, dx)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [17, 501, 1601, 9001])
def test_odd_rows_in_place(width, dtype):
    """dx over dy and y over x: rows share words with rows that another CTA writes."""
    rng = np.random.default_rng(width)
    x = rows_of(rng.normal(0.5, 1.5, (900, width)), dtype)
    dy = rows_of(rng.normal(0, 1, (900, width)), dtype)
    ln = FusedLayerNorm(width)
    y, mean, rstd = ln.forward(x)
    dx, _, _ = ln.backward(dy, x, None, mean, rstd)
    ln.backward(dy, x, None, mean, rstd, dx=dy)
    ln.forward(x, y=x)
    torch.cuda.synchronize()
    assert_guards_intact()
    assert torch.equal(dx, dy) and torch.equal(x, y)


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_weight_and_bias(dtype):
    check(17, 500, dtype, dtype, none=True)


def test_large_mean_keeps_its_variance():
    """Rows whose mean is far above their spread: a variance from squares alone would be lost."""
    check(5, 4096, torch.float32, torch.float32, offset=10.0)


def test_in_place():
    rng = np.random.default_rng(4)
    for width in (100, 4096, 20_003):
        x = rows_of(rng.normal(size=(6, width)), torch.float32)
        dy = rows_of(rng.normal(size=(6, width)), torch.float32)
        ln = FusedLayerNorm(width)
        y, mean, rstd = ln.forward(x)
        dx, _, _ = ln.backward(dy, x, None, mean, rstd)
        z, d = x.clone(), dy.clone()
        ln.backward(d, z, None, mean, rstd, dx=d)
        ln.forward(z, y=z)
        assert torch.equal(z, y) and torch.equal(d, dx)


def test_only_one_of_the_gradients():
    rng = np.random.default_rng(6)
    x = rows_of(rng.normal(size=(40, 300)), torch.float32)
    ln = FusedLayerNorm(300)
    y, mean, rstd = ln.forward(x)
    dx, dw, db = ln.backward(y, x, None, mean, rstd)
    args = (0, 0, 40, y.data_ptr(), 300, x.data_ptr(), 300, None, mean.data_ptr(), rstd.data_ptr())
    for keep in range(2):
        out = [empty(300), empty(300)]
        dx2 = torch.empty_like(dx)
        _capi.adamw_layer_norm_backward(ln.plan, *args, dx2.data_ptr(), 300,
                                        out[0].data_ptr() if keep == 0 else None,
                                        out[1].data_ptr() if keep == 1 else None,
                                        torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out[keep], (dw, db)[keep]) and torch.equal(dx2, dx)


def test_no_rows():
    ln = FusedLayerNorm(64)
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = ln.forward(x)
    dx, dw, db = ln.backward(x, x, None, mean, rstd)
    assert y.shape == (0, 64) and dx.shape == (0, 64)
    assert not dw.any() and not db.any()


def test_gradients_are_the_same_bits_every_time():
    rng = np.random.default_rng(8)
    x = rows_of(rng.normal(size=(5000, 777)), torch.bfloat16)
    dy = rows_of(rng.normal(size=(5000, 777)), torch.bfloat16)
    ln = FusedLayerNorm(777)
    _, mean, rstd = ln.forward(x)
    first = ln.backward(dy, x, None, mean, rstd)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, ln.backward(dy, x, None, mean, rstd)))


def test_non_finite_rows_stay_in_their_rows():
    rng = np.random.default_rng(10)
    for width in (96, 4096):
        a = rng.normal(size=(8, width))
        clean = FusedLayerNorm(width).forward(rows_of(a, torch.float32))[0]
        a[3, 5], a[6, 7] = np.nan, np.inf
        y, mean, rstd = FusedLayerNorm(width).forward(rows_of(a, torch.float32))
        bad = torch.zeros(8, dtype=torch.bool, device="cuda")
        bad[3] = bad[6] = True
        assert torch.equal(y[~bad], clean[~bad]) and torch.isnan(y[3]).all() and torch.isnan(rstd[bad]).all()


def test_offsets_past_32_bits():
    width = 65_537
    rows = 2 ** 31 // width + 3
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    some = [0, rows // 2, rows - 2, rows - 1]
    for t in some:
        x[t] = torch.randn(width, device="cuda", generator=g).to(torch.bfloat16)
    ln = FusedLayerNorm(width)
    y, mean, rstd = ln.forward(x)
    dx, dw, db = ln.backward(x, x, None, mean, rstd)
    sub = x[some].contiguous()
    y2, m2, r2 = ln.forward(sub)
    dx2, dw2, db2 = ln.backward(sub, sub, None, m2, r2)
    assert torch.equal(y[some], y2) and torch.equal(dx[some], dx2) and torch.equal(mean[some], m2)
    # rows of zeros add nothing
    assert torch.allclose(dw.float(), dw2.float(), rtol=2.0 ** -7, atol=1e-4)


def test_differences():
    """dx and dweight against central differences of the library's own forward pass."""
    rng = np.random.default_rng(12)
    a, w, dy = rng.normal(size=(3, 40)), rng.normal(1, 0.3, 40), rng.normal(size=(3, 40))
    ln = FusedLayerNorm(40)
    W = dev(w.astype(np.float32))
    X, DY = rows_of(a, torch.float32), rows_of(dy, torch.float32)
    _, mean, rstd = ln.forward(X, W)
    dx, dw, _ = ln.backward(DY, X, W, mean, rstd)
    loss = lambda x, v: float((ln.forward(x, v)[0].double() * DY.double()).sum())  # noqa: E731
    h = 2.0 ** -7     # y is good to 4e-6, so a quotient to about 40 * 4e-6 / h = 0.02, plus h^2
    for r, c in ((0, 0), (1, 17), (2, 39)):
        up, down = X.clone(), X.clone()
        up[r, c] += h
        down[r, c] -= h
        assert abs((loss(up, W) - loss(down, W)) / (2 * h) - float(dx[r, c])) < 0.02
    for c in (0, 20):
        up, down = W.clone(), W.clone()
        up[c] += h
        down[c] -= h
        assert abs((loss(X, up) - loss(X, down)) / (2 * h) - float(dw[c])) < 0.02


def test_refusals():
    ln = FusedLayerNorm(64)
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="columns"):
        ln.forward(torch.zeros(4, 63, device="cuda"))
    with pytest.raises(TypeError, match="dtype"):
        ln.forward(x.double())
    with pytest.raises(TypeError, match="weight"):
        ln.forward(x, torch.ones(64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError, match="64 elements"):
        ln.forward(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        ln.forward(x.cpu())
    with pytest.raises(ValueError, match="shape"):
        ln.forward(x, y=torch.zeros(4, 32, device="cuda"))
    s = [x.data_ptr()] * 4
    with pytest.raises(AdamWError) as e:
        _capi.adamw_layer_norm_forward(ln.plan, 9, 0, 4, s[0], 64, None, None, s[1], 64, s[2], s[3], None)
    assert e.value.status == _capi.EDTYPE
    with pytest.raises(AdamWError) as e:
        _capi.adamw_layer_norm_forward(ln.plan, 1, 2, 4, s[0], 64, None, None, s[1], 64, s[2], s[3], None)
    assert e.value.status == _capi.EUNSUPPORTED
    with pytest.raises(AdamWError) as e:
        _capi.adamw_layer_norm_forward(ln.plan, 0, 0, 4, s[0], 63, None, None, s[1], 64, s[2], s[3], None)
    assert e.value.status == _capi.EINVAL
    with pytest.raises(AdamWError) as e:
        _capi.adamw_layer_norm_backward(ln.plan, 0, 0, 4, s[0] + 2, 64, s[0], 64, None, s[1], s[2], s[3], 64,
                                        None, None, None)
    assert e.value.status == _capi.EALIGN
