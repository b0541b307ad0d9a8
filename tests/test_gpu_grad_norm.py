"""GPU: the global gradient norm, the scale that clips, and clipping in place,
against the float64 definition.

Tolerance: a run of 64 squares sits in four float32 chains of at most 16, so
its sum is off by at most 18 * 2^-24 relative; the norm is its square root (9)
plus one rounding to float32: 10 * 2^-24 = 6e-7.  2^-20 = 9.5e-7 leaves the
conversion of clip_scale its own rounding.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import AdamWError, FusedAdamW, _capi
from oracle import grad_norm as GN

from _support import assert_guards_intact, bits_equal, dev, empty, host, scalar_f32, scalar_i32, zeros

pytestmark = pytest.mark.gpu
REL = 2.0 ** -20
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def _plan(grads, dtype, shift=0):
    gs = []
    for g in grads:
        t = empty(g.size, dtype, shift)
        t.copy_(torch.from_numpy(g.astype(np.float32)))
        gs.append(t)
    mk = lambda: [zeros(g.size) for g in grads]  # noqa: E731
    opt = FusedAdamW(mk(), gs, mk(), mk(), [0.1] * len(gs))
    return opt, gs


def _wide(gs):
    return [g.float().cpu().numpy().astype(np.float64) for g in gs]


def _run(opt, **kw):
    out = [scalar_f32(-1.0) for _ in range(3)]
    opt.grad_norm(out[0], clip_scale=out[1], found_inf=out[2], **kw)
    torch.cuda.synchronize()
    assert_guards_intact()
    return [float(t.item()) for t in out]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [[1], [7, 0, 1], [8, 16, 256, 2048], [100_003, 33, 5000], [3_000_017]])
def test_norm_matches_float64(sizes, dtype, shift):
    rng = np.random.default_rng(len(sizes) + sum(sizes))
    opt, gs = _plan([rng.normal(0, 1e-2, n) for n in sizes], dtype, shift)
    for max_norm, scale in ((np.inf, None), (0.01, None), (0.01, 128.0), (1e9, 3.0)):
        want = GN.norm_and_clip(_wide(gs), scale or 1.0, max_norm)
        got = _run(opt, max_norm=max_norm, grad_scale=None if scale is None else scalar_f32(scale))
        for g, w in zip(got[:2], want[:2]):
            assert abs(g - w) <= REL * abs(w), (max_norm, scale, got, want)
        assert got[2] == 0.0
        if want[1] == (scale or 1.0):
            assert got[1] == want[1]        # not clipped: the scale itself


def test_empty_plan_has_norm_zero():
    opt, _ = _plan([], torch.float32)
    assert _run(opt, max_norm=1.0) == [0.0, 1.0, 0.0]
    opt.clip_grads(scalar_f32(2.0))


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("dtype", DTYPES)
def test_non_finite_grads_are_found(bad, dtype):
    g = np.full(70_001, 1e-3)
    for at in (0, 35_000, 70_000):
        h = g.copy()
        h[at] = bad
        opt, _ = _plan([np.ones(5), h], dtype)
        norm, scale, found = _run(opt, max_norm=1.0)
        assert found == 1.0
        assert np.isnan(norm) if np.isnan(bad) else norm == np.inf
        assert np.isnan(scale) if np.isnan(bad) else scale == np.inf


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -80, 2.0 ** -130])
def test_squares_outside_float32(size, dtype):
    """Grads whose squares overflow or vanish in float32, alone and beside zeros."""
    g = np.zeros(10_000)
    g[::7] = size
    opt, gs = _plan([g], dtype)
    want = GN.norm_and_clip(_wide(gs))[0]
    got = _run(opt)
    assert want > 0 and abs(got[0] - want) <= REL * want and got[2] == 0.0


def test_norm_past_float32_is_found():
    opt, _ = _plan([np.full(100, 3e38)], torch.float32)
    assert _run(opt)[0] == np.inf and _run(opt)[2] == 1.0


def test_norm_is_the_same_bits_every_time():
    rng = np.random.default_rng(3)
    opt, _ = _plan([rng.normal(size=2_000_001), rng.normal(size=77)], torch.float32)
    assert len({tuple(_run(opt, max_norm=1.0)) for _ in range(20)}) == 1


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
def test_clip_grads_in_place(dtype, shift):
    rng = np.random.default_rng(5)
    opt, gs = _plan([rng.normal(size=n) for n in (100_003, 1, 17, 4096)], dtype, shift)
    before = [g.clone() for g in gs]
    opt.clip_grads(scalar_f32(1.0))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(gs, before))
    scale = scalar_f32(0.0)
    opt.grad_norm(scalar_f32(0.0), max_norm=1.0, clip_scale=scale)
    opt.clip_grads(scale)
    torch.cuda.synchronize()
    assert_guards_intact()
    inv = np.float32(1.0) / np.float32(scale.item())
    for g, b in zip(gs, before):
        want = (b.float() * float(inv)).to(dtype)      # one product, one rounding
        assert torch.equal(g, want)
    assert _run(opt)[0] == pytest.approx(1.0, rel=2e-3)


@pytest.mark.parametrize("dtype", DTYPES)
def test_clipped_step_equals_a_step_on_clipped_grads(dtype):
    """step(grad_scale=clip_scale) is bit for bit the step of grads g * (1 / clip_scale)."""
    rng = np.random.default_rng(9)
    grads = [rng.normal(0, 4, n) for n in (50_000, 33)]
    opt, gs = _plan(grads, dtype)
    norm, scale, found = (scalar_f32(0.0) for _ in range(3))
    opt.grad_norm(norm, max_norm=1.0, grad_scale=scalar_f32(16.0), clip_scale=scale, found_inf=found)
    lr = scalar_f32(1e-3)
    opt.step(lr, scalar_i32(0), grad_scale=scale, found_inf=found)
    inv = np.float32(1.0) / np.float32(scale.item())
    ref_g = [dev(g.float().cpu().numpy() * inv) for g in gs]
    mk = lambda: [zeros(g.numel()) for g in gs]  # noqa: E731
    ps, ms, vs = mk(), mk(), mk()
    FusedAdamW(ps, ref_g, ms, vs, [0.1] * 2).step(lr, scalar_i32(0))
    torch.cuda.synchronize()
    for a, b in zip(opt._keep[0] + opt._keep[2] + opt._keep[3], ps + ms + vs):
        assert bits_equal(host(a), host(b))


@pytest.mark.parametrize("mode", ["q8", "q4", "bf16_rem"])
def test_other_storage_modes(mode):
    rng = np.random.default_rng(2)
    n = 10_001
    g = dev(rng.normal(size=n).astype(np.float32))
    if mode == "bf16_rem":
        opt = FusedAdamW([zeros(n, torch.bfloat16)], [g], [zeros(n)], [zeros(n)], [0.0], mode=mode,
                         param_rems=[zeros(n, torch.int16)])
    else:
        codes = n if mode == "q8" else (n + 1) // 2
        blocks = -(-n // (256 if mode == "q8" else 128))
        opt = FusedAdamW([zeros(n)], [g], [zeros(codes, torch.uint8)], [zeros(codes, torch.uint8)], [0.0],
                         mode=mode, absmax_m=[zeros(blocks)], absmax_v=[zeros(blocks)])
    want = GN.norm_and_clip([host(g).astype(np.float64)])[0]
    assert abs(_run(opt)[0] - want) <= REL * want


def test_other_stream():
    rng = np.random.default_rng(1)
    opt, gs = _plan([rng.normal(size=1_000_003)], torch.float32)
    want = GN.norm_and_clip(_wide(gs))[0]
    s, norm = torch.cuda.Stream(), scalar_f32(0.0)
    s.wait_stream(torch.cuda.current_stream())
    opt.grad_norm(norm, stream=s)
    s.synchronize()
    assert abs(norm.item() - want) <= REL * want


def test_more_than_2_31_elements():
    n = 2 ** 31 + 4097
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[2 ** 31 - 1], g[2 ** 31], g[-1] = 1.0, 2.0, 4.0, 10.0
    p, m = (torch.empty(n, dtype=torch.float32, device="cuda") for _ in range(2))
    opt = FusedAdamW([p], [g], [m], None, [0.0])
    norm, scale = scalar_f32(0.0), scalar_f32(0.0)
    opt.grad_norm(norm, max_norm=5.5, clip_scale=scale)
    opt.clip_grads(scale)
    torch.cuda.synchronize()
    assert norm.item() == 11.0 and scale.item() == pytest.approx(2.0)
    assert [float(g[i]) for i in (0, 1, 2 ** 31 - 1, 2 ** 31, n - 1)] == [0.5, 0.0, 1.0, 2.0, 5.0]
    assert int(torch.count_nonzero(g)) == 4


def test_refusals():
    opt, _ = _plan([np.ones(8)], torch.float32)
    ok = scalar_f32(0.0)
    for max_norm in (0.0, -1.0, float("nan")):
        with pytest.raises(AdamWError) as e:
            opt.grad_norm(ok, max_norm=max_norm)
        assert e.value.status == _capi.EINVAL
    with pytest.raises(AdamWError) as e:
        _capi.adamw_grad_norm(opt.plan, 1.0, None, None, None, None, None)
    assert e.value.status == _capi.EINVAL
    with pytest.raises(AdamWError) as e:
        _capi.adamw_grad_norm(opt.plan, 1.0, None, ok.data_ptr() + 2, None, None, None)
    assert e.value.status == _capi.EALIGN
    with pytest.raises(AdamWError) as e:
        _capi.adamw_clip_grads(opt.plan, None, None)
    assert e.value.status == _capi.EINVAL
