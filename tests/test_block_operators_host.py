"""A block's operators without a GPU: record layouts, and the refusals of the entry points
and of the Python classes, before any device work."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedDropout, FusedGroupNorm, FusedRouter
from adamw_optimizer_step_tensor_gb300 import _capi as C
from adamw_optimizer_step_tensor_gb300 import block_operators as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORDS = (C.adamw_router, C.adamw_channels_last)
NAMES = {"ADAMW_SCORE_SOFTMAX": B._SCORES["softmax"], "ADAMW_SCORE_SIGMOID": B._SCORES["sigmoid"],
         "ADAMW_GROUP_MAX": B._GROUP_SCORES["max"], "ADAMW_GROUP_TOP2": B._GROUP_SCORES["top2"],
         "ADAMW_ACT_NONE": B._ACTIVATIONS["none"], "ADAMW_ACT_SILU": B._ACTIVATIONS["silu"]}


def _status(fn, *args):
    with pytest.raises(C.AdamWError) as e:
        fn(*args)
    return e.value.status


def test_record_layouts_and_names(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "adamw.h"', "int main(void) {"]
    for r in RECORDS:
        lines.append(f'printf("%zu\\n", sizeof({r.__name__}));')
        lines += [f'printf("%zu\\n", offsetof({r.__name__}, {f}));' for f, _ in r._fields_]
    lines += [f'printf("%d\\n", (int){n});' for n in NAMES]
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split()
    want = []
    for r in RECORDS:
        want += [ctypes.sizeof(r)] + [getattr(r, f).offset for f, _ in r._fields_]
    assert [int(v) for v in got] == want + list(NAMES.values())


def test_dropout_refuses():
    def call(dtype=0, rows=4, width=8, x=16, xs=8, r=None, rs=0, y=32, ys=8, p=0.1, step=None):
        return lambda: C.adamw_dropout(dtype, rows, width, x, xs, r, rs, y, ys, p, 1, step, 0, None)

    assert _status(call(dtype=7)) == C.EDTYPE
    for kw in (dict(rows=-1), dict(width=-1), dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(xs=7), dict(ys=7),
               dict(r=64, rs=7), dict(x=None), dict(y=None), dict(y=16, ys=9), dict(r=32, rs=9)):
        assert _status(call(**kw)) == C.EINVAL, kw
    for kw in (dict(x=18), dict(y=17), dict(r=66, rs=8), dict(step=2)):
        assert _status(call(**kw)) == C.EALIGN, kw
    assert _status(call(xs=2 ** 60)) == C.EUNSUPPORTED
    call(rows=0, x=None, y=None)()                 # nothing to do
    call(width=0, x=None, y=None)()


def _router(**kw):
    v = dict(experts=16, top_k=2, groups=4, top_groups=2, score=0, group_score=0, renormalise=1, scale=1.0)
    v.update(kw)
    return C.adamw_router(*v.values())


def test_router_plans_are_checked_first():
    for kw in (dict(experts=0), dict(top_k=0), dict(groups=0), dict(top_groups=0), dict(groups=3), dict(top_groups=5),
               dict(top_k=9), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert _status(C.adamw_router_plan_create, _router(**kw), 8) == C.EINVAL, kw
    assert _status(C.adamw_router_plan_create, _router(), -1) == C.EINVAL
    for kw in (dict(experts=1025), dict(top_k=33), dict(groups=64, experts=128)):
        assert _status(C.adamw_router_plan_create, _router(**kw), 8) == C.EUNSUPPORTED, kw
    assert _status(C.adamw_router_plan_create, _router(), 2 ** 30) == C.EUNSUPPORTED
    assert _status(C.adamw_router_plan_create, _router(score=2), 8) == C.EDTYPE
    assert _status(C.adamw_router_plan_create, _router(group_score=-1), 8) == C.EDTYPE
    lib = C.load()
    assert lib.adamw_router_plan_create(_router(), 8, None) == C.EINVAL
    assert lib.adamw_router_plan_create(None, 8, ctypes.byref(ctypes.c_void_p())) == C.EINVAL


def test_group_norm_plans_are_checked_first():
    for args in ((0, 1, 1, 1e-5, 0), (8, 0, 1, 1e-5, 0), (8, 3, 1, 1e-5, 0), (8, 2, -1, 1e-5, 0), (8, 2, 1, -1.0, 0),
                 (8, 2, 1, float("nan"), 0)):
        assert _status(C.adamw_group_norm_plan_create, *args) == C.EINVAL, args
    assert _status(C.adamw_group_norm_plan_create, 2 ** 16 + 1, 1, 1, 1e-5, 0) == C.EUNSUPPORTED
    assert _status(C.adamw_group_norm_plan_create, 8, 8, 2 ** 38, 1e-5, 0) == C.EUNSUPPORTED
    assert _status(C.adamw_group_norm_plan_create, 8, 2, 1, 1e-5, 2) == C.EDTYPE
    assert C.load().adamw_group_norm_plan_create(8, 2, 1, 1e-5, 0, None) == C.EINVAL


def test_null_plans_are_refused():
    v = C.adamw_channels_last(16, 8, 8)
    assert _status(C.adamw_route, None, 0, 1, 16, 8, None, 16, 16, 16, 16, None) == C.EINVAL
    assert _status(C.adamw_route_backward, None, 0, 1, 16, 8, 16, 16, 16, 8, None) == C.EINVAL
    assert _status(C.adamw_route_balance, None, 16, 0.1, 16, None) == C.EINVAL
    assert _status(C.adamw_route_dispatch, None, 0, 1, 8, 16, 8, 16, 16, 2, 8, None) == C.EINVAL
    assert _status(C.adamw_route_combine, None, 0, 1, 8, 16, 2, 8, 16, None, 16, 8, None) == C.EINVAL
    assert _status(C.adamw_route_combine_backward, None, 0, 1, 8, 16, 8, 16, 2, 8, 16, 16, 16, 8, 16, None) == C.EINVAL
    assert _status(C.adamw_group_norm_forward, None, 0, 0, 1, 1, v, None, None, v, 16, 16, None) == C.EINVAL
    assert _status(C.adamw_group_norm_backward, None, 0, 0, 1, 1, v, v, None, None, 16, 16, v, None, None, None) == C.EINVAL
    assert _status(C.adamw_group_norm_plan_status, None) == C.EINVAL
    assert _status(C.adamw_group_norm_plan_set_wait_limit, None, 0) == C.EINVAL
    C.adamw_router_plan_destroy(None)
    C.adamw_group_norm_plan_destroy(None)


class _Fake:
    """A torch tensor's face over a CPU tensor that says on which GPU it is."""

    is_cuda = True

    def __init__(self, t, device=0):
        self._t, self._device = t, device

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return self._device

    def view(self, *shape):
        return _Fake(self._t.view(*shape), self._device)


@pytest.fixture
def launches(monkeypatch):
    count = []
    for name in ("adamw_dropout", "adamw_route", "adamw_route_backward", "adamw_route_balance", "adamw_route_dispatch",
                 "adamw_route_combine", "adamw_route_combine_backward", "adamw_group_norm_forward",
                 "adamw_group_norm_backward"):
        monkeypatch.setattr(B._capi, name, lambda *args: count.append(args))
    for name in ("adamw_router_plan", "adamw_group_norm_plan"):
        monkeypatch.setattr(B._capi, name + "_create", lambda *args: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(B, "_stream", lambda s: 1)
    return count


def _calls():
    """Every call with its tensors by name."""
    f = lambda *s, dtype=torch.float32: _Fake(torch.zeros(*s, dtype=dtype))  # noqa: E731
    i = lambda *s: f(*s, dtype=torch.int32)  # noqa: E731
    drop, router, norm = FusedDropout(0.1), FusedRouter(4, 8, 2), FusedGroupNorm(8, 2, 4)
    k = lambda: f(4, 2)  # noqa: E731
    v = lambda: f(3, 5, 8)  # noqa: E731
    return [
        (drop.forward, dict(x=f(4, 8), step=i(1), residual=f(4, 8), y=f(4, 8))),
        (drop.backward, dict(dy=f(4, 8), step=i(1), dx=f(4, 8))),
        (router.route, dict(logits=f(4, 8), bias=f(8), weights=k(), ids=i(4, 2), slots=i(4, 2), starts=i(9))),
        (router.backward, dict(dweights=k(), logits=f(4, 8), ids=i(4, 2), dlogits=f(4, 8))),
        (lambda bias, starts: router.balance(bias, starts, 0.1), dict(bias=f(8), starts=i(9))),
        (router.dispatch, dict(x=f(4, 6), slots=i(4, 2), xs=f(8, 6))),
        (router.combine, dict(ys=f(8, 6), slots=i(4, 2), weights=k(), y=f(4, 6))),
        (router.combine_backward, dict(dy=f(4, 6), ys=f(8, 6), slots=i(4, 2), weights=k(), dys=f(8, 6), dweights=k())),
        (norm.forward, dict(x=v(), weight=f(8), bias=f(8), y=v(), mean=f(3, 2), rstd=f(3, 2))),
        (norm.backward, dict(dy=v(), x=v(), weight=f(8), bias=f(8), mean=f(3, 2), rstd=f(3, 2), dx=v(), dweight=f(8),
                             dbias=f(8))),
    ]


def test_every_tensor_s_device_is_checked(launches):
    for call, tensors in _calls():
        call(**tensors)
        assert len(launches) == 1
        for name, t in tensors.items():
            with pytest.raises(ValueError, match=f"^{name} is on device 1, the plan on device 0"):
                call(**{**tensors, name: _Fake(t._t, 1)})
        assert len(launches) == 1
        launches.clear()


def test_every_tensor_s_type_and_shape_are_checked(launches):
    for call, tensors in _calls():
        for name, t in tensors.items():
            with pytest.raises(TypeError):
                call(**{**tensors, name: _Fake(t._t.double())})
            if name in ("x", "dy", "ys") and call.__name__ in ("forward", "backward", "dispatch", "combine"):
                continue                       # sets the shape of the rest
            with pytest.raises(ValueError):
                call(**{**tensors, name: _Fake(torch.zeros(*t._t.shape[:-1], t._t.shape[-1] + 1, dtype=t._t.dtype))})
    assert not launches


def test_strides(launches):
    drop, norm = FusedDropout(0.5), FusedGroupNorm(8, 2, 4)
    t = torch.zeros(6, 4, 16)
    drop.forward(_Fake(t), y=_Fake(t.clone()))
    drop.forward(_Fake(t[:, 0, :8]), y=_Fake(torch.zeros(6, 8)))
    drop.forward(_Fake(t[:, :, 3:9]), y=_Fake(torch.zeros(6, 4, 6)))
    assert [a[1:3] + (a[4],) for a in launches] == [(24, 16, 16), (6, 8, 64), (24, 6, 16)]
    for bad in (t[:, :2, :8], t[0].t()):
        with pytest.raises(ValueError):
            drop.forward(_Fake(bad), y=_Fake(torch.zeros(bad.shape)))
    launches.clear()
    norm.forward(_Fake(t[:, :, 8:]), y=_Fake(torch.zeros(6, 4, 8)), mean=_Fake(torch.zeros(6, 2)), rstd=_Fake(torch.zeros(6, 2)))
    x, y = launches[0][5], launches[0][8]
    assert (x.sample_stride, x.position_stride, y.sample_stride, y.position_stride) == (64, 16, 32, 8)
    with pytest.raises(ValueError, match="contiguous along"):
        norm.forward(_Fake(torch.zeros(6, 8, 4).transpose(1, 2)))


def test_values_are_checked():
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError):
            FusedDropout(p)
    with pytest.raises(ValueError):
        FusedDropout(0.1, site=2 ** 32)
    with pytest.raises(ValueError, match="score"):
        FusedRouter(4, 8, 2, score="tanh")
    with pytest.raises(ValueError, match="group_score"):
        FusedRouter(4, 8, 2, group_score="sum")
    with pytest.raises(ValueError, match="activation"):
        FusedGroupNorm(8, 2, 4, activation="relu")


def test_dropout_refuses_another_current_device(launches, monkeypatch):
    drop = FusedDropout(0.1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    x = _Fake(torch.zeros(4, 8))
    with pytest.raises(RuntimeError, match="not the current one"):
        drop.forward(x, y=x)
    assert not launches
