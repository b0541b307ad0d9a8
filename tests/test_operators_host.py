"""The operators around the step without a GPU: record layouts match the header,
and every entry point refuses bad arguments on the host, before any device work."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedLayerNorm, FusedTokenLoss
from adamw_optimizer_step_tensor_gb300 import _capi as C
from adamw_optimizer_step_tensor_gb300 import operators as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORDS = (C.adamw_logits, C.adamw_policy, C.adamw_preference)


def _status(fn, *args):
    with pytest.raises(C.AdamWError) as e:
        fn(*args)
    return e.value.status


def test_record_layouts(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "adamw.h"', "int main(void) {"]
    for r in RECORDS:
        lines.append(f'printf("%zu\\n", sizeof({r.__name__}));')
        lines += [f'printf("%zu\\n", offsetof({r.__name__}, {f}));' for f, _ in r._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split()
    want = []
    for r in RECORDS:
        want += [ctypes.sizeof(r)] + [getattr(r, f).offset for f, _ in r._fields_]
    assert [int(v) for v in got] == want


def test_null_plans_are_refused():
    z = C.adamw_logits()
    assert _status(C.adamw_grad_norm, None, 1.0, None, 16, None, None, None) == C.EINVAL
    assert _status(C.adamw_clip_grads, None, 16, None) == C.EINVAL
    assert _status(C.adamw_token_logps, None, z, 16, None, None) == C.EINVAL
    assert _status(C.adamw_policy_loss, None, z, C.adamw_policy(), 16, 16, None, 0, None) == C.EINVAL
    assert _status(C.adamw_preference_loss, None, z, C.adamw_preference(), 16, 16, 16, None, 0, None) == C.EINVAL
    assert _status(C.adamw_layer_norm_forward, None, 0, 0, 1, 16, 8, None, None, 16, 8, 16, 16, None) == C.EINVAL
    assert _status(C.adamw_layer_norm_backward, None, 0, 0, 1, 16, 8, 16, 8, None, 16, 16, 16, 8, None,
                   None, None) == C.EINVAL
    C.adamw_loss_plan_destroy(None)
    C.adamw_layer_norm_plan_destroy(None)


def test_plan_sizes_are_checked_first():
    assert _status(C.adamw_loss_plan_create, -1, 0) == C.EINVAL
    assert _status(C.adamw_loss_plan_create, 4, -1) == C.EINVAL
    assert _status(C.adamw_loss_plan_create, 4, 5000) == C.EUNSUPPORTED
    assert _status(C.adamw_layer_norm_plan_create, 0, 1e-5) == C.EINVAL
    for eps in (-1.0, float("nan"), float("inf")):
        assert _status(C.adamw_layer_norm_plan_create, 8, eps) == C.EINVAL
    lib = C.load()
    assert lib.adamw_loss_plan_create(4, 0, None) == C.EINVAL
    assert lib.adamw_layer_norm_plan_create(4, 1e-5, None) == C.EINVAL


class _Fake:
    """A torch tensor's face over a CPU tensor that says it is on the GPU."""

    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_row_strides():
    t = torch.zeros(6, 10)
    assert O._rows("t", _Fake(t)) == 10
    assert O._rows("t", _Fake(t[:, 2:7])) == 10
    assert O._rows("t", _Fake(t[::2])) == 20
    assert O._rows("t", _Fake(t[:1, :3])) == 3       # one row: its stride says nothing
    with pytest.raises(ValueError, match="CUDA matrix"):
        O._rows("t", t)
    with pytest.raises(ValueError, match="contiguous along"):
        O._rows("t", _Fake(t.t()))
    with pytest.raises(ValueError, match="overlapping"):
        O._rows("t", _Fake(t[:1].expand(6, 10)))
    with pytest.raises(TypeError, match="float16"):
        O._rows("t", _Fake(t), torch.float16)
    with pytest.raises(ValueError, match="shape"):
        O._rows("t", _Fake(t), None, (6, 9))


def test_vectors():
    t = torch.zeros(8)
    assert O._vector("v", None, 8) is None
    assert O._vector("v", _Fake(t), 8) == t.data_ptr()
    for bad in (t, _Fake(t[:7]), _Fake(torch.zeros(16)[::2])):
        with pytest.raises(ValueError):
            O._vector("v", bad, 8)
    with pytest.raises(TypeError):
        O._vector("v", _Fake(t.double()), 8)


def test_exports():
    assert FusedTokenLoss is O.FusedTokenLoss and FusedLayerNorm is O.FusedLayerNorm
