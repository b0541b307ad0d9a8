"""GPU: group norm by clusters of two, four and eight CTAs, whose first exchange follows a copy of a few
KB.  Every CTA of a cluster has to have started before another writes to its shared memory: no run shows
that it had, so the order is read from the kernels' text (on the CPU), and the runs show that meeting first
leaves the values as they are.  Bounds: test_gpu_group_norm's."""

import os
import re

import pytest
import torch

from test_gpu_group_norm import check

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "adamw_optimizer_step_tensor_gb300", "csrc")


@pytest.mark.parametrize("file,kernel", [("group_norm.cu", "gn_forward_cluster_kernel"), ("group_norm_backward.cu", "gn_backward_cluster_kernel")])
def test_all_ctas_are_known_to_have_started_before_the_first_exchange(file, kernel):
    text = open(os.path.join(CSRC, file)).read()
    body = text[text.index(f"{kernel}(const GroupNormArgs a, const GnCut c) {{"):]
    body = body[:body.index("\n}\n")]
    calls = re.findall(r"\b(gn_started|gn_all_started|gn_exchange)\(", body)
    assert calls == ["gn_started", "gn_all_started", "gn_exchange"]
    assert body.index("gn_started(") < body.index("for (int64_t sample")


# the clusters that these sizes get, forward or backward: pieces of one element, of 4 and of 16 bytes
SHAPES = {torch.float32: [((1, 414, 7), 1), ((1, 1058, 14), 2), ((1, 161, 64), 1), ((1, 285, 64), 1), ((1, 1462, 7), 1), ((2, 1969, 11), 1),
                          ((1, 1890, 20), 1), ((1, 2583, 24), 1), ((1, 2150, 11), 1), ((2, 5536, 11), 1), ((1, 3032, 24), 1), ((5, 5781, 24), 1)],
          torch.bfloat16: [((1, 263, 22), 2), ((1, 1004, 7), 1), ((1, 329, 40), 2), ((5, 547, 40), 2), ((1, 894, 24), 1), ((2, 1259, 40), 1),
                           ((2, 597, 11), 1), ((1, 1217, 22), 2), ((1, 680, 100), 5), ((2, 1877, 20), 1), ((1, 1123, 40), 1), ((1, 1468, 40), 1),
                           ((1, 3425, 7), 1), ((2, 4959, 11), 1), ((2, 2623, 20), 1), ((2, 6763, 20), 1), ((1, 3114, 64), 1), ((2, 5972, 40), 1)]}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shape,groups", [(d, s, g) for d, v in SHAPES.items() for s, g in v])
def test_clusters_of_every_size(dtype, shape, groups):
    check(shape, groups, dtype, silu=True)
    torch.cuda.synchronize()
