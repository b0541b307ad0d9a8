"""Groups of which one expert is there (the others' logits or biases are -inf, or the group has one): under
"top2" they score that expert's key.  By hand for the definition on the CPU, and on the GPU."""

import os

import numpy as np
import pytest
import torch

from oracle import router as RO

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "adamw.h")
# sigmoid scores of four groups of four; 0: not there.  Sums of two: 0.9 alone, 0.7, 0.8, none.
S = np.array([0.9, 0, 0, 0, 0.3, 0.4, 0.2, 0, 0, 0.35, 0.45, 0.05, 0, 0, 0, 0])
# top_groups, k and the choice
BY_HAND = [(1, 3, [0, -1, -1]), (2, 3, [0, 10, 9]), (3, 6, [0, 10, 5, 9, 4, 6])]


def logits():
    with np.errstate(divide="ignore"):
        return np.log(S) - np.log1p(-S)


@pytest.mark.parametrize("top,k,want", BY_HAND)
def test_the_definition_by_hand(top, k, want):
    for bias in (None, np.full(16, -0.5)):      # below 0, one key is more than the sum of two: 0.4 against -0.3 and -0.2
        ids = RO.choose(logits(), bias, k, "sigmoid", 4, top, "top2")
        assert ids + [-1] * (k - len(ids)) == want
    assert RO.choose(logits(), None, 3, "sigmoid", 4, 1, "max") == [0]


def test_the_header_says_so():
    assert "(of a group with one\n *                       expert that is there: that one's key" in open(HEADER).read()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("top,k,want", BY_HAND)
def test_the_choice_by_hand(top, k, want, dtype):
    from adamw_optimizer_step_tensor_gb300 import FusedRouter
    z = torch.from_numpy(logits()).to(dtype).cuda().expand(9, 16).contiguous()
    for bias in (None, torch.full((16,), -0.5, device="cuda")):
        ids = FusedRouter(9, 16, k, score="sigmoid", groups=4, top_groups=top, group_score="top2").route(z, bias)[1]
        assert ids.tolist() == [want] * 9


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top,k", [(64, 8, 3, 6), (32, 32, 5, 5), (96, 12, 4, 20), (600, 8, 3, 9), (24, 8, 2, 3)])
def test_most_experts_are_not_there(experts, groups, top, k, score):
    from test_gpu_router import check
    rng = np.random.default_rng(experts)
    z = rng.normal(0, 1, (50, experts))
    z[rng.random(z.shape) < 1 - 1.5 * groups / experts] = -np.inf       # one or two of a group
    z[7] = -np.inf
    for bias in (None, -0.4 + 0.01 * rng.integers(-9, 10, experts), np.where(rng.random(experts) < 0.5, -np.inf, 0.25)):
        check(z, bias, k, score, groups, top, "top2")
