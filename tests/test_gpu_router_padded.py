"""GPU: padded rows that share a warp with rows whose choice is made again from 64-bit keys.

Softmax scores with a bias and groups, where the 64-bit keys take the row's sum in 64 bits: a padded
row's is 0.  Teams of 8, 16 and 32 lanes are four, two and one token a warp.  Bounds: test_gpu_router's.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedRouter
from oracle import router as RO

from test_gpu_router import check

pytestmark = pytest.mark.gpu
# experts, groups, top_groups, top_k: teams of 8, 8, 16, 16, 32 lanes, and a warp a token
TEAMS = [(64, 8, 3, 6), (32, 8, 2, 4), (64, 8, 3, 9), (128, 16, 4, 8), (256, 8, 4, 20), (600, 8, 4, 8)]


def rows(tokens, experts, order, seed):
    """Padded rows, rows of equal logits, rows of few values (many ties) and ordinary ones, as `order` names them in turn."""
    rng = np.random.default_rng(seed)
    z = rng.normal(0, 1, (tokens, experts))
    for t in range(tokens):
        kind = order[t % len(order)]
        if kind == "p":
            z[t] = -np.inf
        elif kind == "e":
            z[t] = 0.5
        elif kind == "f":
            z[t] = rng.integers(-1, 2, experts)
    return z


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("experts,groups,top,k", TEAMS)
def test_padded_rows_beside_ties(experts, groups, top, k, group_score):
    constant = np.full(experts, 0.125)
    uneven = 0.125 * np.random.default_rng(experts).integers(0, 3, experts)
    for tokens, order in ((1, "e"), (2, "pe"), (3, "epe"), (7, "pef"), (33, "ppep"), (61, "epfn"), (130, "eeep")):
        z = rows(tokens, experts, order, tokens)
        for bias in (constant, uneven):
            for dtype in (torch.float32, torch.bfloat16):
                ids = check(z, bias, k, "softmax", groups, top, group_score, dtype=dtype)
                assert (ids[np.isneginf(z).all(1)] == -1).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top,k", TEAMS)
def test_padded_rows_beside_keys_closer_than_float32_tells(experts, groups, top, k, score):
    rng = np.random.default_rng(k)
    for seed in range(4):
        z = rng.normal(0, 1, (24, experts)).astype(np.float32)
        z[1::2] = z[0]
        bias = (0.75 - RO.scores(z[0].astype(np.float64), score)).astype(np.float32)
        z[seed::4] = -np.inf
        check(z, bias, k, score, groups, top, "top2")


@pytest.mark.parametrize("experts,groups,top,k", TEAMS)
def test_rows_of_nan_beside_ties(experts, groups, top, k):
    z = torch.from_numpy(rows(50, experts, "epe", 1).astype(np.float32)).cuda()
    z[1::3] = float("nan")
    bias = torch.full((experts,), 0.125, device="cuda")
    router = FusedRouter(50, experts, k, groups=groups, top_groups=top, group_score="top2")
    w, ids, slots, starts = (t.cpu() for t in router.route(z, bias))
    assert w[1::3].isnan().all() and (ids[1::3] == -1).all() and (slots[1::3] == -1).all()
    live = torch.ones(50, dtype=torch.bool)
    live[1::3] = False
    assert torch.equal(ids[live], torch.arange(k, dtype=torch.int32).expand(int(live.sum()), k))
    assert (w[live] - 1 / k).abs().max() <= 2.0 ** -17 / k
    assert int(starts[-1]) == int(live.sum()) * k
