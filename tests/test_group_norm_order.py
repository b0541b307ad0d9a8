"""CPU: what orders memory between a group norm's CTAs, read from the text: no run shows its absence.

One lane of a warp acquires; the others read what it acquired after a barrier of the warp (a shuffle hands the
answer on, but orders no memory)."""

import os
import re

import pytest

TEXT = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "adamw_optimizer_step_tensor_gb300", "csrc",
                         "group_norm.cuh")).read()


def body(name):
    at = TEXT.index(f" {name}(const G")
    return TEXT[at:TEXT.index("\n}\n", at)]


@pytest.mark.parametrize("name,acquires", [("gn_arrive", "atom.add.acq_rel"), ("gn_wait_open", "ld.acquire")])
def test_the_warp_meets_after_its_first_lane_has_acquired(name, acquires):
    text = body(name)
    handed_on = text.rindex("__shfl_sync(")
    assert text.rindex(acquires) < handed_on < text.rindex("__syncwarp();") < text.rindex("return")


def test_the_last_cta_clears_the_words_after_a_fence_on_either_side_of_the_ticket():
    assert re.findall(r"__threadfence|atomicAdd", body("gn_leave")) == ["__threadfence", "atomicAdd", "__threadfence"]
