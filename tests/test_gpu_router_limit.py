"""GPU: as many tokens as a plan takes, 2^31 - 1 with one expert each: every one has its weight, expert,
place and gradient.  A weight is a softmax of two, within 2^-17 (test_gpu_router); a gradient p (dw - dw p),
within 2^-16 of its terms and half a bfloat16 step."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedRouter

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_the_memory_back():
    """The library's plans take memory that torch's cache holds otherwise."""
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens", [2 ** 31 - 1, 2_147_483_612, 2_140_000_000])
def test_tokens_at_the_limit(tokens):
    g = torch.Generator("cuda").manual_seed(tokens % 1000)
    z = torch.empty(tokens, 2, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    z[5] = z[-3] = float("-inf")                 # tokens that go nowhere
    router = FusedRouter(tokens, 2, 1, renormalise=False)
    w = torch.full((tokens, 1), -1.0, device="cuda")
    ids, slots = (torch.full((tokens, 1), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    _, _, _, starts = router.route(z, weights=w, ids=ids, slots=slots)
    dz = router.backward(w, z, ids)              # the weights in place of their gradient
    step, seen = 1 << 27, [0, 0]
    first = starts.tolist()
    assert first[0] == 0 and first[2] == tokens - 2
    for at in range(0, tokens, step):
        part = z[at:at + step].float()
        e, p = ids[at:at + step, 0], w[at:at + step, 0]
        there = part[:, 0] > -float("inf")
        assert torch.equal(e, torch.where(there, (part[:, 1] > part[:, 0]).int(), -1))
        want = torch.where(there, torch.sigmoid((part[:, 1] - part[:, 0]).abs().double()), 0.0)
        assert ((p.double() - want).abs() <= 2.0 ** -17 * want).all()
        for k in range(2):
            mine = e == k
            n = int(mine.sum())
            assert torch.equal(slots[at:at + step, 0][mine], torch.arange(first[k] + seen[k], first[k] + seen[k] + n, device="cuda").int())
            seen[k] += n
        assert (slots[at:at + step, 0][~there] == -1).all()
        # of the chosen one; the other's is its negative
        d = want * (want - want * want)
        got = dz[at:at + step].double()
        for k in range(2):
            dk = torch.where(e == k, d, -d)
            bound = 2.0 ** -8 * dk.abs() + 2.0 ** -15 * want * want + 2.0 ** -126
            assert ((got[:, k] - dk).abs() <= torch.where(there, bound, 0.0)).all()
    assert first[1] == seen[0] and seen[0] + seen[1] == tokens - 2
