"""GPU: group norm in place and over strides of every kind, for each of its kernels (test_group_norm_cuts, on
the CPU, holds the sizes to the kernels named here).  Bounds: test_gpu_group_norm's."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedGroupNorm

from test_gpu_group_norm import check

DTYPES = {torch.float32: 4, torch.bfloat16: 2}
# shift of the first element, elements behind a position's channels, samples inside positions
LAYOUTS = {"padded": (0, 8, False), "odd": (0, 1, False), "shifted": (1, 0, False), "swapped": (0, 0, True), "all": (1, 3, True)}
# sizes, groups, and the kernels of dense tensors: forward and backward, float32 and bfloat16
CASES = [((300, 1, 512), 16, "lanes lanes lanes lanes"), ((40, 6, 96), 4, "row row row row"), ((3, 50, 64), 8, "small small small small"),
         ((8, 700, 320), 32, "cluster cluster cluster cluster"), ((4, 6000, 40), 1, "cluster fused cluster cluster"),
         ((3, 5, 20_000), 1, "fused fused fused fused"), ((4, 20_000, 48), 2, "fused fused cluster fused"),
         ((700, 1, 4104), 1, "fused fused fused fused"), ((9, 9000, 512), 8, "fused fused fused fused")]
SMALL = CASES[:-1]          # few enough elements for the definition


def room(shape, dtype, layout):
    """An empty tensor of that layout."""
    (n, length, c), (shift, pad, swap) = shape, layout
    t = torch.empty(n * length * (c + pad) + shift, dtype=dtype, device="cuda")[shift:]
    return (t.view(length, n, c + pad).transpose(0, 1) if swap else t.view(n, length, c + pad))[:, :, :c]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape,groups", [c[:2] for c in SMALL])
def test_strides(shape, groups, layout, dtype):
    shift, pad, swap = LAYOUTS[layout]
    check(shape, groups, dtype, silu=True, pad=pad, shift=shift, swap=swap)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,groups", [c[:2] for c in CASES])
def test_layouts_on_the_grid_and_in_place_give_the_dense_call_s_bits(shape, groups, dtype):
    """Layouts that leave the pieces as they are leave the cut, and so every sum's order, as it is."""
    n, _, c = shape
    g = torch.Generator("cuda").manual_seed(n)
    x, dy = (torch.randn(shape, device="cuda", generator=g).to(dtype) for _ in range(2))
    w, b = 1 + 0.2 * torch.randn(c, device="cuda", generator=g), 0.2 * torch.randn(c, device="cuda", generator=g)
    norm = FusedGroupNorm(c, groups, n, activation="silu")
    y, mean, rstd = norm.forward(x, w, b)
    back = norm.backward(dy, x, w, b, mean, rstd)
    same = lambda got, want: all(torch.equal(a, t) for a, t in zip(got, want))  # noqa: E731
    for layout in ((0, 0, False), LAYOUTS["padded"], LAYOUTS["swapped"], (8, 8, True)):
        put = lambda t: room(shape, dtype, layout).copy_(t)  # noqa: B023, E731
        assert same(norm.forward(put(x), w, b, y=room(shape, dtype, layout)), (y, mean, rstd))
        z = put(x)
        assert same(norm.forward(z, w, b, y=z), (y, mean, rstd))
        assert same(norm.backward(put(dy), put(x), w, b, mean, rstd, dx=room(shape, dtype, layout)), back)
        z = put(dy)
        assert same(norm.backward(z, put(x), w, b, mean, rstd, dx=z), back)
        z = put(x)
        assert same(norm.backward(put(dy), z, w, b, mean, rstd, dx=z), back)
    # the layouts of a call need not be one
    got = norm.backward(room(shape, dtype, (0, 8, False)).copy_(dy), room(shape, dtype, (0, 0, True)).copy_(x), w, b, mean, rstd,
                        dx=room(shape, dtype, (8, 16, True)))
    assert same(got, back) and norm.status() == 0
