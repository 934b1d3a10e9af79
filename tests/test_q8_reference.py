"""The 64-bit reference of the 8-bit training calls, pinned on the CPU without the library:
torch's own 8-bit types give the same codes, derivatives match differences, and planted
mistakes are seen."""
import math

import pytest
import torch

import q8_reference as ref


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_code_values_are_torchs(fmt):
    got = ref.code_values(fmt)
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(ref.F8[fmt]).double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0, 7, -7), want.nan_to_num(0, 7, -7))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("square", [False, True])
def test_quantise_against_torchs_rounding(fmt, square):
    torch.manual_seed(3)
    x = torch.randn(200, 300) * torch.exp(4 * torch.randn(200, 300))
    q, b = ref.quantise(x, fmt, square)
    f = ref.spread(b, 200, 300, square)
    assert torch.equal((x.double() / f).float().to(ref.F8[fmt]).double(), q)
    top = 448 if fmt == "e4m3" else 57344
    # the least power of two: half of it would not hold the largest element
    a = ref.block_max(x.double(), square)
    s = torch.ldexp(torch.ones_like(a), b - 127)
    assert (a <= top * s).all() and (a > top * s / 2).all()


def test_scale_at_the_borders():
    for fmt, top in [("e4m3", 448.0), ("e5m2", 57344.0)]:
        a = torch.tensor([top, math.nextafter(top, 1e9), top / 2, 0.0, 2.0 ** -149, top * 2.0 ** -110,
                          top * 2.0 ** -111], dtype=torch.float64)
        assert ref.scale_bytes(a, fmt).tolist() == [127, 128, 126, 17, 17, 17, 17]


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_derivative_against_differences(kind):
    g = torch.arange(-9 * 256, 9 * 256 + 1, dtype=torch.float64) / 256  # g +- h is exact
    h = 2.0 ** -10
    f = lambda x: ref.act(x, kind)[0]
    want = (8 * (f(g + h) - f(g - h)) - (f(g + 2 * h) - f(g - 2 * h))) / (12 * h)
    # fourth order: h^4 / 30 times the fifth derivative (below 30), and 18 values, each off by at
    # most 8 steps of 9, over 12 h
    assert (ref.act(g, kind)[1] - want).abs().max() < h ** 4 + 18 * 8 * 9 * 2.0 ** -53 / (12 * h)
    # a derivative without the product rule's second term is far outside that
    wrong = ref.act(g, kind)[0] / g.where(g != 0, torch.ones_like(g))
    assert (wrong - want).abs().max() > 1e-2
