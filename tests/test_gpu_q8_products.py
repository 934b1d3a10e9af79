"""The 8-bit products over every tile, tail, way of summing, format and result type that the
library chooses among: s2r_q8_gemm and s2r_q8_gemm_fast on integers (equality to the bit), the
bound that s2r_q8_gemm_fast states, scales and non-finite values in each of them."""
import math

import pytest
import torch

import count_sketch_aggregation_amd as s2r
import q8_reference as ref
import test_gpu_q8 as q8

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")
DEV = "cuda"
CALLS = {"exact": s2r.s2r_q8_gemm, "fast": s2r.s2r_q8_gemm_fast}
OUTS = ["f32", "bf16", "f16"]


def product(call, M, N, K, a, b, out, with_ws):
    c = q8.wide(M, N, out, fill=7.0)
    ws = q8.workspace(s2r.s2r_q8_gemm_workspace_bytes(M, N, K)) if with_ws else None
    CALLS[call](M, N, K, a, b, s2r.mat(c), workspace=ws)
    assert q8.pad_kept(c, N, 7.0)
    return c[:, :N].cpu()


def cut_bound(va, vb, sa, sb, fa, fb):
    """What s2r_q8_gemm_fast may cut: 7 * 2^-13 times the largest |a b| of every eight neighbours of
    the sum, a nonzero value below its format's normal range counted as the least normal."""
    least = {"e4m3": 2.0 ** -6, "e5m2": 2.0 ** -14}
    up = lambda v, s, f: torch.where(v == 0, 0.0, torch.maximum(v.abs(), least[f] * s))
    K = va.shape[1]
    pad = lambda v: torch.nn.functional.pad(v, (0, ref.up(K, 8) - K)).to(DEV)
    x, y = pad(up(va, sa, fa)), pad(up(vb, sb, fb))
    total = torch.zeros((va.shape[0], vb.shape[0]), dtype=torch.float64, device=DEV)
    for k in range(0, K, 8):
        total += (x[:, None, k:k + 8] * y[None, :, k:k + 8]).amax(2)
    return (7 * 2.0 ** -13 * total).cpu()


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("spread", [0, 4])
@pytest.mark.parametrize("M,N,K", [(40, 200, 700), (300, 300, 1000), (600, 140, 1300)])
def test_fast_product_within_its_bound(M, N, K, spread, fa, fb):
    """The cut products, K additions in fp32, each off by at most a step of a partial sum of at most
    sum |a b|, and one rounding."""
    gp.say(f"gemm fast {M}x{N}x{K} {fa} {fb} spread {spread}")

    def matrix(R, fmt, seed, square):
        g = q8._gen(seed)
        x = torch.randn((R, K), generator=g, dtype=torch.float64) * torch.exp(
            spread * torch.randn((R, K), generator=g, dtype=torch.float64)) / 16
        q, b = ref.quantise(x, fmt, square)
        s = ref.spread(b, R, K, square)
        return q8.stored(q.float().to(ref.F8[fmt]).view(torch.uint8), b, fmt, square), q * s, s

    a, va, sa = matrix(M, fa, 3, False)
    b, vb, sb = matrix(N, fb, 4, True)
    want, mass = va @ vb.t(), va.abs() @ vb.abs().t()
    tol = cut_bound(va, vb, sa, sb, fa, fb) + K * 2.0 ** -23 * mass
    for out in OUTS:
        t = tol + ref.HALF_STEP[out] * (want.abs() + tol) + (2.0 ** -25 if out == "f16" else 0)
        over = want.abs() + tol >= 65504 if out == "f16" else torch.zeros_like(want, dtype=torch.bool)
        for with_ws in (False, True):
            got = product("fast", M, N, K, a, b, out, with_ws).double()
            assert bool((((got - want).abs() <= t) | over).all()), (out, with_ws)
