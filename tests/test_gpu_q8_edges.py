"""The 8-bit training calls where their formulas lose digits if they are computed the obvious
way, and at the ends of their ranges: signalling NaN, the far negative side of GELU, the
derivatives near 1 and at huge arguments, values next to fp32's largest, sums that cancel."""
import math

import pytest
import torch

import count_sketch_aggregation_amd as s2r
import q8_reference as ref
import test_gpu_q8 as q8

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")
DEV = "cuda"
HALF = 2.0 ** -24  # half a step of fp32, relative


# ---------------------------------------------------------------------------------------
# sums of the product


def cancelling(M, N, K, fa):
    """+2^16 and -2^16 next to each other in the sum, and a few multiples of 2^-6 around them:
    every partial sum has 24 bits or fewer, and every result is a small multiple of 2^-6 that all
    three types hold."""
    g = q8._gen(12)
    va, vb = torch.zeros((M, K), dtype=torch.float64), torch.zeros((N, K), dtype=torch.float64)
    big = 2 * (K // 5)
    va[:, big:big + 2] = 2.0 ** 8
    vb[:, big], vb[:, big + 1] = 2.0 ** 8, -2.0 ** 8
    for at in (big + 2, big + 3, (big + 40) % K, (big + 70) % K):
        va[:, at] = 2.0 ** -3 * torch.randint(0, 2, (M,), generator=g)
        vb[:, at] = 2.0 ** -3 * torch.randint(-1, 2, (N,), generator=g)
    code = lambda v, f: v.float().to(ref.F8[f]).view(torch.uint8)
    kb = ref.up(K, 128) // 128
    a = q8.stored(code(va, fa), torch.full((M, kb), 127), fa)
    b = q8.stored(code(vb, "e4m3"), torch.full((ref.up(N, 128) // 128, kb), 127), "e4m3", True)
    return a, b, (va.float() @ vb.float().t()).double()


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", [(1, 140, 400), (30, 140, 400), (40, 140, 1024), (40, 8192, 4100),
                                   (130, 140, 400), (129, 127, 4100), (3000, 1300, 200), (4000, 2100, 130)])
def test_sums_are_fp32_whatever_the_result_is_rounded_to(M, N, K, fa):
    gp.say(f"gemm cancelling {M}x{N}x{K} {fa}")
    a, b, want = cancelling(M, N, K, fa)
    assert len(want.unique()) > 1
    for out in ("f32", "bf16", "f16"):
        for with_ws in (False, True):
            assert torch.equal(q8.gemm(M, N, K, a, b, out, with_ws).double(), want), (out, with_ws)
