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


# Few rows; few rows of a large B (tiles with a workspace, few rows without); and for each size of
# tile: less than a block of the sum, whole blocks, a ragged last one, a cut sum, and more
# tiles than compute units.
SIZES = [(1, 200, 1000), (33, 8192, 4100), (64, 8192, 4096), (65, 70, 40), (130, 257, 384), (300, 300, 1000),
         (129, 127, 4100), (3000, 1300, 100), (3000, 1300, 256), (3000, 1300, 300), (2770, 391, 6200),
         (4100, 2100, 100), (4100, 2100, 256), (4100, 2100, 300), (4100, 4300, 128), (4100, 4300, 300)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_every_tile_on_integers(M, N, K, fa, call):
    """Codes of -2 .. 2 and scales of 1/2, 1 and 2: products of 8 neighbours lie within 2^6 of each
    other, so nothing is cut, and every partial sum is a multiple of 1/4 below 2^22."""
    fb = "e5m2" if (M + K) % 3 == 0 else "e4m3"
    gp.say(f"gemm {call} {M}x{N}x{K} {fa} {fb}")
    a, va = q8.integers(M, K, fa, 1)
    b, vb = q8.integers(N, K, fb, 2, True)
    want = va.float() @ vb.float().t()
    for out in OUTS:
        for with_ws in (False, True):
            got = product(call, M, N, K, a, b, out, with_ws)
            assert torch.equal(got, want.to(ref.DTYPES[out])), (out, with_ws)


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


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("M,N,K", [(3, 140, 1000), (64, 8192, 4100), (70, 140, 1000), (3000, 1300, 300), (4100, 2100, 130)])
def test_scales_far_apart(M, N, K, out, call):
    """One scale for each row of A and each 128 rows of B, over 2^40 for results that hold it:
    every sum is an integer below 2^24 times a power of two."""
    gp.say(f"gemm {call} wide scales {M}x{N}x{K} {out}")
    g = q8._gen(9)
    far = 3 if out == "f16" else 20
    kb, nb = ref.up(K, 128) // 128, ref.up(N, 128) // 128
    ca = torch.randint(-2, 3, (M, K), generator=g)
    cb = torch.randint(-2, 3, (N, K), generator=g)
    ea = torch.randint(-far, far + 1, (M, 1), generator=g)
    eb = torch.randint(-far, far + 1, (nb, 1), generator=g)
    f8 = lambda c: c.float().to(torch.float8_e4m3fn).view(torch.uint8)
    a = q8.stored(f8(ca), (ea + 127).expand(M, kb).contiguous(), "e4m3")
    b = q8.stored(f8(cb), (eb + 127).expand(nb, kb).contiguous(), "e4m3", True)
    want = (ca.float() @ cb.float().t()).double() * torch.exp2(ea.double()) * \
        torch.exp2(eb.double()).repeat_interleave(128, 0)[:N].t()
    for with_ws in (False, True):
        assert torch.equal(product(call, M, N, K, a, b, out, with_ws), want.to(ref.DTYPES[out]))


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("K", [300, 384])
@pytest.mark.parametrize("M,N", [(5, 130), (64, 130), (100, 130), (3000, 1300), (4100, 2100)])
def test_non_finite_values_stay_in_their_row_and_column(M, N, K, out, call):
    """NaN and infinities of A and B, also among the last codes of the sum; codes beyond it are NaN
    in storage and do not count."""
    gp.say(f"gemm {call} non-finite {M}x{N}x{K} {out}")
    a, va = q8.integers(M, K, "e5m2", 5)
    b, vb = q8.integers(N, K, "e5m2", 6, True)
    va, vb = va.float(), vb.float()
    clean = va @ vb.t()
    for r, k, code, v in [(1, K - 1, 0x7F, math.nan), (2, 7, 0x7C, math.inf), (M - 1, 130, 0xFC, -math.inf)]:
        a.codes[r, k], va[r, k] = code, v
    n = N - 2
    b.codes[n, 140], vb[n, 140] = 0x7D, math.nan
    rows, cols = [1, 2, M - 1], [n]
    want = clean.clone()
    for r in rows:
        want[r] = (va[r] * vb).sum(1)
    for c in cols:
        want[:, c] = (va * vb[c]).sum(1)
    want = want.to(ref.DTYPES[out]).float()
    for with_ws in (False, True):
        got = product(call, M, N, K, a, b, out, with_ws).float()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(5, 1e30, -1e30), want.nan_to_num(5, 1e30, -1e30))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("fx", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", [(6200, 2100, 2100), (1700, 4100, 4200)])
def test_weight_gradient_of_large_tiles_in_every_format(M, N, K, fx, kind):
    gp.say(f"wgrad large tiles {M}x{N}x{K} {kind} {fx}")
    if kind == "bf16":
        vy = torch.randint(-3, 4, (M, N), generator=q8._gen(7)).double()
        dy = s2r.mat(q8.wide(M, N, "bf16", x=vy)[:, :N])
    else:
        dy, vy = q8.integers(M, N, kind, 7)
    x, vx = q8.integers(M, K, fx, 8)
    want = vy.float().t() @ vx.float()  # exact: multiples of 1/4 below 2^22
    for with_ws in (False, True):
        assert torch.equal(q8.wgrad(M, N, K, dy, x, with_ws=with_ws).float(), want)


@pytest.mark.parametrize("M,N,K", [(60, 8192, 4100), (129, 127, 4100), (5001, 1000, 1000), (4500, 4300, 1000)])
def test_the_same_bits_every_time(M, N, K):
    """Several tiles to a compute unit, cut sums, few rows: repeated, with other calls in between."""
    gp.say(f"gemm and wgrad repeated {M}x{N}x{K}")
    a, va = q8.ordinary(M, K, "e4m3", 3)
    b, vb = q8.ordinary(N, K, "e4m3", 4, True)
    dy, vy = q8.ordinary(M, N, "e5m2", 5)
    first = {}
    for i in range(6):
        for call in CALLS:
            for out in ("f32", "bf16"):
                got = product(call, M, N, K, a, b, out, True)
                assert torch.equal(got, first.setdefault((call, out), got)), (call, out, i)
        got = q8.wgrad(M, N, K, dy, a)
        assert torch.equal(got, first.setdefault("wgrad", got)), i
