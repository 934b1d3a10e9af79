"""The 4-bit product in tiles of 256 x 256, where the trace has to name them: with and without a ragged end of
the sum, ragged rows and columns, several tiles of several chunks to a workgroup, NaN blocks, ordinary values, every
result type.  Bounds as in test_gpu_q4.py.  And scales over all of their range, in every form of the product."""
import math

import pytest
import torch

import count_sketch_aggregation_amd as s2r
import q4_reference as ref4
import q8_reference as ref
import test_gpu_q4 as q4
import test_gpu_q8 as q8

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")
DEV = "cuda"


def traced(call):
    """The names of the kernels that `call` launches."""
    events = [torch.cuda.Event(enable_timing=True) for _ in range(8)]
    t = s2r.s2r_trace()
    t.capacity, t.count = len(events), 0
    for i, e in enumerate(events):
        e.record()
        t.events[i] = e.cuda_event
    s2r.s2r_diag_trace_attach(t)
    try:
        call()
    finally:
        s2r.s2r_diag_trace_attach(None)
    return [t.names[i].decode() for i in range(t.count)]


def in_large_tiles(M, N, K, a, b, out):
    got = []
    names = traced(lambda: got.append(q4.product(M, N, K, a, b, out, True)))
    assert names == ["k_q4_gemm<256>", "end"], names
    return got[0]


# a sum of one whole chunk of 512, of whole chunks, and with an end of 1 to 511; columns that end inside a lane's eight
# or four; fewer tiles than compute units, as many, and more: a workgroup's second tile is then another's neighbour
LARGE = [(2000, 4500, 1024), (3000, 3001, 513), (2001, 4099, 700), (4000, 3900, 600), (4096, 4096, 4096), (4100, 2100, 2100),
         (8000, 2000, 1100), (5001, 4999, 1100), (9000, 3000, 1536)]


@pytest.mark.parametrize("M,N,K", LARGE)
def test_exact(M, N, K):
    """Partial sums are multiples of 1/16 below 2^17."""
    gp.say(f"q4 gemm 256 exact {M}x{N}x{K}")
    a, va = q4.exact_matrix(M, K, 1)
    b, vb = q4.exact_matrix(N, K, 2)
    want = va.float() @ vb.float().t()
    for out in ("f32", "bf16", "f16"):
        assert torch.equal(in_large_tiles(M, N, K, a, b, out), want.to(ref.DTYPES[out])), out


@pytest.mark.parametrize("M,N,K", [(3000, 3001, 513), (4000, 3900, 600), (2500, 4504, 1536)])
def test_ordinary_values(M, N, K):
    """K additions in fp32, each off by at most a step of a partial sum of at most sum |a b|, and one rounding."""
    gp.say(f"q4 gemm 256 ordinary {M}x{N}x{K}")
    m, v = [], []
    for R, seed in ((M, 3), (N, 4)):
        x = torch.randn((R, K), generator=q8._gen(seed), dtype=torch.float64)
        x *= torch.exp(torch.randn((R, K), generator=q8._gen(seed + 2), dtype=torch.float64))
        code, s = ref4.quantise(x)
        m.append(q4.stored(code, s, seed))
        v.append(ref4.values(code, s))
    want, mass = v[0] @ v[1].t(), v[0].abs() @ v[1].abs().t()
    tol = K * 2.0 ** -23 * mass
    for out in ("f32", "bf16"):
        got = in_large_tiles(M, N, K, *m, out).double()
        assert bool(((got - want).abs() <= tol + ref.HALF_STEP[out] * (want.abs() + tol)).all()), out


@pytest.mark.parametrize("M,N,K", [(3000, 3001, 513), (2000, 4500, 1024)])
def test_nan_blocks_stay_in_their_row_and_column(M, N, K):
    gp.say(f"q4 gemm 256 NaN {M}x{N}x{K}")
    a, va = q4.exact_matrix(M, K, 5)
    b, vb = q4.exact_matrix(N, K, 6)
    a.scales[1, (K - 1) // 32] = 255
    a.scales[M - 1, 0] = 255
    b.scales[N - 2, 3] = 255
    want = va.float() @ vb.float().t()
    want[1], want[M - 1], want[:, N - 2] = math.nan, math.nan, math.nan
    got = in_large_tiles(M, N, K, a, b, "f32")
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(1e9), want.nan_to_num(1e9))


def test_the_same_bits_every_time():
    """Two tiles to some workgroups, repeated, with another product in between."""
    gp.say("q4 gemm 256 repeated")
    M, N, K = 5001, 4999, 1100
    g = q8._gen(7)
    m = [q4.stored(torch.randint(0, 16, (R, K), generator=g), torch.randint(110, 140, (R, -(-K // 32)), generator=g)) for R in (M, N)]
    first = in_large_tiles(M, N, K, *m, "f32")
    for _ in range(3):
        q4.product(300, 300, K, s2r.q4_mat(m[0].codes[:300], m[0].scales[:300]), s2r.q4_mat(m[1].codes[:300], m[1].scales[:300]), "f32", True)
        assert torch.equal(in_large_tiles(M, N, K, *m, "f32"), first)


SCALES = [17, 18, 30, 64, 100, 120, 127, 134, 150, 190, 230, 250, 251, 252]


@pytest.mark.parametrize("M,N,K", [(14, 42, 320), (168, 140, 320), (168, 140, 700), (2001, 4099, 700)])
def test_product_over_all_scales(M, N, K):
    """One product of two nonzero codes in every sum, under all pairs of scales: a power of two times 8 bits, so the
    result is that value in fp32, which infinities and subnormals are too."""
    gp.say(f"q4 gemm all scales {M}x{N}x{K}")
    nb = ref.up(K, 32) // 32
    ca = torch.zeros((M, K), dtype=torch.long)
    ca[torch.arange(M), torch.arange(M) * 37 % K] = 1 + torch.arange(M) % 7
    cb = (1 + torch.arange(N) % 7)[:, None].expand(N, K)
    sa, sb = torch.tensor(SCALES)[torch.arange(M) % 14], torch.tensor(SCALES)[torch.arange(N) // 3 % 14]
    v = ref4.code_values()
    want = v[ca.amax(1)][:, None] * v[cb[:, 0]]
    want = want * torch.exp2((sa - 127).double())[:, None] * torch.exp2((sb - 127).double())
    assert bool((want >= 2.0 ** 128).any()) and bool((want < 2.0 ** -149).any())
    got = q4.product(M, N, K, q4.stored(ca, sa[:, None].expand(M, nb)), q4.stored(cb, sb[:, None].expand(N, nb)), "f32", True)
    assert torch.equal(got, want.float())
