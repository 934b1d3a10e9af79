"""The 4-bit calls on the GPU against the 64-bit reference.  Storage is exact: codes and scales equal
the reference's.  The product is checked on codes and scales whose every partial sum is exact (equality
to the bit) and on ordinary values within the bound of an fp32 sum.  Paddings hold anything on input and a pattern on
output that has to survive."""
import math

import pytest
import torch

import count_sketch_aggregation_amd as s2r
import q4_reference as ref4
import q8_reference as ref
import test_gpu_q8 as q8

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")
DEV = "cuda"
POISON = 0xA5
up = ref.up


def space(rows, cols, pad=16):
    q = torch.full((rows, up(-(-cols // 2), 16) + pad), POISON, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, up(-(-cols // 32), 8) + 8), POISON, dtype=torch.uint8, device=DEV)
    return s2r.q4_mat(q, s)


def unpack(q, cols):
    q = q.cpu()
    return torch.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)[:, :cols].long()


def check(m, R, C, want):
    code, b = want
    n, nb = -(-C // 2), -(-C // 32)
    got = unpack(m.codes[:, :n], C)
    assert torch.equal(m.scales[:, :nb].cpu().long(), b)
    same = (got == code) | ((got % 8 == 0) & (code % 8 == 0))  # a zero's sign is free
    assert bool(same.all())
    assert bool((m.codes[:, n:] == POISON).all()) and bool((m.scales[:, nb:] == POISON).all())
    if C % 2:
        assert bool((m.codes[:, n - 1] >> 4 == 0).all())


def stored(code, b, seed=0):
    """A 4-bit matrix whose padding holds arbitrary codes and NaN scales."""
    R, C = code.shape
    q = torch.randint(0, 256, (R, up(-(-C // 2), 16) + 16), generator=q8._gen(seed), dtype=torch.uint8)
    even = torch.nn.functional.pad(code, (0, C % 2), value=9)
    q[:, :-(-C // 2)] = (even[:, 0::2] | even[:, 1::2] << 4).to(torch.uint8)
    s = torch.full((R, up(b.shape[1], 8) + 8), 255, dtype=torch.uint8)
    s[:, :b.shape[1]] = b.to(torch.uint8)
    return s2r.q4_mat(q.to(DEV), s.to(DEV))


SHAPES = [(1, 1), (1, 33), (3, 64), (33, 129), (64, 640), (130, 1000), (257, 16), (7, 2049), (300, 271)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C", SHAPES)
def test_save_and_load(R, C, dtype):
    gp.say(f"q4 save/load {R}x{C} {dtype}")
    x = q8.awkward(R, C, dtype, R + C)
    m = s2r.mat(q8.wide(R, C, dtype, x=x))
    want, want_t = ref4.quantise(x), ref4.quantise(x.t())
    alone, both, t, t_alone = space(R, C), space(R, C), space(C, R), space(C, R)
    s2r.s2r_q4_save(R, C, m, alone)
    s2r.s2r_q4_save(R, C, m, both, t)
    s2r.s2r_q4_save(R, C, m, None, t_alone)
    for got in (alone, both):
        check(got, R, C, want)
    for got in (t, t_alone):
        check(got, C, R, want_t)
    values = ref4.values(*want)
    for out in ("bf16", "f16", "f32"):
        y = q8.wide(R, C, out, fill=7.0)
        s2r.s2r_q4_load(R, C, alone, s2r.mat(y))
        assert torch.equal(y[:, :C].cpu(), values.to(ref.DTYPES[out])), out
        if out != "f16":
            assert torch.equal(y[:, :C].cpu().double(), values), out
        assert q8.pad_kept(y, C, 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_borders_of_the_grid(dtype):
    """Ties and their neighbours between every two codes, largest magnitudes on both sides of the
    scale's border, and the type's own largest and smallest values."""
    gp.say(f"q4 borders {dtype}")
    t = ref.DTYPES[dtype]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=t)
    near = torch.cat([ties, torch.nextafter(ties, ties.new_zeros(()).expand_as(ties)), torch.nextafter(ties, ties * 2)])
    x = torch.zeros((8, 64), dtype=t)
    x[0, :21], x[0, 31] = near, 6
    x[0, 32:53], x[0, 63] = -near, -6
    x[1, 0], x[1, 32] = 6, torch.nextafter(x.new_tensor(6.0), x.new_tensor(7.0))
    x[2, 0], x[2, 1], x[2, 33] = torch.finfo(t).max, torch.finfo(t).max / 2, -torch.finfo(t).max
    x[3, 0], x[3, 40] = torch.finfo(t).tiny, torch.finfo(t).smallest_normal / 4
    x[4, 3] = 2.0 ** -20 if dtype == "f16" else 2.0 ** -113
    x[5] = -0.0
    x[6, :32] = torch.linspace(-6, 6, 32)
    x[7] = torch.linspace(-48, 47, 64)
    out, out_t = space(8, 64), space(64, 8)
    s2r.s2r_q4_save(8, 64, s2r.mat(q8.wide(8, 64, dtype, x=x)), out, out_t)
    check(out, 8, 64, ref4.quantise(x))
    check(out_t, 64, 8, ref4.quantise(x.t()))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_non_finite_blocks(dtype):
    gp.say(f"q4 non-finite {dtype}")
    x = torch.randn((70, 100), generator=q8._gen(5)).to(ref.DTYPES[dtype])
    x[0, 3], x[1, 40], x[2, 99], x[69, 64] = math.inf, -math.inf, math.nan, math.nan
    out, out_t = space(70, 100), space(100, 70)
    s2r.s2r_q4_save(70, 100, s2r.mat(q8.wide(70, 100, dtype, x=x)), out, out_t)
    check(out, 70, 100, ref4.quantise(x))
    check(out_t, 100, 70, ref4.quantise(x.t()))
    y = q8.wide(70, 100, "f32", fill=7.0)
    s2r.s2r_q4_load(70, 100, out, s2r.mat(y))
    want = ref4.values(*ref4.quantise(x))
    assert torch.equal(y[:, :100].cpu().isnan(), want.isnan())
    assert torch.equal(y[:, :100].cpu().double().nan_to_num(9), want.nan_to_num(9))


def test_load_every_code_under_every_scale():
    gp.say("q4 load every code")
    code = torch.arange(16).repeat(2).expand(237, 32).contiguous()
    b = torch.tensor(list(range(17, 253)) + [255])[:, None]
    m, want = stored(code, b), ref4.values(code, b)
    for out in ("bf16", "f16", "f32"):
        y = q8.wide(237, 32, out, fill=7.0)
        s2r.s2r_q4_load(237, 32, m, s2r.mat(y))
        got = y[:, :32].cpu()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(9), want.to(ref.DTYPES[out]).nan_to_num(9)), out


# ---- product ----------------------------------------------------------------------------------

def product(M, N, K, a, b, out, with_ws):
    c = q8.wide(M, N, out, fill=7.0)
    ws = q8.workspace(s2r.s2r_q4_gemm_workspace_bytes(M, N, K)) if with_ws else None
    s2r.s2r_q4_gemm(M, N, K, a, b, s2r.mat(c), workspace=ws)
    assert q8.pad_kept(c, N, 7.0)
    return c[:, :N].cpu()


def exact_matrix(R, K, seed):
    """Codes of -2 .. 2 in halves under scales of 1/2, 1 and 2."""
    g = q8._gen(seed)
    code = torch.randint(0, 5, (R, K), generator=g) + 8 * torch.randint(0, 2, (R, K), generator=g)
    b = 127 + torch.randint(-1, 2, (R, up(K, 32) // 32), generator=g)
    return stored(code, b, seed), ref4.values(code, b)


SIZES = [(1, 64, 32), (1, 200, 1000), (5, 17, 31), (16, 300, 256), (17, 40, 257), (33, 8192, 4100), (64, 1000, 4096),
         (65, 70, 40), (130, 257, 384), (300, 300, 1000), (129, 127, 4100), (3000, 1300, 100), (3000, 1300, 256),
         (2770, 391, 6200), (4100, 2100, 300), (4100, 2100, 512), (4100, 4300, 130)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_exact(M, N, K):
    """Partial sums are multiples of 1/16 below 2^17 (K * 16 at most), whatever their order."""
    gp.say(f"q4 gemm exact {M}x{N}x{K}")
    a, va = exact_matrix(M, K, 1)
    b, vb = exact_matrix(N, K, 2)
    want = va.float() @ vb.float().t()
    for out in ("f32", "bf16", "f16"):
        for with_ws in (False, True):
            assert torch.equal(product(M, N, K, a, b, out, with_ws), want.to(ref.DTYPES[out])), (out, with_ws)


@pytest.mark.parametrize("M,N,K", [(3, 140, 64), (3, 140, 1000), (40, 200, 700), (300, 300, 96), (300, 300, 1000), (600, 140, 4100)])
@pytest.mark.parametrize("spread", [0, 4])
def test_product_of_ordinary_values(M, N, K, spread):
    """K additions in fp32, each off by at most a step of a partial sum of at most sum |a b|, and one rounding:
    products of codes have 8 bits, so none is cut."""
    gp.say(f"q4 gemm {M}x{N}x{K} spread {spread}")

    def matrix(R, seed):
        g = q8._gen(seed)
        x = torch.randn((R, K), generator=g, dtype=torch.float64)
        x *= torch.exp(spread * torch.randn((R, K), generator=g, dtype=torch.float64)) / 16
        code, b = ref4.quantise(x)
        return stored(code, b, seed), ref4.values(code, b)

    (a, va), (b, vb) = matrix(M, 3), matrix(N, 4)
    want, mass = va @ vb.t(), va.abs() @ vb.abs().t()
    tol = K * 2.0 ** -23 * mass
    for out in ("f32", "bf16", "f16"):
        t = tol + ref.HALF_STEP[out] * (want.abs() + tol) + (2.0 ** -25 if out == "f16" else 0)
        over = want.abs() + tol >= 65504 if out == "f16" else torch.zeros_like(want, dtype=torch.bool)
        for with_ws in (False, True):
            got = product(M, N, K, a, b, out, with_ws).double()
            assert bool((((got - want).abs() <= t) | over).all()), (out, with_ws)


@pytest.mark.parametrize("M,N,K", [(3, 40, 300), (300, 300, 300), (3000, 1300, 290)])
def test_product_of_scales_far_apart(M, N, K):
    """One scale for a row, over 2^40: every sum is a multiple of 1/4 below 2^14 times a power of two."""
    gp.say(f"q4 gemm wide scales {M}x{N}x{K}")
    g = q8._gen(9)
    nb = up(K, 32) // 32
    ca, cb = (torch.randint(0, 16, (R, K), generator=g) for R in (M, N))
    ea, eb = (torch.randint(-20, 21, (R, 1), generator=g) for R in (M, N))
    a, b = (stored(c, (e + 127).expand(-1, nb)) for c, e in ((ca, ea), (cb, eb)))
    v = ref4.code_values()
    want = (v[ca].float() @ v[cb].float().t()).double() * torch.exp2(ea.double()) * torch.exp2(eb.double()).t()
    for with_ws in (False, True):
        assert torch.equal(product(M, N, K, a, b, "f32", with_ws).double(), want)


@pytest.mark.parametrize("M,N,K", [(5, 40, 300), (300, 300, 256), (3000, 1300, 300)])
def test_nan_blocks_stay_in_their_row_and_column(M, N, K):
    gp.say(f"q4 gemm NaN {M}x{N}x{K}")
    a, va = exact_matrix(M, K, 5)
    b, vb = exact_matrix(N, K, 6)
    a.scales[1, (K - 1) // 32] = 255
    a.scales[M - 1, 0] = 255
    b.scales[N - 2, 3] = 255
    want = va.float() @ vb.float().t()
    want[1], want[M - 1], want[:, N - 2] = math.nan, math.nan, math.nan
    for with_ws in (False, True):
        got = product(M, N, K, a, b, "f32", with_ws)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(1e9), want.nan_to_num(1e9))


def test_empty_sum():
    gp.say("q4 gemm K = 0")
    a, b = space(40, 1), space(50, 1)
    for M in (3, 40):
        assert bool((product(M, 50, 0, a, b, "bf16", True) == 0).all())


@pytest.mark.parametrize("M,K,N", [(100, 200, 72), (515, 384, 640)])
def test_a_layers_three_products(M, K, N):
    """Y = X W^T, dX = dY W and dW = dY^T X, the operands saved by one call each."""
    gp.say(f"q4 layer {M}x{K}x{N}")
    x, w, dy = (torch.randn(s, generator=q8._gen(i)).bfloat16() for i, s in enumerate([(M, K), (N, K), (M, N)]))
    m, t = {}, {}
    for name, v in (("x", x), ("w", w), ("dy", dy)):
        m[name], t[name] = s2r.alloc_q4(*v.shape), s2r.alloc_q4(v.shape[1], v.shape[0])
        s2r.s2r_q4_save(*v.shape, s2r.mat(q8.wide(*v.shape, "bf16", x=v)), m[name], t[name])
    v = {n: ref4.values(*ref4.quantise(u)) for n, u in (("x", x), ("w", w), ("dy", dy), ("xt", x.t()), ("wt", w.t()), ("dyt", dy.t()))}
    for P, Q, S, a, b, va, vb in [(M, N, K, m["x"], m["w"], "x", "w"), (M, K, N, m["dy"], t["w"], "dy", "wt"),
                                  (N, K, M, t["dy"], t["x"], "dyt", "xt")]:
        want, mass = v[va] @ v[vb].t(), v[va].abs() @ v[vb].abs().t()
        got = product(P, Q, S, a, b, "f32", True).double()
        assert bool(((got - want).abs() <= S * 2.0 ** -23 * mass + 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("M,N,K", [(3, 300, 1000), (300, 1000, 4096), (900, 700, 600)])
def test_graph_replays_and_other_streams(M, N, K):
    """Storage and product, with a cut sum among them: the same bits eager, on another stream and from every replay of a
    graph, with eager work between the replays."""
    gp.say(f"q4 graph {M}x{N}x{K}")

    def keep(seed):
        g = q8._gen(seed)
        x, w = (torch.randn((r, K), generator=g).bfloat16() for r in (M, N))
        return dict(x=s2r.mat(q8.wide(M, K, "bf16", x=x)[:, :K]), w=s2r.mat(q8.wide(N, K, "bf16", x=w)[:, :K]),
                    xq=s2r.alloc_q4(M, K), xt=s2r.alloc_q4(K, M), wq=s2r.alloc_q4(N, K), y=torch.zeros((M, up(N, 8)), device=DEV),
                    ws=q8.workspace(s2r.s2r_q4_gemm_workspace_bytes(M, N, K)))

    def step(k, stream=None):
        s2r.s2r_q4_save(M, K, k["x"], k["xq"], k["xt"], stream=stream)
        s2r.s2r_q4_save(N, K, k["w"], k["wq"], stream=stream)
        s2r.s2r_q4_gemm(M, N, K, k["xq"], k["wq"], s2r.mat(k["y"][:, :N]), workspace=k["ws"], stream=stream)

    k, other = keep(1), keep(2)
    step(k)
    want = k["y"].clone()
    side = torch.cuda.Stream()
    k["y"].fill_(0)
    torch.cuda.synchronize()
    step(k, side)
    torch.cuda.synchronize()
    assert torch.equal(k["y"][:, :N], want[:, :N])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(k)
    for rep in range(3):
        for t in (k["y"], k["xq"].codes, k["xq"].scales, k["wq"].codes):
            t.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(k["y"][:, :N], want[:, :N]), rep
        step(other)


def test_rows_beyond_four_gib():
    """Codes and results whose offsets do not fit 32 bits: the last rows of a long matrix."""
    gp.say("q4 beyond 4 GiB")
    M, N, K = 1_100_000, 1000, 8192  # 4.5 GB of codes, 4.4 GB of fp32 results
    a = s2r.alloc_q4(M, K)
    a.codes.zero_(), a.scales.fill_(127)
    b, vb = exact_matrix(N, K, 2)
    n = 300
    code = torch.randint(0, 5, (n, K), generator=q8._gen(3)) + 8 * torch.randint(0, 2, (n, K), generator=q8._gen(4))
    a.codes[-n:] = (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8).to(DEV)
    va = ref4.code_values()[code]
    c = torch.empty((M, N), device=DEV)
    s2r.s2r_q4_gemm(M, N, K, a, b, s2r.mat(c))
    assert torch.equal(c[-n:].cpu(), va.float() @ vb.float().t())
    assert bool((c[:-n] == 0).all())
    y = c.view(torch.bfloat16)[:, :K // 8]
    s2r.s2r_q4_load(M, K // 8, a, s2r.mat(y))
    assert torch.equal(y[-n:].cpu().double(), va[:, :K // 8])
    again = s2r.alloc_q4(M, K // 8)
    s2r.s2r_q4_save(M, K // 8, s2r.mat(y), again)
    back = torch.empty((n, K // 8), dtype=torch.bfloat16, device=DEV)
    tail = s2r.q4_mat(again.codes[-n:], again.scales[-n:])
    s2r.s2r_q4_load(n, K // 8, tail, s2r.mat(back))
    assert torch.equal(back.cpu().double(), va[:, :K // 8])


@pytest.mark.parametrize("M", [3, 40, 300])
def test_product_keeps_small_products_beside_large_ones(M):
    """2^12 in one block of the sum and multiples of 2^-11 in every other one: fp32 holds all of it, wherever the
    instruction adds them."""
    gp.say(f"q4 gemm small beside large M={M}")
    N, K = 140, 600
    nb = up(K, 32) // 32
    for big in (0, 3, 5, 18):
        g = q8._gen(big)
        ca, cb = torch.zeros((M, K), dtype=torch.long), torch.zeros((N, K), dtype=torch.long)
        ba, bb = torch.full((M, nb), 127 - 4), torch.full((N, nb), 127 - 5)
        at = torch.arange(nb) * 32 + torch.randint(0, 24, (nb,), generator=g)
        ca[:, at] = torch.randint(0, 2, (M, nb), generator=g)           # 0 or 1/2, times 2^-4
        cb[:, at] = torch.randint(0, 2, (N, nb), generator=g) * (1 + 8 * torch.randint(0, 2, (N, nb), generator=g))
        ca[:, big * 32:big * 32 + 32], cb[:, big * 32:big * 32 + 32] = 0, 0
        ca[:, big * 32 + 7], cb[:, big * 32 + 7] = 6, 6                 # 4, times 2^4
        ba[:, big], bb[:, big] = 127 + 4, 127 + 4
        want = ref4.values(ca, ba) @ ref4.values(cb, bb).t()
        assert len(want.unique()) > 2 and float((want * 2 ** 11).frac().abs().max()) == 0
        a, b = stored(ca, ba), stored(cb, bb)
        for with_ws in (False, True):
            assert torch.equal(product(M, N, K, a, b, "f32", with_ws).double(), want), (big, with_ws)
