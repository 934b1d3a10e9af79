"""The 8-bit training calls on the GPU against the 64-bit reference.

Storage is exact: codes and scales equal the reference's.  The products are checked twice:
on small integers and quarter steps, where every order of the sum gives the same fp32 value
(equality to the bit), and on ordinary values within the bound of an fp32 sum.  Paddings
hold NaN codes on input and a pattern on output that has to survive."""
import math

import pytest
import torch

import count_sketch_aggregation_amd as s2r
import q8_reference as ref

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")
DEV = "cuda"
POISON = 0xA5


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def wide(rows, cols, dtype, pad=16, x=None, fill=math.nan):
    """A [rows][cols] view with its row padding filled; x in it if given."""
    ld = ref.up(cols, 16) + pad
    t = torch.full((rows, ld), fill, dtype=ref.DTYPES[dtype], device=DEV)
    if x is not None:
        t[:, :cols] = x.to(DEV).to(t.dtype)
    return t


def pad_kept(t, cols, fill):
    p = t[:, cols:]
    return bool((p.isnan() if math.isnan(fill) else p == fill).all())


def space(rows, cols, fmt, square=False, pad=16, fill=POISON):
    """An 8-bit matrix of poisoned storage with padded rows and scale rows."""
    sr = ref.up(rows, 128) // 128 if square else rows
    q = torch.full((rows, ref.up(cols, 16) + pad), fill, dtype=torch.uint8, device=DEV)
    s = torch.full((ref.up(cols, 128) // 128, ref.up(sr, 4) + 4), fill, dtype=torch.uint8, device=DEV)
    return s2r.q8_mat(q, s, fmt)


def stored(codes, bytes_, fmt, square=False, pad=16):
    """An 8-bit matrix from codes [R][C] (uint8) and scale bytes [row blocks][column blocks];
    every padding byte is a NaN code or an unused scale of 2^127."""
    m = space(*codes.shape, fmt, square, pad, fill=0x7F)
    m.codes[:, :codes.shape[1]] = codes.to(DEV)
    m.scales.fill_(0xFE)
    m.scales[:, :bytes_.shape[0]] = bytes_.t().to(torch.uint8).to(DEV)
    return m


def check_stored(m, rows, cols, want, fmt, square=False):
    """Codes and scales of m against (code values, bytes), and the padding untouched."""
    q, b = want
    got = ref.code_values(fmt)[m.codes[:, :cols].cpu().int()]
    assert torch.equal(m.scales[:, :b.shape[0]].cpu().t().long(), b)
    assert torch.equal(got.isnan(), q.isnan())
    assert torch.equal(got.nan_to_num(0, 1e9, -1e9), q.nan_to_num(0, 1e9, -1e9))
    assert bool((m.codes[:, cols:] == POISON).all())
    assert bool((m.scales[:, b.shape[0]:] == POISON).all())


def awkward(M, K, dtype, seed):
    """Values over many magnitudes, with blocks of zeros, of subnormals and at the scale's border."""
    g = _gen(seed)
    x = torch.randn((M, K), generator=g, dtype=torch.float64)
    spread = 30 if dtype != "f16" else 4
    x *= torch.exp2(torch.randint(-spread, spread, (M, 1), generator=g).double())
    x[M // 3] = 0
    if K > 3:
        x[M // 2] = 0
        x[M // 2, K // 2] = 448 * 2.0 ** -3
        x[-1, 0] = 449
    x = x.to(ref.DTYPES[dtype])
    if M > 4:
        tiny = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}[dtype]
        x[1] = tiny * 3
        x[2] = (torch.rand((K,), generator=g) * 2.0 ** -113).to(x.dtype)
    return x


SHAPES = [(1, 1), (1, 75), (3, 128), (33, 129), (64, 640), (130, 1000), (257, 16), (7, 2049)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_save_and_load(M, K, dtype, fmt):
    gp.say(f"save/load {M}x{K} {dtype} {fmt}")
    x = awkward(M, K, dtype, M + K)
    out = space(M, K, fmt)
    s2r.s2r_q8_save(M, K, s2r.mat(wide(M, K, dtype, x=x)), out)
    want = ref.quantise(x, fmt)
    check_stored(out, M, K, want, fmt)
    values = want[0] * ref.spread(want[1], M, K, False)
    for t in ("bf16", "f16", "f32"):
        y = wide(M, K, t, fill=7.0)
        s2r.s2r_q8_load(M, K, out, s2r.mat(y))
        assert torch.equal(y[:, :K].cpu(), values.to(ref.DTYPES[t])), t  # exact, or rounded once
        if t != "f16":
            assert torch.equal(y[:, :K].cpu().double(), values), t
        assert pad_kept(y, K, 7.0)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_save_non_finite(fmt, dtype):
    """Infinities and NaN do not move their block's scale and stay non-finite."""
    gp.say(f"save non-finite {fmt} {dtype}")
    x = torch.randn((9, 300), generator=_gen(5)).to(ref.DTYPES[dtype])
    x[0, 3], x[1, 140], x[2, 299], x[3, 0] = math.inf, -math.inf, math.nan, math.nan
    x[3, 1] = math.inf
    x[4, :] = math.nan
    x[5, 128:256] = -math.inf
    out = space(9, 300, fmt)
    s2r.s2r_q8_save(9, 300, s2r.mat(wide(9, 300, dtype, x=x)), out)
    check_stored(out, 9, 300, ref.quantise(x, fmt), fmt)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 127), (40, 300), (300, 40), (257, 1000)])
def test_weight_and_its_transpose(N, K, dtype, fmt):
    gp.say(f"weight {N}x{K} {dtype} {fmt}")
    x = awkward(N, K, dtype, N + K)
    if N > 6:
        x[5, 0], x[6, K - 1] = math.nan, math.inf
    q, b = ref.quantise(x, fmt, True)
    out, out_t = space(N, K, fmt, True), space(K, N, fmt, True)
    s2r.s2r_q8_weight(N, K, s2r.mat(wide(N, K, dtype, x=x)), out, out_t)
    check_stored(out, N, K, (q, b), fmt, True)
    check_stored(out_t, K, N, (q.t(), b.t()), fmt, True)
    alone = space(N, K, fmt, True)
    s2r.s2r_q8_weight(N, K, s2r.mat(wide(N, K, dtype, x=x)), alone)
    assert torch.equal(alone.codes, out.codes) and torch.equal(alone.scales, out.scales)


# ---------------------------------------------------------------------------------------
# products


def integers(R, C, fmt, seed, square=False, most=2):
    """Codes of the integers -most .. most and scales of 1/2, 1 and 2: (stored matrix, fp64 values)."""
    g = _gen(seed)
    v = torch.randint(-most, most + 1, (R, C), generator=g)
    codes = v.float().to(ref.F8[fmt]).view(torch.uint8)
    sr = ref.up(R, 128) // 128 if square else R
    b = torch.randint(126, 129, (sr, ref.up(C, 128) // 128), generator=g)
    return stored(codes, b, fmt, square), v.double() * ref.spread(b, R, C, square)


def ordinary(R, C, fmt, seed, square=False, std=1.0):
    x = torch.randn((R, C), generator=_gen(seed), dtype=torch.float64) * std
    q, b = ref.quantise(x, fmt, square)
    codes = q.float().to(ref.F8[fmt]).view(torch.uint8)
    return stored(codes, b, fmt, square), q * ref.spread(b, R, C, square)


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV) if nbytes else None  # NaNs


def gemm(M, N, K, a, b, out, with_ws):
    c = wide(M, N, out, fill=7.0)
    ws = workspace(s2r.s2r_q8_gemm_workspace_bytes(M, N, K)) if with_ws else None
    s2r.s2r_q8_gemm(M, N, K, a, b, s2r.mat(c), workspace=ws)
    assert pad_kept(c, N, 7.0)
    return c[:, :N].cpu()


GEMMS = [(1, 1, 1), (1, 200, 1000), (2, 16, 128), (5, 31, 129), (16, 64, 256), (17, 100, 384),
         (33, 257, 127), (37, 512, 1024), (64, 128, 2000), (65, 65, 640), (100, 300, 512),
         (129, 127, 4100), (200, 500, 250), (256, 256, 256), (257, 513, 300), (300, 1000, 1152),
         (520, 264, 900), (1030, 700, 520)]


@pytest.mark.parametrize("with_ws", [False, True], ids=["alone", "workspace"])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm_on_integers(M, N, K, with_ws):
    """Every partial sum is a multiple of 1/4 below 2^22: fp32 holds it, in any order."""
    fa = "e5m2" if (M + N) % 3 == 0 else "e4m3"
    gp.say(f"gemm integers {M}x{N}x{K} {fa} ws={with_ws}")
    a, va = integers(M, K, fa, 1)
    b, vb = integers(N, K, "e4m3", 2, True)
    want = va @ vb.t()
    assert torch.equal(gemm(M, N, K, a, b, "f32", with_ws).double(), want)
    for out in ("bf16", "f16"):
        assert torch.equal(gemm(M, N, K, a, b, out, with_ws), want.to(ref.DTYPES[out]))


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 2000), (40, 200, 700), (300, 300, 1000), (600, 520, 1300)])
def test_gemm_on_ordinary_values(M, N, K, fa, fb):
    """Each product is exact in fp32; K of them are added, each addition off by at most one
    step (2^-23: the matrix instruction may cut) of a partial sum of at most sum |a b|; then the result is
    rounded once."""
    gp.say(f"gemm {M}x{N}x{K} {fa} {fb}")
    a, va = ordinary(M, K, fa, 3, std=1e-3)
    b, vb = ordinary(N, K, fb, 4, True, std=0.05)
    want, mass = va @ vb.t(), va.abs() @ vb.abs().t()
    for out in ("f32", "bf16", "f16"):
        # fp16's least step is 2^-24: half of it on top
        tol = K * 2.0 ** -23 * mass + ref.HALF_STEP[out] * want.abs() * 1.01 + \
            (2.0 ** -25 if out == "f16" else 0)
        for with_ws in (False, True):
            got = gemm(M, N, K, a, b, out, with_ws).double()
            assert bool(((got - want).abs() <= tol).all()), (out, with_ws)


@pytest.mark.parametrize("M", [1, 20, 60, 130, 300])
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
def test_gemm_in_fp32_keeps_small_products_beside_large_ones(M, fa):
    """2^16 and 2^-6 among the products of one block of the sum: fp32 holds all of it."""
    gp.say(f"gemm small beside large M={M} {fa}")
    N, K = 140, 400
    g = _gen(12)
    va, vb = torch.zeros((M, K), dtype=torch.float64), torch.zeros((N, K), dtype=torch.float64)
    big = torch.randint(0, K // 2, (1,), generator=g).item() * 2
    va[:, big], vb[:, big] = 2.0 ** 8, 2.0 ** 8
    for at in (big + 1, (big + 7) % K, (big + 40) % K, (big + 190) % K):
        va[:, at] = 2.0 ** -3 * torch.randint(0, 2, (M,), generator=g)
        vb[:, at] = 2.0 ** -3 * torch.randint(-1, 2, (N,), generator=g)
    code = lambda v, f: v.float().to(ref.F8[f]).view(torch.uint8)
    a = stored(code(va, fa), torch.full((M, 4), 127), fa)
    b = stored(code(vb, "e4m3"), torch.full((2, 4), 127), "e4m3", True)
    want = va @ vb.t()
    assert len(want.unique()) > 1
    for with_ws in (False, True):
        assert torch.equal(gemm(M, N, K, a, b, "f32", with_ws).double(), want)


def test_gemm_takes_wide_scales():
    """Scales over the whole range a stored matrix can have, in one row and in one column."""
    gp.say("gemm wide scales")
    M, N, K = 70, 140, 1000
    g = _gen(9)
    ca = torch.randint(-2, 3, (M, K), generator=g)
    cb = torch.randint(-2, 3, (N, K), generator=g)
    ea = torch.randint(-60, 60, (M, 1), generator=g).expand(M, 8).contiguous()
    eb = torch.randint(-50, 50, (2, 1), generator=g).expand(2, 8).contiguous()
    f8 = lambda c: c.float().to(torch.float8_e4m3fn).view(torch.uint8)
    a, b = stored(f8(ca), ea + 127, "e4m3"), stored(f8(cb), eb + 127, "e4m3", True)
    want = (ca.double() * ref.spread(ea + 127, M, K, False)) @ (cb.double() * ref.spread(eb + 127, N, K, True)).t()
    assert torch.equal(gemm(M, N, K, a, b, "f32", True).double(), want)


@pytest.mark.parametrize("M", [3, 100, 300])
def test_gemm_keeps_non_finite_values_in_their_row(M):
    """A NaN of a row of A makes that row of C NaN and leaves the others; infinities follow IEEE."""
    gp.say(f"gemm non-finite M={M}")
    N, K = 130, 300
    a, va = integers(M, K, "e5m2", 5)
    b, vb = integers(N, K, "e4m3", 6, True)
    a.codes[1, 299], a.codes[2, 7] = 0x7F, 0x7C
    va[1, 299], va[2, 7] = math.nan, math.inf
    want = torch.stack([(va[i] * vb).sum(1) for i in range(3)])
    got = gemm(M, N, K, a, b, "f32", True).double()
    assert torch.equal(got[:3].isnan(), want.isnan())
    assert torch.equal(got[:3].nan_to_num(5, 1e30, -1e30), want.nan_to_num(5, 1e30, -1e30))
    assert torch.equal(got[3:], va[3:] @ vb.t())


@pytest.mark.parametrize("K", [100, 128, 300, 512])
def test_gemm_of_many_tiles(K):
    """More tiles than compute units, of one block of the sum and of several, whole and not."""
    M, N = 4500, 4300
    gp.say(f"gemm many tiles {M}x{N}x{K}")
    a, va = integers(M, K, "e4m3", 1)
    b, vb = integers(N, K, "e4m3", 2, True)
    want = va.float() @ vb.float().t()  # exact: multiples of 1/4 below 2^22
    assert torch.equal(gemm(M, N, K, a, b, "f32", True), want)
    assert torch.equal(gemm(M, N, K, a, b, "bf16", False), want.bfloat16())


def test_empty_sums():
    gp.say("empty sums")
    q = s2r.s2r_q8_mat(None, 16, None, 64, 0)
    c = torch.full((40, 48), 3.0, device=DEV)
    s2r.s2r_q8_gemm(40, 33, 0, q, q, s2r.mat(c))
    assert bool((c[:, :33] == 0).all()) and bool((c[:, 33:] == 3).all())
    c.fill_(3.0)
    dy = s2r.s2r_mat(None, 48, s2r.S2R_BF16)
    x = s2r.s2r_q8_mat(None, 64, None, 64, 0)
    s2r.s2r_q8_wgrad(0, 40, 33, dy, x, c, 48)
    assert bool((c[:, :33] == 0).all()) and bool((c[:, 33:] == 3).all())
    c.fill_(3.0)
    s2r.s2r_q8_wgrad(0, 40, 33, dy, x, c, 48, accumulate=True)
    assert bool((c == 3).all())


# ---------------------------------------------------------------------------------------
# weight gradient


def wgrad(M, N, K, dy, x, dw0=None, with_ws=True, lddw=None, off=0):
    """dw [N][K] inside a flat fp32 row at offset `off`, the rest of the row kept."""
    lddw = lddw or K
    flat = torch.full((off + N * lddw + 5,), 7.0, device=DEV)
    body = flat[off:off + N * lddw].view(N, lddw)
    if dw0 is not None:
        body[:, :K] = dw0.to(DEV).float()
    ws = workspace(s2r.s2r_q8_wgrad_workspace_bytes(M, N, K)) if with_ws else None
    s2r.s2r_q8_wgrad(M, N, K, dy, x, flat.data_ptr() + 4 * off, lddw, accumulate=dw0 is not None,
                     workspace=ws)
    assert bool((flat[:off] == 7).all()) and bool((flat[off + N * lddw:] == 7).all())
    assert bool((body[:, K:] == 7).all())
    return body[:, :K].cpu().double()


WGRADS = [(1, 1, 1), (1, 130, 200), (7, 33, 40), (32, 64, 64), (63, 128, 128), (65, 129, 127),
          (200, 40, 300), (333, 256, 256), (1000, 300, 520), (2050, 70, 600), (5001, 100, 65),
          (500, 600, 1000), (700, 257, 255)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", WGRADS)
def test_wgrad_on_integers(M, N, K, kind):
    """Every partial sum is a multiple of 1/4 below 2^22: equality to the bit, whether the sum is
    cut or not, at any offset and with any lddw, alone and added to what was there."""
    fx = "e5m2" if (M + K) % 3 == 0 else "e4m3"
    gp.say(f"wgrad integers {M}x{N}x{K} {kind} {fx}")
    if kind == "bf16":
        vy = torch.randint(-3, 4, (M, N), generator=_gen(7)).double()
        dy = s2r.mat(wide(M, N, "bf16", x=vy)[:, :N])
    else:
        dy, vy = integers(M, N, kind, 7)
    x, vx = integers(M, K, fx, 8)
    want = vy.t() @ vx
    dw0 = torch.randint(-50, 51, (N, K), generator=_gen(9)).double()
    for with_ws in (False, True):
        assert torch.equal(wgrad(M, N, K, dy, x, with_ws=with_ws), want)
        assert torch.equal(wgrad(M, N, K, dy, x, dw0, with_ws, lddw=K + 3, off=3), want + dw0)
        assert torch.equal(wgrad(M, N, K, dy, x, dw0, with_ws, lddw=ref.up(K, 4), off=4), want + dw0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", [(300, 200, 130), (3000, 260, 300)])
def test_wgrad_on_ordinary_values(M, N, K, kind):
    """Products of a bf16 and a stored value are exact in fp32; M additions, each off by at
    most a step."""
    gp.say(f"wgrad {M}x{N}x{K} {kind}")
    if kind == "bf16":
        vy = (torch.randn((M, N), generator=_gen(1)) * 1e-3).bfloat16().double()
        dy = s2r.mat(wide(M, N, "bf16", x=vy)[:, :N])
    else:
        dy, vy = ordinary(M, N, kind, 1, std=1e-3)
    x, vx = ordinary(M, K, "e4m3", 2)
    want, mass = vy.t() @ vx, vy.abs().t() @ vx.abs()
    for with_ws in (False, True):
        got = wgrad(M, N, K, dy, x, with_ws=with_ws)
        assert bool(((got - want).abs() <= M * 2.0 ** -23 * mass).all())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(6200, 2100, 2100), (1700, 4100, 4200)])
def test_wgrad_of_large_tiles(M, N, K, kind):
    """Sizes where the larger tiles are taken: a cut sum, and more tiles than compute units."""
    gp.say(f"wgrad large tiles {M}x{N}x{K} {kind}")
    if kind == "bf16":
        vy = torch.randint(-3, 4, (M, N), generator=_gen(7)).double()
        dy = s2r.mat(wide(M, N, "bf16", x=vy)[:, :N])
    else:
        dy, vy = integers(M, N, kind, 7)
    x, vx = integers(M, K, "e4m3", 8)
    want = vy.float().t() @ vx.float()  # exact: multiples of 1/4 below 2^22
    assert torch.equal(wgrad(M, N, K, dy, x).float(), want)
    dw0 = torch.randint(-50, 51, (N, K), generator=_gen(9)).double()
    assert torch.equal(wgrad(M, N, K, dy, x, dw0, lddw=K + 3, off=3).float(), want + dw0.float())


def test_wgrad_scales_along_the_sum():
    """The checkpoint's scales differ from row to row of the sum, over 2^40."""
    gp.say("wgrad wide scales")
    M, N, K = 40, 20, 300
    g = _gen(11)
    e = torch.randint(-20, 20, (M, 3), generator=g)
    c = torch.randint(1, 3, (M, K), generator=g)
    x = stored(c.float().to(torch.float8_e4m3fn).view(torch.uint8), e + 127, "e4m3")
    vx = c.double() * ref.spread(e + 127, M, K, False)
    sel = torch.zeros((M, N), dtype=torch.float64)   # one row each: nothing is added
    sel[torch.arange(N) * 2, torch.arange(N)] = -1
    got = wgrad(M, N, K, s2r.mat(wide(M, N, "bf16", x=sel)[:, :N]), x)
    assert torch.equal(got, sel.t() @ vx)


@pytest.mark.parametrize("kind", ["bf16", "e5m2"])
def test_scale_padding_may_hold_anything(kind):
    """The scale bytes behind a matrix's last row are not a number; M is not a multiple of 4."""
    gp.say(f"scale padding {kind}")
    M, N, K = 131, 150, 260
    x, vx = integers(M, K, "e4m3", 8)
    x.scales[:, M:] = 0xFF
    if kind == "bf16":
        vy = torch.randint(-3, 4, (M, N), generator=_gen(7)).double()
        dy = s2r.mat(wide(M, N, "bf16", x=vy)[:, :N])
    else:
        dy, vy = integers(M, N, kind, 7)
        dy.scales[:, M:] = 0xFF
    for with_ws in (False, True):
        assert torch.equal(wgrad(M, N, K, dy, x, with_ws=with_ws), vy.t() @ vx)
    b, vb = integers(N, K, "e4m3", 2, True)
    b.scales[:, 2:] = 0xFF
    for out in ("f32", "bf16"):
        assert torch.equal(gemm(M, N, K, x, b, out, True), (vx @ vb.t()).to(ref.DTYPES[out]))


def test_wgrad_keeps_non_finite_values_in_their_row():
    gp.say("wgrad non-finite")
    M, N, K = 100, 140, 150
    vy = torch.randint(1, 4, (M, N), generator=_gen(7)).double()
    vy[99, 3], vy[0, 5] = math.nan, math.inf
    x, vx = integers(M, K, "e4m3", 8)
    got = wgrad(M, N, K, s2r.mat(wide(M, N, "bf16", x=vy)[:, :N]), x)
    want = torch.stack([(vy[:, n:n + 1] * vx).sum(0) for n in range(N)])
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(5, 1e30, -1e30), want.nan_to_num(5, 1e30, -1e30))


# ---------------------------------------------------------------------------------------
# activation


GLUS = [(1, 1), (1, 300), (33, 129), (70, 1000), (5, 2064)]
ACTS = ["silu", "gelu", "gelu_tanh"]


def act_tolerance(g, a, d, kind):
    """Half steps of fp32 (2^-24): the sigmoid's exponential is off by its own 4 and by its
    argument's 2 |z| (z = g, or for gelu_tanh 2 sqrt(2/pi)(g + 0.044715 g^3), itself off by 4
    each), sum, division and products add 8; gelu adds erf's 8 to a value of order one, times
    g.  The derivative adds the same to each of its two terms.  Doubled; and fp32's least
    numbers."""
    z = g.abs() if kind != "gelu_tanh" else 4 * (1.6 * (g.abs() + 0.044715 * g.abs() ** 3))
    n = 2 * (12 + 2 * z)
    extra = 16 * g.abs() if kind == "gelu" else torch.zeros_like(g)
    terms = d.abs() + a.abs() + (g * torch.exp(-g * g / 2)).abs() + (16 if kind == "gelu" else 0)
    return (n * a.abs() + extra) * 2.0 ** -24 + 1e-37, (n * terms) * 2.0 ** -24 + 1e-37


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("M,F", GLUS)
def test_glu(M, F, gated, dtype, kind):
    gp.say(f"glu {M}x{F} {kind} {dtype} gated={gated}")
    fmt = "e5m2" if F % 3 == 0 else "e4m3"
    g = (torch.randn((M, F), generator=_gen(M)) * 4).to(ref.DTYPES[dtype])
    u = torch.randn((M, F), generator=_gen(F)).to(ref.DTYPES[dtype])
    g[0, 0] = 0
    mg = s2r.mat(wide(M, F, dtype, x=g)[:, :F])
    mu = s2r.mat(wide(M, F, dtype, x=u)[:, :F]) if gated else None
    y = wide(M, F, "f32", fill=7.0)
    gq, yq = space(M, F, fmt), space(M, F, "e4m3")
    uq = space(M, F, "e5m2") if gated else None
    s2r.s2r_q8_glu(M, F, kind, mg, mu, gq=gq, uq=uq, y=s2r.mat(y), yq=yq)
    check_stored(gq, M, F, ref.quantise(g, fmt), fmt)
    if gated:
        check_stored(uq, M, F, ref.quantise(u, "e5m2"), "e5m2")
    got = y[:, :F].cpu()
    a, d = ref.act(g.double(), kind)
    tol = act_tolerance(g.double(), a, d, kind)[0]
    want = a * u.double() if gated else a
    tol = tol * (u.double().abs() if gated else 1) + 2.0 ** -24 * want.abs() * 1.01 + 1e-37
    assert bool(((got.double() - want).abs() <= tol).all())
    check_stored(yq, M, F, ref.quantise(got, "e4m3"), "e4m3")  # the same fp32 value, stored
    assert pad_kept(y, F, 7.0)
    for t in ("bf16", "f16"):  # y alone, in 16 bits: the same value rounded
        y16 = wide(M, F, t, fill=7.0)
        s2r.s2r_q8_glu(M, F, kind, mg, mu, y=s2r.mat(y16))
        assert torch.equal(y16[:, :F].cpu(), got.to(ref.DTYPES[t])) and pad_kept(y16, F, 7.0)


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("M,F", GLUS)
def test_glu_grad(M, F, gated, dtype, kind):
    gp.say(f"glu_grad {M}x{F} {kind} {dtype} gated={gated}")
    fmt = "e5m2" if F % 3 == 0 else "e4m3"
    gq, vg = ordinary(M, F, fmt, 1, std=4)
    uq, vu = ordinary(M, F, fmt, 2)
    dy = (torch.randn((M, F), generator=_gen(3)) * 1e-2).to(ref.DTYPES[dtype])
    dg, du = wide(M, F, "f32", fill=7.0), wide(M, F, "f32", fill=7.0)
    dgq, duq = space(M, F, "e5m2"), space(M, F, "e4m3")
    extra = dict(du=s2r.mat(du), duq=duq) if gated else {}
    mdy = s2r.mat(wide(M, F, dtype, x=dy)[:, :F])
    s2r.s2r_q8_glu_grad(M, F, kind, gq, uq if gated else None, mdy, dg=s2r.mat(dg), dgq=dgq, **extra)
    a, d = ref.act(vg, kind)
    ta, td = act_tolerance(vg, a, d, kind)
    t = dy.double()
    k = t * vu if gated else t
    got = dg[:, :F].cpu()
    assert bool(((got.double() - k * d).abs() <= k.abs() * (td + 3 * 2.0 ** -24 * d.abs()) + 1e-37).all())
    check_stored(dgq, M, F, ref.quantise(got, "e5m2"), "e5m2")
    assert pad_kept(dg, F, 7.0)
    if gated:
        got_u = du[:, :F].cpu()
        assert bool(((got_u.double() - t * a).abs() <= t.abs() * (ta + 3 * 2.0 ** -24 * a.abs()) + 1e-37).all())
        check_stored(duq, M, F, ref.quantise(got_u, "e4m3"), "e4m3")
        assert pad_kept(du, F, 7.0)
    dg16 = wide(M, F, "bf16", fill=7.0)
    s2r.s2r_q8_glu_grad(M, F, kind, gq, uq if gated else None, mdy, dg=s2r.mat(dg16))
    assert torch.equal(dg16[:, :F].cpu(), got.bfloat16()) and pad_kept(dg16, F, 7.0)


def test_glu_far_values():
    """Where the exponential over- or underflows: act and its derivative at large |g|, and what
    infinities and NaN give."""
    gp.say("glu far values")
    g = torch.tensor([[-1e30, -200.0, -90.0, 90.0, 200.0, 1e30, math.inf, math.nan, 0.0, -0.0]])
    for kind in ACTS:
        y, d = (torch.zeros((1, 16), device=DEV) for _ in range(2))
        s2r.s2r_q8_glu(1, 10, kind, s2r.mat(wide(1, 10, "f32", x=g)[:, :10]), y=s2r.mat(y))
        y = y[0, :10].cpu()
        assert bool((y[:3].abs() < 1e-35).all()) and y[3:7].tolist() == [90.0, 200.0, float(g[0, 5]), math.inf]
        assert bool(y[7].isnan()) and y[8] == 0 and y[9] == 0
        far = torch.tensor([[-448.0, -100.0, 100.0, 448.0]])
        q = stored(far.to(torch.float8_e4m3fn).view(torch.uint8), torch.tensor([[127]]), "e4m3")
        one = torch.ones((1, 8), device=DEV)
        s2r.s2r_q8_glu_grad(1, 4, kind, q, None, s2r.mat(one), dg=s2r.mat(d))
        assert d[0, :4].cpu().abs().tolist() == [0.0, 0.0, 1.0, 1.0], kind


# ---------------------------------------------------------------------------------------
# how they are called


def test_offsets_beyond_32_bits():
    """Rows that start beyond 2^32 bytes and elements: 2^16 + 300 rows of 2^16."""
    gp.say("offsets beyond 32 bits")
    M, ld, K, N = (1 << 16) + 300, 1 << 16, 64, 16
    x = torch.empty((M, ld), dtype=torch.bfloat16, device=DEV)
    v = torch.randint(-2, 3, (M, K), generator=_gen(1)).double()
    x[:, :K] = v.to(DEV).bfloat16()
    q = torch.empty((M, ld), dtype=torch.uint8, device=DEV)
    s = torch.empty((1, ref.up(M, 4)), dtype=torch.uint8, device=DEV)
    m = s2r.q8_mat(q, s)
    s2r.s2r_q8_save(M, K, s2r.mat(x), m)
    b, vb = integers(N, K, "e4m3", 2, True)
    s2r.s2r_q8_gemm(M, N, K, m, b, s2r.mat(x))          # C over x, which is no longer read
    assert torch.equal(x[:, :N].cpu().double(), (v @ vb.t()).bfloat16().double())
    x[:, :K] = 0
    s2r.s2r_q8_load(M, K, m, s2r.mat(x))
    assert torch.equal(x[:, :K].cpu().double(), v)
    dw = torch.empty((K, K), device=DEV)
    s2r.s2r_q8_wgrad(M, K, K, s2r.mat(x), m, dw, K)
    assert torch.equal(dw.cpu().double(), v.t() @ v)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    s2r.s2r_q8_glu(M, K, "silu", s2r.mat(x), gq=s2r.q8_mat(q2, s2))
    assert torch.equal(q2[:, :K], q[:, :K]) and torch.equal(s2, s)


def _layer(stream, keep):
    """One pass through every call on `stream`, into the buffers of `keep`."""
    k = keep
    M, N, K = k["M"], k["N"], k["K"]
    s2r.s2r_q8_save(M, K, k["x"], k["xq"], stream=stream)
    s2r.s2r_q8_weight(N, K, k["w"], k["wq"], k["wt"], stream=stream)
    s2r.s2r_q8_gemm(M, N, K, k["xq"], k["wq"], k["h"], workspace=k["ws1"], stream=stream)
    s2r.s2r_q8_glu(M, N, "silu", k["h"], gq=k["hq"], yq=k["yq"], stream=stream)
    s2r.s2r_q8_load(M, N, k["yq"], k["y"], stream=stream)
    s2r.s2r_q8_glu_grad(M, N, "silu", k["hq"], None, k["y"], dgq=k["dhq"], stream=stream)
    s2r.s2r_q8_gemm(M, K, N, k["dhq"], k["wt"], k["dx"], workspace=k["ws2"], stream=stream)
    s2r.s2r_q8_wgrad(M, N, K, k["dhq"], k["xq"], k["dw"], K, workspace=k["ws3"], stream=stream)


def _keep(M, N, K, seed=0):
    bf = lambda r, c: torch.zeros((r, c), dtype=torch.bfloat16, device=DEV)
    x = (torch.randn((M, K), generator=_gen(seed))).bfloat16().to(DEV)
    w = (torch.randn((N, K), generator=_gen(seed + 1)) / 20).bfloat16().to(DEV)
    return dict(M=M, N=N, K=K, x=s2r.mat(x), w=s2r.mat(w), xq=s2r.alloc_q8(M, K),
                wq=s2r.alloc_q8(N, K, square=True), wt=s2r.alloc_q8(K, N, square=True),
                h=s2r.mat(bf(M, N)), hq=s2r.alloc_q8(M, N), yq=s2r.alloc_q8(M, N), y=s2r.mat(bf(M, N)),
                dhq=s2r.alloc_q8(M, N, "e5m2"), dx=s2r.mat(bf(M, K)),
                dw=torch.zeros((N, K), device=DEV),
                ws1=workspace(s2r.s2r_q8_gemm_workspace_bytes(M, N, K)),
                ws2=workspace(s2r.s2r_q8_gemm_workspace_bytes(M, K, N)),
                ws3=workspace(s2r.s2r_q8_wgrad_workspace_bytes(M, N, K)))


def _results(k):
    torch.cuda.synchronize()
    return [k["dx"].tensor.clone(), k["dw"].clone(), k["yq"].codes.clone(), k["y"].tensor.clone()]


@pytest.mark.parametrize("M,N,K", [(40, 400, 1024), (600, 512, 640)])
def test_graph_replays_and_other_streams(M, N, K):
    """The same bits eager, again, on another stream and from every replay of a graph, with eager
    work between the replays."""
    gp.say(f"q8 graph {M}x{N}x{K}")
    k = _keep(M, N, K)
    _layer(None, k)
    want = _results(k)

    def clear():
        for t in (k["dx"].tensor, k["dw"], k["yq"].codes, k["y"].tensor):
            t.fill_(5)
        torch.cuda.synchronize()

    def same():
        return all(torch.equal(a, b) for a, b in zip(_results(k), want))

    clear()
    _layer(torch.cuda.current_stream(), k)
    assert same()
    side = torch.cuda.Stream()
    clear()
    _layer(side, k)
    assert same()
    graph = torch.cuda.CUDAGraph()
    clear()
    with torch.cuda.graph(graph):
        _layer(torch.cuda.current_stream(), k)
    other = _keep(M, N, K, seed=50)
    for rep in range(3):
        clear()
        graph.replay()
        assert same(), rep
        _layer(None, other)
        torch.cuda.synchronize()


def test_refusals_reach_python():
    gp.say("q8 refusals")
    k = _keep(8, 32, 48)
    with pytest.raises(s2r.S2RError) as e:
        s2r.s2r_q8_gemm(8, 32, 400, k["xq"], k["wq"], k["h"])
    assert e.value.status == s2r.S2R_ERR_DIM
    with pytest.raises(s2r.S2RError) as e:
        s2r.s2r_q8_wgrad(8, 32, 48, s2r.mat(torch.zeros((8, 32), device=DEV)), k["xq"], k["dw"], 48)
    assert e.value.status == s2r.S2R_ERR_DIM
