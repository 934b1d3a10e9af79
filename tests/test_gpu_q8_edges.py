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


# ---------------------------------------------------------------------------------------
# NaN with a clear quiet bit


SIGNALLING = {"bf16": (torch.int16, [0x7F81, 0x7FBF, -0x7F, -0x41]),  # 0xFF81, 0xFFBF
              "f16": (torch.int16, [0x7C01, 0x7DFF, -0x3FF, -0x201]),
              "f32": (torch.int32, [0x7F800001, 0x7FBFFFFF, -0x7FFFFF, -0x400001])}


def with_signalling_nan(M, K, dtype):
    """Every row: a strong element, and behind it one signalling NaN, at every place of a lane."""
    bits, patterns = SIGNALLING[dtype]
    x = torch.randn((M, K), generator=q8._gen(4)).to(ref.DTYPES[dtype])
    for i in range(M):
        x[i, 0 if i % 2 else (i // 2) % 13] = 300.0 * (-1) ** i
        x.view(bits)[i, (1 + i // 2) % 16 if i % 2 else 13 + i % 3] = patterns[i % 4]
        if K > 200:
            x.view(bits)[i, 128 + (7 * i) % (K - 128)] = patterns[(i + 1) % 4]
    assert bool(x.isnan().any(1).all())
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_signalling_nan_leaves_its_blocks_scale(fmt, dtype):
    gp.say(f"signalling NaN {fmt} {dtype}")
    M, K = 64, 300
    x = with_signalling_nan(M, K, dtype)
    out = q8.space(M, K, fmt)
    s2r.s2r_q8_save(M, K, s2r.mat(q8.wide(M, K, dtype, x=x)), out)
    q8.check_stored(out, M, K, ref.quantise(x, fmt), fmt)
    w, w_t = q8.space(M, K, fmt, True), q8.space(K, M, fmt, True)
    s2r.s2r_q8_weight(M, K, s2r.mat(q8.wide(M, K, dtype, x=x)), w, w_t)
    q, b = ref.quantise(x, fmt, True)
    q8.check_stored(w, M, K, (q, b), fmt, True)
    q8.check_stored(w_t, K, M, (q.t(), b.t()), fmt, True)
    gq, uq = q8.space(M, K, fmt), q8.space(M, K, fmt)
    m = s2r.mat(q8.wide(M, K, dtype, x=x)[:, :K])
    s2r.s2r_q8_glu(M, K, "silu", m, m, gq=gq, uq=uq)
    q8.check_stored(gq, M, K, ref.quantise(x, fmt), fmt)
    q8.check_stored(uq, M, K, ref.quantise(x, fmt), fmt)


# ---------------------------------------------------------------------------------------
# activations


def forward(g, kind):
    """act(g) of a row of fp32 values, in fp32."""
    n = g.numel()
    y = q8.wide(1, n, "f32", fill=7.0)
    s2r.s2r_q8_glu(1, n, kind, s2r.mat(q8.wide(1, n, "f32", x=g[None])[:, :n]), y=s2r.mat(y))
    return y[0, :n].cpu()


def derivative(v):
    """(stored values in fp64, function that gives act' of them in fp32) for a row of multiples of a
    code's step."""
    m, values = v
    n = values.shape[1]

    def of(kind):
        one, d = torch.ones((1, ref.up(n, 8)), device=DEV), q8.wide(1, n, "f32", fill=7.0)
        s2r.s2r_q8_glu_grad(1, n, kind, m, None, s2r.mat(one), dg=s2r.mat(d))
        return d[0, :n].cpu().double()
    return values[0], of


def codes_of(values, byte=127, fmt="e4m3"):
    c = (values / 2.0 ** (byte - 127)).float().to(ref.F8[fmt])
    blocks = ref.up(len(values), 128) // 128
    m = q8.stored(c.view(torch.uint8)[None], torch.full((1, blocks), byte), fmt)
    return m, c.double()[None] * 2.0 ** (byte - 127)


def test_gelu_keeps_its_digits_far_below_zero():
    """g Phi(g) from -13 to 1 against the complementary error function in 64 bits.  Phi(-a) is
    e^(-a^2 / 2) h(a): the exponential is off by 4 half steps and its correction by 1, h's numerator
    and denominator by one for each coefficient (5 and 6), their quotient by 3, two more products by 2:
    21.  Results below fp32's normal range are off by its least number."""
    gp.say("gelu tail")
    g = -torch.arange(0, 13 * 512 + 1, dtype=torch.float64) / 512
    g = torch.cat([g, -g[1:512]]).float()
    want = ref.act(g.double(), "gelu")[0]
    got = forward(g, "gelu").double()
    assert bool(((got - want).abs() <= 21 * HALF * want.abs() + 2.0 ** -148).all())


def test_gelu_of_a_block_far_below_zero():
    """129 columns: the last one is a block of its own, and its scale follows the small value."""
    gp.say("gelu far block")
    M, F = 40, 129
    g = torch.randn((M, F), generator=q8._gen(6))
    g[:, 128] = -4 - torch.arange(M) / 8
    yq = q8.space(M, F, "e4m3")
    s2r.s2r_q8_glu(M, F, "gelu", s2r.mat(q8.wide(M, F, "f32", x=g)[:, :F]), yq=yq)
    want = ref.act(g.double(), "gelu")[0][:, 128]
    code = ref.code_values("e4m3")[yq.codes[:, 128].cpu().int()]
    got = code * torch.exp2(yq.scales[1, :M].cpu().double() - 127)
    # half a step of e4m3, and the value's own error, far below what is left
    assert bool(((got - want).abs() <= 1.001 * 2.0 ** -4 * want.abs()).all())


@pytest.mark.parametrize("kind,lo,hi", [("silu", 4, 17), ("gelu_tanh", 3, 8)])
def test_derivative_keeps_its_digits_where_the_sigmoid_is_near_one(kind, lo, hi):
    """act' = s plus a small term, s = 1 / (1 + e) with e below 0.02.  In half steps: the sum 1 + e and its
    reciprocal 1 each, e's own error (4, for the tanh form 31 with its argument's) times e below
    0.1; the small term, below 0.08 and off by 9 (tanh form: below 0.02 and off by 40), below 0.8;
    the last sum and product 1 each, and what is of second order: below 6."""
    gp.say(f"derivative near one {kind}")
    v = torch.cat([torch.arange(8, 16).double() / 8 * 2.0 ** e for e in range(1, 5)])
    v = v[(v >= lo) & (v <= hi)]
    values, of = derivative(codes_of(v))
    want = ref.act(values, kind)[1]
    assert len(values) > 10
    got = of(kind)
    assert bool(((got - want).abs() <= 6 * HALF * want.abs()).all()), ((got - want) / want / HALF)


@pytest.mark.parametrize("kind", q8.ACTS)
def test_derivative_of_huge_values(kind):
    """0 on the left and 1 on the right, up to the largest that a stored matrix holds."""
    gp.say(f"derivative of huge values {kind}")
    for byte in (127, 160, 187, 190, 220, 239):
        v = torch.tensor([-448.0, -256.0, 256.0, 448.0], dtype=torch.float64) * 2.0 ** (byte - 127)
        values, of = derivative(codes_of(v, byte))
        assert of(kind).abs().tolist() == [0.0, 0.0, 1.0, 1.0], byte


# ---------------------------------------------------------------------------------------
# the ends of the range


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_next_to_the_largest_stay_finite(dtype, fmt):
    """What would round to 2^128 is stored as the largest code below it: still off by at most
    2^-4 (e4m3) or 2^-3 (e5m2) of itself, and finite in bf16 and fp32.  Infinities and NaN stay."""
    gp.say(f"largest values {dtype} {fmt}")
    M, K = 9, 300
    top = {"bf16": 255 * 2.0 ** 120, "f32": (2 - 2.0 ** -23) * 2.0 ** 127}[dtype]
    f = torch.linspace(0.8, 1.0, M * K, dtype=torch.float64).reshape(M, K) * top
    f[:, ::3] *= -1
    f[0, 3] = f[1, 0] = top
    f[2, 0] = -top
    f[3, :200] = torch.linspace(-1, 1, 200) * 1e30
    f[4, 7], f[5, 8], f[6, 9] = math.inf, -math.inf, math.nan
    x = f.to(ref.DTYPES[dtype])
    fin = torch.isfinite(x)
    want = x.double()
    share = 2.0 ** -4 if fmt == "e4m3" else 2.0 ** -3
    least = 2.0 ** -10 if fmt == "e4m3" else 2.0 ** -17  # below the format's normal range, times the scale

    def check(m, rows, cols, back, square):
        got = back.double()
        ok = torch.isfinite(got)
        assert bool(ok[fin].all()) and not bool(ok[~fin].any())
        b = m.scales.cpu().double() - 127
        s = torch.exp2(b[:ref.up(cols, 128) // 128]).t()
        s = (s[:1].expand(rows, -1) if square else s[:rows]).repeat_interleave(128, 1)[:, :cols]
        off = (got - want)[fin].abs()
        assert bool((off <= torch.maximum(share * want[fin].abs(), least * s[fin])).all())

    out = q8.space(M, K, fmt)
    s2r.s2r_q8_save(M, K, s2r.mat(q8.wide(M, K, dtype, x=x)), out)
    for t in ("f32", "bf16"):
        y = q8.wide(M, K, t, fill=7.0)
        s2r.s2r_q8_load(M, K, out, s2r.mat(y))
        check(out, M, K, y[:, :K].cpu(), False)
    gq = q8.space(M, K, fmt)
    s2r.s2r_q8_glu(M, K, "silu", s2r.mat(q8.wide(M, K, dtype, x=x)[:, :K]), gq=gq)
    assert torch.equal(gq.codes, out.codes) and torch.equal(gq.scales, out.scales)
    w = q8.space(M, K, fmt, True)
    s2r.s2r_q8_weight(M, K, s2r.mat(q8.wide(M, K, dtype, x=x)), w)
    code = ref.code_values(fmt)[w.codes[:, :K].cpu().int()]
    scale = torch.exp2(w.scales[:, 0].cpu().double() - 127).repeat_interleave(128)[:K]
    check(w, M, K, (code * scale).float(), True)


def test_the_most_rows():
    """2^28 - 1 rows: more workgroups than one launch holds."""
    gp.say("most rows")
    M, K = (1 << 28) - 1, 16
    x = torch.randint(0, 256, (M, K), dtype=torch.uint8, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    x[x.bitwise_and(0x7F) == 0x7F] = 0
    m = s2r.q8_mat(x, torch.full((1, 1 << 28), 127, dtype=torch.uint8, device=DEV))
    y = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=DEV)
    s2r.s2r_q8_load(M, K, m, s2r.mat(y))
    half = 1 << 27
    for part in (slice(0, half), slice(half, M)):
        assert torch.equal(y[part], x[part].view(torch.float8_e4m3fn).bfloat16())
    back = s2r.alloc_q8(M, K)
    s2r.s2r_q8_save(M, K, s2r.mat(y), back)
    again = torch.empty_like(y)
    s2r.s2r_q8_load(M, K, back, s2r.mat(again))
    for part in (slice(0, half), slice(half, M)):  # a smaller scale holds every value too
        assert torch.equal(again[part], y[part])


# ---------------------------------------------------------------------------------------
# ranges of columns


def columns(m, first, last):
    """Columns first .. last - 1 of an 8-bit matrix, first a multiple of 128."""
    fmt = ["e4m3", "e5m2"][m.format]
    return s2r.q8_mat(m.codes[:, first:last], m.scales[first // 128:ref.up(last, 128) // 128], fmt)


@pytest.mark.parametrize("M,F,D", [(7, 128, 100), (131, 384, 260), (700, 256, 500)])
def test_matrices_side_by_side(M, F, D):
    """A gated layer whose g and u, their checkpoints, their gradients and its weights' transposes
    each lie in one matrix of 2 F columns, the last of which ends the buffer: the same bits as apart, and
    the input gradient dg Wg + du Wu is one product over both halves."""
    gp.say(f"side by side {M}x{F}x{D}")
    g = q8._gen(3)
    bf = lambda r, c: (torch.randn((r, c), generator=g)).bfloat16().to(DEV)
    h, x, dy = bf(M, 2 * F), bf(M, ref.up(D, 8)), bf(M, F)
    halves = lambda t: (s2r.mat(t[:, :F]), s2r.mat(t[:, F:]))
    new = lambda r, c, **k: s2r.alloc_q8(r, c, **k)
    both, grads = new(M, 2 * F), new(M, 2 * F, fmt="e5m2")
    split = lambda m: (columns(m, 0, F), columns(m, F, 2 * F))
    s2r.s2r_q8_glu(M, F, "silu", *halves(h), gq=split(both)[0], uq=split(both)[1])
    s2r.s2r_q8_glu_grad(M, F, "silu", *split(both), s2r.mat(dy), dgq=split(grads)[0], duq=split(grads)[1])
    apart, apart_grads = [new(M, F) for _ in range(2)], [new(M, F, fmt="e5m2") for _ in range(2)]
    s2r.s2r_q8_glu(M, F, "silu", s2r.mat(h[:, :F].contiguous()), s2r.mat(h[:, F:].contiguous()), gq=apart[0], uq=apart[1])
    s2r.s2r_q8_glu_grad(M, F, "silu", *apart, s2r.mat(dy), dgq=apart_grads[0], duq=apart_grads[1])
    for m, parts in ((both, apart), (grads, apart_grads)):
        for half, part in zip(split(m), parts):
            assert torch.equal(half.codes, part.codes) and torch.equal(half.scales[:, :M], part.scales[:, :M])
    # weight gradients from halves: codes, and a bf16 range that ends its buffer
    xq = new(M, D)
    s2r.s2r_q8_save(M, D, s2r.mat(x), xq)
    for i in range(2):
        for one, two in ((split(grads)[i], apart_grads[i]), (halves(h)[i], s2r.mat(h[:, i * F:(i + 1) * F].contiguous()))):
            dw = [torch.zeros((F, D), device=DEV) for _ in range(2)]
            s2r.s2r_q8_wgrad(M, F, D, one, xq, dw[0], D)
            s2r.s2r_q8_wgrad(M, F, D, two, xq, dw[1], D)
            assert torch.equal(*dw)
    # the input gradient
    w = [torch.randn((F, D), generator=g).to(DEV) / 16 for _ in range(2)]
    wq, wt = [new(F, D, square=True) for _ in range(2)], new(D, 2 * F, square=True)
    for i in range(2):
        padded = torch.zeros((F, ref.up(D, 4)), device=DEV)
        padded[:, :D] = w[i]
        s2r.s2r_q8_weight(F, D, s2r.mat(padded), wq[i], split(wt)[i])
    dx = q8.wide(M, D, "f32", fill=7.0)
    s2r.s2r_q8_gemm(M, D, 2 * F, grads, wt, s2r.mat(dx))
    value = lambda m, r, c, square: ref.code_values(["e4m3", "e5m2"][m.format])[m.codes[:, :c].cpu().int()] * ref.spread(
        m.scales.cpu().t().long()[:ref.up(r, 128) // 128 if square else r], r, c, square)
    dv, wv = value(grads, M, 2 * F, False), value(wt, D, 2 * F, True)
    want, mass = dv @ wv.t(), dv.abs() @ wv.abs().t()
    assert bool(((dx[:, :D].cpu().double() - want).abs() <= 2 * F * 2.0 ** -23 * mass).all())
    want_w = torch.cat([(ref.quantise(t.cpu(), "e4m3", True)[0] * ref.spread(ref.quantise(t.cpu(), "e4m3", True)[1], F, D, True)).t()
                        for t in w], 1)
    assert torch.equal(wv, want_w)
    # each half alone, the second one ending its buffer
    for i in range(2):
        y = [q8.wide(M, D, "f32", fill=7.0) for _ in range(2)]
        s2r.s2r_q8_gemm(M, D, F, split(grads)[i], split(wt)[i], s2r.mat(y[0]))
        wti = new(D, F, square=True)
        wti.codes.copy_(split(wt)[i].codes)
        wti.scales.copy_(split(wt)[i].scales)
        s2r.s2r_q8_gemm(M, D, F, apart_grads[i], wti, s2r.mat(y[1]))
        assert torch.equal(y[0][:, :D], y[1][:, :D])
