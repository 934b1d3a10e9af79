"""Layers of experts on the GPU: routing, rows and tokens against plain loops, the experts' products
and weight gradients on integers (equality to the bit) and ordinary values.  Rows that no choice has, paddings and
everything around the outputs hold a pattern that has to survive."""
import math

import pytest
import torch

import count_sketch_aggregation_amd as s2r
import q8_reference as ref
import test_gpu_q8 as q8

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")
DEV = "cuda"
up = ref.up


def choices(T, K, E, seed, drop=0.1):
    """expert [T][K]: some experts liked more, some never chosen, some choices none."""
    g = q8._gen(seed)
    p = torch.rand(E, generator=g) ** 3 + 1e-3
    if E > 3:
        p[torch.randint(0, E, (max(1, E // 4),), generator=g)] = 0
        p[0] = max(float(p[0]), 1e-3)
    expert = torch.multinomial(p, T * K, replacement=True, generator=g).view(T, K).int() if T else torch.zeros((0, K), dtype=torch.int32)
    none = torch.tensor([-1, E, -7, 2 ** 31 - 1], dtype=torch.int64)[torch.randint(0, 4, (T, K), generator=g)].int()
    return torch.where(torch.rand((T, K), generator=g) < drop, none, expert)


def routed(expert, E):
    """first, rows, place by going through the choices."""
    flat = expert.reshape(-1).tolist()
    rows = [0] * E
    for e in flat:
        if 0 <= e < E:
            rows[e] += 1
    first, at = [], 0
    for r in rows:
        first.append(at)
        at += up(r, 4)
    nxt, place = list(first), []
    for e in flat:
        if 0 <= e < E:
            place.append(nxt[e])
            nxt[e] += 1
        else:
            place.append(-1)
    return (torch.tensor(v, dtype=torch.int32) for v in (first, rows, place))


def route(expert, E):
    T, K = expert.shape
    first, rows = (torch.full((E + 2,), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    place = torch.full((T * K + 2,), -9, dtype=torch.int32, device=DEV)
    ws = q8.workspace(s2r.s2r_moe_route_workspace_bytes(T, K, E))
    s2r.s2r_moe_route(T, K, E, expert.to(DEV).contiguous(), first[1:-1], rows[1:-1], place[1:-1].view(T, K), workspace=ws)
    for t in (first, rows, place):
        assert int(t[0]) == -9 and int(t[-1]) == -9
    return first[1:-1], rows[1:-1], place[1:-1].view(T, K)


ROUTES = [(0, 1, 1), (1, 1, 1), (1, 8, 64), (3, 2, 5), (24, 8, 64), (64, 1, 3), (257, 4, 17), (683, 3, 129), (1024, 2, 1024),
          (2049, 1, 128), (1024, 1, 7), (4096, 1, 40), (4097, 1, 40), (1366, 3, 1), (1000, 7, 128), (5000, 8, 200), (4096, 64, 60), (300000, 2, 1000), (70001, 8, 31)]


@pytest.mark.parametrize("T,K,E", ROUTES)
def test_route(T, K, E):
    gp.say(f"route {T}x{K} of {E}")
    expert = choices(T, K, E, T + K)
    for got, want in zip(route(expert, E), routed(expert, E)):
        assert torch.equal(got.cpu().view(-1), want)
    assert T * K == 0 or int(max(routed(expert, E).__next__())) <= s2r.s2r_moe_rows(T, K, E)


@pytest.mark.parametrize("T", [5, 3000])
def test_route_of_one_expert_and_of_none(T):
    gp.say(f"route {T} of one and none")
    for expert in (torch.full((T, 4), 2, dtype=torch.int32), torch.full((T, 4), -1, dtype=torch.int32)):
        for got, want in zip(route(expert, 6), routed(expert, 6)):
            assert torch.equal(got.cpu().view(-1), want)


class Routed:
    """A routing and what the tests need of it on the host."""

    def __init__(self, T, K, E, seed=0, drop=0.1, expert=None):
        self.T, self.K, self.E = T, K, E
        self.expert = choices(T, K, E, seed, drop) if expert is None else expert
        self.first, self.rows, self.place = (v for v in route(self.expert, E))
        self.h = [v.cpu() for v in (self.first, self.rows, self.place)]
        self.R = max(4, s2r.s2r_moe_rows(T, K, E)) + 4
        self.at = self.h[2].reshape(-1).long()
        self.some = self.at >= 0
        self.used = torch.zeros(self.R, dtype=torch.bool)
        self.used[self.at[self.some]] = True
        self.token = torch.arange(T).repeat_interleave(K)
        self.e = s2r.experts(self.first, self.rows)

    def sorted_of(self, per_choice, fill=math.nan):
        """[R][...] rows of values [T K][...], `fill` in the others."""
        out = torch.full((self.R,) + per_choice.shape[1:], fill, dtype=per_choice.dtype)
        out[self.at[self.some]] = per_choice[self.some]
        return out

    def span(self, e):
        f = int(self.h[0][e])
        return slice(f, f + int(self.h[1][e]))


SHAPES = [(1, 1, 1, 1), (5, 3, 4, 33), (24, 8, 64, 1000), (70, 2, 9, 2050), (130, 5, 12, 128), (9, 64, 80, 515), (33, 6, 7, 4097)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,K,E,D", SHAPES)
def test_gather(T, K, E, D, dtype):
    gp.say(f"gather {T}x{K} of {E}, {D} {dtype}")
    m = Routed(T, K, E, T)
    x = q8.awkward(T, D, dtype, T + D)
    src = s2r.mat(q8.wide(T, D, dtype, x=x))
    for fmt in ("e4m3", "e5m2"):
        out, q = q8.wide(m.R, D, dtype, fill=7.0), q8.space(m.R, D, fmt)
        s2r.s2r_moe_gather(T, K, D, src, m.place, m.R, s2r.mat(out), q)
        want = m.sorted_of(x[m.token], 7.0)
        assert torch.equal(out[:, :D].cpu(), want) and q8.pad_kept(out, D, 7.0)
        codes, b = ref.quantise(x, fmt)
        used = m.used
        got = ref.code_values(fmt)[q.codes[:, :D].cpu().int()]
        assert torch.equal(got[used], m.sorted_of(codes[m.token])[used])
        assert torch.equal(q.scales[:, :m.R].cpu().t()[used].long(), m.sorted_of(b[m.token], 0)[used])
        assert bool((q.codes[~used.to(DEV)] == q8.POISON).all()) and bool((q.codes[:, D:] == q8.POISON).all())
        assert bool((q.scales.t()[:m.R][~used.to(DEV)] == q8.POISON).all()) and bool((q.scales[:, m.R:] == q8.POISON).all())
        alone = q8.space(m.R, D, fmt)
        s2r.s2r_moe_gather(T, K, D, src, m.place, m.R, outq=alone)
        assert torch.equal(alone.codes, q.codes) and torch.equal(alone.scales, q.scales)


def rows_of(m, D, dtype, seed):
    """Rows with NaN where no choice is."""
    r = m.sorted_of(torch.randn((m.T * m.K, D), generator=q8._gen(seed)).to(ref.DTYPES[dtype]))
    return r, q8.wide(m.R, D, dtype, x=r)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,K,E,D", SHAPES)
def test_combine(T, K, E, D, dtype):
    """K products and additions in fp32, each off by at most half a step of a partial sum of at most
    sum |w r|, and one rounding."""
    gp.say(f"combine {T}x{K} of {E}, {D} {dtype}")
    m = Routed(T, K, E, T + 1)
    r, buf = rows_of(m, D, dtype, 3)
    w = torch.randn((T, K), generator=q8._gen(4))
    w[~m.some.view(T, K)] = math.nan  # the weight of a choice without a row counts for nothing
    per = torch.where(m.some[:, None], r[m.at.clamp(min=0)].double(), 0.0).view(T, K, D)
    for weight in (w, None):
        f = torch.where(m.some.view(T, K), w.double(), 0.0) if weight is not None else torch.ones((T, K)).double()
        want, mass = (f[..., None] * per).sum(1), (f[..., None] * per).abs().sum(1)
        for out in ("bf16", "f16", "f32"):
            y = q8.wide(T, D, out, fill=7.0)
            s2r.s2r_moe_combine(T, K, D, s2r.mat(buf), m.R, m.place, None if weight is None else w.to(DEV), s2r.mat(y))
            tol = K * 2.0 ** -24 * mass
            tol = tol + ref.HALF_STEP[out] * (want.abs() + tol) + (2.0 ** -25 if out == "f16" else 2.0 ** -140)
            assert bool(((y[:, :D].cpu().double() - want).abs() <= tol).all()), (out, weight is None)
            assert q8.pad_kept(y, D, 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,K,E,D", SHAPES)
def test_combine_grad(T, K, E, D, dtype):
    """drows is one product in fp32 (rounded as its type has it, or stored as s2r_q8_save stores it); dweight has D
    products and additions in fp32, in some order."""
    gp.say(f"combine grad {T}x{K} of {E}, {D} {dtype}")
    m = Routed(T, K, E, T + 2)
    r, buf = rows_of(m, D, dtype, 5)
    dy = torch.randn((T, D), generator=q8._gen(6)).to(ref.DTYPES[dtype])
    src = s2r.mat(q8.wide(T, D, dtype, x=dy))
    w = torch.randn((T, K), generator=q8._gen(7))
    per = torch.where(m.some[:, None], r[m.at.clamp(min=0)].double(), 0.0)
    want_dw = (per * dy.double()[m.token]).sum(1)
    mass = (per * dy.double()[m.token]).abs().sum(1)
    used = m.used
    for weight, fmt, out in [(w, "e5m2", None), (w, "e4m3", "bf16"), (None, None, "f32"), (w, None, "f16"), (w, None, None)]:
        scaled = dy.float()[m.token] * (w.reshape(-1, 1) if weight is not None else 1)
        q = q8.space(m.R, D, fmt) if fmt else None
        g = q8.wide(m.R, D, out, fill=7.0) if out else None
        dw = torch.full((T * K + 2,), 7.0, device=DEV)
        s2r.s2r_moe_combine_grad(T, K, D, src, m.place, m.R, weight=None if weight is None else w.to(DEV),
                                 rows=s2r.mat(buf), drows=None if g is None else s2r.mat(g), drowsq=q,
                                 dweight=dw[1:-1].view(T, K))
        assert float(dw[0]) == 7 and float(dw[-1]) == 7
        assert bool(((dw[1:-1].cpu().double() - want_dw).abs() <= D * 2.0 ** -24 * mass + 2.0 ** -140).all())
        assert bool((dw[1:-1].cpu()[~m.some] == 0).all())
        if g is not None:
            assert torch.equal(g[:, :D].cpu(), m.sorted_of(scaled.to(ref.DTYPES[out]), 7.0)) and q8.pad_kept(g, D, 7.0)
        if q is not None:
            codes, b = ref.quantise(scaled, fmt)
            got = ref.code_values(fmt)[q.codes[:, :D].cpu().int()]
            assert torch.equal(got[used], m.sorted_of(codes)[used])
            assert torch.equal(q.scales[:, :m.R].cpu().t()[used].long(), m.sorted_of(b, 0)[used])
            assert bool((q.codes[~used.to(DEV)] == q8.POISON).all()) and bool((q.codes[:, D:] == q8.POISON).all())


def test_places_of_other_programs():
    """Places beyond the rows count as none; rows in any order."""
    gp.say("places of other programs")
    T, K, D, R = 6, 2, 40, 9
    place = torch.tensor([[8, 0], [9, 3], [-1, 5], [2 ** 31 - 1, -2 ** 31], [1, 10], [2, 4]], dtype=torch.int32, device=DEV)
    x = torch.randn((T, D), generator=q8._gen(1)).bfloat16()
    out = q8.wide(R, D, "bf16", fill=7.0)
    s2r.s2r_moe_gather(T, K, D, s2r.mat(q8.wide(T, D, "bf16", x=x)), place, R, s2r.mat(out))
    want = torch.full((R, D), 7.0).bfloat16()
    for t, k, r in [(0, 0, 8), (0, 1, 0), (1, 1, 3), (2, 1, 5), (4, 0, 1), (5, 0, 2), (5, 1, 4)]:
        want[r] = x[t]
    assert torch.equal(out[:, :D].cpu(), want)
    y = q8.wide(T, D, "f32", fill=7.0)
    s2r.s2r_moe_combine(T, K, D, s2r.mat(out), R, place, None, s2r.mat(y))
    n = torch.tensor([2, 1, 1, 0, 1, 2])[:, None]
    assert torch.equal(y[:, :D].cpu(), n * x.float())


# ---- experts' products ---------------------------------------------------------------------

def expert_weights(E, N, K, fmt, seed, exact=True):
    """Stacked weights with a multiple of 128 rows each: (stored, values [E][N][K], steps)."""
    NS = up(N, 128)
    make = q8.integers if exact else q8.ordinary
    m, v = make(E * NS, K, fmt, seed, True)
    return m, v.view(E, NS, K)[:, :N], (NS * m.ld, NS // 128)


def product(m, N, K, a, b, steps, out):
    c = q8.wide(m.R, N, out, fill=7.0)
    s2r.s2r_q8_gemm_experts(m.R, N, K, m.e, a, b, *steps, s2r.mat(c))
    assert q8.pad_kept(c, N, 7.0)
    assert bool((c[~m.used.to(DEV)] == 7).all())
    return c[:, :N].cpu()


GEMMS = [(1, 1, 1, 1, 1), (1, 2, 4, 40, 129), (16, 4, 32, 200, 1000), (24, 8, 100, 520, 384), (100, 2, 3, 300, 300),
         (400, 3, 5, 257, 127), (1000, 2, 8, 391, 640), (900, 4, 2, 700, 4100), (5000, 2, 6, 520, 256),
         (3000, 4, 40, 1100, 300), (12000, 1, 1000, 130, 200), (6000, 4, 5, 2100, 130),
         # tiles of 256, of few experts and of many, with and without a ragged last block; many experts in tiles of 128
         (8000, 1, 2, 1790, 300), (13800, 1, 70, 500, 256), (13800, 1, 70, 500, 300), (9000, 1, 300, 130, 200)]


@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("T,K,E,N,D", GEMMS)
def test_experts_products_on_integers(T, K, E, N, D, fa, fb):
    """Every partial sum is a multiple of 1/4 below 2^22."""
    gp.say(f"experts gemm {T}x{K} of {E}, {N}x{D} {fa} {fb}")
    m = Routed(T, K, E, 3)
    a, va = q8.integers(m.R, D, fa, 1)
    a.codes[~m.used.to(DEV), :D] = 0x7F  # NaN in rows of no choice
    b, vb, steps = expert_weights(E, N, D, fb, 2)
    want = torch.full((m.R, N), 7.0)
    for e in range(E):
        want[m.span(e)] = va[m.span(e)].float() @ vb[e].float().t()
    for out in ("f32", "bf16", "f16") if fa == fb else ("f32",):
        assert torch.equal(product(m, N, D, a, b, steps, out), want.to(ref.DTYPES[out])), out


@pytest.mark.parametrize("T,K,E,N,D", [(16, 4, 8, 200, 1000), (300, 2, 5, 300, 1000), (2000, 2, 4, 520, 1300)])
def test_experts_products_of_ordinary_values(T, K, E, N, D):
    """As s2r_q8_gemm: D additions in fp32, each off by at most a step of at most sum |a b|."""
    gp.say(f"experts gemm ordinary {T}x{K} of {E}, {N}x{D}")
    m = Routed(T, K, E, 4)
    a, va = q8.ordinary(m.R, D, "e4m3", 3)
    b, vb, steps = expert_weights(E, N, D, "e4m3", 4, exact=False)
    for out in ("f32", "bf16"):
        got = product(m, N, D, a, b, steps, out).double()
        for e in range(E):
            x, w = va[m.span(e)], vb[e]
            want, mass = x @ w.t(), x.abs() @ w.abs().t()
            tol = D * 2.0 ** -23 * mass
            assert bool(((got[m.span(e)] - want).abs() <= tol + ref.HALF_STEP[out] * (want.abs() + tol)).all())


@pytest.mark.parametrize("T", [20, 700])
def test_experts_products_of_transposed_weights(T):
    """One s2r_q8_weight of the stacked weights serves both directions: the transposed copies lie side by
    side."""
    gp.say(f"experts gemm transposed {T}")
    E, N, D = 5, 200, 328
    NS = up(N, 128)
    m = Routed(T, 2, E, 5)
    w = torch.randn((E * NS, D), generator=q8._gen(8))
    b, bt = q8.space(E * NS, D, "e4m3", True), q8.space(D, E * NS, "e4m3", True)
    s2r.s2r_q8_weight(E * NS, D, s2r.mat(q8.wide(E * NS, D, "f32", x=w)), b, bt)
    codes, s = ref.quantise(w, "e4m3", True)
    v = (codes * ref.spread(s, E * NS, D, True)).view(E, NS, D)[:, :N]
    dy, vdy = q8.integers(m.R, N, "e5m2", 9)
    got = product(m, D, N, dy, bt, (NS, NS // 128 * bt.lds), "f32").double()
    for e in range(E):
        want, mass = vdy[m.span(e)] @ v[e], vdy[m.span(e)].abs() @ v[e].abs()
        assert bool(((got[m.span(e)] - want).abs() <= (N * 2.0 ** -23 + 2.0 ** -24) * mass).all())


def wgrad(m, N, K, dy, x, dw0=None, lddw=None, gap=0, off=0):
    lddw = lddw or K
    step = (N - 1) * lddw + K + gap
    flat = torch.full((off + m.E * step + 5,), 7.0, device=DEV)
    view = torch.as_strided(flat, (m.E, N, K), (step, lddw, 1), off)
    kept = torch.ones_like(flat, dtype=torch.bool)
    torch.as_strided(kept, (m.E, N, K), (step, lddw, 1), off).fill_(False)
    if dw0 is not None:
        view.copy_(dw0)
    s2r.s2r_q8_wgrad_experts(m.R, N, K, m.e, dy, x, flat.data_ptr() + 4 * off, lddw, step, accumulate=dw0 is not None)
    assert bool((flat[kept] == 7).all())
    return view.cpu()


WGRADS = [(1, 1, 1, 1, 1), (3, 2, 4, 40, 70), (100, 2, 3, 130, 200), (300, 4, 40, 257, 65), (1501, 2, 8, 500, 258), (900, 4, 5, 300, 2100),
          (3000, 2, 70, 300, 520),
          # 256 x 256 tiles, of many experts and of few
          (1500, 2, 130, 300, 260), (600, 2, 30, 1100, 1000)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("T,K,E,N,D", WGRADS)
def test_experts_weight_gradients_on_integers(T, K, E, N, D, kind):
    """Every partial sum is a multiple of 1/4 below 2^22; rows of no choice hold NaN."""
    gp.say(f"experts wgrad {T}x{K} of {E}, {N}x{D} {kind}")
    m = Routed(T, K, E, 6)
    unused = ~m.used.to(DEV)
    if kind == "bf16":
        vy = torch.randint(-3, 4, (m.R, N), generator=q8._gen(7)).double()
        buf = q8.wide(m.R, N, "bf16", x=vy)
        buf[unused] = math.nan
        dy = s2r.mat(buf[:, :N])
    else:
        dy, vy = q8.integers(m.R, N, kind, 7)
        dy.codes[unused] = 0x7F
    x, vx = q8.integers(m.R, D, "e5m2" if (T + D) % 3 == 0 else "e4m3", 8)
    x.codes[unused] = 0x7F
    want = torch.stack([vy[m.span(e)].float().t() @ vx[m.span(e)].float() for e in range(E)])
    assert torch.equal(wgrad(m, N, D, dy, x), want)
    dw0 = torch.randint(-50, 50, (E, N, D), generator=q8._gen(9)).float().to(DEV)
    assert torch.equal(wgrad(m, N, D, dy, x, dw0, lddw=D + 3, gap=1, off=3), want + dw0.cpu())


def test_experts_without_rows():
    """No choice at all: products write nothing, gradients are zeros, or what was there."""
    gp.say("experts without rows")
    m = Routed(8, 2, 6, expert=torch.full((8, 2), -1, dtype=torch.int32))
    a, _ = q8.integers(m.R, 200, "e4m3", 1)
    b, _, steps = expert_weights(6, 130, 200, "e4m3", 2)
    assert bool((product(m, 130, 200, a, b, steps, "bf16") == 7).all())
    dy, _ = q8.integers(m.R, 130, "e4m3", 3)
    assert bool((wgrad(m, 130, 200, dy, a) == 0).all())
    assert bool((wgrad(m, 130, 200, dy, a, torch.full((6, 130, 200), 5.0, device=DEV)) == 5).all())


@pytest.mark.parametrize("T,E", [(6, 4), (900, 4)])
def test_empty_sums_of_experts(T, E):
    """K == 0 writes zeros to the experts' rows and to no others; M == 0 gives gradients of zeros."""
    gp.say(f"experts, empty sums {T}")
    m = Routed(T, 2, E, 13)
    q = s2r.s2r_q8_mat(None, 16, None, up(m.R, 4), 0)
    c = q8.wide(m.R, 130, "f32", fill=7.0)
    s2r.s2r_q8_gemm_experts(m.R, 130, 0, m.e, q, q, 0, 0, s2r.mat(c))
    want = torch.full((m.R, 130), 7.0)
    want[m.used] = 0
    assert torch.equal(c[:, :130].cpu(), want) and q8.pad_kept(c, 130, 7.0)
    dw = torch.full((E, 40, 36), 3.0, device=DEV)
    none = s2r.s2r_mat(None, 48, s2r.S2R_BF16)
    s2r.s2r_q8_wgrad_experts(0, 40, 36, m.e, none, s2r.s2r_q8_mat(None, 48, None, 4, 0), dw, 36, 40 * 36, accumulate=True)
    assert bool((dw == 3).all())
    s2r.s2r_q8_wgrad_experts(0, 40, 36, m.e, none, s2r.s2r_q8_mat(None, 48, None, 4, 0), dw, 36, 40 * 36)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("T,N", [(60, 300), (1500, 520), (9000, 1000)])
def test_the_same_bits_every_time(T, N):
    """Few rows, tiles, weight gradients, combine's gradients: repeated, with other calls in between."""
    gp.say(f"experts repeated {T}x{N}")
    m, D = Routed(T, 2, 9, 14), 520
    a, _ = q8.ordinary(m.R, D, "e4m3", 3)
    b, _, steps = expert_weights(9, N, D, "e4m3", 4, exact=False)
    dy, _ = q8.ordinary(m.R, N, "e5m2", 5)
    r, buf = rows_of(m, D, "bf16", 5)
    d = s2r.mat(q8.wide(T, D, "bf16", x=torch.randn((T, D), generator=q8._gen(6)))[:, :D])
    first = {}
    for i in range(4):
        for out in ("f32", "bf16"):
            got = product(m, N, D, a, b, steps, out)
            assert torch.equal(got, first.setdefault(out, got)), (out, i)
        got = wgrad(m, N, D, dy, a)
        assert torch.equal(got, first.setdefault("wgrad", got)), i
        dw = torch.zeros((T, 2), device=DEV)
        s2r.s2r_moe_combine_grad(T, 2, D, d, m.place, m.R, rows=s2r.mat(buf), dweight=dw)
        assert torch.equal(dw, first.setdefault("dweight", dw)), i


@pytest.mark.parametrize("T", [4, 900])
def test_rows_beyond_the_matrices_do_not_count(T):
    """first and rows that point beyond M are cut there: the others' results are right."""
    gp.say(f"experts beyond the rows {T}")
    m = Routed(T, 2, 4, 11, drop=0)
    a, va = q8.integers(m.R, 200, "e4m3", 1)
    b, vb, steps = expert_weights(4, 130, 200, "e4m3", 2)
    first, rows = m.first.clone(), m.rows.clone()
    rows[3] = 2 ** 31 - 1
    c = q8.wide(m.R, 130, "f32", fill=7.0)
    s2r.s2r_q8_gemm_experts(m.R, 130, 200, s2r.experts(first, rows), a, b, *steps, s2r.mat(c))
    for e in range(3):
        assert torch.equal(c[m.span(e), :130].cpu(), va[m.span(e)].float() @ vb[e].float().t())
    f = int(first[3])
    assert torch.equal(c[f:, :130].cpu(), va[f:].float() @ vb[3].float().t())
    first[3], rows[3] = 2 ** 31 - 4, 8
    c.fill_(7.0)
    s2r.s2r_q8_gemm_experts(m.R, 130, 200, s2r.experts(first, rows), a, b, *steps, s2r.mat(c))
    assert bool((c[f:] == 7).all())


def test_a_layer_and_its_gradients():
    """Tokens to experts, a product for each, back with weights, and every gradient, against the formulas in
    64 bits on the stored values; the weights' gradient against differences of s2r_moe_combine too."""
    gp.say("layer of experts")
    T, K, E, D, N = 300, 2, 7, 160, 200
    m = Routed(T, K, E, 12)
    x = torch.randn((T, D), generator=q8._gen(1)).bfloat16()
    w = torch.rand((T, K), generator=q8._gen(2))
    b, vb, steps = expert_weights(E, N, D, "e4m3", 3, exact=False)
    xq = q8.space(m.R, D, "e4m3")
    s2r.s2r_moe_gather(T, K, D, s2r.mat(q8.wide(T, D, "bf16", x=x)), m.place, m.R, outq=xq)
    h = q8.wide(m.R, N, "f32", fill=math.nan)
    s2r.s2r_q8_gemm_experts(m.R, N, D, m.e, xq, b, *steps, s2r.mat(h))
    y = q8.wide(T, N, "f32", fill=7.0)
    s2r.s2r_moe_combine(T, K, N, s2r.mat(h), m.R, m.place, w.to(DEV), s2r.mat(y))
    codes, s = ref.quantise(x, "e4m3")
    vx = (codes * ref.spread(s, T, D, False)).requires_grad_()
    ws, vw = w.double().requires_grad_(), vb.double().clone().requires_grad_()
    e = torch.where(m.some, m.expert.reshape(-1).long(), 0)
    per = torch.einsum("td,tnd->tn", vx[m.token], vw[e]) * m.some[:, None]
    want = (per.view(T, K, N) * ws[..., None]).sum(1)
    size = float(want.detach().abs().mean())
    assert float((y[:, :N].cpu().double() - want.detach()).abs().max()) < 1e-4 * size
    dy = torch.randn((T, N), generator=q8._gen(4)).bfloat16()
    want.backward(dy.double())
    g, dw = q8.space(m.R, N, "e5m2"), torch.zeros((T, K), device=DEV)
    dyb = s2r.mat(q8.wide(T, N, "f32", x=dy))
    s2r.s2r_moe_combine_grad(T, K, N, dyb, m.place, m.R, weight=w.to(DEV), rows=s2r.mat(h), drowsq=g, dweight=dw)
    assert float((dw.cpu().double() - ws.grad).abs().max()) < 1e-4 * float(ws.grad.abs().mean())
    # y is linear in the weights: a difference of any size gives their gradient, but for fp32's rounding
    d = torch.zeros((T, K))
    d[:, 1] = 1
    y2 = q8.wide(T, N, "f32", fill=7.0)
    s2r.s2r_moe_combine(T, K, N, s2r.mat(h), m.R, m.place, (w + d).to(DEV), s2r.mat(y2))
    diff = ((y2 - y)[:, :N].cpu().double() * dy.double()).sum(1)
    assert float((diff - dw.cpu().double()[:, 1]).abs().max()) < 1e-4 * float(ws.grad.abs().mean())
    # the experts' gradient, from the stored one of the rows
    gw = wgrad(m, N, D, g, xq)
    stored = ref.code_values("e5m2")[g.codes[:, :N].cpu().int()] * ref.spread(g.scales[:, :m.R].cpu().t().long(), m.R, N, False)
    for e in range(E):
        rows = vx.detach()[m.token][m.some][torch.argsort(m.at[m.some])]
        order = torch.sort(m.at[m.some]).values
        mine = (order >= m.span(e).start) & (order < m.span(e).stop)
        assert float((gw[e].double() - stored[m.span(e)].t() @ rows[mine]).abs().max()) <= 1e-4 * size * 10
        # stored in e5m2 each is off by at most 2^-3, on average by half of that or less
        assert float((gw[e].double() - vw.grad[e]).norm()) <= 2.0 ** -4 * float(vw.grad[e].norm()) + 1e-30
    assert bool((g.codes[~m.used.to(DEV)] == q8.POISON).all())


def test_rows_beyond_four_gib():
    """Rows whose offsets do not fit 32 bits, in every call that goes by rows."""
    gp.say("rows beyond 4 GiB")
    T, K, D, R = 70, 2, 4096, 1_100_000  # 4.5 GB of codes, 9 GB of bf16
    far = R - 200
    place = (far + torch.randperm(T * K, generator=q8._gen(1)).view(T, K)).int().to(DEV)
    x = torch.randn((T, D), generator=q8._gen(2)).bfloat16()
    src = s2r.mat(q8.wide(T, D, "bf16", x=x)[:, :D])
    rows = torch.empty((R, D), dtype=torch.bfloat16, device=DEV)
    q = s2r.alloc_q8(R, D)
    s2r.s2r_moe_gather(T, K, D, src, place, R, s2r.mat(rows), q)
    at = place.long().view(-1)
    per = x[torch.arange(T).repeat_interleave(K)]
    assert torch.equal(rows[at].cpu(), per)
    codes, b = ref.quantise(per, "e4m3")
    assert torch.equal(ref.code_values("e4m3")[q.codes[at][:, :D].cpu().int()], codes)
    assert torch.equal(q.scales[:, at].cpu().t().long(), b)
    y = q8.wide(T, D, "f32", fill=7.0)
    s2r.s2r_moe_combine(T, K, D, s2r.mat(rows), R, place, None, s2r.mat(y))
    assert torch.equal(y[:, :D].cpu(), K * x.float())
    dw = torch.zeros((T, K), device=DEV)
    s2r.s2r_moe_combine_grad(T, K, D, src, place, R, rows=s2r.mat(rows), drowsq=q, dweight=dw)
    want = (x.double() ** 2).sum(1)
    assert bool(((dw.cpu().double() - want[:, None]).abs() <= D * 2.0 ** -24 * want[:, None]).all())
    # two experts on those rows: 100 and 40, then 8 and 4, as few rows and as tiles have them
    v = torch.zeros((R - far, D), dtype=torch.float64)
    v[at.cpu() - far] = codes * ref.spread(b, T * K, D, False)
    w, vw = q8.integers(256, D, "e4m3", 3, True)
    for n0, n1 in ((100, 40), (8, 4)):
        e = s2r.experts(torch.tensor([far, far + n0], dtype=torch.int32, device=DEV), torch.tensor([n0, n1], dtype=torch.int32, device=DEV))
        want = torch.cat([v[:n0] @ vw[:128].t(), v[n0:n0 + n1] @ vw[128:].t()])
        mass = torch.cat([v[:n0].abs() @ vw[:128].abs().t(), v[n0:n0 + n1].abs() @ vw[128:].abs().t()])
        c = torch.empty((R, 128), device=DEV)
        s2r.s2r_q8_gemm_experts(R, 128, D, e, q, w, 128 * w.ld, 1, s2r.mat(c))
        assert bool(((c[far:far + n0 + n1].cpu().double() - want).abs() <= D * 2.0 ** -23 * mass).all())
        dw = torch.empty((2, 64, D), device=DEV)
        s2r.s2r_q8_wgrad_experts(R, 64, D, e, s2r.mat(rows[:, :64]), q, dw, D, 64 * D)
        dy = rows[far:far + n0 + n1, :64].cpu().double()
        for i, (f, n) in enumerate(((0, n0), (n0, n1))):
            want, mass = dy[f:f + n].t() @ v[f:f + n], dy[f:f + n].abs().t() @ v[f:f + n].abs()
            assert bool(((dw[i].cpu().double() - want).abs() <= (n * 2.0 ** -23) * mass + 2.0 ** -140).all())
