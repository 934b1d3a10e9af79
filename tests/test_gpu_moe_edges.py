"""Layers of experts at their edges: sorted matrices without a row to spare, experts' rows anywhere, values that are not
finite, 8-bit rows against s2r_q8_save, and a workspace that two graphs share."""
import math

import pytest
import torch

import count_sketch_aggregation_amd as s2r
import q8_reference as ref
import test_gpu_moe as moe
import test_gpu_q8 as q8

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")
DEV = "cuda"
up = ref.up


@pytest.mark.parametrize("T,K,E", moe.ROUTES[1:])
def test_every_place_is_below_the_promised_rows(T, K, E):
    gp.say(f"rows of {T}x{K} of {E}")
    _, _, place = moe.route(moe.choices(T, K, E, T + K, drop=0), E)
    assert 0 <= int(place.min()) and int(place.max()) < s2r.s2r_moe_rows(T, K, E)


@pytest.mark.parametrize("E", [1, 5, 64, 300])
@pytest.mark.parametrize("each", [1, 5, 65])
def test_no_row_to_spare(E, each):
    """4 n + 1 rows for every expert need as many rows as any choices may: all calls on exactly so many."""
    gp.say(f"no row to spare, {E} experts of {each}")
    T, D, N = E * each, 136, 72
    m = moe.Routed(T, 1, E, expert=(torch.arange(T) % E).int()[:, None])
    R = m.R = s2r.s2r_moe_rows(T, 1, E)
    assert R == E * (each + 3) and int(m.place.max()) == R - 4
    m.used = m.used[:R]
    x, vx = q8.integers(T, D, "e4m3", 1)
    rows = torch.full((R + 4, up(D, 16)), 7.0, dtype=torch.bfloat16, device=DEV)
    q = s2r.alloc_q8(R, D)
    s2r.s2r_moe_gather(T, 1, D, s2r.mat(q8.wide(T, D, "bf16", x=vx)), m.place, R, s2r.mat(rows), q)
    sorted_x = m.sorted_of(vx, 0.0)
    assert torch.equal(rows[:R, :D].cpu()[m.used].double(), sorted_x[m.used]) and bool((rows[R:] == 7).all())
    b, vb, steps = moe.expert_weights(E, N, D, "e4m3", 2)
    c = moe.product(m, N, D, q, b, steps, "f32")
    want = torch.full((R, N), 7.0)
    for e in range(E):
        want[m.span(e)] = sorted_x[m.span(e)].float() @ vb[e].float().t()
    assert torch.equal(c, want)
    dy, vy = q8.integers(R, N, "e4m3", 3)
    got = moe.wgrad(m, N, D, dy, q)
    assert torch.equal(got, torch.stack([vy[m.span(e)].float().t() @ sorted_x[m.span(e)].float() for e in range(E)]))
    y = q8.wide(T, N, "f32", fill=7.0)
    s2r.s2r_moe_combine(T, 1, N, s2r.mat(q8.wide(R, N, "f32", x=c)), R, m.place, None, s2r.mat(y))
    assert torch.equal(y[:, :N].cpu(), want[m.at]) and q8.pad_kept(y, N, 7.0)


@pytest.mark.parametrize("counts,N,D", [([3, 0, 17, 1, 64, 33], 200, 300), ([700, 0, 3, 1300, 257], 391, 200), ([2900, 1, 0, 3100], 1100, 260)])
def test_experts_rows_anywhere(counts, N, D):
    """Rows of experts in another order than theirs, from any multiple of 4 on, with rows of nobody around them."""
    gp.say(f"experts anywhere {counts}")
    E = len(counts)
    first, at = [0] * E, 8
    for e in reversed(range(E)):
        first[e] = at
        at = up(at + counts[e], 4) + 4 * (e % 3)
    m = moe.Routed.__new__(moe.Routed)
    m.E, m.R, m.h = E, at + 6, (first, counts)
    m.used = torch.zeros(m.R, dtype=torch.bool)
    for e in range(E):
        m.used[m.span(e)] = True
    m.e = s2r.experts(*(torch.tensor(v, dtype=torch.int32, device=DEV) for v in (first, counts)))
    a, va = q8.integers(m.R, D, "e4m3", 1)
    a.codes[~m.used.to(DEV), :D] = 0x7F
    b, vb, steps = moe.expert_weights(E, N, D, "e4m3", 2)
    want = torch.full((m.R, N), 7.0)
    for e in range(E):
        want[m.span(e)] = va[m.span(e)].float() @ vb[e].float().t()
    assert torch.equal(moe.product(m, N, D, a, b, steps, "f32"), want)
    dy, vy = q8.integers(m.R, N, "e5m2", 3)
    dy.codes[~m.used.to(DEV), :N] = 0x7F
    want = torch.stack([vy[m.span(e)].float().t() @ va[m.span(e)].float() for e in range(E)])
    assert torch.equal(moe.wgrad(m, N, D, dy, a), want)


def bytes_of(q, m, D):
    """Codes and scales of the rows that some choice has, NaN codes as one."""
    codes, scales = q.codes[:, :D].cpu()[m.used], q.scales[:, :m.R].cpu().t()[m.used]
    nan = codes & 0x7F > 0x7C if q.format == s2r.S2R_E5M2 else codes & 0x7F == 0x7F
    return torch.where(nan, 0x7F, codes), scales


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,K,E,D", [(33, 3, 7, 300), (9, 1, 2, 1100)])
def test_eight_bit_rows_are_those_of_the_save(T, K, E, D, dtype, fmt):
    """Of awkward, infinite and NaN values, with weights of 0, of infinity and NaN among them."""
    gp.say(f"8-bit rows {T}x{K}, {D} {dtype} {fmt}")
    m = moe.Routed(T, K, E, 3)
    x = q8.awkward(T, D, dtype, 5)
    x[0, 3], x[5, 130], x[6, D - 1], x[7, 0] = math.inf, -math.inf, math.nan, torch.finfo(x.dtype).max
    x[8] = math.nan
    w = torch.randn((T, K), generator=q8._gen(6))
    w[1, 0], w[2, 0], w[4, 0], w[7, 0] = 0, math.inf, math.nan, 3
    src = s2r.mat(q8.wide(T, D, dtype, x=x))

    def saved(values, t):
        q = q8.space(m.R, D, fmt)
        s2r.s2r_q8_save(m.R, D, s2r.mat(q8.wide(m.R, D, t, x=m.sorted_of(values, 0.0))), q)
        return bytes_of(q, m, D)

    got = q8.space(m.R, D, fmt)
    s2r.s2r_moe_gather(T, K, D, src, m.place, m.R, outq=got)
    for a, b in zip(bytes_of(got, m, D), saved(x[m.token], dtype)):
        assert torch.equal(a, b)
    got = q8.space(m.R, D, fmt)
    s2r.s2r_moe_combine_grad(T, K, D, src, m.place, m.R, weight=w.to(DEV), drowsq=got)
    for a, b in zip(bytes_of(got, m, D), saved(x.float()[m.token] * w.reshape(-1, 1), "f32")):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,N", [(40, 130), (1500, 520)])
def test_non_finite_rows_stay_in_theirs(T, N):
    """A NaN of one row is in that row's results, in its token's sum and in its expert's gradient, and nowhere else."""
    gp.say(f"non-finite rows {T}x{N}")
    E, K, D = 5, 2, 200
    m = moe.Routed(T, K, E, 8, drop=0.05)
    a, va = q8.integers(m.R, D, "e4m3", 1)
    b, vb, steps = moe.expert_weights(E, N, D, "e4m3", 2)
    spans = [m.span(e) for e in range(E) if m.h[1][e] > 0]
    bad = spans[1].stop - 1
    a.codes[bad, 5] = 0x7F
    want = torch.full((m.R, N), 7.0)
    for e in range(E):
        want[m.span(e)] = va[m.span(e)].float() @ vb[e].float().t()
    want[bad] = math.nan
    c = moe.product(m, N, D, a, b, steps, "f32")
    assert torch.equal(c.isnan(), want.isnan()) and torch.equal(c.nan_to_num(9), want.nan_to_num(9))
    y = q8.wide(T, N, "f32", fill=7.0)
    s2r.s2r_moe_combine(T, K, N, s2r.mat(q8.wide(m.R, N, "f32", x=c)), m.R, m.place, None, s2r.mat(y))
    token = int(m.token[m.at == bad])
    nan = y[:, :N].cpu().isnan()
    assert bool(nan[token].all()) and int(nan.any(1).sum()) == 1
    dy, vy = q8.integers(m.R, N, "e4m3", 3)
    got = moe.wgrad(m, N, D, dy, a)
    for e in range(E):
        want = vy[m.span(e)].float().t() @ va[m.span(e)].float()
        if m.span(e).start <= bad < m.span(e).stop:
            want[:, 5] = math.nan
        assert torch.equal(got[e].isnan(), want.isnan()) and torch.equal(got[e].nan_to_num(9), want.nan_to_num(9))


def test_combine_of_values_that_are_not_finite():
    """Infinities and NaN as fp32 has them, 0 times infinity too, and results beyond fp16."""
    gp.say("combine, not finite")
    T, K, D = 6, 2, 40
    place = torch.arange(T * K, dtype=torch.int32, device=DEV).view(T, K)
    rows = torch.ones((T * K, D))
    rows[0], rows[1], rows[2], rows[4], rows[5], rows[7], rows[8] = math.inf, 1, math.nan, math.inf, -math.inf, math.inf, 60000
    w = torch.ones((T, K))
    w[3, 1], w[4, 0] = 0, 2  # 0 * inf; 2 * 60000
    want = torch.tensor([math.inf, math.nan, math.nan, math.nan, math.inf, 2.0])[:, None].expand(T, D)
    y = q8.wide(T, D, "f16", fill=7.0)
    s2r.s2r_moe_combine(T, K, D, s2r.mat(q8.wide(T * K, D, "f32", x=rows)), T * K, place, w.to(DEV), s2r.mat(y))
    got = y[:, :D].cpu().float()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(9, 8, -8), want.nan_to_num(9, 8, -8))
    # the same rows without a place: nothing of them, and no weight
    place.fill_(-1)
    s2r.s2r_moe_combine(T, K, D, s2r.mat(q8.wide(T * K, D, "f32", x=rows)), T * K, place, torch.full((T, K), math.nan, device=DEV), s2r.mat(y))
    assert bool((y[:, :D] == 0).all())


def test_two_graphs_share_the_sorts_workspace():
    """One after the other on a stream, in any order, each with inputs that change between replays."""
    gp.say("graphs with one workspace")
    sizes = [(5000, 4, 60), (3001, 8, 200)]
    ws = q8.workspace(max(s2r.s2r_moe_route_workspace_bytes(*s) for s in sizes))
    graphs, state = [], []
    for T, K, E in sizes:
        st = [torch.zeros((T, K), dtype=torch.int32, device=DEV)] + [torch.zeros(E, dtype=torch.int32, device=DEV) for _ in range(2)]
        st.append(torch.zeros((T, K), dtype=torch.int32, device=DEV))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s2r.s2r_moe_route(T, K, E, *st, workspace=ws)
        graphs.append(g)
        state.append(st)
    for rep, order in enumerate([(0, 1), (1, 0), (0, 0), (1, 1)]):
        ws.fill_(rep)
        chosen = {i: moe.choices(*sizes[i], rep + i) for i in order}
        for i, c in chosen.items():
            state[i][0].copy_(c)
        torch.cuda.synchronize()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i, c in chosen.items():
            for got, want in zip(state[i][1:], moe.routed(c, sizes[i][2])):
                assert torch.equal(got.cpu().view(-1), want), (rep, i)
