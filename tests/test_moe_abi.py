"""The calls of layers of experts on the CPU: what each refuses, before anything is enqueued, and sizes.
No device is touched."""
import ctypes

import pytest
from test_q8_abi import FAKE, _m, _q, _r, s2r  # noqa: F401


def _e(s2r, first=FAKE, rows=FAKE, experts=4):
    return s2r.s2r_experts(first, rows, experts)


def test_route_refuses(s2r):
    L = s2r.lib()
    call = lambda T=50, K=2, E=8, x=FAKE, f=FAKE, r=FAKE, p=FAKE, ws=None, n=0: L.s2r_moe_route(T, K, E, x, f, r, p, ws, n, None)
    null, dim, align = s2r.S2R_ERR_NULL, s2r.S2R_ERR_DIM, s2r.S2R_ERR_ALIGN
    for bad in ({"x": None}, {"f": None}, {"r": None}, {"p": None}, {"T": 0, "f": None}):
        assert call(**bad) == null
    for bad in ({"K": 0}, {"K": 65}, {"E": 0}, {"E": 1025}, {"T": 1 << 27}, {"T": 1 << 21, "K": 64}, {"T": (1 << 64) - 1}):
        assert call(**bad) == dim
    for bad in ({"x": FAKE + 2}, {"f": FAKE + 1}, {"r": FAKE + 2}, {"p": FAKE + 3}):
        assert call(**bad) == align
    assert call(x=None, K=0) == null and call(K=0, p=FAKE + 2) == dim
    need = s2r.s2r_moe_route_workspace_bytes(100000, 8, 64)
    assert need > 0
    big = lambda ws, n: call(T=100000, K=8, E=64, ws=ws, n=n)
    assert big(None, 0) == s2r.S2R_ERR_WORKSPACE and big(FAKE, need - 1) == s2r.S2R_ERR_WORKSPACE
    assert big(None, need) == s2r.S2R_ERR_WORKSPACE and big(FAKE + 8, need) == align
    assert s2r.s2r_moe_route_workspace_bytes(1, 8, 64) == 0
    for bad in ((1, 0, 1), (1, 1, 0), (1, 65, 1), (1, 1, 1025), (1 << 27, 1, 1)):
        assert s2r.s2r_moe_route_workspace_bytes(*bad) == 0 and s2r.s2r_moe_rows(*bad) == 0


@pytest.mark.parametrize("T,K,E,want", [(0, 1, 5, 0), (1, 1, 1, 4), (1, 8, 64, 32), (3, 1, 2, 8), (100, 2, 3, 208), (5, 1, 1, 8)])
def test_rows(s2r, T, K, E, want):
    assert s2r.s2r_moe_rows(T, K, E) == want


def test_token_calls_refuse(s2r):
    L = s2r.lib()
    T, K, D, R = 50, 2, 200, 120
    null, dim, align = s2r.S2R_ERR_NULL, s2r.S2R_ERR_DIM, s2r.S2R_ERR_ALIGN

    def gather(x=None, p=FAKE, o=None, T=T, K=K, D=D, R=R, q=None):
        return L.s2r_moe_gather(T, K, D, _r(x or _m(s2r)), p, R, _r(o or _m(s2r)), _r(q), None)

    def combine(x=None, p=FAKE, o=None, T=T, K=K, D=D, R=R, w=FAKE):
        return L.s2r_moe_combine(T, K, D, _r(o or _m(s2r)), R, p, w, _r(x or _m(s2r)), None)

    def grad(x=None, p=FAKE, o=None, T=T, K=K, D=D, R=R, w=FAKE, dw=FAKE, q=None):
        return L.s2r_moe_combine_grad(T, K, D, _r(x or _m(s2r)), p, R, w, _r(_m(s2r)), _r(o or _m(s2r)), _r(q), dw, None)

    for f in (gather, combine, grad):
        assert f(p=None) == null
        assert f(x=_m(s2r, data=None)) == null and f(o=_m(s2r, data=None)) == null
        for bad in ({"K": 0}, {"K": 65}, {"T": 1 << 27}, {"R": 1 << 28}, {"D": 1 << 28}, {"D": 257}):
            assert f(**bad) == dim
        assert f(x=_m(s2r, dtype=3)) == dim and f(x=_m(s2r, ld=192)) == dim and f(o=_m(s2r, ld=192)) == dim
        assert f(p=FAKE + 2) == align and f(x=_m(s2r, ld=257)) == align and f(o=_m(s2r, data=FAKE + 8)) == align
    # 8-bit rows are checked as everywhere
    for f in (gather, grad):
        assert f(q=_q(s2r, q=None, lds=120)) == null and f(q=_q(s2r, lds=116)) == dim and f(q=_q(s2r, lds=122)) == align
    m, q = _r(_m(s2r)), _r(_q(s2r, lds=120))
    assert L.s2r_moe_gather(T, K, D, None, FAKE, R, m, None, None) == null
    assert L.s2r_moe_gather(T, K, D, m, FAKE, R, None, None, None) == null
    assert gather(o=_m(s2r, dtype=2)) == dim                       # a copy has its source's type
    assert L.s2r_moe_combine(T, K, D, None, R, FAKE, None, m, None) == null
    assert L.s2r_moe_combine(T, K, D, m, R, FAKE, None, None, None) == null
    assert combine(w=FAKE + 2) == align and grad(w=FAKE + 2) == align and grad(dw=FAKE + 2) == align
    assert L.s2r_moe_combine_grad(T, K, D, m, FAKE, R, None, m, None, None, None, None) == null   # no output
    assert L.s2r_moe_combine_grad(T, K, D, m, FAKE, R, None, None, m, None, FAKE, None) == null   # dweight without rows
    assert L.s2r_moe_combine_grad(T, K, D, m, FAKE, R, None, _r(_m(s2r, dtype=2)), None, q, FAKE, None) == dim
    assert L.s2r_moe_combine_grad(T, K, 0, m, None, R, None, m, None, None, FAKE, None) == null   # empty sums are written


def test_token_calls_with_nothing_to_do(s2r):
    L, ok = s2r.lib(), s2r.S2R_OK
    m = _r(_m(s2r, data=None))
    for T, D, R in [(0, 200, 120), (50, 0, 120), (0, 0, 0)]:
        p = FAKE if T and D else None
        assert L.s2r_moe_gather(T, 2, D, m, p, R, m, None, None) == (ok if T == 0 and R == 0 or D == 0 else s2r.S2R_ERR_NULL)
        assert L.s2r_moe_combine(T, 2, D, m, 0, p, None, m, None) == ok
        assert L.s2r_moe_combine_grad(T, 2, D, m, p, 0, None, None, m, None, None, None) == ok
    assert L.s2r_moe_gather(50, 2, 200, _r(_m(s2r)), FAKE, 0, m, None, None) == ok


def _gemm(s2r, e=None, a=None, b=None, c=None, M=50, N=40, K=200, step=0, sstep=0):
    return s2r.lib().s2r_q8_gemm_experts(M, N, K, _r(e or _e(s2r)), _r(a or _q(s2r)), _r(b or _q(s2r)), step, sstep,
                                         _r(c or _m(s2r)), None)


def _wgrad(s2r, e=None, y=None, x=None, M=50, N=40, K=200, dw=FAKE, ld=200, step=8000, acc=0, y8=None):
    y16 = None if y8 else _r(y or _m(s2r))
    return s2r.lib().s2r_q8_wgrad_experts(M, N, K, _r(e or _e(s2r)), y16, _r(y8), _r(x or _q(s2r)), dw, ld, step, acc, None)


def test_experts_products_refuse(s2r):
    null, dim, align = s2r.S2R_ERR_NULL, s2r.S2R_ERR_DIM, s2r.S2R_ERR_ALIGN
    for f in (_gemm, _wgrad):
        for bad, want in [({"first": None}, null), ({"rows": None}, null), ({"experts": 0}, dim), ({"experts": 1025}, dim),
                          ({"first": FAKE + 2}, align), ({"rows": FAKE + 1}, align)]:
            assert f(s2r, e=_e(s2r, **bad)) == want
        assert f(s2r, M=1 << 28) == dim and f(s2r, N=1 << 28) == dim and f(s2r, K=1 << 28) == dim
    assert _gemm(s2r, a=_q(s2r, q=None)) == null and _gemm(s2r, a=_q(s2r, lds=48)) == dim
    assert _gemm(s2r, b=_q(s2r, scale=None)) == null and _gemm(s2r, b=_q(s2r, ld=192)) == dim
    assert _gemm(s2r, c=_m(s2r, ld=32)) == dim and _gemm(s2r, c=_m(s2r, data=FAKE + 8)) == align
    assert _gemm(s2r, step=8) == align
    assert _wgrad(s2r, dw=None) == null and _wgrad(s2r, x=_q(s2r, q=None)) == null
    assert _wgrad(s2r, y=_m(s2r, dtype=1)) == dim and _wgrad(s2r, y=_m(s2r, dtype=2)) == dim
    assert _wgrad(s2r, ld=199) == dim and _wgrad(s2r, step=7999) == dim and _wgrad(s2r, x=_q(s2r, lds=48)) == dim
    assert _wgrad(s2r, y8=_q(s2r, lds=48)) == dim and _wgrad(s2r, dw=FAKE + 2) == align
    L, e, m, q = s2r.lib(), _r(_e(s2r)), _r(_m(s2r)), _r(_q(s2r))
    for bad in ((None, q, q, m), (e, None, q, m), (e, q, None, m), (e, q, q, None)):
        assert L.s2r_q8_gemm_experts(50, 40, 200, bad[0], bad[1], bad[2], 0, 0, bad[3], None) == null
    assert L.s2r_q8_wgrad_experts(50, 40, 200, None, m, None, q, FAKE, 200, 8000, 0, None) == null
    assert L.s2r_q8_wgrad_experts(50, 40, 200, e, None, None, q, FAKE, 200, 8000, 0, None) == null
    assert L.s2r_q8_wgrad_experts(50, 40, 200, e, m, None, None, FAKE, 200, 8000, 0, None) == null
    assert L.s2r_q8_wgrad_experts(50, 40, 200, e, m, q, q, FAKE, 200, 8000, 0, None) == dim


def test_experts_products_with_nothing_to_do(s2r):
    ok, none, no = s2r.S2R_OK, _m(s2r, data=None), _q(s2r, q=None, scale=None)
    assert _gemm(s2r, M=0, a=no, c=none) == ok and _gemm(s2r, N=0, b=no, c=none) == ok
    assert _wgrad(s2r, N=0, y=none, dw=None) == ok and _wgrad(s2r, K=0, x=no, dw=None) == ok
    assert _wgrad(s2r, M=0, y=none, x=no, acc=1) == ok


def test_python_checks_its_tensors(s2r):
    import torch
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    e = s2r.experts(i(5), i(5))
    assert e.experts == 5 and e.first == e.tensors[0].data_ptr()
    calls = [lambda: s2r.experts(i(4), i(5)), lambda: s2r.experts(i(5).long(), i(5)), lambda: s2r.experts(i(10)[::2], i(5))]
    for bad in ({"expert": i(3, 3)}, {"expert": i(3, 2).long()}, {"first": i(4)}, {"rows": i(6)}, {"place": i(2, 3)},
                {"place": i(3, 4)[:, :2]}):
        a = {"expert": i(3, 2), "first": i(5), "rows": i(5), "place": i(3, 2), **bad}
        calls.append(lambda a=a: s2r.s2r_moe_route(3, 2, 5, **a, stream=0))
    m = s2r.mat(torch.zeros(3, 8))
    calls += [lambda: s2r.s2r_moe_gather(3, 2, 8, m, i(6), 8, m, stream=0),
              lambda: s2r.s2r_moe_combine(3, 2, 8, m, 3, i(3, 2), torch.zeros(3, 2).double(), m, stream=0),
              lambda: s2r.s2r_moe_combine_grad(3, 2, 8, m, i(3, 2), 3, rows=m, dweight=torch.zeros(6), stream=0)]
    for call in calls:
        with pytest.raises(s2r.S2RError) as err:
            call()
        assert err.value.status == s2r.S2R_ERR_DIM
