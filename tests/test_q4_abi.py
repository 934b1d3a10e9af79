"""The 4-bit calls on the CPU: what each refuses, before anything is enqueued, and the reference's own
rounding.  No device is touched."""
import pytest
import torch

import q4_reference as ref4
from test_q8_abi import FAKE, _m, _r, s2r  # noqa: F401


def _q4(s2r, q=FAKE, ld=128, scale=FAKE, lds=16):
    return s2r.s2r_q4_mat(q, ld, scale, lds)


def _calls(s2r):
    L = s2r.lib()

    def save(x=None, o=None, R=50, C=200):
        return L.s2r_q4_save(R, C, _r(x or _m(s2r)), _r(o or _q4(s2r)), None, None)

    def save_t(x=None, o=None, R=50, C=200):
        # the transpose of [C][R]: o has R rows of C
        return L.s2r_q4_save(C, R, _r(x or _m(s2r)), None, _r(o or _q4(s2r)), None)

    def load(x=None, o=None, R=50, C=200):
        return L.s2r_q4_load(R, C, _r(o or _q4(s2r)), _r(x or _m(s2r)), None)

    def gemm_a(x=None, o=None, R=50, C=200):
        return L.s2r_q4_gemm(R, 40, C, _r(o or _q4(s2r)), _r(_q4(s2r)), _r(x or _m(s2r)), None, 0, None)

    def gemm_b(x=None, o=None, R=50, C=200):
        return L.s2r_q4_gemm(40, R, C, _r(_q4(s2r)), _r(o or _q4(s2r)), _r(x or _m(s2r)), None, 0, None)

    return [save, save_t, load, gemm_a, gemm_b]


@pytest.mark.parametrize("which", range(5), ids=["save", "save_t", "load", "gemm_a", "gemm_b"])
def test_refusals(s2r, which):
    f = _calls(s2r)[which]
    null, dim, align = s2r.S2R_ERR_NULL, s2r.S2R_ERR_DIM, s2r.S2R_ERR_ALIGN
    assert f(o=_q4(s2r, q=None)) == null and f(o=_q4(s2r, scale=None)) == null and f(x=_m(s2r, data=None)) == null
    assert f(o=_q4(s2r, ld=96)) == dim                    # 200 columns take 100 bytes
    assert f(o=_q4(s2r, ld=(1 << 22) + 16)) == dim
    assert f(o=_q4(s2r, lds=0)) == dim and f(o=_q4(s2r, lds=(1 << 22) + 8)) == dim
    assert f(o=_q4(s2r, lds=6)) == dim                    # and 7 scales
    assert f(x=_m(s2r, dtype=3)) == dim and f(x=_m(s2r, ld=32)) == dim
    assert f(R=1 << 28) == dim
    assert f(o=_q4(s2r, q=FAKE + 8)) == align and f(o=_q4(s2r, ld=104)) == align
    assert f(o=_q4(s2r, scale=FAKE + 4)) == align and f(o=_q4(s2r, lds=12)) == align
    assert f(x=_m(s2r, data=FAKE + 8)) == align and f(x=_m(s2r, ld=257)) == align
    assert f(o=_q4(s2r, q=None, ld=96)) == null and f(o=_q4(s2r, ld=96, lds=12)) == dim


def test_missing_arguments(s2r):
    L, N = s2r.lib(), s2r.S2R_ERR_NULL
    m, q = _r(_m(s2r)), _r(_q4(s2r))
    assert L.s2r_q4_save(1, 1, None, q, q, None) == N and L.s2r_q4_save(1, 1, m, None, None, None) == N
    assert L.s2r_q4_load(1, 1, None, m, None) == N and L.s2r_q4_load(1, 1, q, None, None) == N
    for a, b, c in ((None, q, m), (q, None, m), (q, q, None)):
        assert L.s2r_q4_gemm(1, 1, 1, a, b, c, None, 0, None) == N


def test_nothing_to_do(s2r):
    L, ok = s2r.lib(), s2r.S2R_OK
    m, q = _r(_m(s2r, data=None)), _r(_q4(s2r, q=None, scale=None))
    for R, C in [(0, 200), (50, 0), (0, 0)]:
        assert L.s2r_q4_save(R, C, m, q, None, None) == ok
        assert L.s2r_q4_load(R, C, q, m, None) == ok
    assert L.s2r_q4_gemm(0, 200, 200, q, _r(_q4(s2r)), m, None, 0, None) == ok
    assert L.s2r_q4_gemm(50, 0, 200, _r(_q4(s2r)), q, m, None, 0, None) == ok


@pytest.mark.parametrize("M,N,K", [(129, 127, 8200), (300, 1000, 4096), (64, 8192, 4100)])
def test_workspace(s2r, M, N, K):
    L = s2r.lib()
    need = s2r.s2r_q4_gemm_workspace_bytes(M, N, K)
    assert s2r.s2r_q4_gemm_workspace_bytes(1 << 28, 1, 1) == 0
    a, c = _q4(s2r, ld=4112, lds=264), _m(s2r, ld=8192)
    if need:
        assert L.s2r_q4_gemm(M, N, K, _r(a), _r(a), _r(c), FAKE, need - 1, None) == s2r.S2R_ERR_WORKSPACE
        assert L.s2r_q4_gemm(M, N, K, _r(a), _r(a), _r(c), FAKE + 8, need, None) == s2r.S2R_ERR_ALIGN


def test_python_descriptors(s2r):
    q = s2r.alloc_q4(130, 201, device="cpu")
    assert q.codes.shape == (130, 112) and q.scales.shape == (130, 8) and (q.ld, q.lds) == (112, 8)
    assert s2r.alloc_q4(1, 257, device="cpu").scales.shape == (1, 16)
    for bad in [lambda: s2r.q4_mat(q.codes.short(), q.scales), lambda: s2r.q4_mat(q.codes.t(), q.scales),
                lambda: s2r.q4_mat(q.codes, q.scales[0])]:
        with pytest.raises(s2r.S2RError) as e:
            bad()
        assert e.value.status == s2r.S2R_ERR_DIM


def test_reference_rounds_to_even_codes():
    x = torch.zeros((2, 32), dtype=torch.float64)
    x[0, :9] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 6])
    x[1, :4] = torch.tensor([6.001, -0.6, 3, 2.0 ** -200])
    code, b = ref4.quantise(x)
    assert b[:, 0].tolist() == [127, 128]
    assert ref4.values(code, b)[0, :9].tolist() == [0, 1, 1, 2, 2, 4, 4, -4, 6]
    assert ref4.values(code, b)[1, :4].tolist() == [6, -1, 3, 0]
