"""The 8-bit training calls on the CPU: what each refuses, before anything is enqueued.  No
device is touched: every call here returns an error, or has nothing to do."""
import ctypes
import os

import pytest

FAKE = 1 << 20  # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def s2r():
    import count_sketch_aggregation_amd as m
    if not os.path.exists(m.LIB_PATH):
        from count_sketch_aggregation_amd import _build
        _build.build()
    return m


def _m(s2r, data=FAKE, ld=256, dtype=0):
    return s2r.s2r_mat(data, ld, dtype)


def _q(s2r, q=FAKE, ld=256, scale=FAKE, lds=64, format=0):
    return s2r.s2r_q8_mat(q, ld, scale, lds, format)


def _r(x):
    return None if x is None else ctypes.byref(x)


def _calls(s2r, M=50, K=200):
    """Every call with an 8-bit matrix `q` and a matrix `m` in each of its places."""
    L = s2r.lib()
    N = 40
    qt = lambda: _q(s2r, ld=256)
    mt = lambda: _m(s2r, ld=256)

    def save(x=None, o=None, M=M, K=K):
        return L.s2r_q8_save(M, K, _r(x or mt()), _r(o or qt()), None)

    def load(x=None, o=None, M=M, K=K):
        return L.s2r_q8_load(M, K, _r(o or qt()), _r(x or mt()), None)

    def weight(x=None, o=None, M=M, K=K):
        return L.s2r_q8_weight(M, K, _r(x or mt()), _r(o or qt()), None, None)

    def gemm_a(x=None, o=None, M=M, K=K):
        return L.s2r_q8_gemm(M, N, K, _r(o or qt()), _r(qt()), _r(x or mt()), None, 0, None)

    def gemm_b(x=None, o=None, M=M, K=K):
        return L.s2r_q8_gemm(N, M, K, _r(qt()), _r(o or qt()), _r(x or mt()), None, 0, None)

    def wgrad_x(x=None, o=None, M=M, K=K):
        return L.s2r_q8_wgrad(M, K, K, _r(x or mt()), None, _r(o or qt()), FAKE, 1000, 0, None, 0,
                              None)

    def glu(x=None, o=None, M=M, K=K):
        return L.s2r_q8_glu(M, K, 0, _r(x or mt()), None, _r(o or qt()), None, None, None, None)

    def glu_grad(x=None, o=None, M=M, K=K):
        return L.s2r_q8_glu_grad(M, K, 0, _r(qt()), None, _r(x or mt()), None, None, _r(o or qt()),
                                 None, None)

    return [save, load, weight, gemm_a, gemm_b, wgrad_x, glu, glu_grad]


NAMES = ["save", "load", "weight", "gemm_a", "gemm_b", "wgrad", "glu", "glu_grad"]


@pytest.mark.parametrize("which", range(len(NAMES)), ids=NAMES)
def test_refusals_of_matrices(s2r, which):
    f = _calls(s2r)[which]
    null, dim, align = s2r.S2R_ERR_NULL, s2r.S2R_ERR_DIM, s2r.S2R_ERR_ALIGN
    assert f(o=_q(s2r, q=None)) == null
    assert f(o=_q(s2r, scale=None)) == null
    assert f(x=_m(s2r, data=None)) == null
    assert f(o=_q(s2r, ld=192)) == dim                      # shorter than a row
    assert f(o=_q(s2r, ld=(1 << 22) + 16)) == dim           # longer than a row may be
    assert f(o=_q(s2r, format=2)) == dim
    assert f(x=_m(s2r, dtype=3)) == dim
    assert f(x=_m(s2r, ld=32)) == dim
    assert f(o=_q(s2r, q=FAKE + 8)) == align
    assert f(o=_q(s2r, ld=264)) == align                    # rows would not stay aligned
    assert f(o=_q(s2r, scale=FAKE + 2)) == align
    assert f(o=_q(s2r, lds=66)) == align
    assert f(x=_m(s2r, data=FAKE + 8)) == align
    assert f(x=_m(s2r, ld=257)) == align
    assert f(M=1 << 28, o=_q(s2r, lds=1 << 28)) == dim
    # a NULL is named before a size, a size before an alignment
    assert f(o=_q(s2r, q=None, ld=192)) == null
    assert f(o=_q(s2r, ld=192, lds=66)) == dim


@pytest.mark.parametrize("which", [0, 1, 3, 5, 6, 7], ids=lambda i: NAMES[i])
def test_refuses_short_scale_rows(s2r, which):
    f = _calls(s2r)[which]
    assert f(o=_q(s2r, lds=48)) == s2r.S2R_ERR_DIM           # 50 rows


def test_square_blocks_need_few_scales(s2r):
    L = s2r.lib()
    w, q = _m(s2r, ld=256), _q(s2r, lds=0)
    assert L.s2r_q8_weight(50, 200, _r(w), _r(q), None, None) == s2r.S2R_ERR_DIM
    # the transposed copy: its own rows and scales are checked, and one format
    good, t = _q(s2r, lds=4), lambda **k: _q(s2r, **{"ld": 64, "lds": 4, **k})
    bad = [(t(q=None), s2r.S2R_ERR_NULL), (t(ld=32), s2r.S2R_ERR_DIM),
           (t(lds=0), s2r.S2R_ERR_DIM), (t(format=1), s2r.S2R_ERR_DIM),
           (t(ld=72), s2r.S2R_ERR_ALIGN)]
    for m, want in bad:
        assert L.s2r_q8_weight(50, 200, _r(w), _r(good), _r(m), None) == want


def test_missing_arguments(s2r):
    L, N = s2r.lib(), s2r.S2R_ERR_NULL
    m, q = _m(s2r), _q(s2r)
    assert L.s2r_q8_save(1, 1, None, _r(q), None) == N
    assert L.s2r_q8_save(1, 1, _r(m), None, None) == N
    assert L.s2r_q8_load(1, 1, None, _r(m), None) == N
    assert L.s2r_q8_weight(1, 1, _r(m), None, None, None) == N
    assert L.s2r_q8_gemm(1, 1, 1, _r(q), None, _r(m), None, 0, None) == N
    assert L.s2r_q8_wgrad(1, 1, 1, None, None, _r(q), FAKE, 1, 0, None, 0, None) == N
    assert L.s2r_q8_wgrad(1, 1, 1, _r(m), None, _r(q), None, 1, 0, None, 0, None) == N
    assert L.s2r_q8_glu(1, 1, 0, _r(m), None, None, None, None, None, None) == N   # no output
    assert L.s2r_q8_glu(1, 1, 0, _r(m), None, None, _r(q), None, None, None) == N  # uq without u
    assert L.s2r_q8_glu_grad(1, 1, 0, _r(q), None, _r(m), None, None, None, None, None) == N
    assert L.s2r_q8_glu_grad(1, 1, 0, _r(q), None, _r(m), None, _r(m), None, None, None) == N
    assert L.s2r_q8_glu_grad(1, 1, 0, _r(q), None, _r(m), None, None, None, _r(q), None) == N


def test_types_that_do_not_go_together(s2r):
    L, D = s2r.lib(), s2r.S2R_ERR_DIM
    m, q = _m(s2r), _q(s2r)
    for dt in (s2r.S2R_F16, s2r.S2R_F32):  # a 16-bit gradient is bf16
        assert L.s2r_q8_wgrad(1, 1, 1, _r(_m(s2r, dtype=dt)), None, _r(q), FAKE, 1, 0, None, 0, None) == D
    assert L.s2r_q8_wgrad(1, 1, 1, _r(m), _r(q), _r(q), FAKE, 1, 0, None, 0, None) == D
    assert L.s2r_q8_wgrad(1, 1, 8, _r(m), None, _r(q), FAKE, 7, 0, None, 0, None) == D
    assert L.s2r_q8_wgrad(1, 1, 1, _r(m), None, _r(q), FAKE + 2, 1, 0, None, 0, None) == s2r.S2R_ERR_ALIGN
    assert L.s2r_q8_glu(1, 1, 0, _r(m), _r(_m(s2r, dtype=2)), _r(q), None, None, None, None) == D
    assert L.s2r_q8_glu(1, 1, 3, _r(m), None, _r(q), None, None, None, None) == D
    assert L.s2r_q8_glu_grad(1, 1, -1, _r(q), None, _r(m), _r(m), None, None, None, None) == D
    assert L.s2r_q8_glu_grad(1, 1, 0, _r(q), _r(_q(s2r, format=1)), _r(m), _r(m), None, None, None, None) == D


def test_workspaces(s2r):
    L = s2r.lib()
    a, b, c = _q(s2r, ld=8192, lds=64), _q(s2r, ld=8192, lds=64), _m(s2r, ld=1024)
    for need, call in [
        (s2r.s2r_q8_gemm_workspace_bytes(64, 1024, 8192),
         lambda ws, n: L.s2r_q8_gemm(64, 1024, 8192, _r(a), _r(b), _r(c), ws, n, None)),
        (s2r.s2r_q8_wgrad_workspace_bytes(8192, 1024, 256),
         lambda ws, n: L.s2r_q8_wgrad(8192, 1024, 256, _r(_m(s2r, ld=1024)), None,
                                      _r(_q(s2r, lds=8192)), FAKE, 256, 0, ws, n, None)),
    ]:
        if need:
            assert call(FAKE, need - 1) == s2r.S2R_ERR_WORKSPACE
            assert call(FAKE + 8, need) == s2r.S2R_ERR_ALIGN
    assert s2r.s2r_q8_gemm_workspace_bytes(1 << 28, 1, 1) == 0
    assert s2r.s2r_q8_wgrad_workspace_bytes(1, 1 << 28, 1) == 0


def test_nothing_to_do(s2r):
    """Empty sizes return before a launch, with no buffers at all."""
    L = s2r.lib()
    m, q = _m(s2r, data=None), _q(s2r, q=None, scale=None)
    for M, K in [(0, 200), (50, 0), (0, 0)]:
        assert L.s2r_q8_save(M, K, _r(m), _r(q), None) == s2r.S2R_OK
        assert L.s2r_q8_load(M, K, _r(q), _r(m), None) == s2r.S2R_OK
        assert L.s2r_q8_weight(M, K, _r(m), _r(q), None, None) == s2r.S2R_OK
        assert L.s2r_q8_glu(M, K, 0, _r(m), None, _r(q), None, None, None, None) == s2r.S2R_OK
        assert L.s2r_q8_glu_grad(M, K, 0, _r(q), None, _r(m), _r(m), None, None, None, None) == s2r.S2R_OK
    assert L.s2r_q8_gemm(0, 200, 200, _r(q), _r(_q(s2r)), _r(m), None, 0, None) == s2r.S2R_OK
    assert L.s2r_q8_wgrad(0, 200, 200, _r(m), None, _r(q), FAKE, 200, 1, None, 0, None) == s2r.S2R_OK


def test_python_descriptors(s2r):
    """Descriptors come from 2-D tensors with unit stride along the rows, and keep them."""
    import torch
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    m = s2r.mat(x[:, :20])
    assert (m.data, m.ld, m.dtype) == (x.data_ptr(), 32, s2r.S2R_BF16) and m.tensor.shape == (4, 20)
    assert s2r.mat(torch.zeros(1, 5)).ld == 5
    for bad in (x.t(), x[0], x.double(), x.view(torch.int16)):
        with pytest.raises(s2r.S2RError) as e:
            s2r.mat(bad)
        assert e.value.status == s2r.S2R_ERR_DIM
    q = s2r.alloc_q8(130, 200, "e5m2", device="cpu")
    assert q.codes.shape == (130, 208) and q.scales.shape == (2, 132) and q.format == s2r.S2R_E5M2
    w = s2r.alloc_q8(130, 200, square=True, device="cpu")
    assert w.scales.shape == (2, 4) and w.lds == 4
    for bad in [lambda: s2r.q8_mat(x, w.scales), lambda: s2r.q8_mat(w.codes, w.scales, "e3m4"),
                lambda: s2r.q8_mat(w.codes.t(), w.scales)]:
        with pytest.raises(s2r.S2RError):
            bad()
    with pytest.raises(s2r.S2RError) as e:
        s2r.s2r_q8_glu(1, 1, "tanh", m, gq=q, stream=0)
    assert e.value.status == s2r.S2R_ERR_DIM


def test_fast_product_refuses_what_the_product_refuses(s2r):
    L = s2r.lib()
    a, b, c = _q(s2r), _q(s2r), _m(s2r)
    bad = [((None, b, c), s2r.S2R_ERR_NULL), ((a, b, None), s2r.S2R_ERR_NULL),
           ((_q(s2r, q=None), b, c), s2r.S2R_ERR_NULL), ((a, _q(s2r, ld=192), c), s2r.S2R_ERR_DIM),
           ((_q(s2r, lds=48), b, c), s2r.S2R_ERR_DIM), ((a, b, _m(s2r, dtype=3)), s2r.S2R_ERR_DIM),
           ((a, b, _m(s2r, data=FAKE + 8)), s2r.S2R_ERR_ALIGN)]
    for call in (L.s2r_q8_gemm, L.s2r_q8_gemm_fast):
        for (x, y, z), want in bad:
            assert call(50, 200, 200, _r(x), _r(y), _r(z), None, 0, None) == want
        assert call(0, 200, 200, _r(a), _r(b), _r(c), None, 0, None) == s2r.S2R_OK


@pytest.mark.parametrize("M,N,K", [(129, 127, 4100), (64, 8192, 4100)])
def test_a_products_workspace_is_checked(s2r, M, N, K):
    """Sizes whose sum is cut: too small and misaligned workspaces are refused, by both products."""
    L = s2r.lib()
    need = s2r.s2r_q8_gemm_workspace_bytes(M, N, K)
    assert need > 0 and need % (4 * M) == 0
    a, b, c = _q(s2r, ld=4112, lds=256), _q(s2r, ld=4112, lds=64), _m(s2r, ld=8192)
    for call in (L.s2r_q8_gemm, L.s2r_q8_gemm_fast):
        assert call(M, N, K, _r(a), _r(b), _r(c), FAKE, need - 1, None) == s2r.S2R_ERR_WORKSPACE
        assert call(M, N, K, _r(a), _r(b), _r(c), FAKE, 1, None) == s2r.S2R_ERR_WORKSPACE
        assert call(M, N, K, _r(a), _r(b), _r(c), FAKE + 8, need, None) == s2r.S2R_ERR_ALIGN


def test_a_weight_gradients_workspace_is_checked(s2r):
    L = s2r.lib()
    need = s2r.s2r_q8_wgrad_workspace_bytes(8192, 1024, 256)
    assert need > 0
    dy, x = _m(s2r, ld=1024), _q(s2r, lds=8192)
    call = lambda ws, n: L.s2r_q8_wgrad(8192, 1024, 256, _r(dy), None, _r(x), FAKE, 256, 0, ws, n, None)
    assert call(FAKE, need - 1) == s2r.S2R_ERR_WORKSPACE
    assert call(FAKE + 8, need) == s2r.S2R_ERR_ALIGN
