"""Strides of weight gradients and steps from expert to expert on the CPU: those whose bytes pass 64 bits are refused, as
-1 is, and do not wrap round to small ones.  No device is touched."""
import pytest
from test_moe_abi import _e, _gemm, _wgrad
from test_q8_abi import FAKE, _m, _q, _r, s2r  # noqa: F401

MINUS = lambda n: (1 << 64) - n


def _dense(s2r, N, ld, M=50):
    return s2r.lib().s2r_q8_wgrad(M, N, 200, _r(_m(s2r)), None, _r(_q(s2r)), FAKE, ld, 1, None, 0, None)


# 2^64 is 2 * 2^63, 39 * (2^64 / 39): what is left of the product may be as small as any
WRAPS = [(2, MINUS(1)), (40, MINUS(1)), (40, MINUS(8000)), (40, MINUS(200)), (3, 1 << 63), (40, (1 << 64) // 39 + 6), (40, 1 << 59)]


@pytest.mark.parametrize("N,ld", WRAPS)
def test_row_strides(s2r, N, ld):
    assert _dense(s2r, N, ld) == s2r.S2R_ERR_DIM
    for experts in (1, 4):
        for step in (8000, MINUS(1)):
            assert _wgrad(s2r, e=_e(s2r, experts=experts), N=N, ld=ld, step=step) == s2r.S2R_ERR_DIM


@pytest.mark.parametrize("experts,step", [(2, MINUS(1)), (4, MINUS(8000)), (3, 1 << 63), (4, (1 << 64) // 3 + 1), (1024, 1 << 54), (5, 1 << 60)])
def test_steps_of_experts(s2r, experts, step):
    assert _wgrad(s2r, e=_e(s2r, experts=experts), step=step) == s2r.S2R_ERR_DIM


@pytest.mark.parametrize("experts,step", [(2, MINUS(16)), (4, MINUS(256)), (3, 1 << 63), (1024, 1 << 55)])
def test_steps_of_weights(s2r, experts, step):
    assert _gemm(s2r, e=_e(s2r, experts=experts), step=step) == s2r.S2R_ERR_DIM
    assert _gemm(s2r, e=_e(s2r, experts=experts), sstep=step) == s2r.S2R_ERR_DIM
    assert _gemm(s2r, e=_e(s2r, experts=experts), sstep=MINUS(1)) == s2r.S2R_ERR_DIM
    none, no = _m(s2r, data=None), _q(s2r, q=None)
    assert _gemm(s2r, e=_e(s2r, experts=1), M=0, a=no, c=none, step=step, sstep=step) == s2r.S2R_OK
    assert _gemm(s2r, e=_e(s2r, experts=experts), M=0, a=no, c=none, step=0, sstep=0) == s2r.S2R_OK
    assert _gemm(s2r, e=_e(s2r, experts=experts), M=0, a=no, c=none, step=48, sstep=1) == s2r.S2R_OK


def test_what_is_not_used_may_be_anything(s2r):
    """One row has no stride and one expert no step; M == 0 with `accumulate` then has nothing to do."""
    none, no = _m(s2r, data=None), _q(s2r, q=None)
    assert s2r.lib().s2r_q8_wgrad(0, 1, 200, _r(none), None, _r(no), FAKE, MINUS(1), 1, None, 0, None) == s2r.S2R_OK
    assert _wgrad(s2r, e=_e(s2r, experts=1), M=0, y=none, x=no, acc=1, step=0) == s2r.S2R_OK
    assert _wgrad(s2r, e=_e(s2r, experts=1), M=0, y=none, x=no, acc=1, step=MINUS(1)) == s2r.S2R_OK
    assert _wgrad(s2r, M=0, y=none, x=no, acc=1, step=1 << 40) == s2r.S2R_OK
    assert _wgrad(s2r, N=0, y=none, dw=None, ld=MINUS(1), step=MINUS(1)) == s2r.S2R_OK
