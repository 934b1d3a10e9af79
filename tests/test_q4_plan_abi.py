"""The workspace of the 4-bit product on the CPU: sizes whose sum is cut, and what is refused there."""
import pytest
from test_q4_abi import _m, _q4, _r
from test_q8_abi import FAKE, s2r  # noqa: F401


@pytest.mark.parametrize("M,N,K", [(129, 127, 8200), (300, 1000, 4096), (64, 8192, 4100)])
def test_long_sums_of_small_results_take_a_workspace(s2r, M, N, K):
    L, need = s2r.lib(), s2r.s2r_q4_gemm_workspace_bytes(M, N, K)
    assert need >= 2 * M * N * 4 and need % (M * 16) == 0  # two parts or more, rows of whole 16 bytes
    a, c = _q4(s2r, ld=4112, lds=264), _m(s2r, ld=8192)
    call = lambda ws, n: L.s2r_q4_gemm(M, N, K, _r(a), _r(a), _r(c), ws, n, None)
    assert call(FAKE, need - 1) == s2r.S2R_ERR_WORKSPACE and call(FAKE, 1) == s2r.S2R_ERR_WORKSPACE
    assert call(FAKE + 8, need) == s2r.S2R_ERR_ALIGN


@pytest.mark.parametrize("M,N,K", [(0, 100, 8192), (100, 0, 8192), (1, 8192, 4096), (32, 64, 8192), (64, 64, 512), (5001, 4999, 1100),
                                   (64, 64, 0), (1 << 28, 1, 1), (1, 1 << 28, 1), (1, 1, 1 << 28)])
def test_and_others_none(s2r, M, N, K):
    assert s2r.s2r_q4_gemm_workspace_bytes(M, N, K) == 0
