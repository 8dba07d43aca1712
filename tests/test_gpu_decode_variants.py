"""The variants of the decoding-step kernels that the calls choose by their sizes: each is run, with and without its
optional operands, under the bounds that tests/test_gpu_decode.py derives."""
import pytest

from tests.test_gpu_decode import _norm_case, _run_norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("M,K", [(3, 8448), (130, 9472), (1, 16128), (2, 16640), (5, 31232), (9, 8192), (2, 8704), (593, 8960),
                                 (600, 16640)])
def test_norm_steps_per_thread(osc, M, K, with_res):
    """One, two and four steps of a thread, the last one whole or not for all threads, few rows and many."""
    X, res, gamma = _norm_case(M, K, M + K)
    _run_norm(osc, X, res if with_res else None, gamma, 1e-6)
