"""Zero matrices: zeros for every positive eps."""
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


@pytest.mark.parametrize("eps", [1e-7, 1e-37, 1e-38, 1e-41])
@pytest.mark.parametrize("m,n", [(40, 60), (60, 40)])
def test_zero_matrix_with_any_positive_eps_gives_zeros(m, n, eps):
    # also where the largest quotient, 2^8 / eps, is past FP32
    assert not fq.fp8q_newton_schulz(torch.zeros(m, n).cuda(), eps=eps).any()
