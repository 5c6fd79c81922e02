"""gemm_norm_backward's bounded wait for a row that several multiprocessors share: it runs out without a fault, shows in
DX alone, and leaves the next calls as they were."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests.test_norm_gpu import back_inputs, run_backward

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


@pytest.fixture
def short_wait():
    gemm.gemm_testing_set_norm_fault(1000)
    yield
    gemm.gemm_testing_set_norm_fault(0)


# clusters of two, four and eight, with one row each and with several
@pytest.mark.parametrize("M,K,dy,h", [(3, 8208, "bf16", "bf16"), (800, 8208, "bf16", "bf16"), (77, 20496, "bf16", "bf16"),
                                      (300, 20496, "bf16", "f32"), (170, 28688, "f32", "f32")])
def test_a_lost_sum_ends_in_nan(M, K, dy, h, short_wait):
    t = back_inputs(M, K, dy, h, seed=M + K)
    gemm.gemm_testing_set_norm_fault(0)
    want = run_backward(M, K, dy, h, "bf16", *t)
    gemm.gemm_testing_set_norm_fault(1000)
    for _ in range(3):
        lost = run_backward(M, K, dy, h, "bf16", *t)
        assert lost[0].isnan().all()             # every cluster's first row is lost, and those behind it
        assert torch.equal(lost[1], want[1]) and torch.equal(lost[2], want[2])
    gemm.gemm_testing_set_norm_fault(0)
    got = run_backward(M, K, dy, h, "bf16", *t)
    assert got[0].isfinite().all() and all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_of_one_multiprocessor_do_not_wait(short_wait):
    t = back_inputs(333, 2064, "bf16", "bf16", seed=1)
    assert run_backward(333, 2064, "bf16", "bf16", "bf16", *t)[0].isfinite().all()
