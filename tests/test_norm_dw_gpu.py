"""gemm_norm_backward's dw where rows could be lost or taken twice: among many rows and row groups, at remainders."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref
from tests.test_norm_dw import DW_REL, SIZES, inputs, terms
from tests.test_norm_gpu import run_backward

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


@pytest.mark.parametrize("M,K,dy,h", SIZES)
def test_every_row_counts(M, K, dy, h):
    DY, H, RS = inputs(M, K, dy, h, seed=M + K)
    got = run_backward(M, K, dy, h, "bf16", DY, None, H, RS, torch.ones(K), again=False)[1]
    t = terms(DY, H, RS)
    ref.assert_within("dw", got, t.sum(0), DW_REL * t.abs().sum(0))
    # alone, a row is rounded twice and added to zeros
    last = (M - 1) // 152 * 152
    for row in {0, 1, M // 2, M // 3, last, M - 34, M - 33, M - 2, M - 1}:
        one = torch.zeros_like(DY)
        one[row] = DY[row]
        got = run_backward(M, K, dy, h, "bf16", one, None, H, RS, torch.ones(K), again=False)[1]
        ref.assert_within(f"row {row}", got, t[row], 3 * ref.U * t[row].abs())


# Terms that are whole numbers below 2^24 in sum: any order of them gives the same bits
@pytest.mark.parametrize("K", [16, 48, 112, 256, 528, 1024, 2064, 4112, 8208, 16400])
@pytest.mark.parametrize("dy,h", [("bf16", "bf16"), ("f32", "f32")])
def test_whole_numbers_sum_exactly(K, dy, h):
    gen = torch.Generator().manual_seed(K)
    most = min(40000, 30_000_000 // K)
    H = torch.randint(1, 4, (most, K), generator=gen).to(ref.TORCH[h])
    DY = torch.randint(-4, 5, (most, K), generator=gen).to(ref.TORCH[dy])
    t = (DY.float() * H.float()).cuda()
    H, DY, W, RS = H.cuda(), DY.cuda(), torch.ones(K, device="cuda"), torch.ones(most, device="cuda")
    rows = {1, 2, 3, 31, 32, 33, 127, 129, 151, 152, 153, 303, 304, 305, 455, 456, 457, 511, 512, 513, 607, 609, 911, 913,
            1216, 1217, 2432, 2433, 4863, 4865, 9727, 9728, 9729, 19455, 19457, 38912, 38913, most - 1, most}
    DX = torch.empty(most, K, dtype=ref.TORCH[h], device="cuda")
    DW, WS = torch.empty(K, device="cuda"), torch.empty(gemm.GEMM_NORM_PARTS, K, device="cuda")
    for M in sorted(r for r in rows if r <= most):
        DW.fill_(float("nan"))
        WS.fill_(float("nan"))
        gemm.gemm_norm_backward(M, K, dy, h, "bf16", DY, None, H, RS, W, DX, DW, None, WS, WS.numel() * 4,
                                torch.cuda.current_stream())
        assert torch.equal(DW.double(), t[:M].double().sum(0)), M
