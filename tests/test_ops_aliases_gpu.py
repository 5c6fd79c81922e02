"""Buffers that may be shared between an input and an output, and inputs that may be left out, in every form of the kernels."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref
from tests.test_gate_gpu import checkpoint, run_backward as gate_backward
from tests.test_norm_dw import DW_REL
from tests.test_norm_gpu import EPS, back_inputs, check_backward, inputs, run_backward, run_forward

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


# a row's threads: part of a warp, whole warps, one to four units each
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(3, 48), (700, 112), (11, 1008), (400, 4096), (5, 16400)])
def test_the_stream_written_in_place_of_x(M, K, t, residual):
    X, R, W = inputs(M, K, t, t, seed=M + K, residual=residual)
    want = run_forward(M, K, t, t, "e4m3", X, R, W)
    X, R, W = X.cuda(), R.cuda() if residual else None, W.cuda()
    Y, SF, RS = torch.empty_like(want[1]), torch.empty_like(want[2]), torch.empty_like(want[3])
    gemm.gemm_norm_run(M, K, t, t, "e4m3", EPS, X, R, W, X, Y, SF, RS, torch.cuda.current_stream())
    assert all(torch.equal(a, b) for a, b in zip((X, Y, SF, RS), want))


# straight to registers, through the ring, several row groups in a CTA, split over two, four and eight CTAs
@pytest.mark.parametrize("M,K,dy,h", [(333, 2064, "bf16", "bf16"), (1000, 2064, "bf16", "bf16"), (700, 4112, "f32", "f32"),
                                      (700, 4096, "bf16", "f32"), (20000, 112, "bf16", "bf16"), (3100, 528, "f32", "f32"),
                                      (800, 8208, "bf16", "bf16"), (500, 8192, "f32", "f32"), (200, 20496, "bf16", "f32"),
                                      (170, 28688, "f32", "f32"), (3, 16384, "f32", "bf16")])
def test_gradient_with_nothing_past_the_norm(M, K, dy, h):
    DY, DH, H, RS, W = back_inputs(M, K, dy, h, seed=M + 5 * K)
    got = run_backward(M, K, dy, h, "bf16", DY, None, H, RS, W)
    check_backward(M, dy, h, "bf16", got, DY, None, H, RS, W)
    *_, dw, dw_size, _ = ref.norm_back(DY, torch.zeros_like(H), H, RS, W)
    ref.assert_within("dw", got[1], dw, DW_REL * dw_size)
    zeros = run_backward(M, K, dy, h, "bf16", DY, torch.zeros_like(DH), H, RS, W)
    assert all(torch.equal(a, b) for a, b in zip(got, zeros))


@pytest.mark.parametrize("M,F", [(1, 16), (77, 2064), (260, 1024)])
@pytest.mark.parametrize("dz", ["bf16", "f32"])
def test_the_gates_operand_in_place_of_its_gradient(M, F, dz):
    CK, SF = checkpoint(M, F, M + F)
    DA = torch.randn(M, F, generator=torch.Generator().manual_seed(3)).bfloat16()
    DZ, A = gate_backward(M, F, "bf16", dz, "bf16", DA, CK, SF)
    both, out = DA.cuda(), torch.empty_like(DZ)
    gemm.gemm_gate_backward(M, F, "bf16", dz, "bf16", both, CK.cuda(), SF.cuda(), out, both, torch.cuda.current_stream())
    assert torch.equal(out, DZ) and torch.equal(both, A)
