"""The gated unit over all of its sigmoid's range, where it is nearly 0 or nearly 1, and the input of the block's second
matrix-vector product that it then makes."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref
from tests.test_gate_gpu import decoded, run_backward, run_forward

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# What the smaller of s and 1 - s may be off by below fp32's normal numbers: one unit of its subnormal ones
SUBNORMAL = 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def test_shut_gates_keep_their_value():
    """s is below fp32's normal numbers from g = -87.3 on, g * s * u is not."""
    F = 4096
    Z = torch.zeros(2, 2 * F)
    Z[0, :F] = torch.linspace(-103, -80, F)
    Z[1, :F] = torch.linspace(-89, -87, F)
    Z[:, F:] = 2.0 ** 100
    A = run_forward(2, F, "f32", "bf16", Z, save=False)[0]
    g, u = Z[:, :F].double(), Z[:, F:].double()
    want = g / (1 + torch.exp(-g)) * u
    # the exponential's two halves below its normal range: twice its error
    tol = ref.half_ulp(want, "bf16") * 1.001 + 2 * ref.sigmoid_rel(g) * want.abs() + 2 * SUBNORMAL * (g * u).abs()
    ref.assert_within("a", A, want, tol)


def test_gradient_of_shut_and_open_gates():
    """At e4m3's values from -112 to 112: 1 - s of an open gate and s of a shut one to their own precision."""
    values = [v * s for v in (8., 9, 10, 11, 12, 13, 14, 16, 18, 20, 22, 24, 26, 28, 30, 32, 40, 48, 56, 64, 72, 80, 88, 96, 104)
              for s in (1, -1)]
    F = 64
    CK = torch.zeros(1, 2 * F, dtype=torch.uint8)
    e4m3 = torch.tensor(values + [0.0] * (F - len(values))).to(torch.float8_e4m3fn)
    assert torch.equal(e4m3[:len(values)].float(), torch.tensor(values))
    CK[0, :F] = e4m3.view(torch.uint8)
    CK[0, F:] = torch.tensor(1.5).to(torch.float8_e4m3fn).view(torch.uint8)
    SF = torch.full((1, 2 * ref.blocks(F)), 127, dtype=torch.uint8)
    DA = torch.full((1, F), 2.0 ** 40)
    DZ, _ = run_backward(1, F, "f32", "f32", "bf16", DA, CK, SF, again=False)
    g, u = decoded(CK, SF, F)
    da = DA.double()
    s, t = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    # s and t are e / (1 + e) or 1 / (1 + e): relative errors of the exponential and five roundings; open gates' t only weighs
    # g t beside 1
    e_rel = (4 + 2 * 1.173 * g.abs()) * 2 * ref.U + 4 * 2 * ref.U
    small = torch.where(g < 0, e_rel, torch.full_like(g, 8 * ref.U))
    du, dg = da * g * s, da * u * s * (1 + g * t)
    lost = torch.where(g < 0, 2 * SUBNORMAL, 0.0) * (da * u * (1 + g.abs())).abs()
    ref.assert_within("du", DZ[:, F:], du, (small + 4 * ref.U) * du.abs() + lost)
    t_rel = torch.where(g < 0, 8 * ref.U, e_rel)
    dg_tol = (small + 8 * ref.U) * (da * u * s).abs() * (1 + g.abs() * t) + t_rel * (da * u * s * g * t).abs() + lost
    ref.assert_within("dg", DZ[:, :F], dg, dg_tol)
