"""gemm_gate_run and gemm_gate_backward against their definitions in 64 bits."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref
from tests.test_norm_gpu import guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def run_forward(M, F, z, a, Z, save=True, stream=None):
    Z = Z.cuda()
    A, a_ok = guarded((M, F), ref.TORCH[a])
    SFA, s_ok = guarded((M, ref.blocks(F)), torch.uint8) if a == "e4m3" else (None, lambda: True)
    CK, c_ok = guarded((M, 2 * F), torch.uint8) if save else (None, lambda: True)
    SFCK, sc_ok = guarded((M, 2 * ref.blocks(F)), torch.uint8) if save else (None, lambda: True)
    torch.cuda.synchronize()
    gemm.gemm_gate_run(M, F, z, a, Z, A, SFA, CK, SFCK, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert a_ok() and s_ok() and c_ok() and sc_ok()
    return A, SFA, CK, SFCK


def make_z(M, F, z, seed):
    gen = torch.Generator().manual_seed(seed)
    Z = torch.randn(M, 2 * F, generator=gen) * 2
    Z[:, ::41] *= 8
    return Z.to(ref.TORCH[z])


SHAPES = [(1, 16), (1, 8192), (3, 48), (130, 32), (77, 2064), (5, 4080), (260, 16), (33, 1024)]


@pytest.mark.parametrize("M,F", SHAPES)
@pytest.mark.parametrize("z", ["bf16", "f32"])
@pytest.mark.parametrize("a", ["e4m3", "bf16", "f16"])
def test_forward(M, F, z, a):
    Z = make_z(M, F, z, M + F)
    A, SFA, CK, SFCK = run_forward(M, F, z, a, Z)
    g, u = Z[:, :F].double(), Z[:, F:].double()
    ref.assert_operand("a", A, SFA, ref.gate(g, u), float(ref.sigmoid_rel(g).max()) + 3 * ref.U, a)
    n = ref.blocks(F)
    for half, codes, scales in ((g, CK[:, :F], SFCK[:, :n]), (u, CK[:, F:], SFCK[:, n:])):
        want = ref.scale_codes(half)
        assert torch.equal(scales.cpu().long(), want)
        assert torch.equal(ref.decode_e4m3(codes), ref.e4m3(half / ref.spread(want, F)))
    lone = run_forward(M, F, z, a, Z, save=False)
    assert torch.equal(lone[0], A) and (SFA is None or torch.equal(lone[1], SFA))


def test_large_gates_and_nonfinite_values():
    """Far from zero the sigmoid is 0 or 1; NaN and infinity reach their own element only."""
    F = 64
    Z = torch.zeros(2, 2 * F)
    Z[0, :F] = torch.linspace(-120, 120, F)
    Z[0, F:] = 3.0
    Z[1] = 1.0
    Z[1, 7] = float("nan")
    Z[1, F + 40] = float("inf")
    A, _, CK, SFCK = run_forward(2, F, "f32", "bf16", Z)
    g, u = Z[:, :F].double(), Z[:, F:].double()
    want = ref.gate(g, u)
    ref.assert_within("a", A, want, ref.half_ulp(want, "bf16") * 1.001 + ref.sigmoid_rel(g) * want.abs() + 1e-35)
    n = ref.blocks(F)
    gq = ref.decode_e4m3(CK[:, :F]) * ref.spread(SFCK[:, :n].cpu(), F)
    uq = ref.decode_e4m3(CK[:, F:]) * ref.spread(SFCK[:, n:].cpu(), F)
    assert gq[1, 7].isnan() and (gq[1, :7] == 1).all() and (gq[1, 8:] == 1).all()
    assert uq.float()[1, 40].isinf() and (uq[1, :32] == 1).all()


def checkpoint(M, F, seed):
    """An 8-bit checkpoint with every kind of code: ordinary ones, subnormals, zeros, the largest."""
    gen = torch.Generator().manual_seed(seed)
    CK = torch.randint(0, 256, (M, 2 * F), generator=gen, dtype=torch.uint8)
    CK[(CK & 127) == 127] = 126
    SF = torch.randint(118, 124, (M, 2 * ref.blocks(F)), generator=gen, dtype=torch.uint8)
    return CK, SF


def run_backward(M, F, da, dz, a, DA, CK, SF, again=True):
    DZ, z_ok = guarded((M, 2 * F), ref.TORCH[dz])
    A, a_ok = guarded((M, F), ref.TORCH[a]) if again else (None, lambda: True)
    torch.cuda.synchronize()
    gemm.gemm_gate_backward(M, F, da, dz, a, DA.cuda(), CK.cuda(), SF.cuda(), DZ, A, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert z_ok() and a_ok()
    return DZ, A


def decoded(CK, SF, F):
    n = ref.blocks(F)
    return (ref.decode_e4m3(CK[:, :F]) * ref.spread(SF[:, :n].cpu(), F),
            ref.decode_e4m3(CK[:, F:]) * ref.spread(SF[:, n:].cpu(), F))


@pytest.mark.parametrize("M,F", SHAPES)
@pytest.mark.parametrize("da,dz,a", [("bf16", "bf16", "bf16"), ("f32", "f32", "f16"), ("bf16", "f32", "bf16"),
                                     ("f32", "bf16", "f16")])
def test_backward(M, F, da, dz, a):
    CK, SF = checkpoint(M, F, M * 3 + F)
    DA = torch.randn(M, F, generator=torch.Generator().manual_seed(8)).to(ref.TORCH[da])
    DZ, A = run_backward(M, F, da, dz, a, DA, CK, SF)
    g, u = decoded(CK, SF, F)
    dg, du, v, dg_tol, du_tol, rel = ref.gate_back(g, u, DA.double())
    # tiny: what a product of subnormals loses
    tiny = 1e-37
    ref.assert_within("dg", DZ[:, :F], dg, ref.half_ulp(dg, dz) * 1.001 + dg_tol + tiny)
    ref.assert_within("du", DZ[:, F:], du, ref.half_ulp(du, dz) * 1.001 + du_tol + tiny)
    ref.assert_within("a", A, v, ref.half_ulp(v, a) * 1.001 + rel * v.abs() + tiny)
    assert torch.equal(run_backward(M, F, da, dz, a, DA, CK, SF, again=False)[0], DZ)


def test_gradient_against_differences():
    """Directional derivatives of sum(da * a) at the checkpoint's values, by central differences in 64 bits."""
    M, F = 4, 112
    Z = make_z(M, F, "f32", 6)
    _, _, CK, SFCK = run_forward(M, F, "f32", "bf16", Z)
    g, u = decoded(CK, SFCK, F)
    assert float((g - Z[:, :F]).abs().max()) < 2.0 ** -4 * float(Z.abs().max())
    DA = torch.randn(M, F, generator=torch.Generator().manual_seed(3))
    DZ, _ = run_backward(M, F, "f32", "f32", "bf16", DA, CK, SFCK)
    gen = torch.Generator().manual_seed(4)
    e = 1e-6
    for _ in range(5):
        vg, vu = (torch.randn(M, F, generator=gen, dtype=torch.float64) for _ in range(2))
        f = lambda s: float((DA.double() * ref.gate(g + s * e * vg, u + s * e * vu)).sum())
        got = DZ.cpu().double() * torch.cat([vg, vu], 1)
        assert abs(float(got.sum()) - (f(1) - f(-1)) / (2 * e)) < 1e-5 * float(got.abs().sum())


def test_rows_past_two_to_the_31_elements():
    M, F = 70000, 16384
    Z = torch.zeros(M, 2 * F, dtype=torch.bfloat16, device="cuda")
    tail = make_z(2, F, "bf16", 1)
    Z[-2:] = tail.cuda()
    A = torch.empty(M, F, dtype=torch.uint8, device="cuda")
    SFA = torch.empty(M, F // 32, dtype=torch.uint8, device="cuda")
    CK = torch.empty(M, 2 * F, dtype=torch.uint8, device="cuda")
    SFCK = torch.empty(M, 2 * F // 32, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream()
    gemm.gemm_gate_run(M, F, "bf16", "e4m3", Z, A, SFA, CK, SFCK, s)
    torch.cuda.synchronize()
    small = run_forward(2, F, "bf16", "e4m3", tail)
    for big, lone in zip((A, SFA, CK, SFCK), small):
        assert torch.equal(big[-2:], lone)
    assert int(CK[-3].max()) == 0
    DZ = Z                                       # the same size, no longer needed
    DA = torch.zeros(M, F, dtype=torch.bfloat16, device="cuda")
    DA[-2:] = 1
    gemm.gemm_gate_backward(M, F, "bf16", "bf16", "bf16", DA, CK, SFCK, DZ, None, s)
    torch.cuda.synchronize()
    lone = run_backward(2, F, "bf16", "bf16", "bf16", DA[-2:].cpu(), CK[-2:].cpu(), SFCK[-2:].cpu(), again=False)[0]
    assert torch.equal(DZ[-2:], lone) and float(DZ[-3].abs().max()) == 0
