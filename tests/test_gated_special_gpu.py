"""NaN and infinities in the gated product's operands, in each of its forms: what they reach, and that they reach nothing else."""
import math

import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import gatedref as gr
from tests import opsref as ref
from tests.test_gated_gpu import ONE, TWO, Out, backward, backward_case, dev, forward, operands
from tests.test_gated_matvec_gpu import case, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


@pytest.mark.parametrize("M,F,K,flags,launches,slices", [
    (300, 96, 512, ONE, 1, 1), (300, 96, 496, ONE, 1, 1), (300, 96, 528, ONE, 2, 1), (300, 160, 512, TWO, 2, 1),
    (300, 160, 80, TWO, 2, 1), (64, 96, 8192, ONE, 1, 8), (64, 96, 8208, ONE, 2, 8)])
def test_nan_codes_and_nan_scales(M, F, K, flags, launches, slices):
    """Scales read as they are and packed ones, single CTAs, slices and pairs: a NaN code or a scale of 255 in X makes its row NaN, in
    W its column."""
    (X, SX, _), (W, SW, _) = operands(M, F, K, "e4m3")
    X, W = X.view(torch.uint8), W.view(torch.uint8)
    plain, odd = Out(M, F, "bf16", True), Out(M, F, "bf16", True)
    with gemm.GatedPlan(M, F, K, "e4m3", "bf16", 1, flags) as plan:
        info = plan.info
        assert (info["launches_per_run"], info["splits"], info["cta_group"]) == (launches, slices, 2 if flags == TWO else 1)
        forward(plan, (dev(X), dev(SX)), (dev(W), dev(SW)), plain)
        last = SX.shape[1] - 1
        X[0, K - 1], X[M - 1, 0], X[40, K // 2] = 0x7F, 0xFF, 0x7F
        SX[7, 0], SX[33, last] = 255, 255
        W[0, 0], W[F + 5, K - 1] = 0x7F, 0xFF           # g of column 0, u of column 5
        SW[F - 1, last], SW[F + 66, last // 2] = 255, 255
        forward(plan, (dev(X), dev(SX)), (dev(W), dev(SW)), odd)
    bad = torch.zeros(M, F, dtype=torch.bool)
    bad[[0, M - 1, 40, 7, 33]] = True
    bad[:, [0, 5, F - 1, 66]] = True
    got, want = odd.A.cpu(), plain.A.cpu()
    assert want.isfinite().all()
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], want[~bad])
    # the checkpoint: g's and u's own columns, and blocks of 32 without one keep their codes and their scales
    ck, n = odd.CK.cpu(), ref.blocks(F)
    nan = torch.zeros(M, 2 * F, dtype=torch.bool)
    nan[[0, M - 1, 40, 7, 33]] = True
    nan[:, [0, F + 5, F - 1, F + 66]] = True
    assert torch.equal((ck & 127) == 127, nan)
    hit = torch.zeros(M, 2 * n, dtype=torch.bool)
    hit[[0, M - 1, 40, 7, 33]] = True
    hit[:, [0, n, (F - 1) // 32, n + 2]] = True
    assert torch.equal(odd.SFCK.cpu()[~hit], plain.SFCK.cpu()[~hit])
    spread = torch.cat([hit[:, :n].repeat_interleave(32, 1)[:, :F], hit[:, n:].repeat_interleave(32, 1)[:, :F]], 1)
    assert torch.equal(ck[~spread], plain.CK.cpu()[~spread])


def same_kinds(got, want):
    """NaN where the definition in 64 bits has NaN, and its infinities with their signs."""
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.where(got.isinf(), torch.sign(got.float()), 0.0), torch.where(want.isinf(), torch.sign(want).float(), 0.0))


def product(x, w):
    """x·wᵀ in doubles, term by term: an infinity times a zero is a NaN."""
    return (x[:, None, :] * w[None, :, :]).sum(2)


@pytest.mark.parametrize("x,w", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("M,F,K", [(1, 40, 272), (7, 40, 1040), (16, 23, 400)])
def test_few_rows(M, F, K, x, w):
    X, (W, SF, wide) = case(M, F, K, x, w)
    base = run(M, F, K, x, w, X, W, SF)
    assert base.isfinite().all()
    for value in (math.nan, math.inf, -math.inf):
        for m, k in ((0, 0), (M - 1, K - 1), (M // 2, K // 2)):
            Y = X.clone()
            Y[m, k] = value
            A = run(M, F, K, x, w, Y, W, SF)
            z = product(Y[m:m + 1].double(), wide)
            same_kinds(A[m:m + 1], ref.gate(z[:, :F], z[:, F:]))
            keep = torch.arange(M) != m
            assert torch.equal(A[keep], base[keep])
        if w == "e4m3":
            continue
        for row, k in ((0, 0), (F + 3, K - 1), (F - 1, K // 2)):
            V = W.clone()
            V[row, k] = value
            A = run(M, F, K, x, w, X, V, SF)
            z = product(X.double(), V.double()[[row % F, F + row % F]])
            same_kinds(A[:, row % F:row % F + 1], ref.gate(z[:, :1], z[:, 1:]))
            keep = torch.arange(F) != row % F
            assert torch.equal(A[:, keep], base[:, keep])


@pytest.mark.parametrize("M,F,N,flags", [(140, 64, 64, ONE), (140, 272, 136, TWO), (64, 64, 2048, 0), (1000, 1296, 72, ONE)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_gradient(kind, M, F, N, flags):
    DY, W2, (CK, SF, g, u) = backward_case(M, F, N, kind)
    with gemm.GatedBackPlan(M, F, N, kind, flags) as plan:
        base, again = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, kind, True)
        DY[3, 0], DY[M - 1, N - 1], DY[20, N // 2] = math.inf, -math.inf, math.nan
        rows = [3, 20, M - 1]
        DZ, A = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, kind, True)
        assert torch.equal(A, again)
        keep = torch.ones(M, dtype=torch.bool)
        keep[rows] = False
        DZ, base = DZ.cpu(), base.cpu()
        assert torch.equal(DZ[keep], base[keep])
        da = product(DY[rows].double(), W2.double().t())
        dg, du = ref.gate_back(g[rows], u[rows], da)[:2]
        same_kinds(DZ[rows], torch.cat([dg, du], 1))
        # a column of W2
        V = W2.clone()
        V[N // 3, F - 2] = math.inf
        DZ, A = backward(plan, dev(DY), dev(V), dev(CK), dev(SF), M, F, kind, True)
        DZ = DZ.cpu()
        assert torch.equal(A, again)
        other = torch.ones(2 * F, dtype=torch.bool)
        other[[F - 2, 2 * F - 2]] = False
        assert torch.equal(DZ[keep][:, other], base[keep][:, other])
        da = product(DY.double(), V.double()[:, F - 2:F - 1].t())
        dg, du = ref.gate_back(g[:, F - 2:F - 1], u[:, F - 2:F - 1], da)[:2]
        same_kinds(DZ[:, ~other], torch.cat([dg, du], 1))
