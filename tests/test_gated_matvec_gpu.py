"""gemm_gated_matvec_run against its definition in 64 bits."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import gatedref as gr
from tests import opsref as ref
from tests.test_norm_gpu import guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def run(M, F, K, x, w, X, W, SF, stream=None):
    A, ok = guarded((M, F), gr.TORCH[x])
    X, W, SF = (None if t is None else t.cuda() for t in (X, W, SF))
    torch.cuda.synchronize()
    gemm.gemm_gated_matvec_run(M, F, K, x, w, x, X, W, SF, A, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert ok()
    return A.cpu()


def case(M, F, K, x, w, seed=0):
    gen = torch.Generator().manual_seed(seed + 5 * M + F + K)
    X = torch.randn(M, K, generator=gen)
    X[:, ::37] *= 8
    X = X.to(gr.TORCH[x])
    return X, gr.rounded(torch.randn(2 * F, K, generator=gen) * K ** -0.5, w)


KINDS = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")]


def check(A, X, wide, kind):
    _, _, want, _, _, tol = gr.gated(X.double(), wide)
    gr.assert_output("a", A, None, want, tol, kind)


@pytest.mark.parametrize("x,w", KINDS)
@pytest.mark.parametrize("M,F,K", [(1, 1, 16), (1, 4096, 1024), (2, 7, 48), (3, 9, 2064), (5, 1040, 272), (8, 17, 8208),
                                   (9, 33, 16), (11, 640, 1040), (16, 8, 32768), (16, 2500, 528), (13, 5, 144)])
def test_matvec(M, F, K, x, w):
    X, (W, SF, wide) = case(M, F, K, x, w)
    A = run(M, F, K, x, w, X, W, SF)
    check(A, X, wide, x)
    assert torch.equal(A, run(M, F, K, x, w, X, W, SF, torch.cuda.Stream()))


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("K", [8, 24, 1000])
def test_rows_of_eight_elements(x, K):
    X, (W, _, wide) = case(3, 50, K, x, x)
    check(run(3, 50, K, x, x, X, W, None), X, wide, x)


@pytest.mark.parametrize("M", [1, 16])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_every_code_and_the_scales_ends(x, M):
    """Every finite e4m3 code, under scales from one end of the range to the other."""
    F, K = 40, 512
    gen = torch.Generator().manual_seed(M)
    W = torch.randint(0, 256, (2 * F, K), generator=gen, dtype=torch.uint8)
    W[(W & 127) == 127] = 126
    X = (torch.randn(M, K, generator=gen) * 2.0 ** -4).to(gr.TORCH[x])
    for low, high in ((100, 120), (0, 40), (127, 145), (130, 136)):
        SF = torch.randint(low, high + 1, (2 * F, K // 32), generator=gen, dtype=torch.uint8)
        wide = ref.decode_e4m3(W) * ref.spread(SF, K)
        g, u, want, tg, tu, tol = gr.gated(X.double(), wide)
        A = run(M, F, K, x, "e4m3", X, W, SF)
        # past the type's largest value it is infinite
        limit = float(torch.finfo(gr.TORCH[x]).max)
        inside = want.abs() + tol < limit
        edge = want.abs() - tol >= limit * (1 + 2.0 ** -8)
        assert A[edge].isinf().all()
        gr.assert_output("a", torch.where(inside, A.double(), 0.0), None, torch.where(inside, want, 0.0),
                         torch.where(inside, tol, 0.0), x)


@pytest.mark.parametrize("x_scale,low,high", [(2.0 ** -100, 190, 215), (2.0 ** 100, 20, 40), (2.0 ** -120, 127, 140), (2.0 ** 60, 60, 75)])
def test_activations_far_from_one(x_scale, low, high):
    """bf16 activations of any magnitude, tokens of a batch far apart, products that only together are ordinary numbers."""
    M, F, K = 11, 24, 640
    gen = torch.Generator().manual_seed(low)
    W = torch.randint(0, 256, (2 * F, K), generator=gen, dtype=torch.uint8)
    W[(W & 127) == 127] = 126
    SF = torch.randint(low, high + 1, (2 * F, K // 32), generator=gen, dtype=torch.uint8)
    X = torch.randn(M, K, generator=gen).double() * x_scale * torch.exp2(-2.0 * torch.arange(M).double())[:, None]
    X = X.to(torch.bfloat16)
    wide = ref.decode_e4m3(W) * ref.spread(SF, K)
    g, u, want, _, _, tol = gr.gated(X.double(), wide)
    A = run(M, F, K, "bf16", "e4m3", X, W, SF)
    # off by 2^-39 of the largest of a token's 128 k, times the weights there
    most = torch.stack([c.abs().amax(1) for c in X.double().split(128, 1)], 1)
    heavy = torch.stack([c.abs().sum(1) for c in wide.split(128, 1)], 1)
    lost = most @ heavy.t() * 2.0 ** -39
    tol = tol + 1.2 * (lost[:, :F] * (u.abs() + lost[:, F:]) + lost[:, F:] * g.abs()) + 1e-42
    limit = float(torch.finfo(torch.bfloat16).max)
    inside = want.abs() + tol < limit
    assert A[want.abs() - tol >= limit * (1 + 2.0 ** -8)].isinf().all()
    gr.assert_output("a", torch.where(inside, A.double(), 0.0), None, torch.where(inside, want, 0.0), torch.where(inside, tol, 0.0),
                     "bf16")


def test_nonfinite_values_stay_their_own():
    M, F, K = 4, 24, 128
    X, (W, SF, _) = case(M, F, K, "bf16", "e4m3")
    base = run(M, F, K, "bf16", "e4m3", X, W, SF)
    odd = W.view(torch.uint8).clone()
    odd[3, 17] = 127                                  # g of column 3
    odd[F + 9, 100] = 255                             # u of column 9
    SF2 = SF.clone()
    SF2[20, 1] = 255                                  # a scale of column 20's g
    A = run(M, F, K, "bf16", "e4m3", X, odd, SF2)
    hit = torch.zeros(F, dtype=torch.bool)
    hit[[3, 9, 20]] = True
    assert A[:, hit].isnan().all() and torch.equal(A[:, ~hit], base[:, ~hit])
    X[2, 5] = float("nan")
    A = run(M, F, K, "bf16", "e4m3", X, W, SF)
    assert A[2].isnan().all() and torch.equal(A[[0, 1, 3]], base[[0, 1, 3]])


def test_agrees_with_the_plan_and_replays():
    """A token through the few-row form and as a row of a batch; captured, it follows new inputs."""
    M, F, K = 16, 528, 1040
    X, (W, SF, wide) = case(M, F, K, "bf16", "bf16")
    X, W = X.cuda(), W.cuda()
    A, B = torch.empty(M, F, dtype=torch.bfloat16, device="cuda"), torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with gemm.GatedPlan(M, F, K) as plan:
        plan.run(X, W, B, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for m in range(M):
                gemm.gemm_gated_matvec_run(1, F, K, "bf16", "bf16", "bf16", X[m], W, None, A[m], stream)
        X2, _ = case(M, F, K, "bf16", "bf16", seed=3)
        X.copy_(X2)
        graph.replay()
        torch.cuda.synchronize()
    check(B.cpu(), case(M, F, K, "bf16", "bf16")[0], wide, "bf16")
    check(A.cpu(), X2, wide, "bf16")
