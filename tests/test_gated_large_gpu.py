"""The gated product, its gradient, its few-row form and the clipping where offsets pass 32 bits: rows and columns at the ends and
around the steps are taken from the outputs and compared with the definitions in 64 bits."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import gatedref as gr
from tests import opsref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def new(*shape, dtype=torch.uint8):
    return torch.full(shape, 0x7f if dtype == torch.uint8 else float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_forward_and_backward_past_32_bits(kind):
    """M x 2F = 4.6e9 codes and values; rows of K and N are short."""
    M, F, K = 70001, 32784, 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=gen, device="cuda").cpu()
    w = torch.randn(2 * F, K, generator=gen, device="cuda").cpu() * K ** -0.5
    (X, SX, xw), (W, SW, ww) = gr.rounded(x, kind), gr.rounded(w, kind)
    X, SX, W, SW = (None if t is None else t.cuda() for t in (X, SX, W, SW))
    n = ref.blocks(F)
    rows = torch.tensor([0, 1, 255, 256, 32766, 32767, 32768, 65498, 65499, 65535, 65536, 65537, M - 2, M - 1])
    A, CK, SFCK = new(M, F, dtype=torch.bfloat16), new(M, 2 * F), new(M, 2 * n)
    with gemm.GatedPlan(M, F, K, kind, "bf16", 1 if kind == "e4m3" else 0) as plan:
        plan.run(X, W, A, SX, SW, None, CK, SFCK, torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert plan.last_status() == gemm.GEMM_OK
    g, u, a, tg, tu, ta = gr.gated(xw[rows], ww)
    ck, sf = CK[rows.cuda()], SFCK[rows.cuda()]
    gr.assert_output("a", A[rows.cuda()], None, a, ta, "bf16")
    gr.assert_output("g", ck[:, :F], sf[:, :n], g, tg, "e4m3")
    gr.assert_output("u", ck[:, F:], sf[:, n:], u, tu, "e4m3")
    assert not torch.isnan(A).any()
    if kind == "e4m3":
        return
    N = 16
    DY = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    W2 = torch.randn(N, F, generator=gen, device="cuda").bfloat16()
    DZ = new(M, 2 * F, dtype=torch.bfloat16)
    with gemm.GatedBackPlan(M, F, N, "bf16") as plan:
        plan.run(DY, W2, CK, SFCK, DZ, A, torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert plan.last_status() == gemm.GEMM_OK
    from tests.test_gated_gpu import check_backward
    wide = [ref.decode_e4m3(ck[:, i * F:(i + 1) * F].cpu()) * ref.spread(sf[:, i * n:(i + 1) * n].cpu().long(), F) for i in (0, 1)]
    check_backward(DZ[rows.cuda()], A[rows.cuda()], DY[rows.cuda()].cpu(), W2.cpu(), wide[0], wide[1], "bf16")
    assert not torch.isnan(DZ).any()


@pytest.mark.parametrize("x,w", [("bf16", "bf16"), ("f16", "e4m3")])
@pytest.mark.parametrize("M", [1, 16])
def test_few_rows_past_32_bits(M, x, w):
    """The largest F: W has 2^21 rows."""
    F, K = 1 << 20, 2064
    gen = torch.Generator(device="cuda").manual_seed(2)
    X = torch.randn(M, K, generator=gen, device="cuda").to(gr.TORCH[x])
    cols = torch.tensor([0, 1, 7, 520191, 520193, 524287, 524288, 1040385, F - 17, F - 2, F - 1])
    picked = torch.cat([cols, cols + F])
    some = torch.randn(len(picked), K, generator=torch.Generator().manual_seed(3)) * K ** -0.5
    q, sf, wide = gr.rounded(some, w)
    W = torch.zeros(2 * F, K, dtype=gr.TORCH[w], device="cuda")
    W.view(torch.uint8)[picked.cuda()] = q.cuda().view(torch.uint8).view(len(picked), -1)
    SF = None
    if w == "e4m3":
        SF = torch.full((2 * F, ref.blocks(K)), 127, dtype=torch.uint8, device="cuda")
        SF[picked.cuda()] = sf.cuda()
    A = new(M, F, dtype=gr.TORCH[x])
    gemm.gemm_gated_matvec_run(M, F, K, x, w, x, X, W, SF, A, torch.cuda.current_stream())
    torch.cuda.synchronize()
    _, _, want, _, _, tol = gr.gated(X.cpu().double(), wide)
    gr.assert_output("a", A[:, cols.cuda()].cpu(), None, want, tol, x)
    A[:, cols.cuda()] = 0
    assert not A.any()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_clip_past_32_bits(kind):
    n = (1 << 32) + 4101 if kind == "bf16" else (1 << 31) + 4101
    t = gr.TORCH["bf16"] if kind == "bf16" else torch.float32
    g = torch.zeros(n, dtype=t, device="cuda")
    at = torch.tensor([0, 5, (1 << 30) + 1, (1 << 31) - 1, (1 << 31) + 3, n - 4097, n - 1], device="cuda")
    g[at] = torch.arange(1, len(at) + 1, device="cuda").to(t)
    h = torch.full((3,), 2.0, device="cuda")
    norm, work = torch.empty(1, device="cuda"), torch.empty(gemm.GEMM_CLIP_WORKSPACE, dtype=torch.uint8, device="cuda")
    want = (sum(i * i for i in range(1, len(at) + 1)) + 12.0) ** 0.5
    # in place; a quarter of the norm: every value below is exact in its type up to the factor's rounding
    gemm.gemm_clip_run(gemm.clip_tensors([(g, g, kind), (h, h, "f32")]), want / 4, norm, work, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= 8 * ref.U * want
    exact = torch.arange(1, len(at) + 1, dtype=torch.float64) / 4
    half = 2.0 ** -8 if kind == "bf16" else ref.U
    assert ((g[at].double().cpu() - exact).abs() <= (half * 1.01 + 12 * ref.U) * exact).all()
    assert ((h.double().cpu() - 0.5).abs() <= 12 * ref.U).all()
    g[at] = 0
    assert not g.any()
