"""Both forms of gemm_clip_run, the single cluster's (up to 64 rows of 4 KiB) and the two kernels', where they can go wrong."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref
from tests.test_clip_gpu import NORM_REL, check, exact_norm, make, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


@pytest.mark.parametrize("sizes", [[], [1], [1025], [5, 1, 2], [1024] * 8, [900] * 9], ids=lambda s: f"{len(s)}_{sum(s)}")
def test_ctas_without_rows_in_many_calls(sizes):
    """CTAs of the cluster that have nothing to load reach the exchange of sums at once: call after call the same norm."""
    calls = 200
    G = make(sizes, ["f32"])
    dev = [g.cuda() for g in G]
    C = [torch.zeros_like(g) for g in dev]
    tensors = gemm.clip_tensors([(g, c, "f32") for g, c in zip(dev, C)])
    norms = torch.zeros(calls, device="cuda")
    work = torch.empty(gemm.GEMM_CLIP_WORKSPACE, dtype=torch.uint8, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        for i in range(calls):
            gemm.gemm_clip_run(tensors, 1e30, norms[i:i + 1], work, stream=stream)
    graph.replay()
    torch.cuda.synchronize()
    assert (norms == norms[0]).all()
    assert abs(float(norms[0]) - exact_norm(G)) <= NORM_REL * exact_norm(G)
    assert all(torch.equal(c.cpu(), g) for c, g in zip(C, G))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2000, 300000], ids=["cluster", "kernels"])
@pytest.mark.parametrize("scale,limits", [(1e-16, (1e-15, 4e-19, 1e-25, 1e-38, 3e-45)), (1e10, (1e9, 4e-19, 1e-25, 1e-30))])
def test_small_limits(scale, limits, n, kind):
    """Elements far below the norm keep their digits where the limit is far below it too: every result that is an ordinary number
    is as exact as in the middle of the range.  (The largest of each piece are such that no sum leaves fp32.)"""
    gen = torch.Generator().manual_seed(n)
    g = scale * torch.pow(10.0, -14.0 * torch.rand(n, generator=gen, dtype=torch.float64))
    g[::4] = scale * (1.0 + torch.rand(len(g[::4]), generator=gen, dtype=torch.float64))
    g = (g * torch.where(torch.rand(n, generator=gen) < 0.5, -1.0, 1.0)).to(ref.TORCH[kind])
    for limit in limits:
        limit = float(torch.tensor(limit))            # as fp32 takes it
        assert limit < exact_norm([g])
        for C in ("new", "same"):
            norm, out = run([g], limit, C)
            check([g], limit, norm, out)
