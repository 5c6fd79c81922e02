"""Both forms of gemm_clip_run, the single cluster's (up to 64 rows of 4 KiB) and the two kernels', where they can go wrong."""
import math

import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref
from tests.test_clip_gpu import check, exact_norm, make, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()

# The most that a norm may be off: a step of 16-bit values adds 8 squares in each of four fp32 sums, one rounding apiece, and joins
# those in two (f32: 4 and two); the sums of the steps carry twice fp32's digits, and become one number by one rounding.  The
# root halves those 11 and rounds once itself.  (Second-order terms: 2^-10 of it.)
NORM = 6.5 * ref.U * (1 + 2.0 ** -10)
FORMS = pytest.mark.parametrize("n", [2003, 300007], ids=["cluster", "kernels"])
KINDS = pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])


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
    assert abs(float(norms[0]) - exact_norm(G)) <= NORM * exact_norm(G)
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


@FORMS
@KINDS
def test_norms_are_as_exact_as_their_sums(kind, n):
    for scale in (1.0, 1e-3):
        for G in (make([n], [kind], scale), make([n, 77, n // 3], [kind, "f32"], scale)):
            want = exact_norm(G)
            norm, _ = run(G, 1.0, None)
            assert abs(norm - want) <= NORM * want


@FORMS
@KINDS
@pytest.mark.parametrize("C", ["new", "same"])
def test_nonfinite_values(C, kind, n):
    """A NaN, an infinity and both, in the tensor's first and last elements and inside, under every kind of limit."""
    big = make([n, 300], [kind, "f32"])
    for at in (0, n // 2, n - 1):
        for value in (math.nan, math.inf, -math.inf):
            G = [g.clone() for g in big]
            G[0][at] = value
            for limit in (0.0, 1.0):
                norm, out = run(G, limit, C)
                if math.isnan(value):
                    assert math.isnan(norm) and all(c.isnan().all() for c in out)
                    continue
                assert norm == math.inf
                hit = torch.zeros(n, dtype=torch.bool)
                hit[at] = True
                assert out[0][hit].isnan().all() and (out[0][~hit] == 0).all() and (out[1] == 0).all()
            norm, out = run(G, math.inf, C)
            if math.isnan(value):
                assert math.isnan(norm) and all(c.isnan().all() for c in out)
            else:
                assert norm == math.inf and all(torch.equal(c, g) for c, g in zip(out, G))
    G[0][0], G[0][n - 1] = math.inf, math.nan
    norm, out = run(G, 1.0, C)
    assert math.isnan(norm) and all(c.isnan().all() for c in out)


@FORMS
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_large_values_beside_tiny_ones(kind, n):
    """One large value among small ones, and the other way round, in one thread's step: scaled by a power of two."""
    for rest, one, at in ((1e-25, 1e22, n // 2), (1e-30, 1e-21, 5), (1e30, 1e-30, 1000), (1e-3, 1e19, n - 9), (3e38, 1e-38, n // 3)):
        g = torch.full((n,), rest).to(ref.TORCH[kind])
        g[at] = one
        want = exact_norm([g])
        for factor in (0.5, 1e-6):
            limit = float(torch.tensor(want * factor))
            if not 1e-38 < limit < 3e38:
                continue
            norm, out = run([g], limit)
            assert abs(norm - want) <= NORM * want if want < 3.4e38 else norm == math.inf
            check([g], limit, norm if want < 3.4e38 else want, out)


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_nonfinite_values_past_the_first_launch(value):
    """A list that goes through several launches: what the later ones find counts for the tensors of all."""
    G = make([1 + i % 97 for i in range(2000)], ["f32", "bf16", "f16"])
    G[1500][0] = value
    norm, out = run(G, 1.0)
    if math.isnan(value):
        assert math.isnan(norm) and all(c.isnan().all() for c in out)
        return
    assert norm == math.inf and out[1500][0].isnan() and (out[1500][1:] == 0).all()
    assert all((c == 0).all() for i, c in enumerate(out) if i != 1500)


@pytest.mark.parametrize("sizes", [[50001, 900, 3], [700001, 5000, 3, 70007], [41] * 1900], ids=["cluster", "kernels", "launches"])
def test_replays_element_by_element(sizes):
    """Clipped, clipped again from there, and the same in place, captured: every element on new inputs."""
    kinds = [("f32", "bf16")[i % 2] for i in range(len(sizes))]
    new = lambda: [torch.empty(n, dtype=ref.TORCH[k], device="cuda") for n, k in zip(sizes, kinds)]
    G, C, C2, C3 = new(), new(), new(), new()
    norms = torch.empty(4, device="cuda")
    work = torch.empty(gemm.GEMM_CLIP_WORKSPACE, dtype=torch.uint8, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        for i, (g, c, limit) in enumerate(((G, C, 0.5), (C, C2, 0.25), (C, C3, math.inf), (C3, C3, 0.25))):
            gemm.gemm_clip_run(gemm.clip_tensors(list(zip(g, c, kinds))), limit, norms[i:i + 1], work, stream=stream)
    for seed in (1, 2):
        host = make(sizes, ["f32", "bf16"], seed=seed)
        for g, h in zip(G, host):
            g.copy_(h)
        graph.replay()
        torch.cuda.synchronize()
        c = [t.cpu() for t in C]
        check(host, 0.5, float(norms[0]), c)
        check(c, 0.25, float(norms[1]), [t.cpu() for t in C2])
        assert float(norms[1]) == float(norms[2]) == float(norms[3])
        assert all(torch.equal(a, b) for a, b in zip(C2, C3))


@pytest.mark.parametrize("sizes", [[3001, 5, 1030, 77, 4097], [200003, 5, 90001, 77, 70001], [3, 41, 5, 16, 1] * 400],
                         ids=["cluster", "kernels", "launches"])
def test_lists_of_every_kind_of_output(sizes):
    """In one list: tensors that only count, in place, written elsewhere, and elsewhere at another place of 16 bytes."""
    G = make(sizes, ["f32", "bf16", "f16"])
    kinds = [("f32", "bf16", "f16")[i % 3] for i in range(len(G))]
    want = exact_norm(G)
    for limit in (0.3 * want, 3.0 * want):
        tensors, outs = [], []
        for i, (g, k) in enumerate(zip(G, kinds)):
            src = g.cuda()
            pool = torch.zeros(g.numel() + 16, dtype=g.dtype, device="cuda")
            c = (None, src, pool[8:8 + g.numel()], pool[1:1 + g.numel()])[i % 4]
            tensors.append((src, c, k))
            outs.append((src, c, pool))
        norm = torch.empty(1, device="cuda")
        work = torch.empty(gemm.GEMM_CLIP_WORKSPACE, dtype=torch.uint8, device="cuda")
        gemm.gemm_clip_run(gemm.clip_tensors(tensors), limit, norm, work, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        written = [i for i, (_, c, _) in enumerate(outs) if c is not None]
        assert abs(float(norm) - want) <= NORM * want
        factor = min(1.0, float(torch.tensor(limit)) / want)
        for i in written:
            g, c, v = G[i], outs[i][1].cpu(), G[i].double() * factor
            if factor == 1.0:
                assert torch.equal(c, g)
            else:
                tol = ref.half_ulp(v, kinds[i]) * (1 + 2.0 ** -10) + (NORM + 3 * ref.U) * v.abs()
                ref.assert_within("c", c, v, tol + 2.0 ** -149)
        for i, (src, c, pool) in enumerate(outs):
            if c is not src:
                assert torch.equal(src.cpu(), G[i])
            start = {2: 8, 3: 1}.get(i % 4)
            rest = pool.clone()
            if start is not None:
                rest[start:start + G[i].numel()] = 0
            assert not rest.any()
