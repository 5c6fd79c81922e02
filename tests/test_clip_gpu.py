"""gemm_clip_run against its definition in 64 bits."""
import math

import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref
from tests.test_norm_gpu import guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# A thread adds at most 32 squares of a step in four fp32 sums of 8 (16-bit types; fused, one rounding apiece) and joins those (two);
# what follows carries twice fp32's digits.  The root halves those 10 and rounds once: 6, and this is no less.
NORM_REL = (19 / 2 + 1) * ref.U


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def run(G, limit, C="new", stream=None):
    """(norm, outputs) of host tensors; C: "new" buffers, "same" (in place) or None."""
    kind = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}
    bufs = [guarded(tuple(g.shape), g.dtype) for g in G]
    for (b, _), g in zip(bufs, G):
        b.copy_(g)
    outs = [guarded(tuple(g.shape), g.dtype) for g in G] if C == "new" else (bufs if C == "same" else [(None, None)] * len(G))
    norm, n_ok = guarded((1,), torch.float32)
    work, w_ok = guarded((gemm.GEMM_CLIP_WORKSPACE,), torch.uint8)
    tensors = gemm.clip_tensors([(b, o, kind[g.dtype]) for (b, _), (o, _), g in zip(bufs, outs, G)])
    torch.cuda.synchronize()
    gemm.gemm_clip_run(tensors, limit, norm, work, stream=stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert n_ok() and w_ok() and all(ok() for _, ok in bufs) and all(ok is None or ok() for _, ok in outs)
    if C != "same":
        assert all(torch.equal(b.cpu().view(torch.uint8), g.view(torch.uint8)) for (b, _), g in zip(bufs, G))
    return float(norm), [None if o is None else o.cpu() for o, _ in outs]


def exact_norm(G):
    return math.sqrt(sum(float(g.double().square().sum()) for g in G))


def check(G, limit, norm, C):
    want = exact_norm(G)
    assert abs(norm - want) <= NORM_REL * want + 1e-46
    factor = min(1.0, limit / want) if want else 1.0
    for g, c in zip(G, C):
        v = g.double() * factor
        if factor == 1.0:
            assert torch.equal(c, g)
        else:                                         # the norm's error, the factor's and the product's roundings
            kind = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[g.dtype]
            ref.assert_within("c", c, v, ref.half_ulp(v, kind) * (1 + 2.0 ** -10) + (NORM_REL + 3 * ref.U) * v.abs() + 2.0 ** -149)


def make(sizes, kinds, scale=1e-2, seed=0):
    gen = torch.Generator().manual_seed(seed + len(sizes))
    return [(torch.randn(n, generator=gen) * scale).to(ref.TORCH[kinds[i % len(kinds)]]) for i, n in enumerate(sizes)]


SIZES = [[1], [0], [], [7], [8, 1, 0, 3], [4096, 4095, 4097], [70000, 16384, 1, 16385, 8192, 3], [600011], [5] * 33, [2049] * 257]


@pytest.mark.parametrize("kinds", [["f32"], ["bf16"], ["f16", "f32", "bf16"]])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}_{sum(s)}")
@pytest.mark.parametrize("factor", [0.3, 3.0])
def test_clip(sizes, kinds, factor):
    G = make(sizes, kinds)
    limit = factor * exact_norm(G) if sum(sizes) else factor
    for C in ("new", "same"):
        norm, out = run(G, limit, C)
        check(G, limit, norm, out)
    norm2, _ = run(G, limit, None)
    assert norm2 == norm


def test_more_tensors_than_a_launch_takes():
    G = make([1 + i % 37 for i in range(2203)], ["f32", "bf16"])
    limit = 0.5 * exact_norm(G)
    flat = {}
    for kind in ("f32", "bf16"):
        own = [g for g in G if g.dtype == ref.TORCH[kind]]
        flat[kind] = torch.cat(own).cuda()
    at = {"f32": 0, "bf16": 0}
    views = []
    for g in G:                                       # one behind the other: of every alignment
        kind = "f32" if g.dtype == torch.float32 else "bf16"
        views.append((flat[kind][at[kind]:at[kind] + g.numel()], kind))
        at[kind] += g.numel()
    out = {k: torch.zeros(v.numel() + 1, dtype=v.dtype, device="cuda") for k, v in flat.items()}
    at = {"f32": 1, "bf16": 1}                        # the outputs a step off the inputs' alignment
    tensors = []
    for v, kind in views:
        tensors.append((v, out[kind][at[kind]:at[kind] + v.numel()], kind))
        at[kind] += v.numel()
    norm = torch.empty(1, device="cuda")
    work = torch.empty(gemm.GEMM_CLIP_WORKSPACE, dtype=torch.uint8, device="cuda")
    gemm.gemm_clip_run(gemm.clip_tensors(tensors), limit, norm, work, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    check(G, limit, float(norm), [t[1].cpu() for t in tensors])
    assert all(float(v[0]) == 0 for v in out.values())


@pytest.mark.parametrize("offset", [1, 3, 4])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_alignments(kind, offset):
    """Tensors that begin anywhere, outputs at the same place of a line and at another one."""
    n = 40003
    base = (torch.randn(n + 16, generator=torch.Generator().manual_seed(offset)) * 0.1).to(ref.TORCH[kind])
    g = base[offset:offset + n]
    limit = 0.25 * exact_norm([g])
    for to in (offset, offset + 1, 0):
        src, dst = base.cuda(), torch.zeros(n + 16, dtype=base.dtype, device="cuda")
        norm = torch.empty(1, device="cuda")
        work = torch.empty(gemm.GEMM_CLIP_WORKSPACE, dtype=torch.uint8, device="cuda")
        gemm.gemm_clip_run(gemm.clip_tensors([(src[offset:offset + n], dst[to:to + n], kind)]), limit, norm, work,
                           stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        check([g], limit, float(norm), [dst[to:to + n].cpu()])
        assert float(dst[:to].abs().sum()) == 0 and float(dst[to + n:].abs().sum()) == 0


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30, 1e-20, 1e18, 1e19, 1e30, 1e38])
def test_range(scale):
    """Squares past fp32's ends: norms and results are as exact as in the middle."""
    for kinds in (["f32"], ["bf16"], ["f32", "bf16"]):
        G = make([3000, 70001], kinds, scale=0.1)
        G = [(g.double() * scale).to(g.dtype) for g in G]
        want = exact_norm(G)
        for limit in (0.5 * want, 1e-3 * want, 1.0, 1e-30):
            if limit > 3e38 or limit < 1e-38:
                continue
            norm, C = run(G, limit)
            if want >= 3.4e38:
                assert norm == math.inf
                norm = want
            limit = float(torch.tensor(limit))        # as fp32 takes it
            check(G, limit, norm if norm > 1e-36 else want, C)


def test_mixed_magnitudes():
    """One large value among small ones, and the other way round, in one thread's piece."""
    g = torch.full((9000,), 1e-25)
    g[4000] = 1e22
    h = torch.full((9000,), 1e-30)
    h[5] = 1e-21
    for t in (g, h):
        norm, C = run([t], exact_norm([t]) * 0.5)
        check([t], float(torch.tensor(exact_norm([t]) * 0.5)), norm, C)


def test_nonfinite_values():
    G = make([5000, 300], ["f32", "bf16"])
    G[1][7] = float("nan")
    norm, C = run(G, 1.0)
    assert math.isnan(norm) and all(c.isnan().all() for c in C)
    G[1][7] = float("inf")
    norm, C = run(G, 1.0)
    assert norm == math.inf
    assert (C[0] == 0).all() and C[1][7].isnan() and (C[1][:7] == 0).all() and (C[1][8:] == 0).all()
    norm, C = run(G, math.inf)
    assert norm == math.inf and torch.equal(C[0], G[0]) and torch.equal(C[1], G[1])
    norm, C = run(make([5000], ["f32"]), 0.0)
    assert norm > 0 and (C[0] == 0).all()
    norm, C = run([torch.zeros(100)], 0.0)
    assert norm == 0 and (C[0] == 0).all()


def test_replays_follow_the_inputs():
    G = [g.cuda() for g in make([50001, 900, 3], ["f32", "bf16"])]
    C = [torch.empty_like(g) for g in G]
    norms = torch.empty(2, device="cuda")
    work = [torch.empty(gemm.GEMM_CLIP_WORKSPACE, dtype=torch.uint8, device="cuda") for _ in range(2)]
    kinds = ["f32", "bf16", "f32"]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        tensors = gemm.clip_tensors(list(zip(G, C, kinds)))
        gemm.gemm_clip_run(tensors, 0.5, norms[:1], work[0], stream=stream)
        again = gemm.clip_tensors([(c, c, k) for c, k in zip(C, kinds)])
        gemm.gemm_clip_run(again, 0.25, norms[1:], work[1], stream=stream)
        del tensors, again                            # the list is read before the call returns
    for seed in (1, 2):
        new = make([50001, 900, 3], ["f32", "bf16"], seed=seed)
        for g, n in zip(G, new):
            g.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        want = exact_norm(new)
        assert abs(float(norms[0]) - want) <= NORM_REL * want
        assert abs(float(norms[1]) - 0.5) <= 2.0 ** -9 * 0.5      # the bf16 tensor is rounded in between
        check([c.cpu() for c in C], 1.0, exact_norm(C), [c.cpu() for c in C])
        assert abs(exact_norm(C) - 0.25) <= 2.0 ** -8 * 0.25
