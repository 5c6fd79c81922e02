"""gemm_gated_run and gemm_gated_back_run against their definitions in 64 bits."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import gatedref as gr
from tests import opsref as ref
from tests.test_norm_gpu import guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ONE, TWO = gemm.GEMM_FLAG_FORCE_1CTA, gemm.GEMM_FLAG_FORCE_2CTA


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def operands(M, F, K, kind, seed=0):
    gen = torch.Generator().manual_seed(seed + 7 * M + F + K)
    x = torch.randn(M, K, generator=gen)
    x[:, ::37] *= 8
    w = torch.randn(2 * F, K, generator=gen) * K ** -0.5
    return gr.rounded(x, kind), gr.rounded(w, kind)


def dev(t):
    return None if t is None else t.cuda()


class Out:
    def __init__(self, M, F, a, keep):
        n = ref.blocks(F)
        self.A, a_ok = guarded((M, F), gr.TORCH[a])
        self.SFA, s_ok = guarded((M, n), torch.uint8) if a == "e4m3" else (None, lambda: True)
        self.CK, c_ok = guarded((M, 2 * F), torch.uint8) if keep else (None, lambda: True)
        self.SFCK, k_ok = guarded((M, 2 * n), torch.uint8) if keep else (None, lambda: True)
        self.intact = lambda: a_ok() and s_ok() and c_ok() and k_ok()


def forward(plan, X, W, out, stream=None):
    torch.cuda.synchronize()
    plan.run(X[0], W[0], out.A, X[1], W[1], out.SFA, out.CK, out.SFCK, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert plan.last_status() == gemm.GEMM_OK
    assert out.intact()


def check(out, x, w, a, keep):
    F = w.shape[0] // 2
    g, u, want, tg, tu, ta = gr.gated(x, w)
    gr.assert_output("a", out.A, out.SFA, want, ta, a)
    if keep:
        n = ref.blocks(F)
        gr.assert_output("g", out.CK[:, :F], out.SFCK[:, :n], g, tg, "e4m3")
        gr.assert_output("u", out.CK[:, F:], out.SFCK[:, n:], u, tu, "e4m3")


def scaled(kind):
    return gemm.GEMM_SCALE_UE8M0_32 if kind == "e4m3" else 0


SHAPES = [(1, 16, 16), (3, 48, 80), (130, 144, 208), (257, 1040, 272), (333, 528, 2064)]


@pytest.mark.parametrize("flags", [0, ONE, TWO])
@pytest.mark.parametrize("a", ["e4m3", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("M,F,K", SHAPES)
def test_forward(M, F, K, kind, a, flags):
    (X, SX, x), (W, SW, w) = operands(M, F, K, kind)
    keep = a != "f16"
    out = Out(M, F, a, keep)
    with gemm.GatedPlan(M, F, K, kind, a, scaled(kind), flags) as plan:
        assert flags == 0 or plan.info["cta_group"] == (1 if flags == ONE else 2)
        forward(plan, (dev(X), dev(SX)), (dev(W), dev(SW)), out)
        check(out, x, w, a, keep)


@pytest.mark.parametrize("K", [8, 72])
def test_rows_of_eight_elements(K):
    """16-bit rows whose length is no multiple of anything but a copy's 16 bytes."""
    (X, _, x), (W, _, w) = operands(200, 32, K, "bf16")
    out = Out(200, 32, "bf16", True)
    with gemm.GatedPlan(200, 32, K, "bf16", "bf16") as plan:
        forward(plan, (dev(X), None), (dev(W), None), out)
    check(out, x, w, "bf16", True)


@pytest.mark.parametrize("flags", [ONE, TWO])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_more_tiles_than_run_at_once(kind, flags):
    M, F, K = 2053, 1168, 144
    (X, SX, x), (W, SW, w) = operands(M, F, K, kind)
    out = Out(M, F, "e4m3", True)
    with gemm.GatedPlan(M, F, K, kind, "e4m3", scaled(kind), flags) as plan:
        assert plan.info["tiles"] * plan.info["cta_group"] > plan.info["grid"]
        forward(plan, (dev(X), dev(SX)), (dev(W), dev(SW)), out)
    check(out, x, w, "e4m3", True)


@pytest.mark.parametrize("flags", [ONE, TWO])
def test_nonfinite_rows_stay_their_own(flags):
    M, F, K = 300, 96, 64
    (X, _, x), (W, _, w) = operands(M, F, K, "bf16")
    plain, odd = Out(M, F, "bf16", True), Out(M, F, "bf16", True)
    with gemm.GatedPlan(M, F, K, "bf16", "bf16", 0, flags) as plan:
        forward(plan, (dev(X), None), (dev(W), None), plain)
        X[7, 3] = float("nan")
        X[131, 5] = float("inf")
        forward(plan, (dev(X), None), (dev(W), None), odd)
    keep = torch.ones(M, dtype=torch.bool)
    keep[[7, 131]] = False
    for name in ("A", "CK", "SFCK"):
        assert torch.equal(getattr(plain, name).cpu()[keep], getattr(odd, name).cpu()[keep])
    assert odd.A[7].isnan().all() and not odd.A[131].isfinite().any()
    assert ((odd.CK[7] & 127) == 127).all()
    g = x[131].clone()
    g[5] = 0
    # x·w with one infinite term: infinite, with the weight's sign (no weight is zero)
    sign = torch.sign(w[:, 5])
    kept = ref.decode_e4m3(odd.CK[131:132]) * torch.cat([ref.spread(odd.SFCK[131:132, :3].cpu(), F),
                                                         ref.spread(odd.SFCK[131:132, 3:].cpu(), F)], 1)
    assert torch.equal(torch.sign(kept[0]), sign) and kept.float().isinf().all()


def test_runs_do_not_depend_on_timing_and_follow_the_stream():
    """The same bits from run to run, on another stream, with other pointers, and from a captured graph replayed on new inputs."""
    M, F, K = 1500, 784, 528
    (X, SX, x), (W, SW, w) = operands(M, F, K, "e4m3")
    X, SX, W, SW = (dev(t) for t in (X, SX, W, SW))
    first, other = Out(M, F, "e4m3", True), Out(M, F, "e4m3", True)
    with gemm.GatedPlan(M, F, K, "e4m3", "e4m3", 1) as plan:
        forward(plan, (X, SX), (W, SW), first)
        check(first, x, w, "e4m3", True)
        side = torch.cuda.Stream()
        forward(plan, (X.clone(), SX.clone()), (W.clone(), SW.clone()), other, side)
        names = ("A", "SFA", "CK", "SFCK")
        assert all(torch.equal(getattr(first, n).view(torch.uint8), getattr(other, n).view(torch.uint8)) for n in names)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.run(X, W, other.A, SX, SW, other.SFA, other.CK, other.SFCK, side)
            plan.run(X, W, other.A, SX, SW, other.SFA, other.CK, other.SFCK, side)
        (X2, SX2, x2), _ = operands(M, F, K, "e4m3", seed=5)
        X.copy_(X2)
        SX.copy_(SX2)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        check(other, x2, w, "e4m3", True)
        assert plan.last_status() == gemm.GEMM_OK


@pytest.mark.parametrize("flags", [ONE, TWO])
@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_a_wait_that_runs_out_is_reported(kind, flags):
    M, F, K = 600, 272, 256
    (X, SX, x), (W, SW, w) = operands(M, F, K, kind)
    X, SX, W, SW = (dev(t) for t in (X, SX, W, SW))
    out = Out(M, F, "bf16", False)
    with gemm.GatedPlan(M, F, K, kind, "bf16", scaled(kind), flags) as plan:
        plan.set_timeout(2_000_000)
        gemm.gemm_testing_set_fault(plan.handle, 1)
        plan.run(X, W, out.A, SX, SW, None, None, None, torch.cuda.current_stream())
        assert plan.last_status() == gemm.GEMM_ERR_TIMEOUT
        gemm.gemm_testing_set_fault(plan.handle, 0)
        plan.set_timeout(1_000_000_000)
        forward(plan, (X, SX), (W, SW), out)
    check(out, x, w, "bf16", False)


def test_plans_refuse_what_is_not_theirs():
    X = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(128, 64, dtype=torch.bfloat16, device="cuda")
    u8 = torch.zeros(64, 128, dtype=torch.uint8, device="cuda")

    def status(f, *args):
        with pytest.raises(gemm.GemmError) as e:
            f(*args)
        return e.value.status

    invalid, unsupported, alignment = gemm.GEMM_ERR_INVALID_ARG, gemm.GEMM_ERR_UNSUPPORTED, gemm.GEMM_ERR_ALIGNMENT
    with gemm.GatedPlan(64, 64, 64, "bf16", "e4m3") as plan, gemm.GatedBackPlan(64, 64, 64, "bf16") as back, \
            gemm.Plan(64, 64, 64, "bf16", "bf16") as product, gemm.GatedPlan(64, 64, 64, "e4m3", "bf16", 1) as mx:
        for p in (plan, back):
            assert status(gemm.gemm_run, p.handle, X, W, None, X) == invalid
            assert status(gemm.gemm_run_host, p.handle, X, W, None, X) == invalid
            assert status(gemm.gemm_chain_run, p.handle, X, W, W, None, X) == invalid
            assert status(gemm.gemm_plan_set_split_k, p.handle, 2) == unsupported
            assert status(gemm.gemm_plan_set_stream_k, p.handle, 1) == unsupported
            assert status(gemm.gemm_plan_set_clock_meter, p.handle, 1) == unsupported
            assert status(gemm.gemm_testing_set_fault, p.handle, 2) == invalid
            p.set_split_k(1)
            p.set_stream_k(False)
        assert status(gemm.gemm_gated_run, back.handle, X, W, None, None, X) == invalid
        assert status(gemm.gemm_gated_run, product.handle, X, W, None, None, X) == invalid
        assert status(gemm.gemm_gated_back_run, plan.handle, X, W, u8, u8, W) == invalid
        for X_, W_, A, SFA, CK, SFCK, want in (
                (None, W, u8, u8, u8, u8, invalid), (X, None, u8, u8, u8, u8, invalid), (X, W, None, u8, u8, u8, invalid),
                (X, W, u8, None, u8, u8, invalid), (X, W, u8, u8, u8, None, invalid),
                (X.data_ptr() + 8, W, u8, u8, u8, u8, alignment), (X, W.data_ptr() + 8, u8, u8, u8, u8, alignment),
                (X, W, u8.data_ptr() + 8, u8, u8, u8, alignment), (X, W, u8, u8, u8.data_ptr() + 8, u8, alignment)):
            assert status(gemm.gemm_gated_run, plan.handle, X_, W_, None, None, A, SFA, CK, SFCK) == want
        assert status(gemm.gemm_gated_run, mx.handle, u8, u8, None, u8, X) == invalid
        assert status(gemm.gemm_gated_run, mx.handle, u8, u8, u8, None, X) == invalid
        for i in range(5):
            args = [X, W, u8, u8, W]
            args[i] = None
            assert status(gemm.gemm_gated_back_run, back.handle, *args) == invalid
        for i in (0, 1, 2, 4):
            args = [X, W, u8, u8, W]
            args[i] = args[i].data_ptr() + 8
            assert status(gemm.gemm_gated_back_run, back.handle, *args) == alignment
        assert status(gemm.gemm_gated_back_run, back.handle, X, W, u8, u8, W, X.data_ptr() + 8) == alignment
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------ backward

def checkpoint(M, F, gen):
    z = torch.randn(M, 2 * F, generator=gen) * 2
    halves = [gr.rounded(z[:, :F], "e4m3"), gr.rounded(z[:, F:], "e4m3")]
    return (torch.cat([h[0].view(torch.uint8) for h in halves], 1), torch.cat([h[1] for h in halves], 1),
            halves[0][2], halves[1][2])


def backward_case(M, F, N, kind, seed=0):
    gen = torch.Generator().manual_seed(seed + M + 3 * F + N)
    DY = (torch.randn(M, N, generator=gen) * 0.1).to(gr.TORCH[kind])
    W2 = (torch.randn(N, F, generator=gen) * N ** -0.5).to(gr.TORCH[kind])
    return DY, W2, checkpoint(M, F, gen)


def backward(plan, DY, W2, CK, SF, M, F, kind, again, stream=None):
    DZ, z_ok = guarded((M, 2 * F), gr.TORCH[kind])
    A, a_ok = guarded((M, F), gr.TORCH[kind]) if again else (None, lambda: True)
    torch.cuda.synchronize()
    plan.run(DY, W2, CK, SF, DZ, A, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert plan.last_status() == gemm.GEMM_OK and z_ok() and a_ok()
    return DZ, A


def check_backward(DZ, A, DY, W2, g, u, kind):
    da, size = gr.product(DY.double(), W2.double().t())
    tol = gr.SUM * size + 1e-37
    dg, du, a, dg_tol, du_tol, rel = ref.gate_back(g, u, da)
    s = torch.sigmoid(g)
    dg_tol = dg_tol + tol * (u * s * (1 + g * torch.sigmoid(-g))).abs()
    du_tol = du_tol + tol * (g * s).abs()
    F = g.shape[1]
    gr.assert_output("dg", DZ[:, :F], None, dg, dg_tol, kind)
    gr.assert_output("du", DZ[:, F:], None, du, du_tol, kind)
    if A is not None:
        gr.assert_output("a", A, None, a, rel * a.abs(), kind)


@pytest.mark.parametrize("flags", [0, ONE, TWO])
@pytest.mark.parametrize("kind,again", [("bf16", True), ("f16", False)])
@pytest.mark.parametrize("M,F,N", [(1, 16, 8), (3, 48, 72), (130, 144, 200), (257, 1040, 264), (333, 528, 2056),
                                   (2053, 1168, 136)])
def test_backward(M, F, N, kind, again, flags):
    DY, W2, (CK, SF, g, u) = backward_case(M, F, N, kind)
    with gemm.GatedBackPlan(M, F, N, kind, flags) as plan:
        DZ, A = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, kind, again)
        check_backward(DZ, A, DY, W2, g, u, kind)
        # the same bits without a, on another stream
        DZ2, _ = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, kind, False, torch.cuda.Stream())
        assert torch.equal(DZ, DZ2)


def test_backward_nonfinite_values_stay_their_own():
    M, F, N = 140, 64, 64
    DY, W2, (CK, SF, g, u) = backward_case(M, F, N, "bf16")
    DY[5, 9] = float("nan")
    CK[20, 3] = 127                                   # a NaN code: its own g alone
    with gemm.GatedBackPlan(M, F, N, "bf16") as plan:
        DZ, A = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, "bf16", True)
    bad = DZ.isnan().cpu()
    want = torch.zeros_like(bad)
    want[5] = True
    want[20, 3] = want[20, F + 3] = True
    assert torch.equal(bad, want)
    assert A.isnan().cpu().nonzero().tolist() == [[20, 3]]


def test_gradients_agree_with_differences():
    """dz, through the two plain products, against differences of the forward definition at the checkpoint."""
    M, F, N = 64, 32, 64
    DY, W2, (CK, SF, g, u) = backward_case(M, F, N, "bf16")
    with gemm.GatedBackPlan(M, F, N, "bf16") as plan:
        DZ, _ = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, "bf16", False)
    loss = lambda g, u: (ref.gate(g, u) @ W2.double().t() * DY.double()).sum()
    step = 1e-6
    for i, j in ((0, 0), (5, 7), (63, 31), (30, 16)):
        for half, base in ((0, g), (1, u)):
            move = torch.zeros_like(base)
            move[i, j] = step
            args = [(g + move, u), (g - move, u)] if half == 0 else [(g, u + move), (g, u - move)]
            want = (loss(*args[0]) - loss(*args[1])) / (2 * step)
            got = float(DZ[i, half * F + j])
            # bf16's half step and the sums' bound; the differences are exact to 1e-8 of the terms
            size = float((DY[i].double().abs() @ W2.double().abs()[:, j]) * max(1.0, abs(u[i, j]), abs(g[i, j])) * 1.1)
            assert abs(got - want) <= 2.0 ** -8 * abs(want) + 2e-5 * size + 1e-7


def test_backward_wait_that_runs_out_is_reported():
    M, F, N = 600, 272, 256
    DY, W2, (CK, SF, g, u) = backward_case(M, F, N, "bf16")
    args = [dev(t) for t in (DY, W2, CK, SF)]
    for flags in (ONE, TWO):
        with gemm.GatedBackPlan(M, F, N, "bf16", flags) as plan:
            plan.set_timeout(2_000_000)
            gemm.gemm_testing_set_fault(plan.handle, 1)
            DZ = torch.empty(M, 2 * F, dtype=torch.bfloat16, device="cuda")
            plan.run(*args, DZ, None, torch.cuda.current_stream())
            assert plan.last_status() == gemm.GEMM_ERR_TIMEOUT
            gemm.gemm_testing_set_fault(plan.handle, 0)
            plan.set_timeout(1_000_000_000)
            DZ, _ = backward(plan, *args, M, F, "bf16", False)
            check_backward(DZ, None, DY, W2, g, u, "bf16")


# ------------------------------------------------------------------------------------------- slices of K

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,F,K,slices", [(40, 80, 8256, 8), (300, 144, 4112, 8), (300, 528, 2064, 4),
                                              (129, 1040, 8224, 4), (520, 784, 4176, 2)])
def test_sliced_tiles(M, F, K, kind, slices):
    """Few tiles: K in slices over a cluster's CTAs, whose sums meet before the unit."""
    K = K if kind == "bf16" else 2 * K
    (X, SX, x), (W, SW, w) = operands(M, F, K, kind)
    out, again = Out(M, F, "e4m3", True), Out(M, F, "e4m3", True)
    with gemm.GatedPlan(M, F, K, kind, "e4m3", scaled(kind)) as plan:
        assert plan.info["splits"] == slices and plan.info["cta_group"] == 1
        forward(plan, (dev(X), dev(SX)), (dev(W), dev(SW)), out)
        forward(plan, (dev(X), dev(SX)), (dev(W), dev(SW)), again)
    check(out, x, w, "e4m3", True)
    for name in ("A", "SFA", "CK", "SFCK"):           # added in a fixed order
        assert torch.equal(getattr(out, name).view(torch.uint8), getattr(again, name).view(torch.uint8))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,F,N,slices", [(40, 80, 8200, 8), (300, 272, 4104, 8), (300, 1040, 4104, 4),
                                              (129, 2064, 8232, 4), (520, 1552, 4176, 2), (520, 1552, 4160, 1),
                                              (300, 528, 8200, 8), (200, 1040, 4096, 4), (256, 2048, 2048, 2),
                                              (33, 528, 3000, 4)])
def test_sliced_backward(M, F, N, kind, slices):
    DY, W2, (CK, SF, g, u) = backward_case(M, F, N, kind)
    with gemm.GatedBackPlan(M, F, N, kind) as plan:
        assert plan.info["splits"] == slices
        DZ, A = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, kind, True)
        check_backward(DZ, A, DY, W2, g, u, kind)
        assert torch.equal(DZ, backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, kind, False)[0])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "back"])
def test_sliced_wait_that_runs_out_is_reported(kind):
    M, F, K = 200, 80, 8192
    if kind == "back":
        DY, W2, (CK, SF, g, u) = backward_case(M, F, K, "bf16")
        args = [dev(t) for t in (DY, W2, CK, SF)]
        plan = gemm.GatedBackPlan(M, F, K)
        run = lambda: plan.run(*args, torch.empty(M, 2 * F, dtype=torch.bfloat16, device="cuda"), None,
                               torch.cuda.current_stream())
    else:
        (X, SX, x), (W, SW, w) = operands(M, F, K, kind)
        X, SX, W, SW = (dev(t) for t in (X, SX, W, SW))
        out = Out(M, F, "bf16", False)
        plan = gemm.GatedPlan(M, F, K, kind, "bf16", scaled(kind))
        run = lambda: plan.run(X, W, out.A, SX, SW, stream=torch.cuda.current_stream())
    with plan:
        assert plan.info["splits"] > 1
        plan.set_timeout(2_000_000)
        gemm.gemm_testing_set_fault(plan.handle, 1)
        run()
        assert plan.last_status() == gemm.GEMM_ERR_TIMEOUT
        gemm.gemm_testing_set_fault(plan.handle, 0)
        plan.set_timeout(1_000_000_000)
        run()
        assert plan.last_status() == gemm.GEMM_OK
    if kind != "back":
        check(out, x, w, "bf16", False)


def test_scales_that_begin_anywhere():
    """The same bits whether the scales' rows are read as they are or packed first."""
    M, F, K = 100, 208, 1536
    (X, SX, x), (W, SW, w) = operands(M, F, K, "e4m3")
    X, SX, W, SW = (dev(t) for t in (X, SX, W, SW))
    outs = [Out(M, F, "e4m3", True) for _ in range(3)]

    def shifted(t, n):
        b = torch.empty(t.numel() + n, dtype=torch.uint8, device="cuda")
        b[n:] = t.view(-1)
        return b[n:]

    with gemm.GatedPlan(M, F, K, "e4m3", "e4m3", 1, ONE) as plan:
        forward(plan, (X, SX), (W, SW), outs[0])
        forward(plan, (X, shifted(SX, 1)), (W, SW), outs[1])
        forward(plan, (X, SX), (W, shifted(SW, 8)), outs[2])
    check(outs[0], x, w, "e4m3", True)
    for o in outs[1:]:
        for name in ("A", "SFA", "CK", "SFCK"):
            assert torch.equal(getattr(outs[0], name).view(torch.uint8), getattr(o, name).view(torch.uint8))


@pytest.mark.parametrize("M,F,K,kind,flags,launches,slices", [
    (4096, 1024, 512, "bf16", TWO, 1, 1), (4096, 1024, 512, "e4m3", TWO, 2, 1),      # pairs take packed scales
    (128, 256, 512, "e4m3", ONE, 1, 1), (128, 256, 528, "e4m3", ONE, 2, 1),          # 17 codes a row: packed
    (64, 128, 8192, "bf16", ONE, 1, 8), (64, 128, 8192, "e4m3", ONE, 1, 8), (64, 128, 8208, "e4m3", ONE, 2, 8)])
def test_what_a_run_launches(M, F, K, kind, flags, launches, slices):
    with gemm.GatedPlan(M, F, K, kind, "bf16", scaled(kind), flags) as plan:
        assert plan.info["launches_per_run"] == launches and plan.info["splits"] == slices


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,F,N,tile,slices", [(1000, 1296, 72, 128, 1), (520, 1040, 648, 64, 1), (129, 4112, 8, 64, 1),
                                               (64, 16, 1000, 64, 2)])
def test_backward_widths_of_single_tiles(M, F, N, kind, tile, slices):
    """Tiles of 64 columns where all of them run at once, else of 128."""
    DY, W2, (CK, SF, g, u) = backward_case(M, F, N, kind)
    with gemm.GatedBackPlan(M, F, N, kind, ONE) as plan:
        assert (plan.info["tile_n"], plan.info["splits"], plan.info["cta_group"]) == (tile, slices, 1)
        DZ, A = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, kind, True)
        check_backward(DZ, A, DY, W2, g, u, kind)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("K", [48, 64, 80, 128, 144, 192, 208, 400])
def test_few_k_blocks_and_many_tiles_of_single_ctas(K, kind):
    """One k-block to several, an odd and an even number, over several tiles of each CTA."""
    M, F = 1100, 2080
    (X, SX, x), (W, SW, w) = operands(M, F, K, kind)
    out = Out(M, F, "bf16", False)
    with gemm.GatedPlan(M, F, K, kind, "bf16", scaled(kind), ONE) as plan:
        assert plan.info["tiles"] > 152
        forward(plan, (dev(X), dev(SX)), (dev(W), dev(SW)), out)
    check(out, x, w, "bf16", False)
    if kind == "bf16":
        DY, W2, (CK, SF, g, u) = backward_case(M, F, K, kind)
        with gemm.GatedBackPlan(M, F, K, kind, ONE) as plan:
            DZ, A = backward(plan, dev(DY), dev(W2), dev(CK), dev(SF), M, F, kind, True)
            check_backward(DZ, A, DY, W2, g, u, kind)
