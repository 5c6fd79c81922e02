"""Calls of the gated product that its documentation allows and that are not everyday ones: plans that wait for their runs, scale codes at
any address, one plan's runs one behind the other."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import gatedref as gr
from tests import opsref as ref
from tests.test_gated_gpu import ONE, TWO, Out, check, dev, operands, scaled
from tests.test_gated_matvec_gpu import case
from tests.test_gated_matvec_gpu import check as check_few
from tests.test_gated_matvec_gpu import run as few

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def shifted(t, n):
    """t at an address that is n bytes past a multiple of 16."""
    b = torch.full((t.numel() + n,), 0xA5, dtype=torch.uint8, device="cuda")
    b[n:] = t.reshape(-1).cuda()
    return b[n:].view(t.shape)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_plans_that_wait(kind):
    M, F, K = 200, 208, 528
    (X, SX, x), (W, SW, w) = operands(M, F, K, kind)
    out = Out(M, F, "bf16", True)
    with gemm.GatedPlan(M, F, K, kind, "bf16", scaled(kind), gemm.GEMM_FLAG_SYNC) as plan:
        assert plan.run(dev(X), dev(W), out.A, dev(SX), dev(SW), None, out.CK, out.SFCK, torch.cuda.Stream()) == gemm.GEMM_OK
        check(out, x, w, "bf16", True)               # no other wait
        plan.set_timeout(2_000_000)
        gemm.gemm_testing_set_fault(plan.handle, 1)
        with pytest.raises(gemm.GemmError) as e:
            plan.run(dev(X), dev(W), out.A, dev(SX), dev(SW), None, out.CK, out.SFCK, torch.cuda.current_stream())
        assert e.value.status == gemm.GEMM_ERR_TIMEOUT and plan.last_status() == gemm.GEMM_OK


@pytest.mark.parametrize("flags", [ONE, TWO])
@pytest.mark.parametrize("n", [1, 2, 4, 8, 15])
def test_scale_codes_anywhere(n, flags):
    """Scale codes in and out begin at any byte."""
    M, F, K = 150, 144, 1024
    (X, SX, x), (W, SW, w) = operands(M, F, K, "e4m3")
    out = Out(M, F, "e4m3", True)
    pool = [torch.full((t.numel() + 64,), 0xA5, dtype=torch.uint8, device="cuda") for t in (out.SFA, out.SFCK)]
    places = [p[16 + n:16 + n + t.numel()].view(t.shape) for p, t in zip(pool, (out.SFA, out.SFCK))]
    with gemm.GatedPlan(M, F, K, "e4m3", "e4m3", 1, flags) as plan:
        plan.run(dev(X), dev(W), out.A, shifted(SX, n), shifted(SW, 16 - n), places[0], out.CK, places[1],
                 torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert plan.last_status() == gemm.GEMM_OK
    for p, t in zip(pool, (out.SFA, out.SFCK)):
        assert (p[:16 + n] == 0xA5).all() and (p[16 + n + t.numel():] == 0xA5).all()
    out.SFA.copy_(places[0])
    out.SFCK.copy_(places[1])
    check(out, x, w, "e4m3", True)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 12])
@pytest.mark.parametrize("M", [3, 12])
def test_few_rows_scale_codes_anywhere(M, n):
    for K in (512, 528):
        F = 136
        X, (W, SF, wide) = case(M, F, K, "bf16", "e4m3")
        A = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
        gemm.gemm_gated_matvec_run(M, F, K, "bf16", "e4m3", "bf16", dev(X), dev(W), shifted(SF, n), A, torch.cuda.current_stream())
        torch.cuda.synchronize()
        check_few(A.cpu(), X, wide, "bf16")


@pytest.mark.parametrize("K", [528, 1024, 8208])
def test_a_plans_runs_one_behind_the_other(K):
    """Packed scales lie in memory of the plan's own: a run packs its own only when the run before has read its."""
    M, F, runs = 100, 208, 12
    ins = [operands(M, F, K, "e4m3", seed=i) for i in range(3)]
    outs = [Out(M, F, "bf16", False) for _ in range(runs)]
    ready = [[dev(t) for t in (X, SX, W, SW)] for (X, SX, _), (W, SW, _) in ins]
    torch.cuda.synchronize()
    with gemm.GatedPlan(M, F, K, "e4m3", "bf16", 1) as plan:
        for i, out in enumerate(outs):
            X, SX, W, SW = ready[i % 3]
            plan.run(X, W, out.A, SX, SW, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert plan.last_status() == gemm.GEMM_OK
    for i, out in enumerate(outs):
        assert out.intact() and torch.equal(out.A, outs[i % 3].A)
        if i < 3:
            check(out, ins[i][0][2], ins[i][1][2], "bf16", False)


def test_operands_written_just_before():
    """Each kernel reads what the one before it in the stream writes, without a wait between: norm, gated product, its gradient, a
    token's form, and the clipping of what they leave."""
    M, F, K = 96, 272, 512
    gen = torch.Generator().manual_seed(3)
    (_, _, _), (W, SW, w) = operands(M, F, K, "e4m3")
    W, SW = dev(W), dev(SW)
    norm_w = torch.ones(K, device="cuda")
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    n = -(-F // 32)
    hs = [torch.randn(M, K, generator=gen).bfloat16().cuda() for _ in range(6)]

    def chain(h, sync):
        wait = torch.cuda.synchronize if sync else (lambda: None)
        s = torch.cuda.current_stream()
        y, sfy, y16, a, ck, sfck = u8(M, K), u8(M, K // 32), bf(16, K), bf(M, F), u8(M, 2 * F), u8(M, 2 * n)
        dz, few, total, work = bf(M, 2 * F), bf(16, F), torch.empty(1, device="cuda"), u8(gemm.GEMM_CLIP_WORKSPACE)
        c = bf(M, 2 * F)
        gemm.gemm_norm_run(M, K, "bf16", "bf16", "e4m3", 1e-6, h, None, norm_w, None, y, sfy, None, s)
        wait()
        plan.run(y, W, a, sfy, SW, None, ck, sfck, s)
        wait()
        back.run(h, w2, ck, sfck, dz, None, s)
        wait()
        gemm.gemm_clip_run(gemm.clip_tensors([(dz, c, "bf16")]), 1.0, total, work, stream=s)
        wait()
        gemm.gemm_norm_run(16, K, "bf16", "bf16", "bf16", 1e-6, h, None, norm_w, None, y16, None, None, s)
        wait()
        gemm.gemm_gated_matvec_run(16, F, K, "bf16", "e4m3", "bf16", y16, W, SW, few, s)
        wait()
        return y, sfy, a, ck, sfck, dz, c, total, few

    w2 = (torch.randn(K, F, generator=gen) * K ** -0.5).bfloat16().cuda()
    with gemm.GatedPlan(M, F, K, "e4m3", "bf16", 1, ONE) as plan, gemm.GatedBackPlan(M, F, K) as back:
        assert plan.info["launches_per_run"] == 1    # scales read as they are
        apart = [chain(h, True) for h in hs]
        together = [chain(h, False) for h in hs]
        torch.cuda.synchronize()
        assert plan.last_status() == back.last_status() == gemm.GEMM_OK
    for x, y in zip(apart, together):
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(x, y))


@pytest.mark.parametrize("M", [2, 11])
@pytest.mark.parametrize("x_scale,low,high", [(2.0 ** -105, 225, 247), (2.0 ** -90, 240, 247), (2.0 ** 110, 10, 24), (2.0 ** 122, 0, 6)])
def test_few_rows_at_the_ends_of_the_weights(x_scale, low, high, M):
    """e4m3 weights up to fp32's largest and down to its smallest against bf16 activations that bring them to ordinary numbers."""
    F, K = 24, 640
    gen = torch.Generator().manual_seed(low)
    W = torch.randint(0, 256, (2 * F, K), generator=gen, dtype=torch.uint8)
    W[(W & 127) == 127] = 126
    SF = torch.randint(low, high + 1, (2 * F, K // 32), generator=gen, dtype=torch.uint8)
    wide = ref.decode_e4m3(W) * ref.spread(SF, K)
    wide = torch.where(wide.abs() > float(torch.finfo(torch.float32).max), 0.0, wide)
    W[wide == 0] = 0
    X = (torch.randn(M, K, generator=gen).double() * x_scale * torch.exp2(-torch.arange(M).double())[:, None]).to(torch.bfloat16)
    g, u, want, _, _, tol = gr.gated(X.double(), wide)
    A = few(M, F, K, "bf16", "e4m3", X, W, SF)
    # off by 2^-39 of the largest of a token's 128 k, times the weights there, and for each of their four blocks by 2^-142 of it
    most = torch.stack([c.abs().amax(1) for c in X.double().split(128, 1)], 1)
    heavy = torch.stack([c.abs().sum(1) for c in wide.split(128, 1)], 1)
    lost = most @ (heavy.t() * 2.0 ** -39 + 4 * 2.0 ** -142)
    tol = tol + 1.2 * (lost[:, :F] * (u.abs() + lost[:, F:]) + lost[:, F:] * g.abs()) + 1e-42
    assert want.isfinite().all() and want.abs().max() < 3e38
    gr.assert_output("a", A, None, want, tol, "bf16")
