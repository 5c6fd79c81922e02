"""gemm_matvec_run against its definition in 64 bits, under the products' accept rule
|D - D_ref| <= 1e-5 sum |x w| + 1e-6 |c| (+ 1 bf16 ulp for bf16 D)."""
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


def make(M, N, K, x, mode, seed=0, c=False, low=120, high=134):
    gen = torch.Generator().manual_seed(seed)
    X = (torch.randn(M, K, generator=gen)).to(ref.TORCH[x])
    B = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8)
    if mode == 1:
        SFB = torch.randint(low, high, (N, K // 32), generator=gen, dtype=torch.uint8)
    else:
        SFB = torch.randint(0, 127, (N, K // 16), generator=gen, dtype=torch.uint8)
    C = torch.randn(M, N, generator=gen) * 10 if c else None
    return X, B, SFB, C


def run(M, N, K, x, d, mode, X, B, SFB, C, stream=None):
    D, ok = guarded((M, N), ref.TORCH[d])
    X, B, SFB = X.cuda(), B.cuda(), SFB.cuda()
    C = None if C is None else C.cuda()
    torch.cuda.synchronize()
    gemm.gemm_matvec_run(M, N, K, x, d, mode, X, B, SFB, C, D, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert ok()
    return D


def check(D, d, X, B, SFB, mode, C):
    want, size = ref.matvec(X, B, SFB, mode, C)
    tol = 1e-5 * size + (0 if C is None else 1e-6 * C.double().abs())
    if d == "bf16":
        tol = tol + 2 * ref.half_ulp(want, "bf16")
    ref.assert_within("d", D, want, tol)


SHAPES = [(1, 1, 32), (1, 16, 32), (2, 17, 64), (3, 33, 96), (1, 256, 128), (4, 100, 160), (5, 1000, 2080), (8, 513, 4096),
          (7, 40, 1056), (9, 130, 288), (16, 300, 8192), (13, 64, 544), (1, 2000, 4096), (11, 5, 32768), (16, 2048, 4128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("mode", [gemm.GEMM_SCALE_UE8M0_32, gemm.GEMM_SCALE_UE4M3_16])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_product(M, N, K, mode, x):
    d = "bf16" if (N + K // 32) % 2 else "f32"
    t = make(M, N, K, x, mode, seed=M + N + K, c=M % 2 == 1)
    check(run(M, N, K, x, d, mode, *t), d, t[0], t[1], t[2], mode, t[3])


# more columns than run at once, K cut over warps and over clusters, activations past one pass
@pytest.mark.parametrize("M,N,K,mode", [(1, 40000, 512, 2), (1, 6001, 16384, 1), (2, 30000, 1056, 1), (3, 9000, 8192, 2), (4, 20000, 4096, 1),
                                        (5, 30000, 2080, 1), (8, 12000, 6144, 2), (8, 1500, 32768, 2), (16, 20000, 2048, 1),
                                        (12, 6000, 8224, 2), (16, 700, 32768, 1), (9, 300, 32736, 2)])
def test_many_columns(M, N, K, mode):
    t = make(M, N, K, "bf16", mode, seed=M + N + K, c=True)
    check(run(M, N, K, "bf16", "f32", mode, *t), "f32", t[0], t[1], t[2], mode, t[3])


@pytest.mark.parametrize("M", range(1, 17))
def test_every_row_count(M):
    for mode in (1, 2):
        t = make(M, 72, 416, "bf16", mode, seed=M, c=True)
        check(run(M, 72, 416, "bf16", "f32", mode, *t), "f32", t[0], t[1], t[2], mode, t[3])


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_wide_ranges(x):
    """Scales over all of their range within a row, activations over many magnitudes, rows of zeros: sums
    are fp32's, element by element."""
    M, N, K = 6, 96, 1024
    X, B, SFB, _ = make(M, N, K, x, 1, seed=5, low=60, high=190)
    gen = torch.Generator().manual_seed(6)
    e = torch.randint(-40, 30, (M, K), generator=gen) if x == "bf16" else torch.randint(-20, 9, (M, K), generator=gen)
    X = (X.float() * torch.exp2(e.float())).to(X.dtype)
    X[4] = 0
    SFB[7] = 0
    SFB[8] = 254
    B[8] = 0
    B[9] = 0
    check(run(M, N, K, x, "f32", 1, X, B, SFB, None), "f32", X, B, SFB, 1, None)


def test_huge_activations_under_tiny_scales():
    """Products that pass fp32's ends on the way come out at their value."""
    M, N, K = 2, 40, 320
    X, B, SFB, _ = make(M, N, K, "bf16", 1, seed=9, low=5, high=12)
    X = (X.float().sign() * 3e38).bfloat16()
    X[1] = X[1] * 2.0 ** -60
    check(run(M, N, K, "bf16", "f32", 1, X, B, SFB, None), "f32", X, B, SFB, 1, None)


def test_outlier_under_a_zero_weight():
    """An activation 2^60 above the others whose weight is zero leaves the others' sum as it is."""
    M, N, K = 2, 32, 256
    X, B, SFB, _ = make(M, N, K, "bf16", 1, seed=8)
    X[:, 100] = 2.0 ** 60
    B[:, 50] &= 0xF0
    check(run(M, N, K, "bf16", "f32", 1, X, B, SFB, None), "f32", X, B, SFB, 1, None)


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("mode", [1, 2])
def test_nonfinite_values(x, mode):
    """Infinity and NaN reach the outputs that take them and no others."""
    M, N, K = 3, 48, 320
    X, B, SFB, _ = make(M, N, K, x, mode, seed=2)
    X[0, 7] = float("inf")
    X[1, 200] = float("nan")
    B[:, 3] = (B[:, 3] & 0x0F) | 0x50            # k = 7 times 3
    B[5, 3] &= 0x0F                              # infinity times zero
    SFB[:, 0] = 120 if mode == 1 else 56
    D = run(M, N, K, x, "f32", mode, X, B, SFB, None).cpu()
    assert D[1].isnan().all() and D[0, 5].isnan()
    other = torch.arange(N) != 5
    assert (D[0][other] == float("inf")).all()
    want, size = ref.matvec(X[2:], B, SFB, mode)
    ref.assert_within("finite row", D[2:], want, 1e-5 * size)


def test_nan_scale():
    M, N, K = 2, 40, 256
    X, B, SFB, _ = make(M, N, K, "bf16", 1, seed=3)
    SFB[11, 5] = 255
    D = run(M, N, K, "bf16", "f32", 1, X, B, SFB, None).cpu()
    assert D[:, 11].isnan().all()
    rest = torch.arange(N) != 11
    assert D[:, rest].isfinite().all()


def test_same_values_as_the_plan():
    """The block-scaled plan and the matrix-vector product on the same buffers: activations that are e2m1
    values with scale 1 are the same operand in both."""
    M, N, K = 8, 256, 512
    _, B, SFB, C = make(M, N, K, "bf16", 1, seed=12, c=True)
    gen = torch.Generator().manual_seed(13)
    A = torch.randint(0, 256, (M, K // 2), generator=gen, dtype=torch.uint8)
    ones = torch.full((M, K // 32), 127, dtype=torch.uint8)
    X = ref.weights(A, ones, 1).bfloat16()
    got = run(M, N, K, "bf16", "f32", 1, X, B, SFB, C)
    D = torch.empty(M, N, device="cuda")
    with gemm.Plan(M, N, K, "e2m1", "f32", gemm.GEMM_SCALE_UE8M0_32) as plan:
        plan.run(A.cuda(), B.cuda(), C.cuda(), D, ones.cuda(), SFB.cuda(), torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert plan.last_status() == gemm.GEMM_OK
    _, size = ref.matvec(X, B, SFB, 1, C)
    ref.assert_within("plan", got, D.cpu().double(), 2e-5 * size + 2e-6 * C.double().abs())


def test_repeatable_on_another_stream_and_in_a_graph():
    M, N, K = 4, 1500, 3104
    t = make(M, N, K, "bf16", 2, seed=4, c=True)
    D = run(M, N, K, "bf16", "f32", 2, *t)
    s = torch.cuda.Stream()
    assert torch.equal(run(M, N, K, "bf16", "f32", 2, *t, stream=s), D)
    X, B, SFB, C = (v.cuda() for v in t)
    out = torch.zeros_like(D)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        gemm.gemm_matvec_run(M, N, K, "bf16", "f32", 2, X, B, SFB, C, out, s)
        g.capture_end()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, D)


def test_weights_past_four_gigabytes():
    M, N, K = 2, 270000, 32768
    B = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda").fill_(0)
    SFB = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    X, tail, sf, _ = make(M, 20, K, "bf16", 1, seed=7)
    B[-20:] = tail.cuda()
    SFB[-20:] = sf.cuda()
    D = torch.empty(M, N, device="cuda")
    gemm.gemm_matvec_run(M, N, K, "bf16", "f32", 1, X.cuda(), B, SFB, None, D, torch.cuda.current_stream())
    torch.cuda.synchronize()
    check(D[:, -20:], "f32", X, tail, sf, 1, None)
    assert float(D[:, :-20].abs().max()) == 0
