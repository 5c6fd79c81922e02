"""gemm_matvec_run on activations of very different magnitudes within a chunk of K, as a gated unit makes them."""
import statistics

import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref
from tests.test_matvec_gpu import check, make, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def gated(M, K, deviation, seed):
    gen = torch.Generator().manual_seed(seed)
    g, u = (torch.randn(M, K, generator=gen) * deviation for _ in range(2))
    return (g * torch.sigmoid(g) * u).bfloat16()


@pytest.mark.parametrize("deviation", [4, 8, 30])
@pytest.mark.parametrize("mode", [gemm.GEMM_SCALE_UE8M0_32, gemm.GEMM_SCALE_UE4M3_16])
@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (2, 77, 1056), (3, 50, 8192), (5, 130, 2080), (8, 48, 4096), (13, 40, 544),
                                   (16, 300, 2048)])
def test_gated_activations(M, N, K, mode, deviation):
    _, B, SFB, C = make(M, N, K, "bf16", mode, seed=M + N, c=True)
    X = gated(M, K, deviation, seed=K)
    check(run(M, N, K, "bf16", "f32", mode, X, B, SFB, C), "f32", X, B, SFB, mode, C)


def one_per_column(K, mode):
    """Weights that are the identity: every output is one activation."""
    B = torch.zeros(K, K // 2, dtype=torch.uint8)
    k = torch.arange(K)
    B[k, k // 2] = torch.where(k % 2 == 0, 0x02, 0x20).to(torch.uint8)           # e2m1's 1
    return B, torch.full((K, K // (32 if mode == 1 else 16)), 127 if mode == 1 else 0x38, dtype=torch.uint8)


# every finite bf16 number, dealt out at random: chunks hold all bands of exponents.  With an odd block at the end too.
@pytest.mark.parametrize("mode", [gemm.GEMM_SCALE_UE8M0_32, gemm.GEMM_SCALE_UE4M3_16])
@pytest.mark.parametrize("M,K", [(16, 4096), (8, 4096), (5, 1056), (4, 4096), (2, 4096), (1, 4096), (1, 2080)])
def test_every_number_comes_out_as_it_is(M, K, mode):
    gen = torch.Generator().manual_seed(M)
    codes = torch.arange(65536)
    codes = codes[(codes & 0x7F80) != 0x7F80][torch.randperm(65280, generator=gen)]
    codes = torch.cat([codes, codes])[:M * K].view(M, K)
    X = torch.where(codes >= 32768, codes - 65536, codes).to(torch.int16).view(torch.bfloat16)
    B, SFB = one_per_column(K, mode)
    D = run(M, K, K, "bf16", "f32", mode, X, B, SFB, None)
    assert torch.equal(D.cpu(), X.float())


@pytest.mark.parametrize("mode", [gemm.GEMM_SCALE_UE8M0_32, gemm.GEMM_SCALE_UE4M3_16])
def test_infinities_among_all_magnitudes(mode):
    """Beside finite values of every band, infinity and NaN reach the outputs that take them."""
    M, K = 2, 512
    B, SFB = one_per_column(K, mode)
    X = (torch.randn(M, K, generator=torch.Generator().manual_seed(1)) * torch.exp2(torch.arange(K) % 240 - 120.0)).bfloat16()
    X[0, 300] = float("-inf")
    X[1, 10] = float("nan")
    D = run(M, K, K, "bf16", "f32", mode, X, B, SFB, None).cpu()
    assert D[0, 300] == float("-inf") and D[0, torch.arange(K) != 300].isnan().all() and D[1].isnan().all()
    B[:, 150] = 0x22                              # every column takes k = 300 (and 301)
    X[1, 10] = 1.0
    D = run(M, K, K, "bf16", "f32", mode, X, B, SFB, None).cpu()
    assert (D[0] == float("-inf")).all() and D[1].isfinite().all()


def test_nan_scale_under_zeros():
    """A NaN scale is NaN whatever it scales."""
    M, N, K = 2, 40, 512
    _, B, SFB, _ = make(M, N, K, "bf16", 1, seed=3)
    X = torch.zeros(M, K).bfloat16()
    SFB[11, 5] = 255
    D = run(M, N, K, "bf16", "f32", 1, X, B, SFB, None).cpu()
    assert D[:, 11].isnan().all() and (D[:, torch.arange(N) != 11] == 0).all()


@pytest.mark.parametrize("M,N,K,mode", [(16, 8192, 8192, 1), (8, 8192, 8192, 2), (4, 8192, 8192, 2), (1, 16384, 8192, 2)])
def test_time_of_gated_activations(M, N, K, mode):
    """Gates far apart cost a small multiple of the ordinary time, not hundreds of times as much."""
    X, B, SFB, _ = make(M, N, K, "bf16", mode, seed=1)
    B, SFB, D = B.cuda(), SFB.cuda(), torch.empty(M, N, device="cuda")
    times = []
    for x in (X.cuda(), gated(M, K, 8, seed=2).cuda()):
        calls = []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                gemm.gemm_matvec_run(M, N, K, "bf16", "f32", mode, x, B, SFB, None, D, torch.cuda.current_stream())
            b.record()
            b.synchronize()
            calls.append(a.elapsed_time(b))
        times.append(statistics.median(calls))
    assert times[1] < 25 * times[0], times
