"""The feed-forward operators one right after another: each may begin while the one before it ends, so that what they
read, write and write again is checked against the same calls with a wait after each, and inside graphs with branches."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


class Block:
    """A feed-forward block of a few rows, forward and backward, on buffers that every step writes anew."""

    def __init__(self, M, K, F):
        gen = torch.Generator().manual_seed(7)
        self.M, self.K, self.F = M, K, F
        new = lambda dtype, *shape: torch.zeros(*shape, dtype=dtype, device="cuda")
        bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        weights = lambda n, k: torch.randint(0, 256, (2, n, k // 2), generator=gen, dtype=u8).cuda()
        self.W = torch.rand(K, generator=gen).cuda() + 0.5
        self.up, self.down = weights(2 * F, K), weights(K, F)
        self.sf_up = torch.full((2 * F, K // 32), 121, dtype=u8, device="cuda")
        self.sf_down = torch.full((K, F // 32), 120, dtype=u8, device="cuda")
        self.start = torch.randn(M, K, generator=gen).to(bf16).cuda()
        self.X, self.H, self.Y, self.RS = new(bf16, M, K), new(bf16, M, K), new(bf16, M, K), new(f32, M)
        self.B1, self.B2 = new(u8, 2 * F, K // 2), new(u8, K, F // 2)
        self.Z, self.A = new(bf16, M, 2 * F), new(bf16, M, F)
        self.CK, self.SFCK = new(u8, M, 2 * F), new(u8, M, 2 * (-(-F // 32)))
        self.DZ, self.DX, self.DW = new(bf16, M, 2 * F), new(bf16, M, K), new(f32, K)
        self.ws = new(f32, M, K)
        self.log = new(f32, 12, K)

    def step(self, i, stream, after=lambda: None, side=None):
        M, K, F = self.M, self.K, self.F
        self.B1.copy_(self.up[i % 2])
        self.B2.copy_(self.down[(i + 1) % 2])
        after()
        gemm.gemm_norm_run(M, K, "bf16", "bf16", "bf16", 1e-6, self.X, self.H, self.W, self.H, self.Y, None, self.RS, stream)
        after()
        gemm.gemm_matvec_run(M, 2 * F, K, "bf16", "bf16", 1, self.Y, self.B1, self.sf_up, None, self.Z, stream)
        after()
        gemm.gemm_gate_run(M, F, "bf16", "bf16", self.Z, self.A, None, self.CK, self.SFCK, stream)
        after()
        if side is not None:                       # a branch that writes what the next call reads
            side.wait_stream(stream)
            with torch.cuda.stream(side):
                self.B2.copy_(self.down[i % 2])
            stream.wait_stream(side)
        else:
            self.B2.copy_(self.down[i % 2])
        after()
        gemm.gemm_matvec_run(M, K, F, "bf16", "bf16", 1, self.A, self.B2, self.sf_down, None, self.X, stream)
        after()
        gemm.gemm_gate_backward(M, F, "bf16", "bf16", "bf16", self.A, self.CK, self.SFCK, self.DZ, self.A, stream)
        after()
        gemm.gemm_norm_backward(M, K, "bf16", "bf16", "bf16", self.X, self.DX, self.H, self.RS, self.W, self.DX, self.DW,
                                self.Y, self.ws, self.ws.numel() * 4, stream)
        after()
        if i % 3 == 0:
            self.X.clamp_(-4, 4)
        self.DX.mul_(0.5)
        self.log[i].copy_(self.DW)
        after()

    def reset(self):
        self.X.copy_(self.start)
        self.H.copy_(self.start)
        self.DX.zero_()
        self.log.zero_()

    def result(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.X, self.H, self.A, self.DZ, self.DX, self.log)]


@pytest.mark.parametrize("M,K,F", [(1, 1024, 512), (5, 2048, 1056), (16, 9216, 1024)])
def test_calls_in_a_row(M, K, F):
    b, stream = Block(M, K, F), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        b.reset()
        for i in range(12):
            b.step(i, stream, after=torch.cuda.synchronize)
        want = b.result()
        assert all(t.isfinite().all() for t in want) and want[5].abs().amax(1).min() > 0
        for _ in range(3):
            b.reset()
            for i in range(12):
                b.step(i, stream)
            assert all(torch.equal(x, y) for x, y in zip(b.result(), want))


@pytest.mark.parametrize("branches", [False, True])
def test_calls_in_a_graph(branches):
    b, stream, side = Block(3, 2048, 1024), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        b.reset()
        for i in range(12):
            b.step(i, stream, after=torch.cuda.synchronize)
        want = b.result()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            b.reset()
            for i in range(12):
                b.step(i, stream, side=side if branches else None)
        for _ in range(3):
            graph.replay()
            assert all(torch.equal(x, y) for x, y in zip(b.result(), want))
