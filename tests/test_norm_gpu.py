"""gemm_norm_run and gemm_norm_backward against their definitions in 64 bits."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm
from tests import opsref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gemm.lib()


def guarded(shape, dtype, margin=64):
    """A buffer inside a larger one filled with a pattern, and a check that the margins keep it."""
    n = 1
    for s in shape:
        n *= s
    full = torch.full(((n + 2 * margin) * torch.empty(0, dtype=dtype).element_size(),), 0xA5, dtype=torch.uint8,
                      device="cuda").view(dtype)
    mid = full[margin:margin + n].view(shape)
    return mid, lambda: bool((full[:margin].view(torch.uint8) == 0xA5).all() and
                             (full[margin + n:].view(torch.uint8) == 0xA5).all())


def inputs(M, K, x, h, seed=0, residual=True):
    gen = torch.Generator().manual_seed(seed)
    X = torch.randn(M, K, generator=gen).to(ref.TORCH[x])
    R = torch.randn(M, K, generator=gen)
    R[:, ::37] *= 20
    W = 1 + 0.3 * torch.randn(K, generator=gen)
    return X, (R.to(ref.TORCH[h]) if residual else None), W


def run_forward(M, K, x, h, y, X, R, W, eps=EPS, keep_h=True, rstd=True, stream=None, in_place=False):
    dev = lambda t: None if t is None else t.cuda()
    X, R, W = dev(X), dev(R), dev(W)
    H, h_ok = guarded((M, K), ref.TORCH[h]) if keep_h else (None, lambda: True)
    if in_place:
        H, h_ok = R, lambda: True
    Y, y_ok = guarded((M, K), ref.TORCH[y])
    SF, sf_ok = guarded((M, ref.blocks(K)), torch.uint8) if y == "e4m3" else (None, lambda: True)
    RS, r_ok = guarded((M,), torch.float32) if rstd else (None, lambda: True)
    torch.cuda.synchronize()
    gemm.gemm_norm_run(M, K, x, h, y, eps, X, R, W, H, Y, SF, RS, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert h_ok() and y_ok() and sf_ok() and r_ok()
    return H, Y, SF, RS


def rounded_sum(X, R, h):
    v = X.float() if R is None else X.float() + R.float()
    return v.to(ref.TORCH[h])


SHAPES = [(1, 16), (1, 4096), (2, 32), (5, 48), (67, 112), (300, 256), (9, 272), (3, 1040), (2, 2064), (7, 4096),
          (3, 4112), (2, 8192), (3, 8208), (2, 16400), (1, 32768)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("y", ["e4m3", "bf16", "f16"])
@pytest.mark.parametrize("x,h", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_forward(M, K, x, h, y):
    residual = (M + K // 16) % 3 != 0
    X, R, W = inputs(M, K, x, h, seed=M * 7 + K, residual=residual)
    H, Y, SF, RS = run_forward(M, K, x, h, y, X, R, W)
    want = rounded_sum(X, R, h)
    assert torch.equal(H.cpu(), want)
    v, rstd = ref.norm(want, W, EPS)
    ref.assert_within("rstd", RS, rstd, ref.NORM_REL * rstd)
    ref.assert_operand("y", Y, SF, v, ref.NORM_REL, y)


@pytest.mark.parametrize("M,K,x,h,y", [(800, 2064, "bf16", "bf16", "e4m3"), (500, 8208, "bf16", "bf16", "bf16"),
                                       (400, 4096, "f32", "bf16", "e4m3"), (2000, 1040, "f32", "f32", "e4m3")])
def test_forward_of_many_rows(M, K, x, h, y):
    X, R, W = inputs(M, K, x, h, seed=K)
    H, Y, SF, RS = run_forward(M, K, x, h, y, X, R, W)
    want = rounded_sum(X, R, h)
    assert torch.equal(H.cpu(), want)
    v, rstd = ref.norm(want, W, EPS)
    ref.assert_within("rstd", RS, rstd, ref.NORM_REL * rstd)
    ref.assert_operand("y", Y, SF, v, ref.NORM_REL, y)


def test_optional_outputs_and_in_place_residual():
    M, K = 11, 1008
    X, R, W = inputs(M, K, "bf16", "bf16", seed=4)
    H, Y, SF, RS = run_forward(M, K, "bf16", "bf16", "e4m3", X, R, W)
    for kw in (dict(keep_h=False), dict(rstd=False), dict(keep_h=False, rstd=False), dict(in_place=True)):
        h2, y2, sf2, _ = run_forward(M, K, "bf16", "bf16", "e4m3", X, R, W, **kw)
        assert torch.equal(Y, y2) and torch.equal(SF, sf2)
        if h2 is not None:
            assert torch.equal(H, h2)


def test_zero_huge_and_nonfinite_rows():
    """A row of zeros gives zeros; a row whose squares overflow fp32 gives rstd 0; NaN and infinity stay
    inside their row; a row with one huge element keeps its scale blocks apart."""
    M, K = 6, 96
    X = torch.zeros(M, K)
    X[1] = torch.linspace(-3, 3, K)
    X[2] = 1e30
    X[3, 5] = float("nan")
    X[4, 40] = float("inf")
    X[5] = torch.linspace(1e-3, 2e-3, K)
    X[5, 33] = 1e6
    W = torch.ones(K)
    _, Y, SF, RS = run_forward(M, K, "f32", "f32", "e4m3", X, None, W)
    y = ref.decode_e4m3(Y) * ref.spread(SF.cpu(), K)
    assert (y[0] == 0).all() and (y[2] == 0).all() and RS[2] == 0
    assert y[3].isnan().all() and y[4, 40].isnan() and (y[4, :40] == 0).all()
    v, rstd = ref.norm(X[[0, 1, 5]], W, EPS)
    ref.assert_operand("finite rows", Y[[0, 1, 5]], SF[[0, 1, 5]], v, ref.NORM_REL, "e4m3")


def test_scale_boundaries():
    """Values at, just below and just above 448 * 2^j, and the smallest and largest ones, through the
    gated unit's checkpoint, which quantises its input as it is."""
    edge = torch.tensor([448.0, 449.0, 447.0, 1.0], dtype=torch.float32)
    up = torch.nextafter(edge[0], torch.tensor(1e9))
    down = torch.nextafter(edge[0], torch.tensor(0.0))
    tops = [edge[0], up, down, 2.0 ** -126, 2.0 ** -140, 3.4e38, 0.0, 7.0, 1.75 * 2.0 ** -119, 1.8 * 2.0 ** -119, 2.0 ** -149]
    F = 32 * len(tops)
    gen = torch.Generator().manual_seed(3)
    g = torch.rand(F, generator=gen) * 2 - 1
    Z = torch.zeros(1, 2 * F)
    for i, t in enumerate(tops):
        Z[0, 32 * i:32 * i + 32] = g[32 * i:32 * i + 32] * float(t)
        Z[0, 32 * i + 13] = -float(t)
    CK = torch.zeros(1, 2 * F, dtype=torch.uint8, device="cuda")
    SF = torch.zeros(1, 2 * len(tops), dtype=torch.uint8, device="cuda")
    A = torch.empty(1, F, dtype=torch.bfloat16, device="cuda")
    gemm.gemm_gate_run(1, F, "f32", "bf16", Z.cuda(), A, None, CK, SF, torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = ref.scale_codes(Z[:, :F].double())
    assert torch.equal(SF.cpu()[:, :len(tops)].long(), want)
    q = ref.e4m3(Z[:, :F].double() / ref.spread(want, F))
    assert torch.equal(ref.decode_e4m3(CK[:, :F]), q)


def test_side_stream_and_graph():
    M, K = 40, 512
    X, R, W = inputs(M, K, "bf16", "bf16", seed=9)
    H, Y, SF, RS = run_forward(M, K, "bf16", "bf16", "e4m3", X, R, W)
    s = torch.cuda.Stream()
    got = run_forward(M, K, "bf16", "bf16", "e4m3", X, R, W, stream=s)
    assert all(torch.equal(a, b) for a, b in zip((H, Y, SF, RS), got))
    X, R, W = X.cuda(), R.cuda(), W.cuda()
    outs = [torch.zeros_like(t) for t in (H, Y, SF, RS)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        gemm.gemm_norm_run(M, K, "bf16", "bf16", "e4m3", EPS, X, R, W, *outs, s)
        g.capture_end()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((H, Y, SF, RS), outs))


def test_rows_past_two_to_the_31_elements():
    M, K = 65600, 32768
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, K, generator=torch.Generator().manual_seed(1)).bfloat16()
    X[-3:] = tail.cuda()
    W = torch.ones(K, device="cuda")
    Y = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    SF = torch.empty(M, K // 32, dtype=torch.uint8, device="cuda")
    gemm.gemm_norm_run(M, K, "bf16", "bf16", "e4m3", EPS, X, None, W, None, Y, SF, None, torch.cuda.current_stream())
    torch.cuda.synchronize()
    v, _ = ref.norm(tail, W.cpu(), EPS)
    ref.assert_operand("tail", Y[-3:], SF[-3:], v, ref.NORM_REL, "e4m3")
    assert int(Y[-4].max()) == 0


# ---------------------------------------------------------------------------------------- backward

def run_backward(M, K, dy, h, y, DY, DH, H, RS, W, again=True, want_dw=True, in_place=False, stream=None):
    dev = lambda t: None if t is None else t.cuda()
    DY, DH, H, RS, W = (dev(t) for t in (DY, DH, H, RS, W))
    DX, x_ok = guarded((M, K), ref.TORCH[h])
    if in_place:
        DX, x_ok = DH, lambda: True
    DW, w_ok = guarded((K,), torch.float32) if want_dw else (None, lambda: True)
    Y, y_ok = guarded((M, K), ref.TORCH[y]) if again else (None, lambda: True)
    parts = min(M, gemm.GEMM_NORM_PARTS)
    WS, ws_ok = guarded((parts, K), torch.float32)
    torch.cuda.synchronize()
    gemm.gemm_norm_backward(M, K, dy, h, y, DY, DH, H, RS, W, DX, DW, Y, WS if want_dw else None,
                            parts * K * 4 if want_dw else 0, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert x_ok() and w_ok() and y_ok() and ws_ok()
    return DX, DW, Y


def back_inputs(M, K, dy, h, seed):
    gen = torch.Generator().manual_seed(seed)
    H = torch.randn(M, K, generator=gen)
    H[:, ::37] *= 20
    H = H.to(ref.TORCH[h])
    W = 1 + 0.3 * torch.randn(K, generator=gen)
    DY = torch.randn(M, K, generator=gen).to(ref.TORCH[dy])
    DH = torch.randn(M, K, generator=gen).to(ref.TORCH[h])
    RS = (1 / torch.sqrt((H.double() ** 2).mean(1) + EPS)).float()
    return DY, DH, H, RS, W


def check_backward(M, dy, h, y, got, DY, DH, H, RS, W):
    DX, DW, Y = got
    zero = torch.zeros_like(H) if DH is None else DH
    dx, size, dw, dw_size, v = ref.norm_back(DY, zero, H, RS, W)
    # a sum of at most 69 adds (as in the forward pass) and some ten roundings of each term
    ref.assert_within("dx", DX, dx, ref.half_ulp(dx, h) * (1 + 2.0 ** -10) + 80 * ref.U * size)
    if DW is not None:
        # rows are added one after another within a CTA and CTAs' sums in turn: never more adds than rows + 8
        ref.assert_within("dw", DW, dw, (M + 12) * ref.U * dw_size)
    if Y is not None:
        ref.assert_operand("y", Y, None, v, 3 * ref.U, y)


@pytest.mark.parametrize("M,K", SHAPES + [(700, 64), (1300, 528)])
@pytest.mark.parametrize("dy,h,y", [("bf16", "bf16", "bf16"), ("f32", "bf16", "f16"), ("f32", "f32", "bf16"),
                                    ("bf16", "f32", "f16")])
def test_backward(M, K, dy, h, y):
    t = back_inputs(M, K, dy, h, seed=M + 3 * K)
    check_backward(M, dy, h, y, run_backward(M, K, dy, h, y, *t), *t)


# more rows than run at once: each CTA walks several, with the next ones on their way
@pytest.mark.parametrize("M,K,dy,h", [(1000, 2064, "bf16", "bf16"), (700, 4112, "f32", "f32"), (600, 8192, "bf16", "bf16"),
                                      (500, 8208, "f32", "bf16"), (330, 16400, "bf16", "f32"), (320, 16400, "bf16", "bf16"),
                                      (310, 32768, "bf16", "bf16"), (305, 32768, "f32", "f32"), (5000, 112, "bf16", "bf16")])
def test_backward_of_many_rows(M, K, dy, h):
    t = back_inputs(M, K, dy, h, seed=M + K)
    got = run_backward(M, K, dy, h, "bf16", *t)
    check_backward(M, dy, h, "bf16", got, *t)
    again = run_backward(M, K, dy, h, "bf16", *t, in_place=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


# rows that several multiprocessors share, each with several of them, and the sizes next to where the sharing changes
@pytest.mark.parametrize("M,K,dy,h", [(800, 8208, "bf16", "bf16"), (700, 9008, "f32", "f32"), (500, 8192, "f32", "f32"),
                                      (500, 7168, "f32", "f32"), (500, 7184, "bf16", "f32"), (77, 12304, "bf16", "bf16"),
                                      (400, 16384, "f32", "f32"), (400, 16384, "f32", "bf16"), (300, 16400, "f32", "f32"),
                                      (200, 20496, "bf16", "f32"), (170, 28688, "f32", "f32"), (76, 16384, "bf16", "bf16")])
def test_backward_of_shared_rows(M, K, dy, h):
    t = back_inputs(M, K, dy, h, seed=M + K)
    got = run_backward(M, K, dy, h, "f16", *t)
    check_backward(M, dy, h, "f16", got, *t)
    again = run_backward(M, K, dy, h, "f16", *t, in_place=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    lone = run_backward(M, K, dy, h, "f16", *t, again=False, want_dw=False)
    assert torch.equal(lone[0], got[0])


# several rows for every CTA, with as many rows at a time as a CTA takes: row groups of part of a warp, of whole warps and
# of warps with idle lanes, and the widths where the last sum of dw changes
@pytest.mark.parametrize("M,K,dy,h", [(20000, 112, "bf16", "bf16"), (10000, 256, "f32", "f32"), (5000, 1024, "bf16", "bf16"),
                                      (3100, 528, "bf16", "f32"), (3100, 2064, "bf16", "bf16"), (1300, 4096, "f32", "bf16"),
                                      (1300, 2432, "bf16", "bf16"), (1300, 2448, "bf16", "bf16"), (700, 4864, "bf16", "bf16"),
                                      (700, 4880, "f32", "f32")])
def test_backward_of_many_row_groups(M, K, dy, h):
    t = back_inputs(M, K, dy, h, seed=M + K)
    got = run_backward(M, K, dy, h, "bf16", *t)
    check_backward(M, dy, h, "bf16", got, *t)
    again = run_backward(M, K, dy, h, "bf16", *t, in_place=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_backward_optional_parts_and_repeatability():
    M, K = 333, 2064
    DY, DH, H, RS, W = back_inputs(M, K, "bf16", "bf16", 5)
    full = run_backward(M, K, "bf16", "bf16", "bf16", DY, DH, H, RS, W)
    again = run_backward(M, K, "bf16", "bf16", "bf16", DY, DH, H, RS, W, in_place=True)
    assert all(torch.equal(a, b) for a, b in zip(full, again))
    lone = run_backward(M, K, "bf16", "bf16", "bf16", DY, DH, H, RS, W, again=False, want_dw=False)
    assert torch.equal(lone[0], full[0]) and lone[1] is None and lone[2] is None
    bare = run_backward(M, K, "bf16", "bf16", "bf16", DY, None, H, RS, W)
    check_backward(M, "bf16", "bf16", "bf16", bare, DY, None, H, RS, W)
    assert torch.equal(bare[1], full[1])


def test_backward_of_no_rows_clears_dw():
    K = 64
    DW = torch.full((K,), 7.0, device="cuda")
    gemm.gemm_norm_backward(0, K, "bf16", "bf16", "bf16", None, None, None, None, None, None, DW, None, None, 0,
                            torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert (DW == 0).all()


def test_gradient_against_differences():
    """Directional derivatives of sum(dy * y) + sum(dh * h) by central differences of the 64-bit definition."""
    M, K = 3, 208
    DY, DH, H, RS, W = back_inputs(M, K, "f32", "f32", 21)
    DX, DW, _ = run_backward(M, K, "f32", "f32", "bf16", DY, DH, H, RS, W, again=False)
    gen = torch.Generator().manual_seed(2)

    def f(h, w):
        return float((DY.double() * ref.norm(h, w, EPS)[0]).sum() + (DH.double() * h).sum())

    h, w, e = H.double(), W.double(), 1e-6
    for _ in range(5):
        v = torch.randn(M, K, generator=gen, dtype=torch.float64)
        want = (f(h + e * v, w) - f(h - e * v, w)) / (2 * e)
        # differences: about 1e-16 * |f| / e + e^2; the kernel: 80 U of the terms' sizes
        assert abs(float((DX.cpu().double() * v).sum()) - want) < 1e-5 * float((DX.cpu().double() * v).abs().sum())
        v = torch.randn(K, generator=gen, dtype=torch.float64)
        want = (f(h, w + e * v) - f(h, w - e * v)) / (2 * e)
        assert abs(float((DW.cpu().double() * v).sum()) - want) < 1e-5 * float((DW.cpu().double() * v).abs().sum())
