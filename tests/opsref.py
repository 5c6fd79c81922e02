"""The feed-forward operators' definitions in 64 bits (torch doubles on the CPU), and the bounds that
fp32 arithmetic and the output's rounding put on a result's distance from them."""
import torch

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.uint8}
U = 2.0 ** -24                                   # fp32's unit roundoff


def blocks(k):
    return -(-k // 32)


def scale_codes(v):
    """UE8M0 codes of rows of doubles: per 32 elements the smallest c >= 0 with max |v| <= 448 * 2^(c - 127)."""
    m, k = v.shape
    p = torch.zeros(m, blocks(k) * 32, dtype=torch.float64)
    p[:, :k] = torch.where(v.isnan(), torch.zeros_like(v), v).abs()
    amax = p.view(m, -1, 32).amax(2)
    c = torch.zeros(amax.shape, dtype=torch.int64)
    for step in (128, 64, 32, 16, 8, 4, 2, 1):   # the largest c - 1 that does not hold it, plus one
        t = c + step
        bad = (t <= 248) & (amax > 448.0 * torch.exp2((t - 1 - 127).double()))
        c = torch.where(bad, t, c)
    return c


def spread(codes, k):
    """The scale of every element of a row of k (the NaN code does not occur in rows this module makes)."""
    return torch.exp2((codes.long() - 127).double()).repeat_interleave(32, 1)[:, :k]


def e4m3(v):
    """Doubles rounded to e4m3's values, ties to even; past 448 it saturates, as the kernels' conversion does."""
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.copysign((a / step).round() * step, v)


def decode_e4m3(codes):
    c = codes.cpu().to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, torch.exp2((e - 7).double()) * (1 + m / 8))
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(c >= 128, -v, v)


def half_ulp(ref, kind):
    """Half the spacing of a type's values at |ref| (its rounding error)."""
    if kind == "f32":
        return ref.abs() * U
    p, emin = (8, -126) if kind == "bf16" else (11, -14)
    a = ref.abs()
    _, e = torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))
    e = torch.where(a > 0, (e - 1).clamp(min=emin), torch.full_like(e, emin))
    return torch.exp2((e - p).double())


def assert_within(name, got, ref, tol):
    got, ref = got.double().cpu(), ref.double()
    bad = ~((got - ref).abs() <= tol) & ~(got == ref) & ~(got.isnan() & ref.isnan())
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got {got[i]!r}, "
                             f"want {ref[i]!r}, off by {float((got - ref).abs()[i])}, allowed {float(tol[i])}")


def assert_operand(name, y, sf, ref, rel, kind):
    """An operand (codes and scales, or 16 bits) against its 64-bit values, computed to within rel * |ref|."""
    if kind != "e4m3":
        assert_within(name, y, ref, half_ulp(ref, kind) * (1 + 2.0 ** -10) + rel * ref.abs())
        return
    k = ref.shape[1]
    low, high = scale_codes(ref * (1 - rel)), scale_codes(ref * (1 + rel))
    c = sf.cpu().to(torch.int64)
    assert ((c >= low) & (c <= high)).all(), f"{name}: {int(((c < low) | (c > high)).sum())} scale codes"
    s = spread(c, k)
    _, e = torch.frexp((ref / s).abs().clamp(min=2.0 ** -6))
    tol = torch.exp2((e - 1).double() - 4) * s * (1 + 2.0 ** -10) + rel * ref.abs()
    assert_within(name, decode_e4m3(y.view(torch.uint8)) * s, ref, tol)


# ------------------------------------------------------------------------------------------- norm

def norm(h, w, eps):
    h, w = h.double(), w.double()
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


# A sum of K squares runs over at most 32 adds in a thread, 5 in a warp and 32 over warps, all of one sign; the
# root halves its error; mean, eps, root, reciprocal and the two products round once each.
NORM_REL = (69 / 2 + 8) * U


def norm_back(dy, dh, h, rstd, w):
    dy, dh, h, rstd, w = (t.double() for t in (dy, dh, h, rstd, w))
    n, g = h * rstd[:, None], dy * w
    c = (g * n).mean(1, keepdim=True)
    dx = dh + rstd[:, None] * (g - n * c)
    size = dh.abs() + rstd[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    return dx, size, (dy * n).sum(0), (dy * n).abs().sum(0), n * w


# ------------------------------------------------------------------------------------------- gate

def sigmoid_rel(g):
    """Relative error of 1 / (1 + exp(-g)) with the fast fp32 exponential (2 + 1.173 |x| units of 2^-23) and
    division (2 units)."""
    s = torch.sigmoid(g)
    return ((2 + 1.173 * g.abs()) * (1 - s) + 4) * 2 * U


def gate(g, u):
    return g * torch.sigmoid(g) * u


def gate_back(g, u, da):
    """dg, du, a and the sizes their errors scale with."""
    s = torch.sigmoid(g)
    t = torch.sigmoid(-g)
    dg, du = da * u * s * (1 + g * t), da * g * s
    # an error of s also moves 1 - s: by rel * s
    rel = sigmoid_rel(g) + 8 * U
    dg_tol = rel * (da * u * s).abs() * (1 + g.abs() * t + g.abs() * s) + rel * dg.abs()
    return dg, du, g * s * u, dg_tol, rel * du.abs(), rel


# ----------------------------------------------------------------------------------------- matvec

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def weights(B, SFB, mode):
    """N x K doubles of packed e2m1 codes and their scales."""
    b = B.cpu().to(torch.int64)
    n, k = b.shape[0], b.shape[1] * 2
    codes = torch.stack([b & 15, b >> 4], 2).view(n, k)
    w = E2M1[codes & 7] * torch.where(codes >= 8, -1.0, 1.0).double()
    c = SFB.cpu().to(torch.int64)
    if mode == 1:
        s = torch.exp2((c - 127).double())
        s = torch.where(c == 255, torch.full_like(s, float("nan")), s)
    else:
        s = decode_e4m3(c & 127)
    return w * s.repeat_interleave(k // s.shape[1], 1)


def matvec(X, B, SFB, mode, C=None):
    """D and sum |x w| in doubles."""
    x, w = X.cpu().double(), weights(B, SFB, mode)
    d = x @ w.t()
    return (d if C is None else d + C.cpu().double()), x.abs() @ w.abs().t()
