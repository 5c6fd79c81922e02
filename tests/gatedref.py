"""The gated product, its gradient and the clipping in 64 bits, with the bounds on a result's distance from them.

Products meet the library's bound on sums: |z - exact| <= 1e-5 * sum |x w|.  What follows the sums adds its own roundings."""
import torch

from tests import opsref as ref

TORCH = dict(ref.TORCH, e4m3=torch.float8_e4m3fn)
SUM = 1e-5


def rounded(v, kind):
    """An operand in a type, with its scales where it has some: (codes, scales or None, its values in doubles)."""
    if kind != "e4m3":
        t = v.to(TORCH[kind])
        return t, None, t.double()
    codes = ref.scale_codes(v.double())
    s = ref.spread(codes, v.shape[1])
    q = (v.double() / s).float().to(torch.float8_e4m3fn)
    return q, codes.to(torch.uint8), q.double() * s


def product(x, w):
    """x·wᵀ and sum |x w| in doubles (on the GPU: the sizes are a CPU's seconds)."""
    x, w = x.cuda(), w.cuda()
    return (x @ w.t()).cpu(), (x.abs() @ w.abs().t()).cpu()


def gated(x, w):
    """g, u, a of doubles and the bounds on their distance before any rounding of the outputs."""
    F = w.shape[0] // 2
    z, size = product(x, w)
    tol = SUM * size + 1e-37
    g, u = z[:, :F], z[:, F:]
    tg, tu = tol[:, :F], tol[:, F:]
    a = ref.gate(g, u)
    # |silu'| <= 1.1; the sigmoid's own error and three products
    ta = 1.1 * tg * (u.abs() + tu) + (g * torch.sigmoid(g)).abs() * tu + (ref.sigmoid_rel(g) + 4 * ref.U) * a.abs()
    return g, u, a, tg, tu, ta


def assert_output(name, got, scales, want, tol, kind):
    """An output (codes and scales, or 16 bits) against its 64-bit values, computed to within tol."""
    if kind != "e4m3":
        ref.assert_within(name, got, want, ref.half_ulp(want.abs() + tol, kind) * (1 + 2.0 ** -10) + tol)
        return
    # every element of a block may move its maximum
    low, high = ref.scale_codes((want.abs() - tol).clamp(min=0)), ref.scale_codes(want.abs() + tol)
    c = scales.cpu().to(torch.int64)
    assert ((c >= low) & (c <= high)).all(), f"{name}: {int(((c < low) | (c > high)).sum())} scale codes"
    s = ref.spread(c, want.shape[1])
    _, e = torch.frexp(((want.abs() + tol) / s).clamp(min=2.0 ** -6))
    step = torch.exp2((e - 1).double() - 4) * s * (1 + 2.0 ** -10)
    ref.assert_within(name, ref.decode_e4m3(got.view(torch.uint8)) * s, want, step + tol)
