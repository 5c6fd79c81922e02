"""How far the norm's dw may be from its 64-bit value, and that a row left out or taken twice lies outside of it."""
import pytest

from tests import opsref as ref

torch = pytest.importorskip("torch")

# Adds one after another: a thread's rows (at most twenty at the tests' sizes: the fewest groups of threads are clusters of
# eight, of which fifteen or more run at once), a CTA's row groups (at most 64 at more than one row per thread), the CTAs'
# sums (at most sixteen in a lane of the last kernel, then 32); each term is rounded twice.  That is below 168 U = 1e-5.
DW_REL = 1e-5

# rows, columns, dy, h: those of the kernel's tests whose sums have the most terms, and rows split over CTAs
SIZES = [(20000, 112, "bf16", "bf16"), (10000, 256, "f32", "f32"), (5000, 1024, "bf16", "bf16"), (5000, 112, "bf16", "bf16"),
         (3100, 528, "bf16", "f32"), (1300, 4096, "f32", "bf16"), (1000, 2064, "bf16", "bf16"), (800, 8208, "bf16", "bf16"),
         (400, 16384, "f32", "f32"), (305, 32768, "f32", "f32")]


def inputs(M, K, dy, h, seed):
    gen = torch.Generator().manual_seed(seed)
    H = torch.randn(M, K, generator=gen)
    H[:, ::37] *= 20
    H = H.to(ref.TORCH[h])
    DY = torch.randn(M, K, generator=gen).to(ref.TORCH[dy])
    RS = (1 / torch.sqrt((H.double() ** 2).mean(1) + 1e-5)).float()
    return DY, H, RS


def terms(DY, H, RS):
    return DY.double() * H.double() * RS.double()[:, None]


@pytest.mark.parametrize("M,K,dy,h", SIZES)
def test_every_row_shows(M, K, dy, h):
    t = terms(*inputs(M, K, dy, h, seed=M + K)).abs()
    # the planted mistake is the row's own terms; the result itself may be off by the tolerance the other way
    assert (t > 2 * DW_REL * t.sum(0)).any(1).all()
