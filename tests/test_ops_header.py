"""What the header says of the feed-forward operators' arguments is what they do."""
import os
import re

import pytest

from blackwell_tensor_core_tma_gb300 import build, gemm

P = 4096                                         # stands for an aligned pointer; nothing is launched
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def text():
    build.build()
    full = open(os.path.join(ROOT, "include", "gb300gemm.h")).read()
    return re.sub(r"\s+\*?\s*", " ", full[full.index("The feed-forward block around the product"):])


def status(f, *args):
    with pytest.raises(gemm.GemmError) as e:
        f(*args)
    return e.value.status


def test_alignment_of_scale_codes(text):
    """The codes that need no alignment are named, and the matrix-vector product's are not among them."""
    free = re.search(r"16-byte aligned \(GEMM_ERR_ALIGNMENT\) except RSTD and the scale codes of the norm and the gate \(([^)]*)\)",
                     text).group(1).split(", ")
    assert free == ["SFY", "SFA", "SFCK"]
    for off in (1, 8):
        assert status(gemm.gemm_matvec_run, 1, 64, 64, "bf16", "bf16", 1, P, P, P + off, P, P) == gemm.GEMM_ERR_ALIGNMENT


def test_bounds_of_sizes(text):
    assert "Any N from 1 to (2^31 - 1) / 16 (GEMM_ERR_INVALID_ARG)" in text
    assert "it is at most 2^31 - 1 (GEMM_ERR_INVALID_ARG)" in text
    invalid = gemm.GEMM_ERR_INVALID_ARG
    assert status(gemm.gemm_matvec_run, 1, (2 ** 31 - 1) // 16 + 1, 64, "bf16", "bf16", 1, P, P, P, P, P) == invalid
    assert status(gemm.gemm_matvec_run, 1, (2 ** 31 - 1) // 16, 64, "bf16", "bf16", 1, P, P, P + 1, P, P) == \
        gemm.GEMM_ERR_ALIGNMENT
    M = 2 ** 31
    assert status(gemm.gemm_norm_run, M, 64, "bf16", "bf16", "bf16", 1e-6, P, P, P, P, P) == invalid
    assert status(gemm.gemm_norm_backward, M, 64, "bf16", "bf16", "bf16", P, P, P, P, P, P) == invalid
    assert status(gemm.gemm_gate_run, M, 64, "bf16", "bf16", P, P) == invalid
    assert status(gemm.gemm_gate_backward, M, 64, "bf16", "bf16", "bf16", P, P, P, P) == invalid


def test_order_of_sums(text):
    """dw's groups of rows, and the product's slices of K, follow from how many clusters run at once."""
    assert "the GPU's SM count and (rows split over CTAs) how many clusters the GPU runs at once" in text
    assert "the GPU's SM count alone" not in text
