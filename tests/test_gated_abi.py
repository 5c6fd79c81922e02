"""The gated product, its few-row form and the clipping refuse bad arguments before they touch a device."""
import os
import re

import pytest

from blackwell_tensor_core_tma_gb300 import build, gemm
from tests.test_ops_abi import ALIGNMENT, INVALID, P, ROOT, UNSUPPORTED, refused


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gemm.lib()


def test_workspace_matches_the_header():
    text = open(os.path.join(ROOT, "include", "gb300gemm.h")).read()
    assert int(re.search(r"#define GEMM_CLIP_WORKSPACE (\d+)", text).group(1)) == gemm.GEMM_CLIP_WORKSPACE


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(M=0)), (INVALID, dict(F=0)), (INVALID, dict(K=-8)), (INVALID, dict(M=1 << 31)), (INVALID, dict(F=(1 << 20) + 16)),
    (INVALID, dict(K=1 << 31)), (INVALID, dict(M=(1 << 31) - 1, F=1 << 20)), (INVALID, dict(block_scaled=3)), (INVALID, dict(ab=9)),
    (INVALID, dict(flags=6)), (UNSUPPORTED, dict(ab="f32")), (UNSUPPORTED, dict(ab="e4m3")), (UNSUPPORTED, dict(ab="e2m1", block_scaled=1)),
    (UNSUPPORTED, dict(block_scaled=1)), (UNSUPPORTED, dict(ab="e4m3", block_scaled=2)), (UNSUPPORTED, dict(a="f32")),
    (ALIGNMENT, dict(F=24)), (ALIGNMENT, dict(K=20)), (ALIGNMENT, dict(ab="e4m3", block_scaled=1, K=24)),
])
def test_gated_plan_refuses(status, change):
    a = dict(M=64, F=64, K=64, ab="bf16", a="bf16", block_scaled=0, flags=0)
    refused(status, gemm.gemm_gated_plan_create, *(a | change).values())


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(M=0)), (INVALID, dict(F=-16)), (INVALID, dict(N=0)), (INVALID, dict(F=(1 << 20) + 16)), (INVALID, dict(flags=6)),
    (INVALID, dict(ab=7)), (UNSUPPORTED, dict(ab="f32")), (UNSUPPORTED, dict(ab="e4m3")), (ALIGNMENT, dict(F=40)),
    (ALIGNMENT, dict(N=12)),
])
def test_gated_back_plan_refuses(status, change):
    a = dict(M=64, F=64, N=64, ab="bf16", flags=0)
    refused(status, gemm.gemm_gated_back_plan_create, *(a | change).values())


def test_no_plan():
    refused(INVALID, gemm.gemm_gated_run, None, P, P, None, None, P)
    refused(INVALID, gemm.gemm_gated_back_run, None, P, P, P, P, P)


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(M=-1)), (INVALID, dict(F=0)), (INVALID, dict(F=(1 << 20) + 1)), (INVALID, dict(K=0)), (INVALID, dict(X=None)),
    (INVALID, dict(W=None)), (INVALID, dict(SFW=None)), (INVALID, dict(A=None)), (UNSUPPORTED, dict(M=17)),
    (UNSUPPORTED, dict(K=32784)), (UNSUPPORTED, dict(x="f32")), (UNSUPPORTED, dict(w="f16")), (UNSUPPORTED, dict(w="e2m1")),
    (UNSUPPORTED, dict(a="f16")), (ALIGNMENT, dict(K=40)), (ALIGNMENT, dict(w="bf16", K=12)), (ALIGNMENT, dict(X=P + 8)),
    (ALIGNMENT, dict(W=P + 8)), (ALIGNMENT, dict(A=P + 2)),
])
def test_gated_matvec_refuses(status, change):
    a = dict(M=1, F=64, K=64, x="bf16", w="e4m3", a="bf16", X=P, W=P, SFW=P, A=P)
    refused(status, gemm.gemm_gated_matvec_run, *(a | change).values())


def test_no_rows_is_no_work():
    assert gemm.gemm_gated_matvec_run(0, 64, 64, "bf16", "e4m3", "bf16", None, None, None, None) == gemm.GEMM_OK


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(limit=-1.0)), (INVALID, dict(limit=float("nan"))), (INVALID, dict(NORM=None)), (INVALID, dict(workspace=None)),
    (INVALID, dict(bytes=16383)), (INVALID, dict(n=-1)), (INVALID, dict(n=(1 << 40) + 1)), (INVALID, dict(g=None)),
    (UNSUPPORTED, dict(type="e4m3")), (UNSUPPORTED, dict(type="e2m1")), (UNSUPPORTED, dict(count=2100)),
    (ALIGNMENT, dict(g=P + 2)), (ALIGNMENT, dict(c=P + 1)), (ALIGNMENT, dict(type="bf16", g=P + 1)),
    (ALIGNMENT, dict(NORM=P + 2)), (ALIGNMENT, dict(workspace=P + 8)),
])
def test_clip_refuses(status, change):
    a = dict(g=P, c=P, type="f32", n=64, limit=1.0, NORM=P, workspace=P, bytes=16384, count=1) | change
    if a["count"] > 1:
        a["n"] = 1 << 40                              # together past what chunks are counted in
    tensors = gemm.clip_tensors([(P, None, "f32", 8)] + [(a["g"], a["c"], a["type"], a["n"])] * a["count"])
    refused(status, gemm.gemm_clip_run, tensors, a["limit"], a["NORM"], a["workspace"], a["bytes"])


def test_clip_list_takes_contiguous_tensors_of_its_type():
    torch = pytest.importorskip("torch")
    g = torch.zeros(8, 8)
    for bad in ((g[:, ::2], None, "f32"), (g, g[:4], "f32"), (g, g.half(), "f32"), (g, None, "bf16")):
        with pytest.raises(ValueError):
            gemm.clip_tensors([bad])
    assert len(gemm.clip_tensors([(g, None, "f32"), (g, g, "f32")])) == 2


@pytest.mark.parametrize("sizes", [((1 << 31) - 256, 16, 16), (1, 16, (1 << 31) - 256), (1, (1 << 20) + 16, 16), (1 << 30, 1 << 20, 16)])
def test_sizes_past_what_is_counted(sizes):
    refused(INVALID, gemm.gemm_gated_plan_create, *sizes, "bf16", "bf16", 0, 0)
    refused(INVALID, gemm.gemm_gated_back_plan_create, *sizes, "bf16", 0)
