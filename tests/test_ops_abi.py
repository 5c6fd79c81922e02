"""The feed-forward operators refuse bad arguments before they touch a device."""
import os
import re

import pytest

from blackwell_tensor_core_tma_gb300 import build, gemm

P = 4096                                         # stands for an aligned pointer; nothing is launched
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gemm.lib()


def refused(status, f, *args):
    with pytest.raises(gemm.GemmError) as e:
        f(*args)
    assert e.value.status == status


INVALID, UNSUPPORTED, ALIGNMENT = gemm.GEMM_ERR_INVALID_ARG, gemm.GEMM_ERR_UNSUPPORTED, gemm.GEMM_ERR_ALIGNMENT


def test_workspace_rows_match_the_header():
    text = open(os.path.join(ROOT, "include", "gb300gemm.h")).read()
    assert int(re.search(r"#define GEMM_NORM_PARTS (\d+)", text).group(1)) == gemm.GEMM_NORM_PARTS


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(M=-1)), (INVALID, dict(K=0)), (INVALID, dict(K=-16)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(X=None)), (INVALID, dict(W=None)), (INVALID, dict(Y=None)),
    (INVALID, dict(SFY=None)), (UNSUPPORTED, dict(x="f16")), (UNSUPPORTED, dict(h="e4m3")), (UNSUPPORTED, dict(y="f32")),
    (UNSUPPORTED, dict(y="e2m1")), (UNSUPPORTED, dict(K=32784)), (ALIGNMENT, dict(K=40)), (ALIGNMENT, dict(X=P + 8)),
    (ALIGNMENT, dict(R=P + 2)), (ALIGNMENT, dict(W=P + 4)), (ALIGNMENT, dict(H=P + 8)), (ALIGNMENT, dict(Y=P + 1)),
])
def test_norm_refuses(status, change):
    a = dict(M=4, K=64, x="bf16", h="bf16", y="e4m3", eps=1e-6, X=P, R=P, W=P, H=P, Y=P, SFY=P, RSTD=P)
    refused(status, gemm.gemm_norm_run, *(a | change).values())


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(M=-1)), (INVALID, dict(K=0)), (INVALID, dict(DY=None)), (INVALID, dict(H=None)), (INVALID, dict(RSTD=None)),
    (INVALID, dict(W=None)), (INVALID, dict(DX=None)), (INVALID, dict(workspace=None)),
    (INVALID, dict(bytes=4 * 64 * 4 - 4)), (INVALID, dict(M=100000)), (UNSUPPORTED, dict(dy="f16")),
    (UNSUPPORTED, dict(h="f16")), (UNSUPPORTED, dict(y="e4m3")), (UNSUPPORTED, dict(K=65536)), (ALIGNMENT, dict(K=72)),
    (ALIGNMENT, dict(DY=P + 8)), (ALIGNMENT, dict(DH=P + 8)), (ALIGNMENT, dict(DX=P + 8)), (ALIGNMENT, dict(DW=P + 4)),
    (ALIGNMENT, dict(Y=P + 8)), (ALIGNMENT, dict(workspace=P + 8)),
])
def test_norm_backward_refuses(status, change):
    a = dict(M=4, K=64, dy="bf16", h="bf16", y="bf16", DY=P, DH=P, H=P, RSTD=P, W=P, DX=P, DW=P, Y=P, workspace=P,
             bytes=4 * 64 * 4)
    refused(status, gemm.gemm_norm_backward, *(a | change).values())


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(M=-1)), (INVALID, dict(F=0)), (INVALID, dict(F=(1 << 20) + 16)), (INVALID, dict(Z=None)),
    (INVALID, dict(A=None)), (INVALID, dict(SFA=None)), (INVALID, dict(SFCK=None)), (UNSUPPORTED, dict(z="f16")),
    (UNSUPPORTED, dict(a="f32")), (ALIGNMENT, dict(F=24)), (ALIGNMENT, dict(Z=P + 8)), (ALIGNMENT, dict(A=P + 8)),
    (ALIGNMENT, dict(CK=P + 8)),
])
def test_gate_refuses(status, change):
    a = dict(M=4, F=64, z="bf16", a="e4m3", Z=P, A=P, SFA=P, CK=P, SFCK=P)
    refused(status, gemm.gemm_gate_run, *(a | change).values())


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(M=-1)), (INVALID, dict(F=0)), (INVALID, dict(DA=None)), (INVALID, dict(CK=None)), (INVALID, dict(SFCK=None)),
    (INVALID, dict(DZ=None)), (UNSUPPORTED, dict(da="f16")), (UNSUPPORTED, dict(dz="e4m3")), (UNSUPPORTED, dict(a="e4m3")),
    (ALIGNMENT, dict(F=24)), (ALIGNMENT, dict(DA=P + 8)), (ALIGNMENT, dict(CK=P + 8)), (ALIGNMENT, dict(DZ=P + 8)),
    (ALIGNMENT, dict(A=P + 8)),
])
def test_gate_backward_refuses(status, change):
    a = dict(M=4, F=64, da="bf16", dz="bf16", a="bf16", DA=P, CK=P, SFCK=P, DZ=P, A=P)
    refused(status, gemm.gemm_gate_backward, *(a | change).values())


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(M=-1)), (INVALID, dict(N=0)), (INVALID, dict(K=0)), (INVALID, dict(mode=3)), (INVALID, dict(mode=-1)),
    (INVALID, dict(X=None)), (INVALID, dict(B=None)), (INVALID, dict(SFB=None)), (INVALID, dict(D=None)),
    (UNSUPPORTED, dict(M=17)), (UNSUPPORTED, dict(K=32800)), (UNSUPPORTED, dict(x="f32")), (UNSUPPORTED, dict(x="e2m1")),
    (UNSUPPORTED, dict(d="f16")), (UNSUPPORTED, dict(mode=0)), (ALIGNMENT, dict(K=48)), (ALIGNMENT, dict(X=P + 8)),
    (ALIGNMENT, dict(B=P + 8)), (ALIGNMENT, dict(SFB=P + 1)), (ALIGNMENT, dict(C=P + 4)), (ALIGNMENT, dict(D=P + 4)),
])
def test_matvec_refuses(status, change):
    a = dict(M=1, N=64, K=64, x="bf16", d="bf16", mode=1, X=P, B=P, SFB=P, C=P, D=P)
    refused(status, gemm.gemm_matvec_run, *(a | change).values())


def test_no_rows_is_no_work():
    assert gemm.gemm_norm_run(0, 64, "bf16", "bf16", "e4m3", 1e-6, None, None, None, None, None) == gemm.GEMM_OK
    assert gemm.gemm_norm_backward(0, 64, "bf16", "bf16", "bf16", None, None, None, None, None, None) == gemm.GEMM_OK
    assert gemm.gemm_gate_run(0, 64, "bf16", "e4m3", None, None) == gemm.GEMM_OK
    assert gemm.gemm_gate_backward(0, 64, "bf16", "bf16", "bf16", None, None, None, None) == gemm.GEMM_OK
    assert gemm.gemm_matvec_run(0, 64, 64, "bf16", "bf16", 1, None, None, None, None, None) == gemm.GEMM_OK


def test_norm_fault_refuses_a_negative_limit():
    refused(INVALID, gemm.gemm_testing_set_norm_fault, -1)
    gemm.gemm_testing_set_norm_fault(0)
