"""Orders within kernels that a run cannot show to be kept, read from their source: a call may come out right without them."""
import os
import re

from blackwell_tensor_core_tma_gb300 import build


def source(name):
    """A file's code without its comments."""
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, name):
    """The definition of a kernel: what stands between its braces."""
    begin = text.index("{", text.index(")", text.index(name + "(")))
    depth = 0
    for i in range(begin, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[begin:i]
    raise AssertionError(name)


def test_no_store_to_a_cta_that_has_not_begun():
    """The clipping's cluster: every CTA arrives as it begins, and waits for the others before it stores to them."""
    code = body(source("gemm_clip.cu"), "clip_few_kernel")
    arrive, wait, store = (code.find(s) for s in ("cluster_arrive()", "cluster_wait()", "st.shared::cluster"))
    assert 0 <= arrive < code.index("wait_for_previous()")
    assert arrive < wait < store
    # and once more behind the stores, before the sums are read
    assert store < code.find("cluster_arrive()", store) < code.find("cluster_wait()", store) < code.index("all.add(")
    assert code.count("cluster_arrive()") == code.count("cluster_wait()") == 2


def test_no_load_may_be_moved_ahead_of_the_wait_for_earlier_kernels():
    """A kernel that begins while the one before it still writes: no load that takes its data to be the same all through."""
    names = [n for n in sorted(os.listdir(build.CSRC)) if "wait_for_previous()" in source(n)]
    assert {"gemm_gated.cuh", "gemm_gated_matvec.cu", "gemm_clip.cu", "gemm_norm.cu", "gemm_gate.cu", "gemm_matvec.cu"} <= set(names)
    for name in names:
        assert not re.search(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc\b|const\s[^;,{}()]*\*\s*__restrict__", source(name)), name
