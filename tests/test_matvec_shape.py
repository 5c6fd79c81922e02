"""The matrix-vector product's launch, worked out on the host: one pass over the weights for every size that the entry
point takes."""
import pytest

from blackwell_tensor_core_tma_gb300 import build, gemm


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gemm.lib()


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("mode", [gemm.GEMM_SCALE_UE8M0_32, gemm.GEMM_SCALE_UE4M3_16])
def test_every_size_takes_one_pass(mode, x):
    for M in range(1, 17):
        for K in range(32, 32769, 32):
            chunks = -(-K // 256)
            grid, cluster, slices, smem = gemm.gemm_testing_matvec_shape(M, 700, K, x, mode)
            assert 0 < grid <= 152 and grid % cluster == 0 and cluster * slices <= chunks and smem <= 226 * 1024


def test_sizes_that_need_large_clusters():
    """Sixteen rows of 32768 need more than half of a cluster of eight; without one the product is refused as a whole."""
    for M in (13, 16):
        assert gemm.gemm_testing_matvec_shape(M, 700, 32768, "bf16", 1)[1] > 4
        with pytest.raises(gemm.GemmError) as e:
            gemm.gemm_testing_matvec_shape(M, 700, 32768, "bf16", 1, largest_cluster=4)
        assert e.value.status == gemm.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("change", [dict(M=0), dict(M=17), dict(N=0), dict(K=48), dict(K=32800), dict(x="f32"), dict(mode=0),
                                    dict(c=0), dict(c=9)])
def test_refusals(change):
    a = dict(M=1, N=64, K=64, x="bf16", mode=1, c=8) | change
    with pytest.raises(gemm.GemmError) as e:
        gemm.gemm_testing_matvec_shape(*a.values())
    assert e.value.status == gemm.GEMM_ERR_INVALID_ARG
