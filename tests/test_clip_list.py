"""Lists that gemm_clip_run cannot take are refused as they are laid out."""
import pytest

from blackwell_tensor_core_tma_gb300 import gemm

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kind", ["e4m3", "e2m1", gemm.GEMM_E4M3, 17])
def test_a_type_without_a_norm(kind):
    """As a tensor of another type is: by the error that says what the tensor's is."""
    for g in (torch.zeros(8), torch.zeros(8, dtype=torch.uint8), torch.zeros(8).to(torch.float8_e4m3fn)):
        with pytest.raises(ValueError):
            gemm.clip_tensors([(g, None, kind)])
