"""How the training calls behave as Python functions, through the C++ binding and through ctypes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", params=["fast", "ctypes"])
def moe(request):
    from mixture_experts_grouped_fp32_gb300 import moe as m
    m.load()
    fast = m._fast
    if request.param == "fast" and fast is None:
        pytest.skip("_moe_fast.so was not built here")
    m._fast = fast if request.param == "fast" else None
    yield m
    m._fast = fast


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_a_failed_allocation_is_torchs_error(moe):
    """Callers catch torch.OutOfMemoryError (to retry with less): 34 GB of output under a limit of 14."""
    a, b, offs = z(1 << 20, 8), z(1, 8, 8192), torch.tensor([0, 1 << 20], dtype=torch.int32, device="cuda")
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.05)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            moe.grouped_mm(a, b, offs, out_dtype=F32)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert moe.grouped_mm(a[:8], b, offs.clamp_max(8)).shape == (8, 8192)
