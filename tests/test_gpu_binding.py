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


STUB = r"""
#include <stddef.h>
#include <time.h>
#define API __attribute__((visibility("default")))
API volatile int entered, go;
/* Waits up to 3 s for another thread of the interpreter to set `go`. */
API int moe_swiglu() {
    struct timespec ms = {0, 1000000};
    entered = 1;
    for (int i = 0; i < 3000 && !go; ++i) nanosleep(&ms, NULL);
    return go ? 0 : 99;
}
API int moe_swiglu_backward() { return 0; }
API int moe_block_norm() { return 0; }
API int moe_block_norm_backward() { return 0; }
API size_t moe_block_norm_backward_workspace_size() { return 0; }
API int moe_grouped_mm() { return 0; }
API int moe_grouped_mm_wgrad() { return 0; }
API size_t moe_grouped_mm_workspace_size() { return 0; }
API int moe_adamw_step() { return 0; }
"""


def test_other_threads_run_during_a_call(tmp_path):
    """A call that waits (here in a library that stands in for the real one) does not hold the interpreter lock."""
    import ctypes
    import shutil
    import subprocess
    import threading
    import time

    from mixture_experts_grouped_fp32_gb300 import moe as m
    m.load()
    fast = pytest.importorskip("mixture_experts_grouped_fp32_gb300._moe_fast")
    if not shutil.which("gcc"):
        pytest.skip("no gcc")
    src, lib = tmp_path / "stub.c", tmp_path / "libstub.so"
    src.write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    stub = ctypes.CDLL(str(lib))
    entered, go = (ctypes.c_int.in_dll(stub, n) for n in ("entered", "go"))
    gu, result = z(4, 16), []
    fast.init(str(lib))
    try:
        caller = threading.Thread(target=lambda: result.append(fast.swiglu(gu, None)))
        caller.start()
        end = time.time() + 10
        while not entered.value and time.time() < end:
            time.sleep(0.001)
        go.value = 1
        caller.join()
    finally:
        fast.init(m.LIB_PATH)
    assert isinstance(result[0], torch.Tensor), "the call held the lock until it gave up"
