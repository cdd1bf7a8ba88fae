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


def versions(ts):
    return [t._version for t in ts]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("device_step", [False, True])
def test_adamw_raises_the_versions_of_parameters_and_copies(moe, bits, device_step):
    p = [torch.ones(300, device="cuda"), torch.ones(7, device="cuda")]
    g, copies = [torch.ones_like(t) for t in p], [t.bfloat16() for t in p]
    state = list(zip(*(moe.adamw_state(t, bits) for t in p)))
    written = [*p, *copies]  # (the moments are the optimizer's own: no graph has them)
    before, grads = versions(written), versions(g)
    kw = {"step_tensor": torch.ones(1, dtype=torch.int32, device="cuda")} if device_step else {}
    if bits == 8:
        kw.update(m_scales=list(state[2]), v_scales=list(state[3]))
    moe.adamw_step(p, g, list(state[0]), list(state[1]), lr=1e-3, copies=copies, **kw)
    assert all(a > b for a, b in zip(versions(written), before)) and versions(g) == grads


def test_a_graph_that_saved_a_parameter_notices_its_step(moe):
    p = torch.ones(16, device="cuda", requires_grad=True)
    loss = (p * p).sum()  # saves p
    s = moe.adamw_state(p.detach())
    moe.adamw_step([p], [torch.ones(16, device="cuda")], [s[0]], [s[1]], lr=1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_that_are_given_count_as_written(moe):
    offs = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    a, b, gu, x, w = z(4, 8), z(1, 8, 16), z(4, 16), z(4, 8), z(8, dtype=F32)
    rows = z(4, dtype=F32)
    calls = {
        "grouped_mm": lambda o: moe.grouped_mm(a, b, offs, out=o[0]),
        "grouped_mm_wgrad": lambda o: moe.grouped_mm_wgrad(a, z(4, 16), offs, out=o[0], accumulate=True),
        "swiglu": lambda o: moe.swiglu(gu, h=o[0]),
        "swiglu_backward": lambda o: moe.swiglu_backward(gu, a, rows, dgu=o[0], dw=o[1], h=o[2]),
        "block_norm": lambda o: moe.block_norm(x, w, a, w, y=o[0], n=o[1]),
    }
    outs = {"grouped_mm": [z(4, 16)], "grouped_mm_wgrad": [z(1, 8, 16, dtype=F32)], "swiglu": [z(4, 8)],
            "swiglu_backward": [z(4, 16), z(4, dtype=F32), z(4, 8)], "block_norm": [z(4, 8), z(4, 8)]}
    for name, call in calls.items():
        before = versions(outs[name])
        call(outs[name])
        assert all(n > o for n, o in zip(versions(outs[name]), before)), name
    assert versions([a, b, gu, x, w, rows]) == [0] * 6


def test_inference_tensors_have_no_versions_to_raise(moe):
    with torch.inference_mode():
        p, g, m, v = (torch.ones(16, device="cuda") for _ in range(4))
        moe.adamw_step([p], [g], [m], [v], lr=1e-3)
        out = torch.ones(1, 8, 16, device="cuda")
        moe.grouped_mm_wgrad(z(4, 8), z(4, 16), torch.tensor([0, 4], dtype=torch.int32, device="cuda"), out=out)
    moe.adamw_step([p], [g], [m], [v], lr=1e-3)
    assert (p < 1).all() and (out == 0).all()
