"""Refusals of the training operators, without a GPU: the C entry points return before any CUDA call."""
import ctypes
import os

import pytest

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_grouped_fp32_gb300 import build, moe
    if not os.path.exists(moe.LIB_PATH):
        build.build()
    return moe.load()


def _err(lib):
    return lib.moe_last_error_string().decode()


@pytest.mark.parametrize("M,K,N,E,fragment", [
    (-1, 64, 64, 4, "M = -1"),
    (4, 60, 64, 4, "K = 60"),
    (4, 0, 64, 4, "K = 0"),
    (4, 64, 65544, 4, "N = 65544"),
    (4, 64, 12, 4, "N = 12"),
    (4, 64, 64, 0, "E = 0"),
    (4, 64, 64, 257, "E = 257"),
])
def test_grouped_mm_refuses_shapes(lib, M, K, N, E, fragment):
    assert lib.moe_grouped_mm(P, P, P, M, K, N, E, 0, P, 1, None, 0, None, None) == -1
    assert fragment in _err(lib)
    assert lib.moe_grouped_mm_wgrad(P, P, P, M, K, N, E, P, 1, 0, None, 0, None, None) == -1
    assert fragment in _err(lib)
    assert lib.moe_grouped_mm_workspace_size(0, M, K, N, E) == 0


def test_grouped_mm_refuses_pointers_and_workspaces(lib):
    mm = lambda a=P, b=P, o=P, out=P, ws=None, n=0, M=4, K=64: lib.moe_grouped_mm(
        a, b, o, M, K, 64, 4, 0, out, 1, ws, n, None, None)
    for kw in ({"a": None}, {"b": None}, {"o": None}, {"out": None}):
        assert mm(**kw) == -1 and "null" in _err(lib)
    for kw in ({"a": ODD}, {"b": ODD}, {"out": ODD}, {"ws": ODD}, {"o": ODD}):
        assert mm(**kw) == -1 and "aligned" in _err(lib)
    need = lib.moe_grouped_mm_workspace_size(0, 2, 8192, 64, 4)
    assert need > 0
    assert mm(ws=P, n=need - 1, M=2, K=8192) == -3
    assert lib.moe_grouped_mm_wgrad(P, P, P, 4, 64, 64, 4, P, 0, 1, None, 0, None, None) == -1
    assert "accumulate" in _err(lib)
    assert mm(M=0) == 0  # no rows: nothing to do, and no CUDA call
    assert lib.moe_grouped_mm_wgrad(P, P, P, 0, 64, 64, 4, P, 1, 1, None, 0, None, None) == 0
    assert lib.moe_grouped_mm_workspace_size(3, 4, 64, 64, 4) == 0


def test_python_refuses_before_the_library():
    import torch

    from mixture_experts_grouped_fp32_gb300 import moe
    a, b, o = torch.zeros(4, 64).bfloat16(), torch.zeros(2, 64, 8).bfloat16(), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        moe.grouped_mm(a, b, o)
    with pytest.raises(ValueError, match="CUDA"):
        moe.grouped_mm_wgrad(a, a, o)
