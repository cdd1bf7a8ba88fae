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


def test_swiglu_refuses(lib):
    assert lib.moe_swiglu(P, None, 4, 60, P, None) == -1 and "f = 60" in _err(lib)
    assert lib.moe_swiglu(P, None, -1, 64, P, None) == -1 and "M = -1" in _err(lib)
    assert lib.moe_swiglu(None, None, 4, 64, P, None) == -1 and "null" in _err(lib)
    assert lib.moe_swiglu(ODD, None, 4, 64, P, None) == -1 and "aligned" in _err(lib)
    assert lib.moe_swiglu(None, None, 0, 64, None, None) == 0
    bwd = lambda gu=P, dh=P, w=None, M=4, f=64, dgu=P, dw=None, h=None: lib.moe_swiglu_backward(
        gu, dh, w, M, f, dgu, dw, h, None)
    for kw in ({"gu": None}, {"dh": None}, {"dgu": None}):
        assert bwd(**kw) == -1 and "null" in _err(lib)
    for kw in ({"gu": ODD}, {"dh": ODD}, {"dgu": ODD}, {"h": ODD}, {"w": ODD}, {"dw": ODD}):
        assert bwd(**kw) == -1 and "aligned" in _err(lib)
    assert bwd(f=65544) == -1 and bwd(M=0) == 0


def test_block_norm_refuses(lib):
    fwd = lambda x=P, h=P, w_pre=P, w_post=P, gate=None, tgate=None, res=None, T=4, d=64, eps=1e-6, y=P, n=P: \
        lib.moe_block_norm(x, 1, h, w_pre, w_post, gate, tgate, res, T, d, eps, y, n, None)
    for kw, word in (({"d": 60}, "d = 60"), ({"d": 65544}, "d = 65544"), ({"T": -1}, "T = -1"),
                     ({"eps": -1.0}, "eps"), ({"eps": float("nan")}, "eps"), ({"w_post": None}, "w_post"),
                     ({"h": None}, "belong"), ({"n": None}, "together"), ({"w_pre": None}, "together"),
                     ({"x": None}, "null"), ({"x": ODD}, "aligned"), ({"gate": ODD}, "aligned"),
                     ({"tgate": ODD}, "aligned"), ({"y": None, "w_pre": None, "n": None}, "null")):
        assert fwd(**kw) == -1 and word in _err(lib), kw
    assert fwd(T=0) == 0
    need = lib.moe_block_norm_backward_workspace_size(4, 64)
    assert need == 4 * 3 * 64 * 4 and lib.moe_block_norm_backward_workspace_size(4, 60) == 0

    def bwd(x=P, h=P, dy=P, dn=P, w_pre=P, w_post=P, gate=None, tgate=None, res=None, T=4, d=64, dx=P, dh=P,
            dw_pre=None, dw_post=None, dgate=None, dtgate=None, dres=None, ws=P, n=need):
        return lib.moe_block_norm_backward(x, 0, h, dy, dn, w_pre, w_post, gate, tgate, res, T, d, 1e-6, dx, dh,
                                           dw_pre, dw_post, dgate, dtgate, dres, ws, n, None)
    for kw, word in (({"d": 12}, "d = 12"), ({"w_pre": None}, "dn needs"), ({"dgate": P}, "NULL"), ({"dres": P}, "NULL"),
                     ({"dtgate": P}, "NULL"), ({"dx": None}, "null"), ({"dh": None}, "null"),
                     ({"dy": None, "dn": None}, "null"), ({"dn": None, "dw_pre": P}, "needs dn"),
                     ({"h": None, "w_post": None, "dw_post": P}, "belong"), ({"dh": ODD}, "aligned"),
                     ({"dw_post": ctypes.c_void_p(3)}, "aligned")):
        assert bwd(**kw) == -1 and word in _err(lib), kw
    assert bwd(n=need - 1) == -3 and bwd(ws=None) == -3
    assert bwd(T=0) == 0


def test_adamw_refuses(lib):
    import numpy as np

    from mixture_experts_grouped_fp32_gb300 import moe

    def call(bits=32, count=1, betas=(0.9, 0.99), eps=1e-8, lr=1e-3, wd=0.1, step=1, table=True, **entry):
        t = np.zeros(1, moe._ADAMW_ENTRY)
        for k, v in {"param": 1 << 20, "grad": 1 << 20, "m": 1 << 20, "v": 1 << 20, "n": 10, **entry}.items():
            t[k] = v
        return lib.moe_adamw_step(t.ctypes.data if table else None, count, 0, 1, bits, lr, *betas, eps, wd, step, None,
                                  None, None)
    for kw, word in (({"bits": 16}, "state_bits"), ({"count": -1}, "count"), ({"betas": (1.0, 0.9)}, "betas"),
                     ({"betas": (0.9, -0.1)}, "betas"), ({"eps": -1.0}, "eps"), ({"lr": float("inf")}, "finite"),
                     ({"wd": float("nan")}, "finite"), ({"step": 0}, "step = 0"), ({"table": False}, "null"),
                     ({"param": 0}, "null"), ({"m": 0}, "null"), ({"bits": 8}, "null"), ({"param": (1 << 20) + 2}, "aligned"),
                     ({"grad": (1 << 20) + 1}, "aligned"), ({"v": (1 << 20) + 2}, "aligned"),
                     ({"copy": (1 << 20) + 1}, "aligned"), ({"n": (1 << 40) + 1}, "outside")):
        assert call(**kw) == -1 and word in _err(lib), kw
    assert call(count=0) == 0


def test_python_refusals_of_the_other_operators():
    import torch

    from mixture_experts_grouped_fp32_gb300 import moe
    t = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.swiglu(t.bfloat16())
    with pytest.raises(ValueError, match="CUDA"):
        moe.block_norm(t, torch.zeros(64))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        moe.block_norm(t.half())
    with pytest.raises(ValueError, match="CUDA"):
        moe.adamw_step([t], [t], [t], [t], lr=1e-3)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        moe.adamw_step([t.half()], [t], [t], [t], lr=1e-3)
    with pytest.raises(ValueError, match="m_scales"):
        moe.adamw_step([t], [t], [t.to(torch.float8_e4m3fn)], [t.to(torch.float8_e4m3fn)], lr=1e-3)
    with pytest.raises(ValueError, match="8 or 32"):
        moe.adamw_state(t, 16)
    q = moe.adamw_state(t, 8)
    assert q[0].dtype is torch.float8_e4m3fn and q[2].shape == (1,) and (q[3] == 1).all()
    assert moe.adamw_step([], [], [], [], lr=1e-3) is None
