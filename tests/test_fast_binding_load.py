"""The C++ binding is used only with the torch that it was built against (its view of a tensor is that torch's)."""
import ctypes
import os

import pytest
import torch

from mixture_experts_grouped_fp32_gb300 import moe


@pytest.fixture
def fresh(monkeypatch):
    """A binding that has not loaded the library yet."""
    if not os.path.exists(os.path.join(os.path.dirname(moe.LIB_PATH), "_moe_fast.so")):
        pytest.skip("_moe_fast.so was not built here")
    for name, value in (("_lib", None), ("_fast", None), ("_fns", {})):
        monkeypatch.setattr(moe, name, value)


def test_used_with_its_own_torch(fresh):
    moe.load()
    assert moe._fast is not None and moe._fast.torch_version == torch.__version__


def test_not_used_with_another_torch(fresh, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert isinstance(moe.load(), ctypes.CDLL)
    assert moe._fast is None
