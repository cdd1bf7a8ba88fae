"""Operands of the training calls that are not where the call launches (the current device), a status word or a
workspace in host memory: refused by name, before the library is called.  Stand-ins for CUDA tensors: no GPU."""
import pytest
import torch

from mixture_experts_grouped_fp32_gb300 import moe

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Fake:
    """A contiguous CUDA tensor as the binding sees it."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, *shape, dtype=BF16, on=0, cuda=True):
        self.shape, self.dtype, self.on, self.is_cuda = torch.Size(shape), dtype, on, cuda
        self.nbytes = self.numel() * dtype.itemsize

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.on if self.is_cuda else -1

    def data_ptr(self):
        return 1 << 20


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """No launches: the library's calls are noted."""
    made = []
    monkeypatch.setattr(moe, "_fast", None)
    monkeypatch.setattr(moe, "_call", lambda name, *a: made.append(name))
    monkeypatch.setattr(moe, "_stream", lambda s: None)
    monkeypatch.setattr(moe, "_wrote", lambda *ts: None, raising=False)
    monkeypatch.setattr(moe, "grouped_mm_workspace_size", lambda *a: 0)
    monkeypatch.setattr(moe, "_several", True, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return made


def mm(a=0, b=0, o=0, out=0, status=None, workspace=None):
    return moe.grouped_mm(Fake(4, 8, on=a), Fake(2, 8, 16, on=b), Fake(3, dtype=I32, on=o), out=Fake(4, 16, on=out),
                          status=status, workspace=workspace)


def wgrad(a=0, g=0, out=0, status=None, workspace=None):
    return moe.grouped_mm_wgrad(Fake(4, 8, on=a), Fake(4, 16, on=g), Fake(3, dtype=I32),
                                out=Fake(2, 8, 16, dtype=F32, on=out), status=status, workspace=workspace)


def norm(x=0, h=0, w=0, y=0, n=0):
    v = lambda on=0: Fake(8, dtype=F32, on=on)
    return moe.block_norm(Fake(4, 8, on=x), v(w), Fake(4, 8, on=h), v(), y=Fake(4, 8, on=y), n=Fake(4, 8, on=n))


def test_operands_of_the_current_device_pass(calls):
    mm(status=Fake(1, dtype=I32), workspace=Fake(64, dtype=U8))
    wgrad(status=Fake(3, dtype=I32))
    norm()
    moe.swiglu(Fake(4, 16), Fake(4, dtype=F32), h=Fake(4, 8))
    assert calls == ["moe_grouped_mm", "moe_grouped_mm_wgrad", "moe_block_norm", "moe_swiglu"]


@pytest.mark.parametrize("call,where", [(mm, "a"), (mm, "b"), (mm, "o"), (mm, "out"), (wgrad, "a"), (wgrad, "g"),
                                        (wgrad, "out"), (norm, "x"), (norm, "h"), (norm, "w"), (norm, "y"), (norm, "n")])
def test_another_device_is_refused(calls, call, where):
    with pytest.raises(ValueError, match="is on device 1, the current one is 0"):
        call(**{where: 1})
    assert not calls


@pytest.mark.parametrize("call", [mm, wgrad])
def test_status_words_and_workspaces_must_be_on_the_device(calls, call):
    for status in (Fake(1, dtype=I32, cuda=False), Fake(1, dtype=F32), Fake(0, dtype=I32), torch.zeros(1, dtype=I32)):
        with pytest.raises(ValueError, match="status must be a CUDA int32"):
            call(status=status)
    with pytest.raises(ValueError, match="status is on device 1"):
        call(status=Fake(1, dtype=I32, on=1))
    with pytest.raises(ValueError, match="workspace must be a contiguous CUDA"):
        call(workspace=torch.zeros(64, dtype=U8))
    with pytest.raises(ValueError, match="workspace is on device 1"):
        call(workspace=Fake(64, dtype=U8, on=1))
    assert not calls


def test_norm_backward_workspace(calls, monkeypatch):
    monkeypatch.setattr(moe, "_empty", lambda shape, dtype, device, stream: Fake(*shape, dtype=dtype))
    x = Fake(4, 8)
    moe.block_norm_backward(x, dy=x, workspace=Fake(64, dtype=U8))
    assert calls == ["moe_block_norm_backward"]
    for ws in (torch.zeros(64, dtype=U8), Fake(64, dtype=U8, on=1)):
        with pytest.raises(ValueError, match="workspace"):
            moe.block_norm_backward(x, dy=x, workspace=ws)
