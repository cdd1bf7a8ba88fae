"""The norms over as many rows as the calls accept, where T plus the number of thread blocks passes 2^31: every
row of the outputs is written, and equals that of a small call of the same rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
MOST = 2 ** 31 - 1025


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_fp32_gb300 import moe as m
    yield m
    torch.cuda.empty_cache()


def inputs(T, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(T, 8, dtype=BF16, device="cuda").uniform_(-1, 1, generator=gen)


def unwritten(t, step=1 << 26):
    return sum(int(t[r:r + step].isnan().any(1).sum()) for r in range(0, t.shape[0], step))


def test_block_norm(moe):
    x, h, w = inputs(MOST, 1), inputs(MOST, 2), torch.rand(8, device="cuda") + 0.5
    y, n = (torch.full((MOST, 8), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    moe.block_norm(x, w, h, w, y=y, n=n)
    assert unwritten(y) == 0 and unwritten(n) == 0
    for lo in (0, 1 << 30, MOST - 5000):
        rows = slice(lo, lo + 5000)
        for a, b in zip((y, n), moe.block_norm(x[rows].clone(), w, h[rows].clone(), w)):
            assert torch.equal(a[rows], b)


def test_block_norm_without_a_block(moe):
    x, w = inputs(MOST, 1), torch.rand(8, device="cuda") + 0.5
    n = torch.full((MOST, 8), float("nan"), dtype=BF16, device="cuda")
    moe.block_norm(x, w, n=n)
    assert unwritten(n) == 0
    assert torch.equal(n[-5000:], moe.block_norm(x[-5000:].clone(), w)[1])


def test_block_norm_backward(moe):
    x, dn, w = inputs(MOST, 1), inputs(MOST, 2), torch.rand(8, device="cuda") + 0.5
    g = moe.block_norm_backward(x, dn=dn, w_pre=w)
    for lo in (0, 1 << 30, MOST - 5000):
        rows = slice(lo, lo + 5000)
        assert torch.equal(g["x"][rows], moe.block_norm_backward(x[rows].clone(), dn=dn[rows].clone(), w_pre=w)["x"])
