"""The gradient that the last block of a layer-norm stack gets is the output's, dropped and rounded to bf16 once."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = torch.float64


@pytest.mark.parametrize("p", [0.0, 0.1, 0.4])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_the_last_blocks_gradient_is_rounded_once(p, dt):
    """Half a step of bf16 (2^-8 of the value), and the fp32 product of the dropout before it (two roundings of 2^-24: the
    factor's and the product's) where the stream has 32 bits.  A second rounding to bf16 would be off by up to 2^-7."""
    from mixture_experts_grouped_fp32_gb300 import moe
    from mixture_experts_grouped_fp32_gb300.train import MoEStack
    g = torch.Generator("cuda").manual_seed(3)
    stack = MoEStack(2, 64, 64, 8, 2, norm="layer", dropout=p, seed=9)
    x, dx = torch.randn(300, 64, generator=g, device="cuda").to(dt), torch.randn(300, 64, generator=g, device="cuda").to(dt)
    got, inner = [], stack._experts_backward

    def watched(dc, *rest):
        got.append(dc.clone())
        return inner(dc, *rest)
    stack._experts_backward = watched
    before = dx.clone()
    stack.backward(dx, stack.forward(x)[1])
    assert torch.equal(dx, before)
    keep = moe.dropout(torch.ones(300, 64, device="cuda"), p, 9, 1).ne(0)
    cut = round(p * 65536)
    want = torch.where(keep, dx.to(D) * (65536 / (65536 - cut)), 0.0)
    assert got[0].dtype is torch.bfloat16 and torch.equal(got[0].ne(0), want.ne(0))
    assert (got[0].to(D) - want).abs().le((2.0 ** -8 + 2.0 ** -22) * want.abs()).all()
