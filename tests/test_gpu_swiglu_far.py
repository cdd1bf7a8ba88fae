"""SwiGLU and its gradient where exp(-g) comes near the largest fp32 value: g from -104 to -80 with large u.

exp(g) is below the smallest normal number from g = -87.3 on and has steps of 2^-149 there; the kernel's values are
that number, off by one step at most, times |g u| and a factor near one, rounded once to bf16 (2^-8)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, D = torch.bfloat16, torch.float64


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("u", [1.0, -3e20, 1e37])
def test_far_negative_gates(u, weighted):
    from mixture_experts_grouped_fp32_gb300 import moe
    g = torch.cat([torch.linspace(-104, -80, 505), torch.tensor([-88.0, -87.5, -88.5])]).to(BF16)
    f = -(-g.numel() // 8) * 8
    g = torch.nn.functional.pad(g, (0, f - g.numel()), value=-88.0)
    gu = torch.cat([g, torch.full((f,), u).to(BF16)])[None]
    dh = torch.full((1, f), 0.5).to(BF16)
    w = torch.tensor([0.75]) if weighted else None
    dev = lambda t: None if t is None else t.cuda()
    x = gu.to(D).requires_grad_()
    w64 = torch.tensor([0.75 if weighted else 1.0], dtype=D, requires_grad=True)
    ref = w64[:, None] * x[:, :f] * torch.exp(x[:, :f]) / (1 + torch.exp(x[:, :f])) * x[:, f:]
    ref.backward(dh.to(D))
    size = (x.detach()[:, :f] * x.detach()[:, f:]).abs()

    def near(got, want, scale, what):
        off = (got.cpu().to(D) - want).abs()
        # (1 + 2^-18 for the few fp32 operations; bf16's own steps below its normal numbers are 2^-133)
        bound = (2.0 ** -8 + 2.0 ** -18) * want.abs() + 2.0 ** -148 * scale + 2.0 ** -134
        assert (off <= bound).all(), f"{what}: {float((off / bound).max())} of the bound at g = {g[int((off / bound).argmax()) % f]}"

    h = moe.swiglu(dev(gu), dev(w))
    near(h, ref.detach(), size, "h")
    dgu, dw, h2 = moe.swiglu_backward(dev(gu), dev(dh), dev(w), want_h=True)
    assert torch.equal(h, h2)
    scale = torch.cat([size * 2, x.detach()[:, :f].abs()], 1)  # |dg| <= |u| s (1 + |g|)
    near(dgu, x.grad, scale, "dgu")
    if weighted:
        want = float(w64.grad)
        assert abs(float(dw[0]) - want) <= 2.0 ** -18 * float((dh.to(D) * ref.detach() / 0.75).abs().sum()) + \
            2.0 ** -148 * float(size.sum()) + 2.0 ** -134


def test_ordinary_gates_near_zero_and_signs():
    """Both branches meet at zero, and the sigmoid of g and of -g add up to one."""
    from mixture_experts_grouped_fp32_gb300 import moe
    g = torch.tensor([0.0, -0.0, 2.0 ** -130, -2.0 ** -130, 1e-3, -1e-3, 5.0, -5.0]).to(BF16)
    gu = torch.cat([g, torch.ones(8, dtype=BF16)])[None].cuda()
    h = moe.swiglu(gu)[0].cpu().to(D)
    want = g.to(D) / (1 + torch.exp(-g.to(D)))
    assert ((h - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs() + 2.0 ** -134).all()
    assert float(h[0]) == 0 and float(h[1]) == 0
