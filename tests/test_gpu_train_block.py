"""The operators together: a stack of MoE blocks against the same network in 64-bit autograd, and the
training example, eager and from a graph.

Tolerance of the gradients, by the 2-norm: a path from the output to a gradient passes up to sixteen
tensors that are rounded to bf16 (x's normed form, gu, h, dc, dh, dgu, dn in each of two blocks), each
by at most 2^-8 of the value: 16 * 2^-8."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D = torch.float64


def reference(stack, x, dx, choices):
    """Output and gradients in 64 bits, with the routing choices given."""
    ps = [{k: (stack.weights[l][k] if k in stack.weights[l] else v).to(D).requires_grad_() for k, v in p.items()}
          for l, p in enumerate(stack.params)]
    rms = lambda t: torch.sqrt((t * t).mean(1, keepdim=True) + stack.eps)
    x = x.to(D).requires_grad_()
    y, f = x, stack.f
    for p, idx in zip(ps, choices):
        n = p["w_pre"] * y / rms(y)
        w = torch.softmax(torch.gather(n @ p["w_router"], 1, idx.long()), 1)
        c = torch.zeros_like(y)
        for j in range(idx.shape[1]):
            gu = torch.einsum("td,tdf->tf", n, p["w_gate_up"][idx[:, j].long()])
            h = torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
            c = c + w[:, j:j + 1] * torch.einsum("tf,tfd->td", h, p["w_down"][idx[:, j].long()])
        y = p["res_scale"] * y + p["gate"] * p["w_post"] * c / rms(c)
    y.backward(dx.to(D))
    return y.detach(), x.grad, [{k: v.grad for k, v in p.items()} for p in ps]


@pytest.mark.parametrize("T,d,f,E,k", [(37, 64, 72, 8, 2), (1, 128, 64, 4, 1), (130, 256, 136, 16, 4)])
def test_stack_against_64_bits(T, d, f, E, k):
    from mixture_experts_grouped_fp32_gb300 import moe
    from mixture_experts_grouped_fp32_gb300.train import MoEStack
    stack = MoEStack(2, d, f, E, k, seed=5)
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, d, generator=g, device="cuda")
    dx = torch.randn(T, d, generator=g, device="cuda")
    for p in stack.params:
        for v in ("w_pre", "w_post", "gate", "res_scale"):
            p[v].add_(0.1 * torch.randn(d, generator=g, device="cuda"))
    y, saved = stack.forward(x)
    gx, grads = stack.backward(dx, saved)
    ry, rgx, rgrads = reference(stack, x, dx, [s[2][1] for s in saved])
    near = lambda a, b, what: torch.linalg.norm(a.double() - b) <= 16 * 2.0 ** -8 * torch.linalg.norm(b) or \
        pytest.fail(f"{what}: off by {float(torch.linalg.norm(a.double() - b) / torch.linalg.norm(b)):.3e}")
    near(y, ry, "y")
    near(gx, rgx, "dx")
    for l in range(2):
        assert set(grads[l]) == set(rgrads[l])
        for name in grads[l]:
            if k == 1 and name == "w_router":  # one choice: its weight is 1 whatever the logits
                continue
            near(grads[l][name], rgrads[l][name], f"{name} of block {l}")
    assert moe.get_device_error(stack.status) == 0


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_moe", os.path.join(ROOT, "examples", "train_moe.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_training_lowers_the_loss(example, bits):
    losses = example.train(steps=60, tokens=256, d=128, f=128, state_bits=bits, report=lambda s: None)
    assert all(l == l for l in losses)
    assert losses[-1] < 0.7 * losses[0]


def test_graph_replays_the_eager_steps(example):
    """The kernels add in fixed orders, so captured steps give the eager steps' losses bit for bit, but for
    torch's own products of the router (which may choose another algorithm under capture)."""
    kw = dict(steps=12, tokens=128, d=128, f=128, report=lambda s: None)
    eager, graph = example.train(**kw), example.train(graph=True, **kw)
    assert max(abs(a - b) for a, b in zip(eager, graph)) <= 1e-3 * eager[0]
