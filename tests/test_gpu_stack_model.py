"""Embedding, layer norm, dropout and routing by scores as they are used together: stacks of MoE blocks against the same
networks in 64-bit autograd, with the choices and masks given, and the training example with them.

Tolerance of the gradients, by the 2-norm, as for the plain stack: a path from the output to a gradient passes up to
eighteen tensors that are rounded to bf16 (n, gu, h, c, dc, dh, dgu, dn in each of two blocks, twice for the last block's
dc), each by at most 2^-8 of the value: 18 * 2^-8."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D = torch.float64


def reference(stack, x, dx, choices, masks):
    """Output and gradients in 64 bits; `masks` multiply the blocks' outputs."""
    ps = [{k: (stack.weights[l][k] if k in stack.weights[l] else v).to(D).requires_grad_() for k, v in p.items()}
          for l, p in enumerate(stack.params)]
    rms = lambda t: torch.sqrt((t * t).mean(1, keepdim=True) + stack.eps)
    if stack.vocab is not None:
        x = y = (ps[0]["w_embed"][x.long()] * stack.embed_scale)
        x.retain_grad()
    else:
        x = y = x.to(D).requires_grad_()
    f, r, extra = stack.f, stack.router, 0.0

    def normed(t, p):
        if stack.norm == "rms":
            return p["w_pre"] * t / rms(t)
        m = t - t.mean(1, keepdim=True)
        return p["w_pre"] * m / rms(m) + p["b_pre"]
    for p, idx, mask in zip(ps, choices, masks):
        n = normed(y, p)
        logits = n @ p["w_router"]
        if r is None:
            w = torch.softmax(torch.gather(logits, 1, idx.long()), 1)
        else:
            s = torch.softmax(logits, 1) if r["scoring"] == "softmax" else torch.sigmoid(logits)
            w = torch.gather(s, 1, idx.long())
            w = r["scale"] * (w / w.sum(1, keepdim=True) if r["renormalize"] else w)
            load = torch.bincount(idx.view(-1).long(), minlength=stack.E).to(D) / idx.numel()
            extra = extra + r["balance"] * stack.E * (load * s.mean(0)).sum()
        c = torch.zeros_like(y)
        for j in range(idx.shape[1]):
            gu = torch.einsum("td,tdf->tf", n, p["w_gate_up"][idx[:, j].long()])
            h = torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
            c = c + w[:, j:j + 1] * torch.einsum("tf,tfd->td", h, p["w_down"][idx[:, j].long()])
        c = c * mask
        y = y + c if stack.norm == "layer" else p["res_scale"] * y + p["gate"] * p["w_post"] * c / rms(c)
    ((y * dx.to(D)).sum() + extra).backward()
    return y.detach(), x.grad, [{k: v.grad for k, v in p.items()} for p in ps]


SIGMOID = dict(scoring="sigmoid", n_group=4, topk_group=2, scale=2.5, bias_rate=0.01)
CASES = [  # T, d, f, E, k, options
    (37, 64, 72, 8, 2, dict(norm="layer")),
    (130, 128, 136, 16, 4, dict(norm="layer", dropout=0.25, router=dict(scoring="softmax", renormalize=False, scale=2.0), vocab=50)),
    (65, 256, 64, 16, 3, dict(norm="layer", dropout=0.1, router={**SIGMOID, "balance": 0.5})),
    (33, 64, 64, 8, 2, dict(norm="rms", dropout=0.5, router=dict(scoring="softmax", balance=1.0), vocab=11)),
    (1, 64, 64, 8, 2, dict(norm="layer", dropout=0.3, vocab=3)),
]


@pytest.mark.parametrize("T,d,f,E,k,options", CASES)
def test_stack_against_64_bits(T, d, f, E, k, options):
    from mixture_experts_grouped_fp32_gb300 import moe
    from mixture_experts_grouped_fp32_gb300.train import MoEStack
    stack = MoEStack(2, d, f, E, k, seed=5, **options)
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, d, generator=g, device="cuda") if stack.vocab is None else \
        torch.randint(0, stack.vocab, (T,), generator=g, device="cuda")
    dx = torch.randn(T, d, generator=g, device="cuda")
    for p in stack.params:
        for v in ("w_pre", "b_pre", "w_post", "gate", "res_scale"):
            if v in p:
                p[v].add_(0.1 * torch.randn(d, generator=g, device="cuda"))
    for b in stack.biases:
        if b is not None:
            b.add_(0.05 * torch.randn(E, generator=g, device="cuda"))
    stack.mask_number.fill_(6)
    y, saved = stack.forward(x)
    gx, grads = stack.backward(dx, saved)
    masks = [moe.dropout(torch.ones(T, d, device="cuda"), stack.p, stack.seed, 6 + l).to(D) for l in range(2)]
    ry, rgx, rgrads = reference(stack, x, dx, [s[2][1] for s in saved], masks)
    near = lambda a, b, what: torch.linalg.norm(a.double() - b) <= 18 * 2.0 ** -8 * torch.linalg.norm(b) or \
        pytest.fail(f"{what}: off by {float(torch.linalg.norm(a.double() - b) / torch.linalg.norm(b)):.3e}")
    near(y, ry, "y")
    near(gx, rgx, "dx")
    for l in range(2):
        assert set(grads[l]) == set(rgrads[l])
        for name in grads[l]:
            near(grads[l][name], rgrads[l][name], f"{name} of block {l}")
    assert moe.get_device_error(stack.status) == 0
    before = [b.clone() if b is not None else None for b in stack.biases]
    stack.step(grads)
    assert stack.mask_number.item() == (8 if stack.p else 6)
    for b, old, load in zip(stack.biases, before, stack.loads):
        if b is not None:
            assert load.sum() == T * k and torch.equal(torch.sign(b - old), torch.sign(load.sum() / E - load))


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_other_passes_between_a_forward_pass_and_its_backward_pass(norm):
    """The masks and loads of a pass are its own; one that does not train changes neither."""
    from mixture_experts_grouped_fp32_gb300.train import MoEStack
    new = lambda: MoEStack(2, 64, 64, 8, 2, norm=norm, dropout=0.25, router=dict(balance=0.5, bias_rate=0.1))
    g = torch.Generator("cuda").manual_seed(2)
    x, other, dx = (torch.randn(T, 64, generator=g, device="cuda") for T in (40, 70, 40))
    a, b = new(), new()
    ya, saved = a.forward(x)
    want = a.backward(dx, saved)
    yb, saved = b.forward(x)
    assert torch.equal(ya, yb)
    loads = [t.clone() for t in b.loads]
    plain = b.forward(other, train=False)[0]
    assert all(torch.equal(s, t) for s, t in zip(loads, b.loads)) and b.mask_number.item() == 2
    assert torch.equal(plain, b.forward(other, train=False)[0])
    trained = b.forward(other)[0]
    assert b.mask_number.item() == 4 and not torch.equal(plain, trained) and not torch.equal(trained, b.forward(other)[0])
    got = b.backward(dx, saved)
    assert torch.equal(got[0], want[0])
    for s, t in zip(got[1], want[1]):
        assert all(torch.equal(s[k], t[k]) for k in t)
    out, saved = b.forward(x, train=False)
    assert all(torch.isfinite(v).all() for s in b.backward(dx, saved)[1] for v in s.values())


def test_options_that_there_are_not():
    from mixture_experts_grouped_fp32_gb300.train import MoEStack
    with pytest.raises(ValueError, match="norm must be"):
        MoEStack(1, 64, 64, 4, 1, norm="batch")
    with pytest.raises(ValueError, match="router has no"):
        MoEStack(1, 64, 64, 4, 1, router=dict(score="softmax"))


def test_a_token_outside_the_vocabulary_is_reported():
    from mixture_experts_grouped_fp32_gb300 import moe
    from mixture_experts_grouped_fp32_gb300.train import MoEStack
    stack = MoEStack(1, 64, 64, 4, 1, vocab=10, norm="layer")
    stack.forward(torch.tensor([1, 10, 2], device="cuda"))
    assert moe.get_device_error(stack.status) == moe.STATUS_BAD_TOKEN


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_moe", os.path.join(ROOT, "examples", "train_moe.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("options", [
    dict(norm="layer", dropout=0.1, scoring="sigmoid", groups=4, kept=2, bias_rate=1e-3, balance=0.01, vocab=100),
    dict(dropout=0.2, scoring="softmax", balance=0.1)])
def test_graph_replays_the_eager_steps(example, options):
    """The kernels add in fixed orders and the masks follow the step on the device, so captured steps give the eager steps'
    losses bit for bit, but for torch's own products of the router (which may choose another algorithm under capture)."""
    kw = dict(steps=12, tokens=128, d=128, f=128, report=lambda s: None, **options)
    eager, graph = example.train(**kw), example.train(graph=True, **kw)
    assert all(a == a for a in eager)
    assert max(abs(a - b) for a, b in zip(eager, graph)) <= 1e-3 * eager[0]
