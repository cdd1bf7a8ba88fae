"""Train a small stack of MoE blocks to imitate another one, on one GB300.

    python examples/train_moe.py [--steps 50] [--tokens 512] [--layers 2] [--d 256] [--f 512]
                                 [--experts 8] [--top-k 2] [--state-bits 8|32] [--graph]
                                 [--norm rms|layer] [--dropout 0.1] [--scoring softmax|sigmoid]
                                 [--groups 4 --kept 2] [--bias-rate 1e-3] [--balance 0.01] [--vocab 1000]

Every step draws inputs, runs forward, backward and AdamW with this package's kernels and prints the mean
squared error.  With --graph the whole step is captured once and replayed.  --scoring replaces the softmax router (with
groups, a bias that follows the loads, a balancing loss); --vocab makes the stacks read tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_grouped_fp32_gb300 import moe  # noqa: E402
from mixture_experts_grouped_fp32_gb300.train import MoEStack  # noqa: E402


def train(steps=50, tokens=512, layers=2, d=256, f=512, experts=8, top_k=2, state_bits=32, graph=False, lr=3e-3,
          norm="rms", dropout=0.0, scoring=None, groups=1, kept=1, bias_rate=0.0, balance=0.0, vocab=None, report=print):
    """Returns the losses of all steps (a device tensor is read once, at the end)."""
    if scoring is None and (groups, kept, bias_rate, balance) != (1, 1, 0.0, 0.0):
        raise ValueError("groups, kept, bias_rate and balance are options of a router by scores: give scoring")
    router = None if scoring is None else dict(scoring=scoring, n_group=groups, topk_group=kept, bias_rate=bias_rate,
                                               balance=balance)
    teacher = MoEStack(layers, d, f, experts, top_k, seed=1, norm=norm, vocab=vocab)
    student = MoEStack(layers, d, f, experts, top_k, state_bits=state_bits, seed=2, norm=norm, dropout=dropout,
                       router=router, vocab=vocab)
    gen = torch.Generator("cuda").manual_seed(3)
    if vocab is None:
        batches = torch.randn(8, tokens, d, generator=gen, device="cuda")
    else:
        batches = torch.randint(0, vocab, (8, tokens), generator=gen, device="cuda")
    targets = torch.stack([teacher.forward(x)[0] for x in batches])
    x, target = torch.empty_like(batches[0]), torch.empty_like(targets[0])
    loss = torch.zeros((), device="cuda")

    def one_step():
        y, saved = student.forward(x)
        diff = y - target
        loss.copy_(diff.square().mean())
        _, grads = student.backward(diff * (2.0 / diff.numel()), saved)
        student.step(grads, lr=lr)

    losses = torch.zeros(steps, device="cuda")
    replay = None
    for i in range(steps):
        x.copy_(batches[i % 8])
        target.copy_(targets[i % 8])
        if graph and i == 2:  # two eager steps warm everything up
            replay = torch.cuda.CUDAGraph()
            with torch.cuda.graph(replay):
                one_step()
        if replay is not None:
            replay.replay()
        else:
            one_step()
        losses[i] = loss
    status = moe.get_device_error(student.status)
    if status:
        raise RuntimeError(f"a kernel reported device status {status:#x}")
    losses = losses.tolist()
    for i in range(0, steps, max(1, steps // 10)):
        report(f"step {i:4d}  mean squared error {losses[i]:.5f}")
    report(f"step {steps - 1:4d}  mean squared error {losses[-1]:.5f}")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--d", type=int, default=256)
    ap.add_argument("--f", type=int, default=512)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    ap.add_argument("--graph", action="store_true")
    ap.add_argument("--lr", type=float, default=3e-3)
    ap.add_argument("--norm", default="rms", choices=("rms", "layer"))
    ap.add_argument("--dropout", type=float, default=0.0)
    ap.add_argument("--scoring", choices=("softmax", "sigmoid"))
    ap.add_argument("--groups", type=int, default=1)
    ap.add_argument("--kept", type=int, default=1)
    ap.add_argument("--bias-rate", type=float, default=0.0)
    ap.add_argument("--balance", type=float, default=0.0)
    ap.add_argument("--vocab", type=int)
    train(**vars(ap.parse_args()))


if __name__ == "__main__":
    main()
