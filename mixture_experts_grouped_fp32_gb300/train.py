"""A stack of MoE blocks trained with this package's kernels: forward, backward and AdamW.

Block l takes the residual stream x [T, d] and its normed form n:

    c    = experts(n)                                    routed SwiGLU experts, weights from the router
    x    = res * x + gate * (w_post * c / rms(c))        norm after the block, gate, residual scale
    n    = w_pre[l + 1] * x / rms(x)                     the next block's norm, in the same kernel

and experts(n) is: route the fp32 logits n @ w_router, sort the assignments by expert (``moe.permute``),
grouped product with w_gate_up, SwiGLU weighted by the routing weights, grouped product with w_down, sum
of a token's rows (``moe.combine`` with weights 1).  Every backward step is the same kernels' gradient.

The operators take no part in torch's autograd: ``backward`` is written out, as the forward pass is.  The
router's product, its gradients and the gradient of its softmax are torch operations in fp32 (with
``torch.backends.cuda.matmul.allow_tf32`` the products run in TF32, and close choices of experts may differ).

Parameters are fp32 with bf16 copies of the expert weights for the products; ``step`` updates both in
one launch.  Nothing synchronises with the host and the step number lives on the device, so forward,
backward and step can be captured into one CUDA graph (``examples/train_moe.py --graph``).
"""
from __future__ import annotations

import torch

from . import moe

VECTORS = ("w_pre", "w_post", "gate", "res_scale")


class MoEStack:
    """``layers`` MoE blocks of width ``d`` (a multiple of 64) with ``E`` experts of width ``f`` (of 8),
    ``top_k`` of them per token."""

    def __init__(self, layers: int, d: int, f: int, E: int, top_k: int, state_bits: int = 32, device="cuda",
                 seed: int = 0, eps: float = 1e-6):
        self.layers, self.d, self.f, self.E, self.top_k, self.eps = layers, d, f, E, top_k, eps
        g = torch.Generator(device).manual_seed(seed)
        randn = lambda *s, scale: torch.randn(*s, generator=g, device=device) * scale
        ones = lambda: torch.ones(d, device=device)
        self.params, self.weights = [], []  # fp32 parameters, and the bf16 copies the products read
        for _ in range(layers):
            p = {"w_pre": ones(), "w_post": ones(), "gate": ones(), "res_scale": ones(),
                 "w_router": randn(d, E, scale=d ** -0.5),
                 "w_gate_up": randn(E, d, 2 * f, scale=d ** -0.5),
                 "w_down": randn(E, f, d, scale=f ** -0.5)}
            self.params.append(p)
            self.weights.append({k: p[k].bfloat16() for k in ("w_gate_up", "w_down")})
        self.state_bits = state_bits
        self._list = [(p, w.get(k), k) for p, w in zip(self.params, self.weights) for k in p]
        self._state = [moe.adamw_state(p[k], state_bits) for p, _, k in self._list]
        self.step_number = torch.zeros(1, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)  # device-side errors of the kernels

    # ----------------------------------------------------------------------------------------------
    def _experts(self, n, p, w):
        """The routed experts of one block: (c bf16 [T, d], what the backward pass needs)."""
        logits = n.float() @ p["w_router"]
        idx, wt = moe.route(logits, self.top_k)
        _, offsets, _, dest, rows = moe.permute(idx, n, self.E, status=self.status)
        where = dest.view(-1).long()
        w_rows = torch.empty(where.numel(), dtype=torch.float32, device=n.device)
        w_rows[where] = wt.view(-1)  # the routing weight of each sorted row
        gu = moe.grouped_mm(rows, w["w_gate_up"], offsets, status=self.status)
        h = moe.swiglu(gu, w_rows)
        y = moe.grouped_mm(h, w["w_down"], offsets, out_dtype=torch.float32, status=self.status)
        c = moe.combine(y, torch.ones_like(wt), dest, status=self.status)
        return c, (n, idx, wt, offsets, dest, where, rows, w_rows, gu)

    def _experts_backward(self, dc, saved, p, w):
        """(gradient of n as bf16, gradients of the block's router and expert weights)."""
        n, idx, wt, offsets, dest, where, rows, w_rows, gu = saved
        dy = moe.permute(idx, dc, self.E, status=self.status)[4]  # dc's rows in the experts' order
        dh = moe.grouped_mm(dy, w["w_down"], offsets, transpose_b=True, status=self.status)
        dgu, dw_rows, h = moe.swiglu_backward(gu, dh, w_rows, want_h=True)
        g = {"w_down": moe.grouped_mm_wgrad(h, dy, offsets, status=self.status),
             "w_gate_up": moe.grouped_mm_wgrad(rows, dgu, offsets, status=self.status)}
        d_rows = moe.grouped_mm(dgu, w["w_gate_up"], offsets, transpose_b=True, out_dtype=torch.float32,
                                status=self.status)
        dn = moe.combine(d_rows, torch.ones_like(wt), dest, status=self.status)
        # The routing weights are a softmax over the chosen logits.
        dw = dw_rows[where].view_as(wt)
        d_chosen = wt * (dw - (wt * dw).sum(1, keepdim=True))
        d_logits = torch.zeros(n.shape[0], self.E, device=n.device).scatter_(1, idx.long(), d_chosen)
        g["w_router"] = n.float().t() @ d_logits
        return (dn.float() + d_logits @ p["w_router"].t()).bfloat16(), g

    # ----------------------------------------------------------------------------------------------
    def forward(self, x):
        """x [T, d] fp32 or bf16 (the residual stream's type) -> (x after the last block, saved)."""
        _, n = moe.block_norm(x, self.params[0]["w_pre"], eps=self.eps)
        saved = []
        for l, (p, w) in enumerate(zip(self.params, self.weights)):
            c, kept = self._experts(n, p, w)
            saved.append((x, c, kept))
            nxt = self.params[l + 1]["w_pre"] if l + 1 < self.layers else None
            x, n = moe.block_norm(x, nxt, h=c, w_post=p["w_post"], gate=p["gate"], res_scale=p["res_scale"],
                                  eps=self.eps)
        return x, saved

    def backward(self, dx, saved):
        """From the gradient of the output: (gradient of x, a list of the blocks' gradients by name)."""
        grads = [{} for _ in range(self.layers)]
        dn = None
        for l in reversed(range(self.layers)):
            p, w = self.params[l], self.weights[l]
            x, c, kept = saved[l]
            nxt = self.params[l + 1]["w_pre"] if l + 1 < self.layers else None
            g = moe.block_norm_backward(x, dx, dn, w_pre=nxt, h=c, w_post=p["w_post"], gate=p["gate"],
                                        res_scale=p["res_scale"], eps=self.eps)
            if nxt is not None:
                grads[l + 1]["w_pre"] = g["w_pre"]
            dx = g["x"]
            grads[l].update({k: g[k] for k in ("w_post", "gate", "res_scale")})
            dn, ge = self._experts_backward(g["h"], kept, p, w)
            grads[l].update(ge)
        g = moe.block_norm_backward(saved[0][0], dx, dn, w_pre=self.params[0]["w_pre"], eps=self.eps)
        grads[0]["w_pre"] = g["w_pre"]
        return g["x"], grads

    def step(self, grads, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.95, eps: float = 1e-8,
             weight_decay: float = 0.1, factors=None):
        """One AdamW step on every parameter and its bf16 copy; ``factors`` as for ``moe.adamw_step``."""
        self.step_number.add_(1)
        by_param = {id(p): g for p, g in zip(self.params, grads)}
        have = [(p[k], by_param[id(p)][k], s, w) for (p, w, k), s in zip(self._list, self._state)]
        args = dict(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay, step_tensor=self.step_number,
                    factors=factors)
        for group in ([a for a in have if a[3] is not None], [a for a in have if a[3] is None]):
            scales = [a[2][2:] for a in group] if self.state_bits == 8 else None
            moe.adamw_step([a[0] for a in group], [a[1] for a in group], [a[2][0] for a in group],
                           [a[2][1] for a in group], m_scales=scales and [s[0] for s in scales],
                           v_scales=scales and [s[1] for s in scales],
                           copies=[a[3] for a in group] if group[0][3] is not None else None, **args)
