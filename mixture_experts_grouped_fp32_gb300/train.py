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

With ``norm="layer"`` the blocks have layer norms before them and nothing after:

    x    = x + dropout(c)
    n    = w_pre[l + 1] * (x - mean(x)) / std(x) + b_pre[l + 1]     in one kernel with the addition

``dropout`` (either norm) zeroes elements of c; the masks are functions of the seed, the block and
``mask_number`` on the device, which every forward pass counts up and keeps, so that its backward pass has the
same masks and a replayed graph new ones.  ``router`` replaces the softmax router by ``moe.route_scores`` and its
gradient: scoring, n_group, topk_group, renormalize and scale as for that call; bias_rate, the step by which
a bias that steers the choice follows the experts' loads of the last forward pass (there is one if it is not 0);
balance, the weight of a loss E * sum_e load_e * mean score_e on each block.  ``forward(x, train=False)`` drops
nothing and records no loads.  With ``vocab`` the stack reads tokens:
x = scale * w_embed[ids], and ids take the place of x in ``forward``.

Parameters are fp32 with bf16 copies of the expert weights for the products; ``step`` updates both in
one launch.  Nothing synchronises with the host and the step number lives on the device, so forward,
backward and step can be captured into one CUDA graph (``examples/train_moe.py --graph``).
"""
from __future__ import annotations

import torch

from . import moe

VECTORS = ("w_pre", "w_post", "gate", "res_scale")
ROUTER = dict(scoring="softmax", n_group=1, topk_group=1, renormalize=True, scale=1.0, bias_rate=0.0, balance=0.0)


class MoEStack:
    """``layers`` MoE blocks of width ``d`` (a multiple of 64) with ``E`` experts of width ``f`` (of 8),
    ``top_k`` of them per token."""

    def __init__(self, layers: int, d: int, f: int, E: int, top_k: int, state_bits: int = 32, device="cuda",
                 seed: int = 0, eps: float = 1e-6, norm: str = "rms", dropout: float = 0.0, router: dict | None = None,
                 vocab: int | None = None, embed_scale: float | None = None):
        if norm not in ("rms", "layer"):
            raise ValueError(f"norm must be 'rms' or 'layer', got {norm!r}")
        if router is not None and set(router) - set(ROUTER):
            raise ValueError(f"router has no {sorted(set(router) - set(ROUTER))}")
        self.layers, self.d, self.f, self.E, self.top_k, self.eps = layers, d, f, E, top_k, eps
        self.norm, self.p, self.seed, self.vocab = norm, dropout, seed, vocab
        self.embed_scale = float(d) ** 0.5 if embed_scale is None else embed_scale
        self.router = None if router is None else {**ROUTER, **router}
        g = torch.Generator(device).manual_seed(seed)
        randn = lambda *s, scale: torch.randn(*s, generator=g, device=device) * scale
        ones = lambda: torch.ones(d, device=device)
        self.params, self.weights = [], []  # fp32 parameters, and the bf16 copies the products read
        for _ in range(layers):
            p = {"w_pre": ones(), "w_post": ones(), "gate": ones(), "res_scale": ones()} if norm == "rms" else \
                {"w_pre": ones(), "b_pre": torch.zeros(d, device=device)}
            p.update(w_router=randn(d, E, scale=d ** -0.5), w_gate_up=randn(E, d, 2 * f, scale=d ** -0.5),
                     w_down=randn(E, f, d, scale=f ** -0.5))
            self.params.append(p)
            self.weights.append({k: p[k].bfloat16() for k in ("w_gate_up", "w_down")})
        if vocab is not None:
            self.params[0]["w_embed"] = randn(vocab, d, scale=d ** -0.5)
        # The bias that steers each block's choice and the loads that it follows; the number of the masks.
        steered = self.router is not None and self.router["bias_rate"] != 0
        self.biases = [torch.zeros(E, device=device) if steered else None for _ in range(layers)]
        self.loads = [torch.zeros(E, dtype=torch.int32, device=device) for _ in range(layers)]
        self.mask_number = torch.zeros(1, dtype=torch.int64, device=device)
        self.state_bits = state_bits
        self._list = [(p, w.get(k), k) for p, w in zip(self.params, self.weights) for k in p]
        self._state = [moe.adamw_state(p[k], state_bits) for p, _, k in self._list]
        self.step_number = torch.zeros(1, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)  # device-side errors of the kernels

    # ----------------------------------------------------------------------------------------------
    def _scoring(self):
        return {k: self.router[k] for k in ("scoring", "renormalize", "scale")}

    def _experts(self, n, p, w, l=0, train=True):
        """The routed experts of block l: (c bf16 [T, d], what the backward pass needs)."""
        logits = n.float() @ p["w_router"]
        if self.router is None:
            idx, wt = moe.route(logits, self.top_k)
        else:
            idx, wt, _ = moe.route_scores(logits, self.top_k, bias=self.biases[l], n_group=self.router["n_group"],
                                          topk_group=self.router["topk_group"], **self._scoring())
        counts, offsets, _, dest, rows = moe.permute(idx, n, self.E, status=self.status)
        if self.router is not None and train:
            self.loads[l].copy_(counts)
        where = dest.view(-1).long()
        w_rows = torch.empty(where.numel(), dtype=torch.float32, device=n.device)
        w_rows[where] = wt.view(-1)  # the routing weight of each sorted row
        gu = moe.grouped_mm(rows, w["w_gate_up"], offsets, status=self.status)
        h = moe.swiglu(gu, w_rows)
        y = moe.grouped_mm(h, w["w_down"], offsets, out_dtype=torch.float32, status=self.status)
        c = moe.combine(y, torch.ones_like(wt), dest, status=self.status)
        return c, (n, idx, wt, offsets, dest, where, rows, w_rows, gu, logits, counts)

    def _experts_backward(self, dc, saved, p, w):
        """(gradient of n as bf16, gradients of the block's router and expert weights)."""
        n, idx, wt, offsets, dest, where, rows, w_rows, gu, logits, counts = saved
        dy = moe.permute(idx, dc, self.E, status=self.status)[4]  # dc's rows in the experts' order
        dh = moe.grouped_mm(dy, w["w_down"], offsets, transpose_b=True, status=self.status)
        dgu, dw_rows, h = moe.swiglu_backward(gu, dh, w_rows, want_h=True)
        g = {"w_down": moe.grouped_mm_wgrad(h, dy, offsets, status=self.status),
             "w_gate_up": moe.grouped_mm_wgrad(rows, dgu, offsets, status=self.status)}
        d_rows = moe.grouped_mm(dgu, w["w_gate_up"], offsets, transpose_b=True, out_dtype=torch.float32,
                                status=self.status)
        dn = moe.combine(d_rows, torch.ones_like(wt), dest, status=self.status)
        dw = dw_rows[where].view_as(wt)
        if self.router is None:  # the routing weights are a softmax over the chosen logits
            d_chosen = wt * (dw - (wt * dw).sum(1, keepdim=True))
            d_logits = torch.zeros(n.shape[0], self.E, device=n.device).scatter_(1, idx.long(), d_chosen)
        else:
            T = n.shape[0]  # (the loss' load is a number: its gradient goes through the scores)
            dscores = counts * (self.router["balance"] * self.E / (T * T * self.top_k)) if \
                self.router["balance"] and T else None
            d_logits = moe.route_scores_backward(logits, idx, dw, dscores, **self._scoring())
        g["w_router"] = n.float().t() @ d_logits
        return (dn.float() + d_logits @ p["w_router"].t()).bfloat16(), g

    # ----------------------------------------------------------------------------------------------
    def _masks(self, l, number):
        """The dropout of block l's output; number: the forward pass' mask_number, None for no dropout."""
        return dict(p=0.0, seed=0) if number is None else dict(p=self.p, seed=self.seed, offset=l, offset_tensor=number)

    def forward(self, x, train: bool = True):
        """x [T, d] fp32 or bf16 (the residual stream's type), or ids [T] int32 or int64 with ``vocab`` (an fp32 stream)
        -> (x after the last block, saved)."""
        number = None
        if self.p and train:
            number = self.mask_number.clone()
            self.mask_number.add_(self.layers)
        ids = None
        if self.vocab is not None:
            ids, x = x, moe.embed(x, self.params[0]["w_embed"], self.embed_scale, status=self.status)
        saved = []
        layer = self.norm == "layer"
        if layer:
            _, n, stats = moe.layer_norm(x, self.params[0]["w_pre"], self.params[0]["b_pre"], eps=self.eps)
        else:
            _, n = moe.block_norm(x, self.params[0]["w_pre"], eps=self.eps)
        for l, (p, w) in enumerate(zip(self.params, self.weights)):
            c, kept = self._experts(n, p, w, l, train)
            nxt = self.params[l + 1] if l + 1 < self.layers else None
            if layer:
                saved.append((x, stats, kept, ids, number))
                if nxt is None:
                    x = moe.dropout(c, residual=x, **self._masks(l, number))
                else:
                    x, n, stats = moe.layer_norm(x, nxt["w_pre"], nxt["b_pre"], h=c, eps=self.eps,
                                                 **self._masks(l, number))
                continue
            if number is not None:
                c = moe.dropout(c, **self._masks(l, number))
            saved.append((x, c, kept, ids, number))
            x, n = moe.block_norm(x, nxt and nxt["w_pre"], h=c, w_post=p["w_post"], gate=p["gate"],
                                  res_scale=p["res_scale"], eps=self.eps)
        return x, saved

    def backward(self, dx, saved):
        """From the gradient of the output: (gradient of x, or of the embedding's rows, a list of the blocks' gradients by
        name; that of w_embed is in the first block's)."""
        grads = [{} for _ in range(self.layers)]
        dx = self._backward_layer(dx, saved, grads) if self.norm == "layer" else self._backward_rms(dx, saved, grads)
        if self.vocab is not None:
            grads[0]["w_embed"] = moe.embed_backward(saved[0][3], dx, self.vocab, self.embed_scale, status=self.status)
        return dx, grads

    def _backward_layer(self, dx, saved, grads):
        number = saved[0][4]
        # (dropped in the stream's type: rounded to bf16 once)
        dc = dx if number is None else moe.dropout(dx, **self._masks(self.layers - 1, number))
        dc = dc.bfloat16()
        for l in reversed(range(self.layers)):
            p, w = self.params[l], self.weights[l]
            x, stats, kept = saved[l][:3]
            dn, ge = self._experts_backward(dc, kept, p, w)
            g = moe.layer_norm_backward(x, stats, dn, dx, p["w_pre"], p["b_pre"], want_h=l > 0,
                                        **self._masks(l - 1, number))
            dx, dc = g["x"], g["h"]
            grads[l].update(ge, w_pre=g["weight"], b_pre=g["bias"])
        return dx

    def _backward_rms(self, dx, saved, grads):
        dn = None
        for l in reversed(range(self.layers)):
            p, w = self.params[l], self.weights[l]
            x, c, kept = saved[l][:3]
            nxt = self.params[l + 1]["w_pre"] if l + 1 < self.layers else None
            g = moe.block_norm_backward(x, dx, dn, w_pre=nxt, h=c, w_post=p["w_post"], gate=p["gate"],
                                        res_scale=p["res_scale"], eps=self.eps)
            if nxt is not None:
                grads[l + 1]["w_pre"] = g["w_pre"]
            dx = g["x"]
            grads[l].update({k: g[k] for k in ("w_post", "gate", "res_scale")})
            number = saved[l][4]
            dc = g["h"] if number is None else moe.dropout(g["h"], **self._masks(l, number))
            dn, ge = self._experts_backward(dc, kept, p, w)
            grads[l].update(ge)
        g = moe.block_norm_backward(saved[0][0], dx, dn, w_pre=self.params[0]["w_pre"], eps=self.eps)
        grads[0]["w_pre"] = g["w_pre"]
        return g["x"]

    def step(self, grads, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.95, eps: float = 1e-8,
             weight_decay: float = 0.1, factors=None):
        """One AdamW step on every parameter and its bf16 copy; ``factors`` as for ``moe.adamw_step``."""
        self.step_number.add_(1)
        for bias, load in zip(self.biases, self.loads):
            if bias is not None:  # towards the experts that have fewer tokens than the mean
                bias.add_(torch.sign(load.sum() / self.E - load), alpha=self.router["bias_rate"])
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
