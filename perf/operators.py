"""Cases of the training operators around the Mixture-of-Experts layer, for measuring them.

Four operators, which one training step of an MoE block runs together:

  mm       products grouped by expert over ragged row segments: forward (weights [E, K, N]), input
           gradient (weights read transposed) and weight gradient (reduction over the ragged rows)
  swiglu   h = w * silu(g) * u from the joined [M, 2f] pre-activations, and its gradient
  norm     root-mean-square norms after and before a block, with its gate and residual scale, and
           their gradient
  adamw    one AdamW step over many tensors, with its moments in 32 bits or in 8

`listed()` names the cases, `draw()` gives more of the same ranges, `prepare()` makes what a program
has in hand, `run()` makes one call — in plain torch operations in 32 bits, or with `own` through
this package — and `exact()` restates the operator's definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF16, "f32": F32}
BLOCK = 256  # elements that share one scale of an 8-bit moment


# -------------------------------------------------------------------------------------------------
# cases
# -------------------------------------------------------------------------------------------------
def listed():
    return [
        # the smallest layer: the forward product of 128 assignments, where launch latency counts
        dict(name="mm_fwd_tiny", op="mm", way="fwd", M=128, K=256, N=1024, E=8, active=8, skew=0.0, out="bf16"),
        # serving one token with top-2: two rows stream two experts' down weights
        dict(name="mm_fwd_one_token", op="mm", way="fwd", M=2, K=14336, N=4096, E=8, active=2, skew=0.0, out="f32"),
        # a training batch of 4096 tokens, top-2: the gate+up product, bound by the tensor cores
        dict(name="mm_fwd_batch", op="mm", way="fwd", M=8192, K=4096, N=28672, E=8, active=8, skew=0.0, out="bf16"),
        # input gradient with sizes that are no multiple of a tile and a third of the experts empty
        dict(name="mm_dgrad_odd", op="mm", way="dgrad", M=3001, K=2888, N=1544, E=24, active=16, skew=1.2, out="f32"),
        # weight gradient of many small experts (2048 tokens, top-8 of 256): written bytes count
        dict(name="mm_wgrad_experts", op="mm", way="wgrad", M=16384, K=2048, N=7168, E=256, active=240, skew=1.2,
             out="bf16", accumulate=False),
        # serving: the activation of one token's eight assignments
        dict(name="swiglu_fwd_token", op="swiglu", way="fwd", M=8, f=2048, weighted=True),
        # training: the gradient for 4096 tokens, top-2, with h recomputed for the weight gradient
        dict(name="swiglu_bwd_batch", op="swiglu", way="bwd", M=8192, f=14336, weighted=True, want_h=True),
        # serving: the norms around one token's block
        dict(name="norm_fwd_token", op="norm", way="fwd", T=1, d=4096, x="bf16", post=True, pre=True, gate=True,
             tgate=False, res=True),
        # a training batch with the residual stream in 32 bits
        dict(name="norm_fwd_batch", op="norm", way="fwd", T=4096, d=7168, x="f32", post=True, pre=True, gate=True,
             tgate=True, res=True),
        # its gradient with the residual stream in 16 bits
        dict(name="norm_bwd_batch", op="norm", way="bwd", T=4096, d=4096, x="bf16", post=True, pre=True, gate=True,
             tgate=True, res=True),
        # optimizer step of master weights in 32 bits, gradients in 16, few large tensors and many small
        dict(name="adamw32", op="adamw", bits=32, p="f32", g="bf16", copy=True, tensors=40, largest=1 << 25),
        # the same with 8-bit moments over a few hundred tensors, gradients in 32 bits
        dict(name="adamw8", op="adamw", bits=8, p="f32", g="f32", copy=False, tensors=300, largest=1 << 24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mm", "mm", "swiglu", "norm", "adamw"])
    if op == "mm":
        way = rng.choice(["fwd", "dgrad", "wgrad"])
        while True:
            M, K, N, E = _log(rng, 1, 16384), 8 * _log(rng, 4, 1792), 8 * _log(rng, 4, 3584), _log(rng, 1, 256)
            c = dict(op=op, way=way, M=M, K=K, N=N, E=E, active=min(M, rng.randint(max(1, E // 2), E)),
                     skew=round(rng.uniform(0.0, 1.2), 3), out=rng.choice(["bf16", "f32"]))
            if way == "wgrad":
                c["accumulate"] = c["out"] == "f32" and rng.random() < 0.5
            cost = work(c)  # no more than the listed products' 1.92 TFLOP, and their 7.8 GB
            if cost["flops"] <= 2.0 * 8192 * 4096 * 28672 and cost["bytes"] <= 7.8e9:
                return c
    if op == "swiglu":
        way = rng.choice(["fwd", "bwd"])
        while True:
            M, f = _log(rng, 1, 16384), 8 * _log(rng, 8, 1792)
            if M * f <= 8192 * 14336:
                break
        c = dict(op=op, way=way, M=M, f=f, weighted=rng.random() < 0.7)
        if way == "bwd":
            c["want_h"] = rng.random() < 0.5
        return c
    if op == "norm":
        way = rng.choice(["fwd", "bwd"])
        while True:
            T, d = _log(rng, 1, 16384), 8 * _log(rng, 8, 1024)
            if T * d <= 4096 * 7168:
                break
        post = rng.random() < 0.8
        return dict(op=op, way=way, T=T, d=d, x=rng.choice(["bf16", "f32"]), post=post,
                    pre=(not post) or rng.random() < 0.8, gate=post and rng.random() < 0.7,
                    tgate=post and rng.random() < 0.5, res=post and rng.random() < 0.7)
    bits = rng.choice([32, 8])
    tensors = _log(rng, 2, 300)
    # `largest` such that the tensors (a geometric series down to one element) hold at most 280 M
    largest = _log(rng, 64, (1 << 24) if tensors > 40 else (1 << 25))
    p = rng.choice(["bf16", "f32"])
    return dict(op=op, bits=bits, p=p, g=rng.choice(["bf16", "f32"]), copy=p == "f32" and rng.random() < 0.5,
                tensors=tensors, largest=largest)


def _sizes(case):
    """Elements of each tensor: a geometric series from `largest` down to one, odd sizes among them."""
    n, big = case["tensors"], case["largest"]
    return [max(1, int(big ** (1 - i / max(1, n - 1))) - (i % 3 if i else 0)) for i in range(n)]


def work(case):
    op = case["op"]
    if op == "mm":
        M, K, N, E, act = (case[k] for k in ("M", "K", "N", "E", "active"))
        so = DT[case["out"]].itemsize
        flops = 2.0 * M * K * N
        if case["way"] == "wgrad":
            return {"bytes": 2 * M * (K + N) + E * K * N * so * (2 if case["accumulate"] else 1) + 4 * (E + 1),
                    "flops": flops}
        return {"bytes": 2 * M * K + 2 * act * K * N + M * N * so + 4 * (E + 1), "flops": flops}
    if op == "swiglu":
        M, f, w = case["M"], case["f"], case["weighted"]
        if case["way"] == "fwd":
            return {"bytes": 3 * 2 * M * f + 4 * M * w, "flops": 6.0 * M * f}
        return {"bytes": (5 + case["want_h"]) * 2 * M * f + 8 * M * w, "flops": 16.0 * M * f}
    if op == "norm":
        T, d, sx = case["T"], case["d"], DT[case["x"]].itemsize
        vec = 4 * d * (case["pre"] + case["post"] + case["gate"] + case["res"]) + 4 * T * case["tgate"]
        if case["way"] == "fwd":
            return {"bytes": T * d * (sx + (2 + sx) * case["post"] + 2 * case["pre"]) + vec, "flops": 12.0 * T * d}
        # x, dy (and h, dn) read; dx (and dh) written
        return {"bytes": T * d * (3 * sx + 4 * case["post"] + 2 * case["pre"]) + 2 * vec, "flops": 30.0 * T * d}
    n = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4
    scales = 0 if case["bits"] == 32 else 16 * sum(-(-s // BLOCK) for s in _sizes(case))
    per = 2 * DT[case["p"]].itemsize + DT[case["g"]].itemsize + state + 2 * case["copy"]
    return {"bytes": n * per + scales, "flops": 16.0 * n}


# -------------------------------------------------------------------------------------------------
# inputs
# -------------------------------------------------------------------------------------------------
def _offsets(case, seed):
    """Row segments of the experts: `active` experts share the rows, popularity ~ rank**-skew."""
    rng = np.random.default_rng(seed)
    M, E, act = case["M"], case["E"], case["active"]
    p = np.arange(1, act + 1, dtype=np.float64) ** -case["skew"]
    counts = 1 + rng.multinomial(M - act, p / p.sum())
    full = np.zeros(E, np.int64)
    full[rng.permutation(E)[:act]] = counts
    return [0] + [int(v) for v in np.cumsum(full)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)

    def randn(*shape, dtype=BF16, scale=1.0, mean=0.0):
        t = torch.randn(*shape, generator=g, device=dev, dtype=dtype)
        t = t.mul_(scale) if scale != 1.0 else t
        return t.add_(mean) if mean else t

    s = {"case": case}
    if case["op"] == "mm":
        M, K, N, E = (case[k] for k in ("M", "K", "N", "E"))
        offs = _offsets(case, seed)
        s["host_offsets"] = offs
        s["offsets"] = torch.tensor(offs, dtype=torch.int32, device=dev)
        s["a"] = randn(M, K)
        if case["way"] == "wgrad":
            s["g"] = randn(M, N, scale=0.01)
            if case["accumulate"]:
                s["grad"] = randn(E, K, N, dtype=F32, scale=0.1)
        else:
            s["b"] = randn(E, K, N, scale=0.02) if case["way"] == "fwd" else randn(E, N, K, scale=0.02)
    elif case["op"] == "swiglu":
        M, f = case["M"], case["f"]
        s["gu"] = randn(M, 2 * f, scale=1.5)
        s["w"] = torch.rand(M, generator=g, device=dev) if case["weighted"] else None
        if case["way"] == "bwd":
            s["dh"] = randn(M, f, scale=0.1)
    elif case["op"] == "norm":
        T, d, xt = case["T"], case["d"], DT[case["x"]]
        s["x"] = randn(T, d, dtype=xt, scale=2.0)
        s["h"] = randn(T, d, scale=0.5) if case["post"] else None
        s["w_pre"] = randn(d, dtype=F32, scale=0.1, mean=1.0) if case["pre"] else None
        s["w_post"] = randn(d, dtype=F32, scale=0.1, mean=1.0) if case["post"] else None
        s["gate"] = randn(d, dtype=F32, scale=0.2, mean=0.5) if case["gate"] else None
        s["tgate"] = torch.rand(T, generator=g, device=dev) if case["tgate"] else None
        s["res"] = randn(d, dtype=F32, scale=0.05, mean=1.0) if case["res"] else None
        if case["way"] == "bwd":
            s["dy"] = randn(T, d, dtype=xt, scale=0.1)
            s["dn"] = randn(T, d, scale=0.1) if case["pre"] else None
    else:
        # The tensors are pieces of flat buffers, each starting at a multiple of BLOCK elements.
        sizes, bits, at, pieces = _sizes(case), case["bits"], 0, []
        for n in sizes:
            pieces.append((at, n))
            at += -(-n // BLOCK) * BLOCK
        ends = torch.tensor([lo + n for lo, n in pieces], device=dev)
        gaps = torch.tensor([-n % BLOCK for n in sizes], device=dev)
        first = torch.repeat_interleave(ends - (gaps.cumsum(0) - gaps), gaps)
        unused = first + torch.arange(first.numel(), device=dev)  # elements between the pieces

        def flat(dtype, scale):
            t = randn(at, dtype=dtype, scale=scale)
            t[unused] = 0
            return t

        cut = lambda t: [t[lo:lo + n] for lo, n in pieces]
        cut_scales = lambda t: [t[lo // BLOCK:-(-(lo + n) // BLOCK)] for lo, n in pieces]
        b = {"p": flat(DT[case["p"]], 0.02), "m": flat(F32, 0.001), "v": flat(F32, 0.001).square_()}
        s["flat_grads"] = flat(DT[case["g"]], 0.001)
        s["grads"] = cut(s["flat_grads"])
        s["copy"] = None
        if case["copy"]:
            b["copy"] = torch.zeros(at, dtype=BF16, device=dev)
            s["copy"] = cut(b["copy"])
        if bits == 8:
            for k, t in (("m", b["m"]), ("v", b["v"].sqrt())):
                q, b[k + "_scale"] = _codes(t.view(-1, BLOCK), k == "v")
                b[k] = q.view(-1)
                s[k + "_scale"] = cut_scales(b[k + "_scale"])
        s["p"], s["m"], s["v"] = cut(b["p"]), cut(b["m"]), cut(b["v"])
        s["all"] = b
    return s


# -------------------------------------------------------------------------------------------------
# plain forms
# -------------------------------------------------------------------------------------------------
def _codes(b, root):
    """8-bit floating (4 exponent bits, 3 of mantissa) codes of blocks and a scale for each: the largest
    magnitude goes to 448; a block below 2^-100 is zero. Roots (of the second moment) that are not zero
    keep at least the smallest code, so that a step is never divided by a root lost to rounding."""
    big = b.abs().amax(1, keepdim=True)
    some = big >= 2.0 ** -100
    some = some | big.isnan()
    scale = torch.where(some, big * (1.0 / 448.0), torch.ones_like(big))
    q = b * torch.where(some, scale.reciprocal(), torch.zeros_like(big))
    if root:
        q = torch.where((b > 0) & some, q.clamp_min(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn), scale.view(-1)


def _values(codes, scales):
    """What 8-bit codes stand for, in 32 bits."""
    return (codes.float().view(-1, BLOCK) * scales.view(-1, 1)).view(-1)


HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=100)


def _adamw_flat(p, g, m, v, h):
    """New parameter, first moment and root of the second from 32-bit values; v is the second moment."""
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + (g * (1.0 - h["beta2"])) * g
    r = v.sqrt()
    bc1, bc2 = 1.0 - h["beta1"] ** h["step"], 1.0 - h["beta2"] ** h["step"]
    up = (m * (h["lr"] / bc1)) / (r * (1.0 / math.sqrt(bc2)) + h["eps"])
    return p * (1.0 - h["lr"] * h["weight_decay"]) - up, m, v, r


def _norm_plain(s):
    c = s["case"]
    f = lambda k: None if s.get(k) is None else s[k].float()
    x, h, w_pre, w_post, gate, tgate, res = (f(k) for k in ("x", "h", "w_pre", "w_post", "gate", "tgate", "res"))
    eps = 1e-6
    one = torch.ones((), device=x.device)
    gc, gt, rs = (one if gate is None else gate), (one if tgate is None else tgate[:, None]), (one if res is None else res)
    if h is not None:
        rh = (h.square().mean(1, keepdim=True) + eps).rsqrt()
        hh = h * rh
        y = rs * x + (gc * gt) * (hh * w_post)
    else:
        y = x
    if w_pre is not None:
        ry = (y.square().mean(1, keepdim=True) + eps).rsqrt()
        yh = y * ry
    if c["way"] == "fwd":
        out = {}
        if h is not None:
            out["y"] = y.to(s["x"].dtype)
        if w_pre is not None:
            out["n"] = (yh * w_pre).to(BF16)
        return out
    dy, out = f("dy"), {}
    if w_pre is not None:
        dn = f("dn")
        t = dn * w_pre
        dy = dy + ry * (t - yh * (t * yh).mean(1, keepdim=True))
        out["dw_pre"] = (dn * yh).sum(0)
    out["dx"] = (rs * dy).to(s["x"].dtype)
    if h is not None:
        z = hh * w_post
        dz = dy * (gc * gt)
        out["dw_post"] = (dz * hh).sum(0)
        t = dz * w_post
        out["dh"] = (rh * (t - hh * (t * hh).mean(1, keepdim=True))).to(BF16)
        if gate is not None:
            out["dgate"] = (dy * gt * z).sum(0)
        if tgate is not None:
            out["dtgate"] = (dy * gc * z).sum(1)
        if res is not None:
            out["dres"] = (dy * x).sum(0)
    return out


def _run_plain(s):
    c = s["case"]
    if c["op"] == "mm":
        # One product for each expert with its rows: padding all experts to the fullest one's rows
        # would be a single batched product of several times the work.
        seg = list(zip(s["host_offsets"][:-1], s["host_offsets"][1:]))
        a, out = s["a"], DT[c["out"]]
        if c["way"] == "wgrad":
            d = s["grad"] if c["accumulate"] else torch.empty(c["E"], c["K"], c["N"], dtype=out, device=a.device)
            for e, (lo, hi) in enumerate(seg):
                p = a[lo:hi].float().t() @ s["g"][lo:hi].float()
                if c["accumulate"]:
                    d[e].add_(p)
                else:
                    d[e].copy_(p)
            return d
        b = s["b"] if c["way"] == "fwd" else s["b"].transpose(1, 2)
        return torch.cat([a[lo:hi].float() @ b[e].float() for e, (lo, hi) in enumerate(seg) if hi > lo]).to(out)
    if c["op"] == "swiglu":
        g, u = s["gu"].float().chunk(2, 1)
        w = s["w"][:, None] if s["w"] is not None else torch.ones((), device=g.device)
        sg = 1.0 / (1.0 + (-g).exp())
        if c["way"] == "fwd":
            return (w * (g * sg * u)).to(BF16)
        dh = s["dh"].float()
        out = {"dgu": torch.cat([w * dh * u * sg * (1.0 + g * (1.0 - sg)), w * dh * g * sg], 1).to(BF16)}
        if s["w"] is not None:
            out["dw"] = (dh * (g * sg * u)).sum(1)
        if c["want_h"]:
            out["h"] = (w * (g * sg * u)).to(BF16)
        return out
    if c["op"] == "norm":
        return _norm_plain(s)
    # On the flat buffers that the tensors are pieces of: what lies between them is zero and stays so.
    b, g = s["all"], s["flat_grads"].float()
    if c["bits"] == 32:
        new, m, v, _ = _adamw_flat(b["p"].float(), g, b["m"], b["v"], HYPER)
        b["m"].copy_(m)
        b["v"].copy_(v)
    else:
        new, m, _, r = _adamw_flat(b["p"].float(), g, _values(b["m"], b["m_scale"]),
                                   _values(b["v"], b["v_scale"]).square(), HYPER)
        for name, t, root in (("m", m, False), ("v", r, True)):
            q, sc = _codes(t.view(-1, BLOCK), root)
            b[name].copy_(q.view(-1))
            b[name + "_scale"].copy_(sc)
    b["p"].copy_(new)
    if c["copy"]:
        b["copy"].copy_(new)
    return s["all"]


def _run_own(s):
    from mixture_experts_grouped_fp32_gb300 import moe as m
    c = s["case"]
    if c["op"] == "mm":
        if c["way"] == "wgrad":
            if c["accumulate"]:
                return m.grouped_mm_wgrad(s["a"], s["g"], s["offsets"], out=s["grad"], accumulate=True)
            return m.grouped_mm_wgrad(s["a"], s["g"], s["offsets"], out_dtype=DT[c["out"]])
        return m.grouped_mm(s["a"], s["b"], s["offsets"], transpose_b=c["way"] == "dgrad", out_dtype=DT[c["out"]])
    if c["op"] == "swiglu":
        if c["way"] == "fwd":
            return m.swiglu(s["gu"], s["w"])
        dgu, dw, h = m.swiglu_backward(s["gu"], s["dh"], s["w"], want_h=c["want_h"])
        return {k: v for k, v in (("dgu", dgu), ("dw", dw), ("h", h)) if v is not None}
    if c["op"] == "norm":
        args = dict(w_pre=s["w_pre"], h=s["h"], w_post=s["w_post"], gate=s["gate"], token_gate=s["tgate"],
                    res_scale=s["res"], eps=1e-6)
        if c["way"] == "fwd":
            y, n = m.block_norm(s["x"], **args)
            return {k: v for k, v in (("y", y), ("n", n)) if v is not None}
        d = m.block_norm_backward(s["x"], s["dy"], s["dn"], **args)
        names = (("dx", "x"), ("dh", "h"), ("dw_pre", "w_pre"), ("dw_post", "w_post"), ("dgate", "gate"),
                 ("dtgate", "token_gate"), ("dres", "res_scale"))
        return {k: d[v] for k, v in names if d[v] is not None}
    m.adamw_step(s["p"], s["grads"], s["m"], s["v"], m_scales=s.get("m_scale"), v_scales=s.get("v_scale"),
                 copies=s["copy"], **HYPER)
    return s["all"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# -------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["op"] == "mm":
        M, K, N, E = (case[k] for k in ("M", "K", "N", "E"))
        res = torch.zeros(E, K, N, dtype=D, device="cuda") if case["way"] == "wgrad" else \
            torch.zeros(M, N, dtype=D, device="cuda")
        for e in range(E):
            rows = slice(s["host_offsets"][e], s["host_offsets"][e + 1])
            a = s["a"][rows].to(D)
            if case["way"] == "wgrad":
                torch.mm(a.T, s["g"][rows].to(D), out=res[e])
                if case["accumulate"]:
                    res[e] += s["grad"][e]
            elif a.shape[0]:
                w = s["b"][e].to(D)
                torch.mm(a, w if case["way"] == "fwd" else w.T, out=res[rows])
        return res
    leaf = lambda t: None if t is None else t.to(D).requires_grad_()
    if case["op"] == "swiglu":
        gu, w = leaf(s["gu"]), leaf(s["w"])
        f = case["f"]
        h = torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
        h = h if w is None else w.unsqueeze(1) * h
        if case["way"] == "fwd":
            return h.detach()
        h.backward(s["dh"].to(D))
        out = {"dgu": gu.grad}
        if w is not None:
            out["dw"] = w.grad
        if case["want_h"]:
            out["h"] = h.detach()
        return out
    if case["op"] == "norm":
        v = {k: leaf(s[k]) for k in ("x", "h", "w_pre", "w_post", "gate", "tgate", "res")}
        rms = lambda t: torch.sqrt((t * t).sum(-1, keepdim=True) / t.shape[-1] + 1e-6)
        y = v["x"]
        if v["h"] is not None:
            z = v["w_post"] * v["h"] / rms(v["h"])
            z = z if v["gate"] is None else z * v["gate"]
            z = z if v["tgate"] is None else z * v["tgate"].unsqueeze(1)
            y = (y if v["res"] is None else y * v["res"]) + z
        n = None if v["w_pre"] is None else v["w_pre"] * y / rms(y)
        if case["way"] == "fwd":
            out = {} if v["h"] is None else {"y": y.detach()}
            return out if n is None else {**out, "n": n.detach()}
        total = (y * s["dy"].to(D)).sum()
        if n is not None:
            total = total + (n * s["dn"].to(D)).sum()
        total.backward()
        names = dict(x="dx", h="dh", w_pre="dw_pre", w_post="dw_post", gate="dgate", tgate="dtgate", res="dres")
        return {names[k]: t.grad for k, t in v.items() if t is not None}
    b1, b2, t = HYPER["beta1"], HYPER["beta2"], HYPER["step"]
    # On the flat buffers: what lies between the pieces is zero throughout, and stays zero.
    b = s["all"]
    g = s["flat_grads"].to(D)
    wide = lambda k: (b[k].float().to(D).view(-1, BLOCK) * b[k + "_scale"].to(D)[:, None]).view(-1)
    m, v = (b["m"].to(D), b["v"].to(D)) if case["bits"] == 32 else (wide("m"), wide("v") ** 2)
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    hat = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + HYPER["eps"])
    p = b["p"].to(D)
    p = p - HYPER["lr"] * (HYPER["weight_decay"] * p + hat)
    out = {"p": p, "m": m, "v": v}
    if case["copy"]:
        out["copy"] = p
    if case["bits"] == 8:  # the scaled values before their rounding to 8 bits
        for k, val in (("m", m), ("v", v.sqrt())):
            q = val.view(-1, BLOCK)
            top = q.abs().max(dim=1, keepdim=True).values / 448
            out[k + "_scale"] = torch.where(top > 0, top, 1.0).view(-1)
            out[k] = (q / torch.where(top > 0, top, 1.0)).view(-1)
    return out
