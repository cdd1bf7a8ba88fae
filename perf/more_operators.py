"""Cases of the operators around a stack of MoE blocks that reads tokens, for measuring them.

Four operators, which one training step of such a stack runs together:

  embed    rows of an embedding table by token ids, scaled; and the table's gradient, in which the
           rows of equal tokens are summed (written whole, or added to a gradient that is there)
  norm     layer norm of a residual stream after a block's output has been added to it (with
           dropout on that output), and its gradient with the sums for the weight and the bias
  dropout  zeroing by the bits of a counter-based generator (Philox4x32 with ten rounds, from
           "Parallel random numbers: as easy as 1, 2, 3", Salmon et al., SC 2011), with a residual
           to add to; the mask is a function of seed and offset and is never stored
  route    routing to experts: softmax or sigmoid scores, a bias that steers the choice, groups,
           top-k, weights with or without renormalisation; and the gradient of the logits

`listed()` names the cases, `draw()` gives more of the same ranges, `prepare()` makes what a program
has in hand, `run()` makes one call — in plain torch operations in 32 bits, or with `own` through
this package — and `exact()` restates the operator's definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DT = {"bf16": BF16, "f32": F32}
MASK32 = 0xFFFFFFFF
SEED, OFFSET = 0x243F6A8885A308D3, 5
EPS = 1e-5


# -------------------------------------------------------------------------------------------------
# cases
# -------------------------------------------------------------------------------------------------
def listed():
    return [
        # the smallest layer's router: 64 tokens over 8 experts, where launch latency counts
        dict(name="route_fwd_small", op="route", way="fwd", T=64, E=8, k=2, scoring="softmax", bias=False, groups=1,
             kept=1, renorm=True, scale=1.0, logits="f32", scores=False),
        # a training batch over 256 experts: sigmoid scores, balancing bias, 4 of 8 groups
        dict(name="route_fwd_groups", op="route", way="fwd", T=16384, E=256, k=8, scoring="sigmoid", bias=True,
             groups=8, kept=4, renorm=True, scale=2.5, logits="f32", scores=False),
        # the gradient of a softmax router without renormalisation, with a balancing loss on the scores
        dict(name="route_bwd_dense", op="route", way="bwd", T=16001, E=160, k=6, scoring="softmax", bias=False,
             groups=1, kept=1, renorm=False, scale=1.0, logits="f32", dscores="expert"),
        # one token of a serving step: the stream takes the block's output and is normed
        dict(name="norm_fwd_token", op="norm", way="fwd", T=1, d=4096, x="bf16", h=True, p=0.0, bias=True),
        # a training batch with the residual stream in 32 bits and dropout on the block's output
        dict(name="norm_fwd_batch", op="norm", way="fwd", T=8192, d=7168, x="f32", h=True, p=0.1, bias=True),
        # the gradient of a training batch with the stream in 16 bits
        dict(name="norm_bwd_batch", op="norm", way="bwd", T=8192, d=4096, x="bf16", h=True, p=0.1, bias=True),
        # rows of an odd width, ragged tokens, a plain layer norm without a bias
        dict(name="norm_bwd_odd", op="norm", way="bwd", T=3001, d=2891, x="bf16", h=False, p=0.0, bias=False),
        # dropout on the smallest layer's activations
        dict(name="dropout_small", op="dropout", rows=64, cols=256, x="bf16", residual="", p=0.1),
        # dropout on a batch of hidden activations
        dict(name="dropout_batch", op="dropout", rows=8192, cols=14336, x="bf16", residual="", p=0.1),
        # a prompt's tokens looked up in a table of 32-bit parameters of odd height
        dict(name="embed_fwd_batch", op="embed", way="fwd", T=8192, V=50001, d=7168, table="f32", out="bf16", skew=1.0,
             ids="i64"),
        # the table's gradient of a training batch, written whole
        dict(name="embed_bwd_whole", op="embed", way="bwd", T=16384, V=131072, d=4096, dy="bf16", out="f32", skew=1.0,
             ids="i32", add=False),
        # a later micro-batch of odd sizes: added to the gradient that is there
        dict(name="embed_bwd_added", op="embed", way="bwd", T=12001, V=50001, d=1028, dy="bf16", out="f32", skew=1.2,
             ids="i64", add=True),
    ]


MOST_BYTES = 2.29e9  # what a drawn case may move at the most: the table's gradient above


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "dropout", "embed"])
    while True:
        way = rng.choice(["fwd", "bwd"])
        if op == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            E = groups * _log(rng, max(1, 4 // groups), 256 // groups)
            kept = rng.randint(1, groups)
            c = dict(op=op, way=way, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, min(8, kept * E // groups)),
                     scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, kept=kept,
                     renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), logits=rng.choice(["f32", "bf16"]))
            if way == "fwd":
                c["scores"] = rng.random() < 0.4
            else:
                c["dscores"] = rng.choice(["", "expert", "token"])
        elif op == "norm":
            h = rng.random() < 0.7
            c = dict(op=op, way=way, T=_log(rng, 1, 16384), d=_log(rng, 32, 16384), x=rng.choice(["bf16", "f32"]), h=h,
                     p=rng.choice([0.0, 0.1, 0.35]) if h else 0.0, bias=rng.random() < 0.7)
        elif op == "dropout":
            c = dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 1, 16384), x=rng.choice(["bf16", "f32"]),
                     residual=rng.choice(["", "bf16", "f32"]), p=round(rng.uniform(0.0, 0.6), 3))
        else:
            c = dict(op=op, way=way, T=_log(rng, 1, 32768), V=_log(rng, 64, 262144), d=_log(rng, 16, 8192))
            if way == "fwd":
                c.update(table=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]))
            else:
                c.update(dy=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]))
                c["add"] = c["out"] == "f32" and rng.random() < 0.5
            c.update(skew=round(rng.uniform(0.0, 1.2), 3), ids=rng.choice(["i32", "i64"]))
            if c["V"] * c["d"] * 4 > MOST_BYTES:  # (a gradient that is added to is held whole too)
                continue
        if work(c)["bytes"] <= MOST_BYTES:
            return c


def _popularity(case):
    """Share of each token: rank**-skew, low ids most frequent."""
    p = np.arange(1, case["V"] + 1, dtype=np.float64) ** -case["skew"]
    return p / p.sum()


def _distinct(case):
    """Expected number of distinct tokens."""
    return float(-np.expm1(case["T"] * np.log1p(-np.minimum(_popularity(case), 1 - 1e-12))).sum())


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        read = T * E * DT[case["logits"]].itemsize
        if case["way"] == "fwd":
            return {"bytes": read + 4 * E * case["bias"] + 8 * T * k + 4 * T * E * case["scores"], "flops": 4.0 * T * E}
        dense = case["dscores"] or not case["renorm"]  # else the chosen logits alone are read
        read = read if dense and not (case["scoring"] == "sigmoid" and not case["dscores"]) else \
            T * k * DT[case["logits"]].itemsize
        ds = {"": 0, "expert": 4 * E, "token": 4 * T * E}[case["dscores"]]
        return {"bytes": read + T * E * DT[case["logits"]].itemsize + 8 * T * k + ds, "flops": 8.0 * T * E}
    if op == "norm":
        T, d, sx, h = case["T"], case["d"], DT[case["x"]].itemsize, case["h"]
        vec = 4 * d * (1 + case["bias"])
        if case["way"] == "fwd":
            return {"bytes": T * d * (sx + (2 + sx) * h + 2) + 8 * T + vec, "flops": 10.0 * T * d}
        # the stream, dy and dn read; dx (and dh) written
        return {"bytes": T * d * (3 * sx + 2 + 2 * h) + 8 * T + vec + 4 * d, "flops": 16.0 * T * d}
    if op == "dropout":
        n, sx = case["rows"] * case["cols"], DT[case["x"]].itemsize
        sr = DT[case["residual"]].itemsize if case["residual"] else 0
        return {"bytes": n * (sx + sr + (sr or sx)), "flops": 2.0 * n}
    T, V, d = case["T"], case["V"], case["d"]
    ids = T * (8 if case["ids"] == "i64" else 4)
    some = _distinct(case) * d
    if case["way"] == "fwd":
        return {"bytes": ids + some * DT[case["table"]].itemsize + T * d * DT[case["out"]].itemsize, "flops": 1.0 * T * d}
    so = DT[case["out"]].itemsize
    return {"bytes": ids + T * d * DT[case["dy"]].itemsize + (some * 2 * so if case["add"] else 1.0 * V * d * so),
            "flops": 1.0 * T * d}


# -------------------------------------------------------------------------------------------------
# inputs
# -------------------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)

    def randn(*shape, dtype=BF16, scale=1.0, mean=0.0):
        t = torch.randn(*shape, generator=g, device=dev, dtype=dtype)
        t = t.mul_(scale) if scale != 1.0 else t
        return t.add_(mean) if mean else t

    s = {"case": case, "seed": SEED + seed}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # experts of unequal popularity, which the bias partly evens out
        taste = randn(E, dtype=F32, scale=0.7)
        s["logits"] = (randn(T, E, dtype=F32) + taste).to(DT[case["logits"]])
        s["bias"] = (taste * -0.1 + randn(E, dtype=F32, scale=0.01)) if case["bias"] else None
        if case["way"] == "bwd":
            s["idx"], _ = _choose(s)  # what the forward pass chose
            s["dw"] = randn(T, k, dtype=F32, scale=0.1)
            s["dscores"] = {"": None, "expert": randn(E, dtype=F32, scale=0.01),
                            "token": randn(T, E, dtype=F32, scale=0.01) if case["dscores"] == "token" else None}[
                                case["dscores"]]
    elif case["op"] == "norm":
        T, d, xt = case["T"], case["d"], DT[case["x"]]
        s["x"] = randn(T, d, dtype=xt, scale=2.0, mean=0.25)
        s["weight"] = randn(d, dtype=F32, scale=0.1, mean=1.0)
        s["bias"] = randn(d, dtype=F32, scale=0.1) if case["bias"] else None
        if case["way"] == "fwd":
            s["h"] = randn(T, d, scale=0.5) if case["h"] else None
        else:  # x is the stream that the forward pass normed, stats are its mean and 1 / standard deviation
            wide = s["x"].to(F64)
            s["stats"] = torch.stack([wide.mean(1), (wide.var(1, correction=0) + EPS).rsqrt()], 1).float()
            s["dn"], s["dy"] = randn(T, d, scale=0.1), randn(T, d, dtype=xt, scale=0.1)
    elif case["op"] == "dropout":
        n = (case["rows"], case["cols"])
        s["x"] = randn(*n, dtype=DT[case["x"]])
        s["residual"] = randn(*n, dtype=DT[case["residual"]], scale=2.0) if case["residual"] else None
    else:
        T, V, d = case["T"], case["V"], case["d"]
        cdf = torch.from_numpy(_popularity(case).cumsum()).to(dev)
        ids = torch.searchsorted(cdf, torch.rand(T, generator=g, device=dev, dtype=F64)).clamp_(max=V - 1)
        s["ids"] = ids.to(torch.int64 if case["ids"] == "i64" else torch.int32)
        s["scale"] = float(d) ** 0.5
        if case["way"] == "fwd":
            s["table"] = randn(V, d, dtype=DT[case["table"]], scale=0.02)
        else:
            s["dy"] = randn(T, d, dtype=DT[case["dy"]], scale=0.01)
            if case["add"]:
                s["grad"] = randn(V, d, dtype=F32, scale=0.1)
    return s


# -------------------------------------------------------------------------------------------------
# plain forms
# -------------------------------------------------------------------------------------------------
def _scores(logits, scoring):
    if scoring == "sigmoid":
        return 1.0 / (1.0 + (-logits).exp())
    e = (logits - logits.amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True)


def _first(c, k):
    """Indices of the k largest of each row, in falling order; of equal ones the lowest first."""
    return c.sort(dim=1, descending=True, stable=True).indices[:, :k]


def _choose(s):
    """The experts of each token. Scores next to one another have to be told apart: 64 bits."""
    c, logits = s["case"], s["logits"].to(F64)
    if s["bias"] is None and c["groups"] == 1:
        return _first(logits, c["k"]).int(), None
    pick = _scores(logits, c["scoring"])
    if s["bias"] is not None:
        pick = pick + s["bias"].to(F64)
    if c["groups"] > 1:
        T, G, size = c["T"], c["groups"], c["E"] // c["groups"]
        q = min(size, max(1, c["k"] // c["kept"]))
        best = pick.view(T, G, size).sort(dim=2, descending=True).values[:, :, :q].sum(2)
        keep = torch.zeros(T, G, dtype=torch.bool, device=pick.device).scatter_(1, _first(best, c["kept"]), True)
        pick = pick.masked_fill(~keep.repeat_interleave(size, 1), -math.inf)
    return _first(pick, c["k"]).int(), None


def _route_plain(s):
    c, l = s["case"], s["logits"].float()
    p = _scores(l, c["scoring"])
    if c["way"] == "fwd":
        idx, _ = _choose(s)
        w = p.gather(1, idx.long())
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        out = {"idx": idx, "w": w * c["scale"]}
        if c["scores"]:
            out["scores"] = p
        return out
    idx, dw = s["idx"].long(), s["dw"] * c["scale"]
    if c["renorm"]:
        chosen = p.gather(1, idx)
        total = chosen.sum(1, keepdim=True)
        r = chosen / total
        dw = (dw - (r * dw).sum(1, keepdim=True)) / total
    dp = torch.zeros_like(p).scatter_(1, idx, dw)
    if s["dscores"] is not None:
        dp = dp + s["dscores"]
    if c["scoring"] == "sigmoid":
        d = dp * p * (1.0 - p)
    else:
        d = p * (dp - (p * dp).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _philox(n, seed, offset, device):
    """The generator's 16-bit pieces for n elements, eight to a block of counter (block, offset)."""
    block = torch.arange((n + 7) // 8, dtype=torch.int64, device=device)
    c = [block & MASK32, block >> 32, torch.full_like(block, offset & MASK32), torch.full_like(block, offset >> 32)]
    k = [seed & MASK32, (seed >> 32) & MASK32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64-bit products (modulo 2^64)
        c = [((b >> 32) & MASK32) ^ c[1] ^ k[0], b & MASK32, ((a >> 32) & MASK32) ^ c[3] ^ k[1], a & MASK32]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    words = torch.stack(c, 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n]


def _kept(shape, p, seed, device):
    """Which elements stay, and what they are multiplied by: p counts in 65536ths."""
    cut = round(p * 65536)
    return (_philox(math.prod(shape), seed, OFFSET, device) >= cut).view(shape), 65536.0 / (65536 - cut)


def _dropped(t, p, seed):
    if p == 0.0:
        return t
    keep, up = _kept(t.shape, p, seed, t.device)
    return torch.where(keep, t * up, torch.zeros_like(t))


def _norm_plain(s):
    c, w = s["case"], s["weight"]
    if c["way"] == "fwd":
        out, y = {}, s["x"].float()
        if c["h"]:
            out["y"] = (y + _dropped(s["h"].float(), c["p"], s["seed"])).to(s["x"].dtype)
            y = out["y"].float()
        mean = y.mean(1, keepdim=True)
        r = ((y - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
        n = (y - mean) * r * w
        if s["bias"] is not None:
            n = n + s["bias"]
        return {**out, "n": n.to(BF16), "stats": torch.cat([mean, r], 1)}
    mean, r = s["stats"][:, :1], s["stats"][:, 1:]
    dn, yh = s["dn"].float(), (s["x"].float() - mean) * r
    g = dn * w
    dx = s["dy"].float() + r * (g - g.mean(1, keepdim=True) - yh * (g * yh).mean(1, keepdim=True))
    out = {"dx": dx.to(s["x"].dtype), "dweight": (dn * yh).sum(0)}
    if s["bias"] is not None:
        out["dbias"] = dn.sum(0)
    if c["h"]:
        out["dh"] = _dropped(dx, c["p"], s["seed"]).to(BF16)
    return out


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _route_plain(s)
    if c["op"] == "norm":
        return _norm_plain(s)
    if c["op"] == "dropout":
        t = _dropped(s["x"].float(), c["p"], s["seed"])
        if s["residual"] is not None:
            return (s["residual"].float() + t).to(s["residual"].dtype)
        return t.to(s["x"].dtype)
    if c["way"] == "fwd":
        return (s["table"][s["ids"].long()].float() * s["scale"]).to(DT[c["out"]])
    dy = s["dy"].float() * s["scale"]
    if c["add"]:
        return s["grad"].index_add_(0, s["ids"], dy)
    return torch.zeros(c["V"], c["d"], device=dy.device).index_add_(0, s["ids"], dy).to(DT[c["out"]])


def _run_own(s):
    from mixture_experts_grouped_fp32_gb300 import moe as m
    c = s["case"]
    if c["op"] == "route":
        kw = dict(scoring=c["scoring"], renormalize=c["renorm"], scale=c["scale"])
        if c["way"] == "fwd":
            idx, w, scores = m.route_scores(s["logits"], c["k"], bias=s["bias"], n_group=c["groups"],
                                            topk_group=c["kept"], want_scores=c["scores"], **kw)
            return {"idx": idx, "w": w, "scores": scores} if c["scores"] else {"idx": idx, "w": w}
        return m.route_scores_backward(s["logits"], s["idx"], s["dw"], dscores=s["dscores"], **kw)
    if c["op"] == "norm":
        drop = dict(p=c["p"], seed=s["seed"], offset=OFFSET) if c["p"] else {}
        if c["way"] == "fwd":
            y, n, stats = m.layer_norm(s["x"], s["weight"], s["bias"], h=s["h"], eps=EPS, **drop)
            return {"y": y, "n": n, "stats": stats} if c["h"] else {"n": n, "stats": stats}
        g = m.layer_norm_backward(s["x"], s["stats"], s["dn"], dy=s["dy"], weight=s["weight"], bias=s["bias"],
                                  want_h=c["h"], **drop)
        names = (("dx", "x"), ("dweight", "weight"), ("dbias", "bias"), ("dh", "h"))
        return {k: g[v] for k, v in names if g[v] is not None}
    if c["op"] == "dropout":
        return m.dropout(s["x"], c["p"], seed=s["seed"], offset=OFFSET, residual=s["residual"])
    if c["way"] == "fwd":
        return m.embed(s["ids"], s["table"], scale=s["scale"], out_dtype=DT[c["out"]])
    if c["add"]:
        return m.embed_backward(s["ids"], s["dy"], c["V"], scale=s["scale"], out=s["grad"], accumulate=True)
    return m.embed_backward(s["ids"], s["dy"], c["V"], scale=s["scale"], out_dtype=DT[c["out"]])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# -------------------------------------------------------------------------------------------------
def _random_pieces(n, seed, offset):
    """The generator once more, from its definition, in unsigned arithmetic on 16-bit limbs."""
    i = torch.arange(-(-n // 8), device="cuda", dtype=torch.int64)

    def mul(x, m):  # (high, low) words of x * m
        xl, xh, ml, mh = x % 65536, x // 65536, m % 65536, m // 65536
        ll, mid = xl * ml, xl * mh + xh * ml
        low = ll + (mid % 65536) * 65536
        return xh * mh + mid // 65536 + low // 2 ** 32, low % 2 ** 32

    x0, x1, x2, x3 = i % 2 ** 32, i // 2 ** 32, i * 0 + offset % 2 ** 32, i * 0 + offset // 2 ** 32
    key0, key1 = seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32
    for r in range(10):
        r0, r1 = (key0 + r * 0x9E3779B9) % 2 ** 32, (key1 + r * 0xBB67AE85) % 2 ** 32
        h0, l0 = mul(x0, 0xD2511F53)
        h1, l1 = mul(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = h1 ^ x1 ^ r0, l1, h0 ^ x3 ^ r1, l0
    out = torch.empty(i.numel(), 8, dtype=torch.int32, device="cuda")
    for j, word in enumerate((x0, x1, x2, x3)):
        out[:, 2 * j], out[:, 2 * j + 1] = word % 65536, word // 65536
    return out.flatten()[:n]


def _without_dropped(t, p, seed):
    """t in 64 bits with elements zeroed, the others divided by their probability to stay."""
    if not p:
        return t
    cut = int(p * 65536 + 0.5)
    gone = _random_pieces(t.numel(), seed, OFFSET).view(t.shape) < cut
    return (t / (1 - cut / 65536)).masked_fill(gone, 0)


def _best(rows, k):
    """The k largest of each row one by one, the lowest index of equal ones."""
    rows, found = rows.clone(), []
    place = torch.arange(rows.shape[1], device=rows.device)
    for _ in range(k):
        top = rows.max(1, keepdim=True).values
        i = torch.where(rows == top, place, rows.shape[1]).min(1).values
        found.append(i)
        rows[place == i[:, None]] = -math.inf
    return torch.stack(found, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "route":
        l = s["logits"].to(F64).requires_grad_(c["way"] == "bwd")
        p = torch.sigmoid(l) if c["scoring"] == "sigmoid" else torch.softmax(l, 1)
        if c["way"] == "bwd":
            w = p.gather(1, s["idx"].long())
            w = c["scale"] * (w / w.sum(1, keepdim=True) if c["renorm"] else w)
            total = (w * s["dw"].to(F64)).sum()
            if s["dscores"] is not None:
                total = total + (p * s["dscores"].to(F64)).sum()
            return torch.autograd.grad(total, l)[0]
        pick = p if s["bias"] is None else p + s["bias"].to(F64)
        G = c["groups"]
        if G > 1:
            size = c["E"] // G
            parts = pick.unflatten(1, (G, size))
            many = max(1, min(size, c["k"] // c["kept"]))
            score = parts.topk(many, dim=2).values.sum(2)
            chosen = _best(score, c["kept"])
            inside = (torch.arange(G, device=l.device)[None, :, None] == chosen[:, None, :]).any(2)
            pick = torch.where(inside[:, :, None], parts, -math.inf).flatten(1)
        elif s["bias"] is None:
            pick = l
        idx = _best(pick, c["k"])
        w = p.gather(1, idx)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
        out = {"idx": idx.int(), "w": c["scale"] * w}
        if c["scores"]:
            out["scores"] = p
        return out
    if c["op"] == "norm":
        x, w = s["x"].to(F64), s["weight"].to(F64)
        if c["way"] == "fwd":
            out = {}
            if c["h"]:
                out["y"] = x + _without_dropped(s["h"].to(F64), c["p"], s["seed"])
                x = out["y"].to(s["x"].dtype).to(F64)  # the norm is that of the stream as stored
            mean = x.mean(1)
            std = torch.sqrt(x.var(1, correction=0) + EPS)
            n = w * (x - mean[:, None]) / std[:, None]
            out["n"] = n if s["bias"] is None else n + s["bias"].to(F64)
            out["stats"] = torch.stack([mean, 1 / std], 1)
            return out
        dn = s["dn"].to(F64)
        yh = (x - s["stats"][:, 0, None].to(F64)) * s["stats"][:, 1, None].to(F64)
        out = {"dweight": torch.einsum("td,td->d", dn, yh)}
        a = torch.einsum("td,d->t", dn, w) / c["d"]
        b = torch.einsum("td,td,d->t", dn, yh, w) / c["d"]
        dx = s["dy"].to(F64) + s["stats"][:, 1, None].to(F64) * (dn * w - a[:, None] - yh * b[:, None])
        out = {"dx": dx, **out}
        if s["bias"] is not None:
            out["dbias"] = dn.sum(0)
        if c["h"]:
            out["dh"] = _without_dropped(dx, c["p"], s["seed"])
        return out
    if c["op"] == "dropout":
        t = _without_dropped(s["x"].to(F64), c["p"], s["seed"])
        return t if s["residual"] is None else s["residual"].to(F64) + t
    if c["way"] == "fwd":
        return s["table"].index_select(0, s["ids"].long()).to(F64) * s["scale"]
    # Row by row of the sorted tokens: sums of runs as differences would lose digits, so a product
    # with each block of tokens' incidence is taken instead, over the distinct tokens.
    res = s["grad"].to(F64) if c["add"] else torch.zeros(c["V"], c["d"], dtype=F64, device="cuda")
    seen, which = torch.unique(s["ids"].long(), return_inverse=True)
    part = torch.zeros(seen.numel(), c["d"], dtype=F64, device="cuda")
    for lo in range(0, c["T"], 2048):
        rows, local = torch.unique(which[lo:lo + 2048], return_inverse=True)
        hit = torch.zeros(rows.numel(), local.numel(), dtype=F64, device="cuda")
        hit[local, torch.arange(local.numel(), device="cuda")] = s["scale"]
        part[rows] += hit @ s["dy"][lo:lo + 2048].to(F64)
    res[seen] += part
    return res
