"""SwiGLU with row weights, the norms around a block and AdamW against their formulas in 64 bits, and
their gradients against differences of the forward formulas.

Tolerances: a bf16 output is rounded once, by at most 2^-8 of the value (half a step); what is computed
in fp32 before it is allowed 2^-18 of the magnitudes that are added (a dozen operations and sums of at
most a few thousand terms in blocks, each off by 2^-24 of them; exponentials by a few units of 2^-24)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, D = torch.bfloat16, torch.float32, torch.float64
FP32_SLACK = 2.0 ** -18


@pytest.fixture(scope="module", params=["fast", "ctypes"])
def moe(request):
    """The binding with its C++ calls, and with ctypes alone."""
    from mixture_experts_grouped_fp32_gb300 import moe as m
    m.load()
    fast = m._fast
    if request.param == "fast" and fast is None:
        pytest.skip("_moe_fast.so was not built here")
    m._fast = fast if request.param == "fast" else None
    yield m
    m._fast = fast


def check(got, ref, mag, what):
    """|got - ref| <= 2^-18 mag (+ 2^-8 |ref| for bf16); not-finite values equal."""
    got = got.detach().cpu()
    ref, mag = ref.detach().cpu(), mag.detach().cpu().expand(ref.shape)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bound = FP32_SLACK * mag + (2.0 ** -8 * ref.abs() if got.dtype == BF16 else 0) + 1e-30
    off = (got.double() - ref).abs()
    bad = ~(off <= bound) & ~(got.double().isnan() & ref.isnan()) & ~(got.double() == ref)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((off / bound)[bad].max())} of the bound"


# ------------------------------------------------------------------------------------------------
# SwiGLU
# ------------------------------------------------------------------------------------------------
def swiglu64(gu, w):
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    h = g / (1 + torch.exp(-g)) * u
    return h if w is None else w[:, None] * h


@pytest.mark.parametrize("M,f", [(1, 8), (1, 2048), (3, 264), (17, 512), (40, 2056), (5, 14336), (700, 64)])
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu(moe, M, f, weighted):
    gen = torch.Generator().manual_seed(M + f)
    gu = (3 * torch.randn(M, 2 * f, generator=gen)).to(BF16)
    dh = torch.randn(M, f, generator=gen).to(BF16)
    w = torch.rand(M, generator=gen) if weighted else None
    dev = lambda t: None if t is None else t.cuda()
    gu64, w64 = gu.to(D).requires_grad_(), None if w is None else w.to(D).requires_grad_()
    ref = swiglu64(gu64, w64)
    ref.backward(dh.to(D))
    check(moe.swiglu(dev(gu), dev(w)), ref, ref.abs(), "h")
    dgu, dw, h = moe.swiglu_backward(dev(gu), dev(dh), dev(w), want_h=True)
    check(h, ref, ref.abs(), "h of the backward pass")
    # dg adds w dh u s and w dh u s g (1 - s); |g| <= 20 here
    g, u = gu64.detach()[:, :f], gu64.detach()[:, f:]
    ww = 1.0 if w is None else w.to(D)[:, None]
    mag = torch.cat([(ww * dh.to(D) * u).abs() * (1 + g.abs()) * torch.sigmoid(g), gu64.grad[:, f:].abs()], 1)
    check(dgu, gu64.grad, mag, "dgu")
    if weighted:
        check(dw, w64.grad, (dh.to(D) * swiglu64(gu64.detach(), None)).abs().sum(1), "dw")
    else:
        assert dw is None
    assert moe.swiglu_backward(dev(gu), dev(dh), dev(w))[2] is None


def test_swiglu_far_values(moe):
    """Gates far from zero: silu goes to g on one side and to 0 on the other, its derivative to 1 and 0."""
    g = torch.tensor([-1e30, -200.0, -100.0, -89.0, 0.0, 89.0, 200.0, 1e30]).to(BF16)
    gu = torch.cat([g, torch.full((8,), 0.5).to(BF16)])[None].cuda()
    h = moe.swiglu(gu)[0].float().cpu()
    assert torch.allclose(h, torch.where(g > 0, 0.5 * g, 0).float(), rtol=2.0 ** -8, atol=1e-30)
    dgu, _, _ = moe.swiglu_backward(gu, torch.ones(1, 8, dtype=BF16, device="cuda"))
    assert dgu.isfinite().all()
    assert torch.allclose(dgu[0, :8].float().cpu(), torch.tensor([0, 0, 0, 0, 0.25, 0.5, 0.5, 0.5]), atol=1e-30)


def test_swiglu_difference(moe):
    """The gradient against central differences of the kernel's own forward pass, summed over h in 64 bits.
    With steps of 1/8 the cubic term is below 2^-7, and h's rounding (2^-8 of values below 4) adds 2^-4."""
    g = torch.linspace(-4, 4, 64).to(BF16)
    u = torch.linspace(1, -1, 64).to(BF16)
    dgu, _, _ = moe.swiglu_backward(torch.cat([g, u])[None].cuda(), torch.ones(1, 64, dtype=BF16, device="cuda"))
    up, dn = (g.float() + 0.125).to(BF16), (g.float() - 0.125).to(BF16)
    hs = [moe.swiglu(torch.cat([t, u])[None].cuda())[0].double().cpu() for t in (up, dn)]
    slope = (hs[0] - hs[1]) / (up.double() - dn.double())
    assert (slope - dgu[0, :64].double().cpu()).abs().max() < 2.0 ** -4 + 4 * 2 * 2.0 ** -8 / 0.25


# ------------------------------------------------------------------------------------------------
# norms around a block
# ------------------------------------------------------------------------------------------------
def norm64(v, eps):
    rms = lambda t: torch.sqrt((t * t).mean(1, keepdim=True) + eps)
    y = v["x"]
    if v["h"] is not None:
        z = v["w_post"] * v["h"] / rms(v["h"])
        for k, s in (("gate", lambda t: t), ("token_gate", lambda t: t[:, None])):
            if v[k] is not None:
                z = z * s(v[k])
        y = (y if v["res_scale"] is None else v["res_scale"] * y) + z
    return y, None if v["w_pre"] is None else v["w_pre"] * y / rms(y)


def norm_inputs(T, d, xt, post, pre, gates, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    v = dict.fromkeys(("x", "h", "w_pre", "w_post", "gate", "token_gate", "res_scale"))
    v["x"] = r(T, d).to(xt)
    if post:
        v["h"], v["w_post"] = (0.3 * r(T, d)).to(BF16), 1 + 0.2 * r(d)
        if gates:
            v["gate"], v["token_gate"], v["res_scale"] = r(d), torch.rand(T, generator=g), 1 + 0.1 * r(d)
    if pre:
        v["w_pre"] = 1 + 0.2 * r(d)
    return v, r(T, d).to(xt), r(T, d).to(BF16)


NORM_SHAPES = [(1, 8), (1, 4096), (2, 264), (5, 2048), (7, 2056), (33, 512), (3, 7168), (5, 5120), (460, 4104),
               (2, 8192), (2, 8200), (2, 16384), (1, 20480), (1, 65536), (700, 72),
               (153, 8), (2500, 264), (1000, 640), (611, 1000)]


@pytest.mark.parametrize("post,pre,gates", [(True, True, True), (True, True, False), (True, False, True),
                                            (False, True, False)])
@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("T,d", NORM_SHAPES)
def test_block_norm(moe, T, d, xt, post, pre, gates):
    v, dy, dn = norm_inputs(T, d, xt, post, pre, gates)
    dev = {k: None if t is None else t.cuda() for k, t in v.items()}
    v64 = {k: None if t is None else t.to(D).requires_grad_() for k, t in v.items()}
    y, n = norm64(v64, 1e-6)
    gy, gn = moe.block_norm(**dev)
    with torch.no_grad():
        # y adds res x and the gated norm: ymag is the sum of their magnitudes (y itself may cancel)
        rms = lambda t: torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6)
        part = v64["x"].abs() if v64["res_scale"] is None else (v64["x"] * v64["res_scale"]).abs()
        ymag = part + (y - (v64["x"] if v64["res_scale"] is None else v64["x"] * v64["res_scale"])).abs()
    if post:
        check(gy, y, ymag, "y")
    else:
        assert gy is None
    if pre:
        check(gn, n, v64["w_pre"].detach().abs() * ymag / rms(y.detach()), "n")
    else:
        assert gn is None
    loss = (y * dy.to(D)).sum() + ((n * dn.to(D)).sum() if pre else 0)
    loss.backward()
    grads = moe.block_norm_backward(dy=dy.cuda(), dn=dn.cuda() if pre else None, **dev)
    with torch.no_grad():
        # magnitudes: every row gradient adds a few terms of size |dn| w / rms and their row means
        e = (dn.to(D) * v64["w_pre"]).abs() if pre else torch.zeros(T, d, dtype=D)
        yh = ymag / rms(y)
        magD = dy.to(D).abs() + (e + yh * (e * yh).mean(1, keepdim=True)) / rms(y) * 2
        magx = magD * (1 if v64["res_scale"] is None else v64["res_scale"].abs())
        check(grads["x"], v64["x"].grad, magx, "dx")
        if pre:
            check(grads["w_pre"], v64["w_pre"].grad, (dn.to(D).abs() * yh).sum(0) * 2, "dw_pre")
        if post:
            hh = (v64["h"] / rms(v64["h"])).abs()
            one = torch.ones((), dtype=D)
            gate = one if v64["gate"] is None else v64["gate"].abs()
            tg = one if v64["token_gate"] is None else v64["token_gate"][:, None]
            wp = v64["w_post"].abs()
            q = magD * gate * wp
            check(grads["h"], v64["h"].grad, tg * (q + hh * (q * hh).mean(1, keepdim=True)) / rms(v64["h"]) * 2, "dh")
            A = (magD * tg * hh).sum(0) * 2
            check(grads["w_post"], v64["w_post"].grad, gate * A, "dw_post")
            if gates:
                check(grads["gate"], v64["gate"].grad, wp * A, "dgate")
                check(grads["token_gate"], v64["token_gate"].grad, (q * hh).sum(1) * 2, "dtgate")
                check(grads["res_scale"], v64["res_scale"].grad, (magD * v64["x"].abs()).sum(0) * 2, "dres")


def test_block_norm_zero_rows_and_missing_gradients(moe):
    """A row of zeros has norm eps alone; dy or dn may be missing; y may be written over x."""
    v, dy, dn = norm_inputs(4, 264, F32, True, True, True)
    v["x"][1] = 0
    v["h"][1] = 0
    dev = {k: t.cuda() for k, t in v.items()}
    y, n = moe.block_norm(**dev)
    assert (y[1] == 0).all() and (n[1] == 0).all()
    both = moe.block_norm_backward(dy=dy.cuda(), dn=dn.cuda(), **dev)
    assert all(g.isfinite().all() for g in both.values())
    only_y = moe.block_norm_backward(dy=dy.cuda(), **dev)
    assert only_y["w_pre"] is None
    only_n = moe.block_norm_backward(dn=dn.cuda(), **dev)
    zero = moe.block_norm_backward(dy=torch.zeros_like(dy).cuda(), dn=dn.cuda(), **dev)
    for k in both:
        assert torch.equal(only_n[k], zero[k])
        if k not in ("w_pre", "h"):  # linear in (dy, dn); rows scaled by up to 1/sqrt(eps)
            total = only_y[k] + only_n[k]
            assert torch.allclose(both[k], total, rtol=1e-4, atol=1e-4 * float(total.abs().max()))
    x = dev["x"].clone()
    y2, n2 = moe.block_norm(**{**dev, "x": x}, y=x)
    assert y2 is x and torch.equal(x, y) and torch.equal(n2, n)
    again = moe.block_norm_backward(dy=dy.cuda(), dn=dn.cuda(), **dev)
    assert all(torch.equal(both[k], again[k]) for k in both)
    none = {k: t[:0].contiguous() if k in ("x", "h", "token_gate") else t for k, t in dev.items()}
    g = moe.block_norm_backward(dy=dy[:0].cuda(), dn=dn[:0].cuda(), **none)
    assert g["x"].shape == (0, 264) and all((g[k] == 0).all() for k in ("w_pre", "w_post", "gate", "res_scale"))


@pytest.mark.parametrize("xt", [BF16, F32])
def test_block_norm_of_tensors_aligned_to_16_bytes(moe, xt):
    """Pieces of larger buffers that start at 16 bytes past a multiple of 32: the same results."""
    v, dy, dn = norm_inputs(9, 264, xt, True, True, True, seed=2)

    def moved(t):
        skip = 16 // t.element_size()
        buf = torch.zeros(t.numel() + skip, dtype=t.dtype, device="cuda")
        buf[skip:].copy_(t.reshape(-1))
        return buf[skip:].view(t.shape)
    at = {k: t.cuda() for k, t in v.items()}
    off = {k: t.cuda() if k == "token_gate" else moved(t) for k, t in v.items()}
    for a, b in zip(moe.block_norm(**at), moe.block_norm(**off)):
        assert torch.equal(a, b)
    ga = moe.block_norm_backward(dy=dy.cuda(), dn=dn.cuda(), **at)
    gb = moe.block_norm_backward(dy=moved(dy), dn=moved(dn), **off)
    assert all(torch.equal(ga[k], gb[k]) for k in ga)
    y = moved(torch.zeros(9, 264, dtype=xt))
    assert torch.equal(moe.block_norm(**at, y=y)[0], moe.block_norm(**at)[0])


def test_block_norm_difference(moe):
    """Directional derivatives against central differences of the kernel's forward pass (fp32 stream)."""
    v, dy, _ = norm_inputs(6, 256, F32, True, False, True, seed=4)
    dev = {k: None if t is None else t.cuda() for k, t in v.items()}
    grads = moe.block_norm_backward(dy=dy.cuda(), **dev)
    g = torch.Generator().manual_seed(1)
    for k in ("x", "w_post", "gate", "token_gate", "res_scale"):
        step = torch.randn(v[k].shape, generator=g).cuda()
        ys = [moe.block_norm(**{**dev, k: dev[k] + s * step})[0].double() for s in (0.5, -0.5)]
        slope = float(((ys[0] - ys[1]) * dy.cuda().double()).sum())  # y is linear in each of these
        want = float((grads[k].double() * step.double()).sum())
        size = float(((ys[0].abs() + ys[1].abs()) * dy.cuda().double().abs()).sum())
        assert abs(slope - want) <= 1e-6 * size, k


# ------------------------------------------------------------------------------------------------
# AdamW
# ------------------------------------------------------------------------------------------------
H = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 255, 256, 257, 2048, 2049, 5000, 0, 70001]


def adamw64(p, g, m, v, step, lr=1e-2, factor=1.0):
    g = g.to(D) * factor
    m = 0.9 * m + 0.1 * g
    v = 0.95 * v + 0.05 * g * g
    hat = (m / (1 - 0.9 ** step)) / (torch.sqrt(v / (1 - 0.95 ** step)) + 1e-8)
    return p.to(D) * (1 - lr * 0.1) - lr * hat, m, v


def code32(b, root):
    """The 8-bit form of [blocks, 256] values as documented, in fp32 torch operations on the CPU."""
    big = b.abs().amax(1, keepdim=True)
    some = ~(big < 2.0 ** -100)
    scale = torch.where(some, big * torch.tensor(1.0 / 448.0), torch.ones(()))
    q = b * torch.where(some, 1.0 / scale, torch.zeros(()))
    if root:
        q = torch.where((b > 0) & some, q.clamp_min(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn), scale.view(-1)


def blocks(t):
    return torch.nn.functional.pad(t, (0, -t.numel() % 256)).view(-1, 256)


@pytest.mark.parametrize("shift", [0, 1, 3, 4])
@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_adamw32(moe, pt, gt, shift):
    g = torch.Generator().manual_seed(1)
    # shift: pieces that start off the alignment of 16 bytes (1, 3), or off that of 32 (4)
    make = lambda n, dt, f: f(torch.randn(n + shift, generator=g)).to(dt)
    ps = [make(n, pt, lambda t: t) for n in SIZES]
    gs = [make(n, gt, lambda t: 0.1 * t) for n in SIZES]
    ms = [make(n, F32, lambda t: 0.1 * t) for n in SIZES]
    vs = [make(n, F32, lambda t: 0.01 * t * t) for n in SIZES]
    dev = [[t.cuda() for t in l] for l in (ps, gs, ms, vs)]
    copies = [torch.zeros(n + shift, dtype=BF16, device="cuda") for n in SIZES]
    cut = lambda l: [t[shift:] for t in l]
    moe.adamw_step(*[cut(l) for l in dev], step=3, copies=cut(copies), **H)
    for p, gr, m, v, dp, dg, dm, dv, c in zip(ps, gs, ms, vs, *dev, copies):
        want, wm, wv = adamw64(p[shift:], gr[shift:], m[shift:].to(D), v[shift:].to(D), 3)
        mag = p[shift:].double().abs() + 2 * H["lr"] * (m[shift:].double().abs() + gr[shift:].double().abs()) / \
            (torch.sqrt(wv) + 1e-8) + H["lr"]
        check(dp[shift:], want, mag, "p")
        check(c[shift:], want, mag, "copy")
        check(dm[shift:], wm, m[shift:].double().abs() + gr[shift:].double().abs(), "m")
        check(dv[shift:], wv, wv, "v")
        for t, before in ((dp, p), (dm, m), (dv, v)):
            assert torch.equal(t[:shift].cpu(), before[:shift])  # the neighbours stay


@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("pt,gt", [(F32, BF16), (BF16, F32)])
def test_adamw8(moe, pt, gt, shift):
    """8-bit moments: values from codes, a 64-bit step, and codes of the result — equal to the documented
    coding of the kernel's own fp32 moments, which torch computes bit for bit."""
    g = torch.Generator().manual_seed(2)
    lists = {k: [] for k in ("p", "g", "m", "v", "ms", "vs")}
    for n in SIZES:
        lists["p"].append(torch.randn(n + shift, generator=g).to(pt).cuda()[shift:])
        lists["g"].append((0.1 * torch.randn(n + shift, generator=g)).to(gt).cuda()[shift:])
        for k, root in (("m", False), ("v", True)):
            val = 0.1 * torch.randn(n, generator=g) * torch.exp(3 * torch.randn(n, generator=g))
            q, s = code32(blocks(val.abs() if root else val), root)
            buf = torch.zeros(n + shift, dtype=torch.float8_e4m3fn, device="cuda")
            buf[shift:].copy_(q.view(-1)[:n])
            lists[k].append(buf[shift:])
            lists[k + "s"].append(s.cuda())
    before = {k: [t.cpu().clone() for t in l] for k, l in lists.items()}
    moe.adamw_step(lists["p"], lists["g"], lists["m"], lists["v"], step=5, m_scales=lists["ms"], v_scales=lists["vs"], **H)
    for i, n in enumerate(SIZES):
        b = {k: l[i] for k, l in before.items()}
        val = lambda k: (blocks(b[k].float()) * b[k + "s"][:, None]).view(-1)[:n]
        m32, r32, g32 = val("m"), val("v"), b["g"].float()
        v32 = r32 * r32
        want, _, wv = adamw64(b["p"], b["g"], m32.to(D), v32.to(D), 5)
        mag = b["p"].double().abs() + 2 * H["lr"] * (m32.double().abs() + g32.double().abs()) / (torch.sqrt(wv) + 1e-8) + 0.01
        check(lists["p"][i], want, mag, "p")
        f = lambda c: torch.tensor(c, dtype=F32)
        m32 = m32 * f(0.9) + g32 * f(1 - 0.9)
        v32 = v32 * f(0.95) + (g32 * f(1 - 0.95)) * g32
        for k, t, root in (("m", m32, False), ("v", v32.sqrt(), True)):
            q, s = code32(blocks(t), root)
            assert torch.equal(lists[k + "s"][i].cpu(), s), (k, n)
            assert torch.equal(lists[k][i].cpu().view(torch.uint8), q.view(-1)[:n].view(torch.uint8)), (k, n)


def test_adamw8_fresh_zero_and_nonfinite_blocks(moe):
    p = torch.zeros(1024, device="cuda")
    state = moe.adamw_state(p, 8)
    g = torch.zeros(1024, device="cuda")
    g[256:512] = 1e-33  # the moments stay below 2^-100: zero
    g[600] = float("nan")
    g[800] = 3.0
    g[801] = 1e-9       # a root far below the block's largest keeps the smallest code
    step = lambda: moe.adamw_step([p], [g], [state[0]], [state[1]], step=1, m_scales=[state[2]], v_scales=[state[3]], **H)
    step()
    assert (state[0][:512].float() == 0).all() and (state[2][:2] == 1).all() and (state[3][:2] == 1).all()
    assert state[0][512:768].float().isnan().all() and state[2][2].isnan() and p[600].isnan()
    assert float(state[1][801].float()) == 2.0 ** -9 and float(state[1][802].float()) == 0
    assert abs(float(p[800]) + H["lr"]) < 1e-6  # the first step is lr times the sign
    g.zero_()
    q = p.clone()
    step()
    assert (p[768:] - q[768:]).abs().max() < 2 * H["lr"]  # no element divides by a vanished root


def test_adamw_device_step_factors_and_graph(moe):
    """The step number and the factors read on the device: a captured step replays as later steps."""
    gen = torch.Generator().manual_seed(3)
    p0, g = torch.randn(3000, generator=gen), 0.1 * torch.randn(3000, generator=gen)
    p, m, v = p0.cuda(), torch.zeros(3000, device="cuda"), torch.zeros(3000, device="cuda")
    t = torch.ones(1, dtype=torch.int32, device="cuda")
    factors = torch.tensor([0.5, 2.0], device="cuda")
    gd = g.cuda()
    run = lambda: moe.adamw_step([p], [gd], [m], [v], step_tensor=t, factors=factors, **H)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.add_(1)
        run()
    graph.replay()
    factors.copy_(torch.tensor([1.0, 0.5]))
    graph.replay()
    torch.cuda.synchronize()
    want, wm, wv = p0.to(D), torch.zeros(3000, dtype=D), torch.zeros(3000, dtype=D)
    for step, (c, l) in enumerate([(0.5, 2.0), (0.5, 2.0), (1.0, 0.5)], 1):
        want, wm, wv = adamw64(want, g, wm, wv, step, lr=H["lr"] * l, factor=c)
    check(p, want, p0.double().abs() + 0.2, "p")
    check(m, wm, wm.abs(), "m")


def test_adamw_many_tensors(moe):
    """More tensors than one launch's table holds."""
    gen = torch.Generator().manual_seed(4)
    n = 900
    sizes = np.random.default_rng(0).integers(1, 400, n)
    mk = lambda s: [s * torch.randn(int(k), generator=gen) for k in sizes]
    ps, gs = mk(1.0), mk(0.1)
    dp, dg = [t.cuda() for t in ps], [t.cuda() for t in gs]
    dm, dv = ([torch.zeros_like(t) for t in dp] for _ in range(2))
    moe.adamw_step(dp, dg, dm, dv, step=1, **H)
    for i in range(n):
        want, wm, _ = adamw64(ps[i], gs[i], torch.zeros(1, dtype=D), torch.zeros(1, dtype=D), 1)
        check(dp[i], want, ps[i].double().abs() + 0.02, f"p {i}")
