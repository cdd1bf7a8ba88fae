"""Routing by scores and its gradient against the definition in 64 bits.

Tolerances.  A weight is a quotient of scores: expf is off by 2 units in the last place at the most (4 half units of
2^-24), its argument's rounding adds |l - top| 2^-24 (below 16 for the logits here), the additions of up to 21 terms,
a quotient and the scale one each, for numerator and denominator: below 64 2^-24 = 2^-18 of the value in all.  A
gradient is such factors times D - sum(s D), whose terms are off by as much of |D| + sum(s |D|): 2^-17 of those, and
half a step of the type that it is stored in.  Below 2^-126 fp32 has no relative accuracy: 2^-126 is added."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", params=["fast", "ctypes"])
def moe(request):
    from mixture_experts_grouped_fp32_gb300 import moe as m
    m.load()
    fast = m._fast
    if request.param == "fast" and fast is None:
        pytest.skip("_moe_fast.so was not built here")
    m._fast = fast if request.param == "fast" else None
    yield m
    m._fast = fast


def scores_of(l, scoring):
    """fp64 scores; a row of -inf has scores 0."""
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = l.max(1, keepdim=True).values
    e = torch.where(top == -INF, 0.0, torch.exp(l - top))
    return torch.where(top == -INF, 0.0, e / e.sum(1, keepdim=True))


def best(rows, k):
    """The k best, one row after another: numbers by size, then NaN, equal ones by index."""
    out = []
    for r in rows.tolist():
        order = sorted(range(len(r)), key=lambda e: (r[e] != r[e], -r[e] if r[e] == r[e] else 0.0, e))
        out.append(order[:k])
    return torch.tensor(out)


def reference(logits, k, scoring, bias, groups, kept, renorm, scale):
    l = logits.to(D).cpu()
    s = scores_of(l, scoring)
    if bias is None and groups == 1:
        idx = best(l, k)
    else:
        c = s if bias is None else s + bias.to(D).cpu()
        if groups > 1:
            T, E = c.shape
            parts = c.view(T, groups, E // groups)
            q = min(E // groups, max(1, k // kept))
            total = parts.sort(2, descending=True).values[:, :, :q].sum(2)
            keep = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, best(total, kept), True)
            c = torch.where(keep[:, :, None], parts, -INF).reshape(T, E)
        idx = best(c, k)
    w = s.gather(1, idx)
    if renorm:  # (shares of sigmoids by their logarithms: 1 / (1 + e^-l) is 0 in fp64 too from l = -709 on)
        logs = l.gather(1, idx)
        if scoring == "sigmoid":
            logs = logs.clamp_max(0) - torch.log1p(torch.exp(-logs.abs()))
        top = logs.max(1, keepdim=True).values
        e = torch.where(top == -INF, 0.0, torch.exp(logs - top))
        w = torch.where(top == -INF, 0.0, e / e.sum(1, keepdim=True))
    return idx, scale * w, s


SHAPES = [  # T, E, k, groups, kept
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 8, 2, 1, 1), (33, 17, 3, 1, 1), (129, 64, 8, 4, 2), (40, 64, 6, 8, 3),
    (7, 65, 8, 1, 1), (130, 96, 8, 3, 2), (65, 160, 6, 8, 4), (257, 256, 8, 8, 4), (31, 256, 8, 1, 1), (19, 255, 5, 5, 2),
    (21, 256, 8, 32, 2), (9, 32, 4, 32, 8), (12, 24, 8, 2, 2), (300, 128, 1, 4, 1), (50, 248, 7, 31, 9),
]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,kept", SHAPES)
def test_forward(moe, T, E, k, groups, kept, scoring, with_bias):
    g = torch.Generator("cuda").manual_seed(T * 1000 + E)
    for dt in (F32, BF16):  # (of bf16 logits many are equal)
        logits = (torch.randn(T, E, generator=g, device="cuda") * 2).to(dt)
        bias = torch.randn(E, generator=g, device="cuda") * 0.1 if with_bias else None
        for renorm, scale, want in ((True, 2.5, False), (False, 1.0, True)):
            idx, w, s = moe.route_scores(logits, k, scoring, bias, groups, kept, renorm, scale, want)
            ridx, rw, rs = reference(logits, k, scoring, bias, groups, kept, renorm, scale)
            assert idx.dtype is torch.int32 and torch.equal(idx.cpu().long(), ridx)
            assert (w.cpu().to(D) - rw).abs().le(2.0 ** -18 * rw + 2.0 ** -126).all()
            assert (s is not None) == want
            if want:
                assert (s.cpu().to(D) - rs).abs().le(2.0 ** -18 * rs + 2.0 ** -126).all()


def test_scores_that_fp32_cannot_tell_apart(moe):
    """Neighbours by 2^-20 of a unit under a bias, far sigmoids, and groups whose sums differ by as little."""
    g = torch.Generator("cuda").manual_seed(1)
    T, E = 400, 64
    near = torch.randn(T, 1, generator=g, device="cuda") + torch.randint(0, 64, (T, E), generator=g, device="cuda") * 2.0 ** -20
    far = 17 + torch.randn(T, E, generator=g, device="cuda")  # 1 / (1 + e^-17): fp32 holds few values there
    bias = torch.randint(0, 4, (E,), generator=g, device="cuda") * 2.0 ** -22
    for logits in (near, far, torch.zeros(T, E, device="cuda")):
        for scoring in ("softmax", "sigmoid"):
            for b, groups, kept in ((bias, 1, 1), (bias, 8, 3), (None, 8, 3), (bias + 1e4, 1, 1)):
                got = moe.route_scores(logits, 6, scoring, b, groups, kept)[0]
                assert torch.equal(got.cpu().long(), reference(logits, 6, scoring, b, groups, kept, True, 1.0)[0])


def test_masked_experts_and_empty_rows(moe):
    l = torch.randn(6, 40, device="cuda")
    l[0, 3:] = -INF       # three experts left for four slots
    l[1] = -INF           # none
    l[2, ::2] = torch.finfo(F32).min
    l[3] = torch.finfo(F32).min
    l[4] = -200.0         # sigmoids below what fp32 holds
    l[5, 7] = INF
    zero = torch.zeros(40, device="cuda")
    for scoring in ("softmax", "sigmoid"):
        rows = 6 if scoring == "sigmoid" else 5  # (a softmax over +inf is NaN: below)
        for bias, groups, kept in ((None, 1, 1), (zero, 1, 1), (zero, 4, 2)):
            for renorm in (True, False):
                idx, w, s = moe.route_scores(l[:rows].contiguous(), 4, scoring, bias, groups, kept, renorm, 1.0, True)
                ridx, rw, rs = reference(l[:rows], 4, scoring, bias, groups, kept, renorm, 1.0)
                assert torch.equal(idx.cpu().long(), ridx)
                assert (w.cpu().to(D) - rw).abs().le(2.0 ** -18 * rw + 2.0 ** -126).all()
                assert (s.cpu().to(D) - rs).abs().le(2.0 ** -18 * rs + 2.0 ** -126).all()
                assert w[1].eq(0).all()
                dw = torch.randn(rows, 4, device="cuda")
                d = moe.route_scores_backward(l[:rows].contiguous(), idx, dw, zero + 1, scoring, renorm)
                assert d.isfinite().all() and d[1].eq(0).all()


@pytest.mark.parametrize("low", [-INF, torch.finfo(F32).min, -1e9])
def test_experts_masked_by_the_bias_or_the_logits(moe, low):
    g = torch.Generator("cuda").manual_seed(6)
    for E, groups, kept, k in ((256, 8, 4, 8), (64, 4, 2, 3), (160, 8, 8, 6), (32, 8, 2, 6)):
        logits = torch.randn(300, E, generator=g, device="cuda")
        bias = torch.randn(E, generator=g, device="cuda") * 0.1
        for gone in (torch.arange(0, E, 3), torch.arange(0, E // groups), torch.arange(0, E - k), torch.arange(1, E)):
            b, l = bias.clone(), logits.clone()
            b[gone.cuda()] = low
            l[:, gone.cuda()] = low
            for scoring in ("softmax", "sigmoid"):
                for x, y in ((logits, b), (l, bias), (l, None)):
                    for n, m in ((1, 1), (groups, kept)):
                        idx, w, _ = moe.route_scores(x, k, scoring, y, n, m)
                        ridx, rw, _ = reference(x, k, scoring, y, n, m, True, 1.0)
                        assert torch.equal(idx.cpu().long(), ridx)
                        assert (w.cpu().to(D) - rw).abs().le(2.0 ** -18 * rw + 2.0 ** -126).all()


def test_nan_ranks_last_and_reaches_its_weights(moe):
    l = torch.randn(3, 12, device="cuda")
    l[0, 2] = NAN
    l[1, :11] = NAN
    l[2] = NAN
    idx, w, _ = moe.route_scores(l, 3)
    assert torch.equal(idx.cpu().long(), best(l.cpu(), 3))
    assert w[0].isfinite().all() and w[1:].isnan().all()
    idx, w, s = moe.route_scores(l, 3, renormalize=False, want_scores=True)
    assert torch.equal(idx.cpu().long(), best(l.cpu(), 3)) and w.isnan().all() and s.isnan().all()
    idx, w, _ = moe.route_scores(l, 3, "sigmoid", torch.zeros(12, device="cuda"), 3, 2)
    assert (idx >= 0).all() and (idx < 12).all() and all(len(set(r)) == 3 for r in idx.tolist())
    l[0, 2] = INF
    _, w, s = moe.route_scores(l[:1].contiguous(), 3, renormalize=False, want_scores=True)
    assert w.isnan().all() and s.isnan().all()


def gradient(logits, idx, dw, ds, scoring, renorm, scale):
    l = logits.to(D).cpu().requires_grad_()
    s = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 1)
    total = l.sum() * 0
    if dw is not None:
        w = s.gather(1, idx.cpu().long())
        w = w / w.sum(1, keepdim=True) if renorm else w
        total = total + (scale * w * dw.to(D).cpu()).sum()
    if ds is not None:
        total = total + (s * ds.to(D).cpu()).sum()
    return torch.autograd.grad(total, l)[0], s.detach()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 8, 2), (33, 17, 3), (129, 64, 8), (7, 65, 8), (257, 256, 8), (64, 250, 4),
                                   (65, 28, 4), (33, 100, 4), (130, 160, 6), (31, 188, 8), (9, 150, 5), (17, 240, 8)])
def test_backward(moe, T, E, k, scoring, renorm):
    g = torch.Generator("cuda").manual_seed(T + E)
    for dt in (F32, BF16):
        logits = (torch.randn(T, E, generator=g, device="cuda") * 2).to(dt)
        idx = moe.route_scores(logits, k, scoring)[0]
        dw = torch.randn(T, k, generator=g, device="cuda")
        for ds in (None, torch.randn(E, generator=g, device="cuda"), torch.randn(T, E, generator=g, device="cuda")):
            for give in (dw, None):
                if give is None and ds is None:
                    continue
                got = moe.route_scores_backward(logits, idx, give, ds, scoring, renorm, 1.5)
                want, s = gradient(logits, idx, give, ds, scoring, renorm, 1.5)
                size = torch.zeros(T, E, dtype=D)
                if give is not None:
                    part = s.gather(1, idx.cpu().long())
                    part = 1.5 * (part / part.sum(1, keepdim=True) if renorm else part)
                    total = (part * give.cpu().abs()).sum(1, keepdim=True)
                    size.scatter_add_(1, idx.cpu().long(), part * (give.cpu().abs() + total))
                    size += s * total
                if ds is not None:
                    a = ds.cpu().to(D).abs().expand(T, E)
                    size += s * (a + (s * a).sum(1, keepdim=True))
                step = torch.finfo(dt).eps / 2
                assert got.dtype is dt
                assert (got.cpu().to(D) - want).abs().le(2.0 ** -17 * size + step * want.abs() + 2.0 ** -126).all()


def test_backward_is_the_slope_of_forward(moe):
    """Differences of the forward call's weights and scores, fp32 logits in steps of 2^-8: the weights' rounding (2^-18,
    above) over the step is 2^-10, and the step's own error is h^2 / 6 times a third derivative that is below 2."""
    g = torch.Generator("cuda").manual_seed(5)
    l = torch.randn(9, 20, generator=g, device="cuda")
    dw, ds = torch.randn(9, 4, generator=g, device="cuda"), torch.randn(20, generator=g, device="cuda")
    h = 2.0 ** -8
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx = moe.route_scores(l, 4, scoring)[0]
            grad = moe.route_scores_backward(l, idx, dw, ds, scoring, renorm, 2.0)

            def loss(t):  # with the choice of the middle: weights from all scores
                s = moe.route_scores(t, 1, scoring, want_scores=True)[2].to(D)
                w = s.gather(1, idx.long())
                w = 2.0 * (w / w.sum(1, keepdim=True) if renorm else w)
                return (w * dw).sum(1) + (s * ds).sum(1)
            for e in range(20):
                up, down = l.clone(), l.clone()
                up[:, e] += h
                down[:, e] -= h
                slope = (loss(up) - loss(down)) / (2 * h)
                size = 2 * dw.abs().sum(1) + ds.abs().sum()
                assert (slope - grad[:, e]).abs().le((2.0 ** -10 + h * h) * size).all()


@pytest.mark.parametrize("E", [10, 12, 100, 130])
def test_experts_given_twice_and_out_of_range(moe, E):
    l, dw = torch.randn(4, E, device="cuda"), torch.randn(4, 3, device="cuda")
    idx = torch.tensor([[1, 1, 1], [2, -1, E], [-1, E + 89, -7], [9, 0, 9]], dtype=torch.int32, device="cuda")
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = moe.route_scores_backward(l, idx, dw, scoring=scoring, renormalize=renorm)
            assert got[2].eq(0).all()
            for t, cols in ((0, [0, 1, 2]), (1, [0]), (3, [0, 1, 2])):
                want, _ = gradient(l[t:t + 1], idx[t:t + 1, cols], dw[t:t + 1, cols], None, scoring, renorm, 1.0)
                assert (got[t:t + 1].cpu().to(D) - want).abs().max() <= 2.0 ** -17 * dw[t].abs().sum()


def test_given_outputs_streams_and_empty(moe):
    l = torch.randn(5, 12, device="cuda")
    want = moe.route_scores(l, 2, "sigmoid", want_scores=True)
    outs = (torch.empty(5, 2, dtype=torch.int32, device="cuda"), torch.empty(5, 2, device="cuda"), torch.empty(5, 12, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.route_scores(l, 2, "sigmoid", idx=outs[0], w=outs[1], scores=outs[2], stream=side)
    side.synchronize()
    assert all(a is b for a, b in zip(got, outs)) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(t._version > 0 for t in outs)
    none = l[:0]
    idx, w, s = moe.route_scores(none, 2, want_scores=True)
    assert idx.shape == (0, 2) and w.shape == (0, 2) and s.shape == (0, 12)
    assert moe.route_scores_backward(none, idx, w).shape == (0, 12)


def test_unaligned_logits(moe):
    flat = torch.randn(1 + 7 * 30, device="cuda").bfloat16()
    l = flat[1:].view(7, 30)
    assert l.data_ptr() % 4 == 2
    a, b = moe.route_scores(l, 3, "sigmoid", want_scores=True), moe.route_scores(l.clone(), 3, "sigmoid", want_scores=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_logits_beyond_32_bits(moe):
    T, E = 2 ** 31 // 256 + 100, 256
    l, ends = torch.zeros(T, E, dtype=BF16, device="cuda"), [*range(20), *range(T - 50, T)]
    l[ends] = torch.randn(70, E, device="cuda").bfloat16()
    bias = torch.randn(E, device="cuda") * 0.1
    idx, w, _ = moe.route_scores(l, 8, "sigmoid", bias, 8, 4)
    want = moe.route_scores(l[ends], 8, "sigmoid", bias, 8, 4)
    assert torch.equal(idx[ends], want[0]) and torch.equal(w[ends], want[1])
    assert idx[20:T - 50].eq(idx[20]).all()
    dw = torch.zeros(T, 8, device="cuda")
    dw[ends] = torch.randn(70, 8, device="cuda")
    got = moe.route_scores_backward(l, idx, dw, scoring="sigmoid")
    assert torch.equal(got[ends], moe.route_scores_backward(l[ends], idx[ends], dw[ends], scoring="sigmoid"))
    assert got[20:T - 50].count_nonzero() == 0


@pytest.mark.parametrize("E,k,groups,kept", [(64, 6, 1, 1), (256, 8, 8, 4), (100, 3, 1, 1)])
def test_two_streams_at_once_and_a_replayed_graph(moe, E, k, groups, kept):
    g = torch.Generator("cuda").manual_seed(E)
    sets = [torch.randn(2000, E, generator=g, device="cuda") for _ in range(2)]
    sets[1][:, 1] = sets[1][:, 0]  # (contested rows)
    bias, dw = torch.randn(E, generator=g, device="cuda") * 0.1, torch.randn(2000, k, generator=g, device="cuda")

    def both(l):
        idx, w, s = moe.route_scores(l, k, "softmax", bias, groups, kept, want_scores=True)
        return [idx, w, s, moe.route_scores_backward(l, idx, dw, bias, "softmax")]
    want = [both(l) for l in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both(sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept_outputs = both(sets[0])
    sets[0].copy_(sets[1])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(kept_outputs, want[1]))
