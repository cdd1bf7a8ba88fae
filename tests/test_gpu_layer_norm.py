"""Layer norm after a residual, with dropout, and its gradient, against 64 bits.

Tolerances, with u = 2^-24.  A sum over a row of d <= 65536 values passes through fewer than 64 additions one after
another (up to 32 in a thread, 5 in a warp, 5 over the warps), so it is off by 64 u = 2^-18 of the sum of the terms'
sizes at the most; the mean by 2^-18 mean|y|, 1 / std by 2^-18 of itself beyond what the mean's error brings (of second
order).  So n before its rounding is off by 2^-18 |weight| (|yh| + mean|y| / std) + u |bias| and a few u, and by half a
step of bf16 (2^-8) after it.  The gradients alike; column sums over T rows add fewer than 64 rows one after another in
a block and fewer than 32 blocks and runs, so 2^-17 of the sum of sizes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
EPS = 1e-5


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


def randn(g, *shape, dtype=F32, scale=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale + mean).to(dtype)


def check_norm(y, weight, bias, n, stats, eps=EPS):
    """n and stats against the norm of y (fp64 on the device)."""
    y = y.to(D)
    w = weight.to(D) if weight is not None else 1.0
    b = bias.to(D) if bias is not None else torch.zeros((), dtype=D, device="cuda")
    mean = y.mean(1, keepdim=True)
    r = 1 / ((y - mean).square().mean(1, keepdim=True) + eps).sqrt()
    yh = (y - mean) * r
    size = y.abs().mean(1, keepdim=True)
    assert (stats[:, :1].to(D) - mean).abs().le(2.0 ** -18 * size).all()
    assert (stats[:, 1:].to(D) / r - 1).abs().le(2.0 ** -17 + (2.0 ** -18 * size * r) ** 2).all()
    want = w * yh + b
    slack = 2.0 ** -17 * abs(w) * (yh.abs() + size * r) + 2.0 ** -22 * b.abs()
    assert (n.to(D) - want).abs().le(2.0 ** -8 * want.abs() + slack * 1.01).all()


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (9, 33), (4, 256), (7, 264), (700, 96), (33, 1000), (301, 1024), (5, 2891),
          (160, 4096), (3, 4104), (1, 7168), (311, 7168), (6, 8190), (5, 8192), (400, 6091),
          (1216, 2072), (1300, 2891), (2, 8200), (3, 16384), (2, 20001), (2, 65536)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(moe, T, d, dt):
    g = torch.Generator("cuda").manual_seed(T * 100 + d)
    x, h = randn(g, T, d, dtype=dt, scale=2, mean=0.5), randn(g, T, d, dtype=BF16)
    w, b = randn(g, d, scale=0.2, mean=1), randn(g, d, scale=0.2)
    y, n, stats = moe.layer_norm(x, w, b)
    assert y is None and n.dtype is BF16 and stats.dtype is F32
    check_norm(x, w, b, n, stats)
    for p in (0.0, 0.3):
        y, n, stats = moe.layer_norm(x, w, None, h=h, p=p, seed=7, offset=3)
        assert y.dtype is dt
        assert torch.equal(y, moe.dropout(h, p, 7, 3, residual=x))
        check_norm(y, w, None, n, stats)
    y, n, stats = moe.layer_norm(x, None, b, h=h, eps=0.5)
    want = x.to(D) + h.to(D)
    assert (y.to(D) - want).abs().le(STEP[dt] * want.abs() + 2.0 ** -24 * want.abs()).all()
    check_norm(y, None, b, n, stats, eps=0.5)


@pytest.mark.parametrize("d", [64, 100, 7168, 20000])
def test_far_means_outliers_and_constant_rows(moe, d):
    """A mean a thousand times the deviation, one value far from all others, and no deviation at all."""
    g = torch.Generator("cuda").manual_seed(d)
    x = randn(g, 4, d)
    x[0] += 1000
    x[1, 0] = 1e4
    x[2, d - 1] = -1e4
    x[3] = 3.0
    y, n, stats = moe.layer_norm(x)
    check_norm(x[:3], None, None, n[:3], stats[:3])
    assert n[3].eq(0).all() and stats[3, 0] == 3.0
    assert abs(stats[3, 1].item() * EPS ** 0.5 - 1) < 2.0 ** -20


def test_infinities_and_nan_stay_in_their_rows(moe):
    for d in (40, 41, 9000):
        x = torch.randn(5, d, device="cuda")
        clean = moe.layer_norm(x)[1]
        x[1, 3], x[3, d - 1] = float("inf"), float("nan")
        n = moe.layer_norm(x)[1]
        assert torch.equal(n[::2], clean[::2]) and n[1].isnan().all() and n[3].isnan().all()


def test_what_is_dropped_is_not_there(moe):
    """Infinities and NaN of h in dropped places leave no trace."""
    g = torch.Generator("cuda").manual_seed(2)
    for d in (64, 67):
        x, h = randn(g, 50, d), randn(g, 50, d, dtype=BF16, mean=10, scale=0.1)
        gone = moe.dropout(h, 0.5, 1, 2).eq(0)
        bad = h.masked_fill(gone, float("nan"))
        for a, b in zip(moe.layer_norm(x, h=h, p=0.5, seed=1, offset=2), moe.layer_norm(x, h=bad, p=0.5, seed=1, offset=2)):
            assert torch.equal(a, b)


def backward(x, stats, dn, dy, weight):
    x, dn = x.to(D), dn.to(D)
    yh = (x - stats[:, :1].to(D)) * stats[:, 1:].to(D)
    g = dn * weight.to(D) if weight is not None else dn
    a, b = g.mean(1, keepdim=True), (g * yh).mean(1, keepdim=True)
    dx = (dy.to(D) if dy is not None else 0.0) + stats[:, 1:].to(D) * (g - a - yh * b)
    size = (dy.to(D).abs() if dy is not None else 0.0) + stats[:, 1:].to(D) * (
        g.abs() + g.abs().mean(1, keepdim=True) + yh.abs() * (g * yh).abs().mean(1, keepdim=True))
    return dx, size, (dn * yh).sum(0), (dn * yh).abs().sum(0), dn.sum(0), dn.abs().sum(0)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,d", SHAPES)
def test_backward(moe, T, d, dt):
    g = torch.Generator("cuda").manual_seed(T * 100 + d + 1)
    x, dy = randn(g, T, d, dtype=dt, scale=2, mean=0.5), randn(g, T, d, dtype=dt, scale=0.1)
    dn, w = randn(g, T, d, dtype=BF16, scale=0.1), randn(g, d, scale=0.2, mean=1)
    stats = moe.layer_norm(x)[2]
    for weight, give, want_h, p in ((w, dy, False, 0.0), (w, dy, True, 0.25), (None, None, True, 0.0), (w, None, False, 0.0)):
        bias = w if weight is None else None
        got = moe.layer_norm_backward(x, stats, dn, give, weight, bias, want_h, p, 11, 4)
        dx, size, dw, dw_size, db, db_size = backward(x, stats, dn, give, weight)
        assert got["x"].dtype is dt and (got["x"].to(D) - dx).abs().le(STEP[dt] * dx.abs() + 2.0 ** -17 * size).all()
        assert (got["h"] is not None) == want_h and (got["weight"] is None) == (weight is None)
        if weight is not None:
            assert got["bias"] is None and (got["weight"].to(D) - dw).abs().le(2.0 ** -17 * dw_size).all()
        else:
            assert (got["bias"].to(D) - db).abs().le(2.0 ** -17 * db_size).all()
        if want_h:
            stays = moe.dropout(torch.ones(T, d, device="cuda"), p, 11, 4).to(D)
            assert (got["h"].to(D) - dx * stays).abs().le(stays * (2.0 ** -8 * dx.abs() + 2.0 ** -16 * size)).all()


def test_backward_is_the_slope_of_forward(moe):
    """Differences of sum(dn n + dy y) computed from the forward call's stats (n itself is bf16), in steps of h = 2^-6:
    the stats' errors, 2^-18 of values below 4, over the step are 2^-10 of the terms' sum, the step's own h^2."""
    g = torch.Generator("cuda").manual_seed(3)
    T, d, h = 3, 24, 2.0 ** -6
    x, w = randn(g, T, d), randn(g, d, scale=0.2, mean=1)
    dn, dy = randn(g, T, d, dtype=BF16), randn(g, T, d)

    def loss(t):
        s = moe.layer_norm(t, w)[2].to(D)
        return ((t.to(D) - s[:, :1]) * s[:, 1:] * w * dn + t.to(D) * dy).sum(1)
    grad = moe.layer_norm_backward(x, moe.layer_norm(x, w)[2], dn, dy, w)["x"]
    size = (dn.abs().sum(1) + dy.abs().sum(1)).to(D)
    for c in range(d):
        up, down = x.clone(), x.clone()
        up[:, c] += h
        down[:, c] -= h
        assert ((loss(up) - loss(down)) / (2 * h) - grad[:, c]).abs().le((2.0 ** -10 + 4 * h * h) * size).all()


def test_same_result_on_every_run_and_in_graphs(moe):
    g = torch.Generator("cuda").manual_seed(9)
    x, dn, h = randn(g, 2000, 520), randn(g, 2000, 520, dtype=BF16), randn(g, 2000, 520, dtype=BF16)
    w = randn(g, 520)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def both():
        y, n, stats = moe.layer_norm(x, w, w, h=h, p=0.2, seed=5, offset=1, offset_tensor=step)
        b = moe.layer_norm_backward(y, stats, dn, x, w, w, True, 0.2, 5, 1, step)
        return [y, n, stats, *b.values()]
    first = both()
    assert all(torch.equal(a, b) for a, b in zip(first, both()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for i in range(3):
        step.fill_(i)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(kept, both())), i
    step.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, kept)) and not torch.equal(kept[0], moe.layer_norm(x, w, w, h=h, p=0.2, seed=5, offset=2)[0])


def test_weights_off_the_widest_loads(moe):
    g = torch.Generator("cuda").manual_seed(14)
    flat, x = randn(g, 4 * 4200, scale=0.2, mean=1), randn(g, 40, 4096, dtype=BF16)
    dn = randn(g, 40, 4096, dtype=BF16)
    for off in (1, 2, 4, 12):
        w, b = flat[off:off + 4096], flat[8400 + off:8400 + off + 4096]
        _, n, stats = moe.layer_norm(x, w, b)
        check_norm(x, w, b, n, stats)
        got = moe.layer_norm_backward(x, stats, dn, None, w)["x"]
        dx, size = backward(x, stats, dn, None, w)[:2]
        assert (got.to(D) - dx).abs().le(2.0 ** -8 * dx.abs() + 2.0 ** -17 * size).all()


def test_unaligned_tensors_in_place_and_no_rows(moe):
    g = torch.Generator("cuda").manual_seed(4)
    flat = randn(g, 1 + 6 * 48, dtype=BF16)
    x = flat[1:].view(6, 48)
    want = moe.layer_norm(x.clone())
    got = moe.layer_norm(x)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])  # (sums in the same order)
    h = randn(g, 6, 48, dtype=BF16)
    y, n, stats = moe.layer_norm(x.clone(), h=h, p=0.1, seed=1)
    mine = x.clone()
    y2, n2, _ = moe.layer_norm(mine, h=h, p=0.1, seed=1, y=mine)
    assert y2 is mine and torch.equal(mine, y) and torch.equal(n, n2)
    e = x[:0]
    y, n, stats = moe.layer_norm(e, h=h[:0])
    assert y.shape == (0, 48) and n.shape == (0, 48) and stats.shape == (0, 2)
    grads = moe.layer_norm_backward(e, stats, n, weight=torch.ones(48, device="cuda"), bias=torch.ones(48, device="cuda"))
    assert grads["weight"].eq(0).all() and grads["bias"].eq(0).all() and grads["x"].shape == (0, 48)


@pytest.mark.parametrize("T,d", [(600_001, 3581), (524_500, 4104)])
def test_elements_beyond_32_bits(moe, T, d):
    """The first and the last rows of more than 2^31 elements."""
    g = torch.Generator("cuda").manual_seed(d)
    assert T * d > 2 ** 31
    x, dn = torch.zeros(T, d, dtype=BF16, device="cuda"), torch.zeros(T, d, dtype=BF16, device="cuda")
    w = randn(g, d, scale=0.2, mean=1)
    ends = [*range(9), *range(T - 9, T)]
    x[ends], dn[ends] = randn(g, 18, d, dtype=BF16, scale=2, mean=0.5), randn(g, 18, d, dtype=BF16)
    _, n, stats = moe.layer_norm(x, w)
    check_norm(x[ends], w, None, n[ends], stats[ends])
    assert n[9:T - 9].count_nonzero() == 0
    del n
    got = moe.layer_norm_backward(x, stats, dn, None, w)
    dx, size, dw, dw_size, _, _ = backward(x[ends], stats[ends], dn[ends], None, w)
    assert (got["x"][ends].to(D) - dx).abs().le(2.0 ** -8 * dx.abs() + 2.0 ** -17 * size).all()
    assert got["x"][9:T - 9].count_nonzero() == 0
    assert (got["weight"].to(D) - dw).abs().le(2.0 ** -17 * dw_size).all()


@pytest.mark.parametrize("T,d", [(50, 256), (1300, 2891), (40, 8200), (90, 12288), (30, 16384), (3, 65536)])
def test_two_streams_at_once_and_a_replayed_graph(moe, T, d):
    g = torch.Generator("cuda").manual_seed(d)
    sets = [(randn(g, T, d, dtype=BF16), randn(g, T, d, dtype=BF16), randn(g, d)) for _ in range(2)]

    def both(x, h, w, stream=None):
        y, n, stats = moe.layer_norm(x, w, w, h=h, p=0.25, seed=3, stream=stream)
        return [y, n, stats, *moe.layer_norm_backward(y, stats, h, x, w, w, True, 0.25, 3, stream=stream).values()]
    want = [both(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = [both(*s) for s in sets]
    for r in kept:
        for t in r:
            t.zero_()
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(a, b) for r, v in zip(kept, want) for a, b in zip(r, v))
