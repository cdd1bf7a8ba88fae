"""Grouped products and their gradients (moe_grouped_mm, moe_grouped_mm_wgrad) against the formulas in
64 bits.

Tolerance, elementwise: the bf16 operands' products are exact in fp32; a sum of n of them is off by at
most n * 2^-23 of the sum of their magnitudes (each fp32 addition, rounded or truncated, by 2^-23 of a
partial sum at most), plus, for a bf16 output, half a step of the value (2^-8 of it)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

COUNTS = {
    "mixed": [0, 1, 15, 16, 17, 0, 33, 64, 65, 129],
    "long": [257, 0, 600, 256, 3],
    "empty": [0, 0, 0],
    "one": [1],
    "single_row_late": [0, 0, 1],
    "even": [32, 32, 64, 48],
    "segment_ends": [63, 127, 128, 31, 2, 47],
}


def _inputs(counts, K, N, way, seed=0, lead=0, trail=0):
    g = torch.Generator().manual_seed(seed)
    M = lead + sum(counts) + trail
    offs = torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + lead, dtype=torch.int32)
    a = torch.randn(M, K, generator=g).bfloat16()
    shape = {"fwd": (len(counts), K, N), "dgrad": (len(counts), N, K), "wgrad": (M, N)}[way]
    return a, torch.randn(*shape, generator=g).bfloat16(), offs


def _reference(a, b, offs, way):
    """The products in 64 bits, and the sums of the magnitudes of what they add."""
    a, b = a.double(), b.double()
    E = len(offs) - 1
    if way == "wgrad":
        out = torch.stack([a[offs[e]:offs[e + 1]].T @ b[offs[e]:offs[e + 1]] for e in range(E)])
        mag = torch.stack([a[offs[e]:offs[e + 1]].abs().T @ b[offs[e]:offs[e + 1]].abs() for e in range(E)])
        return out, mag
    w = b if way == "fwd" else b.transpose(1, 2)
    out, mag = (torch.zeros(a.shape[0], w.shape[2], dtype=torch.float64) for _ in range(2))
    for e in range(E):
        r = slice(int(offs[e]), int(offs[e + 1]))
        out[r], mag[r] = a[r] @ w[e], a[r].abs() @ w[e].abs()
    return out, mag


def _check(got, ref, mag, n, what):
    got = got.cpu()
    bound = n * 2.0 ** -23 * mag + (2.0 ** -8 * ref.abs() if got.dtype == torch.bfloat16 else 0) + 1e-30
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((off / bound).max())} of the bound"


def _run(moe, a, b, offs, way, **kw):
    a, b, offs = a.cuda(), b.cuda(), offs.cuda()
    if way == "wgrad":
        return moe.grouped_mm_wgrad(a, b, offs, **kw)
    return moe.grouped_mm(a, b, offs, transpose_b=way == "dgrad", **kw)


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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("K,N", [(64, 256), (8, 8), (72, 264), (328, 520), (128, 16), (256, 320),
                                 (512, 64)])
@pytest.mark.parametrize("counts", list(COUNTS))
def test_products(moe, counts, K, N, way, dtype):
    a, b, offs = _inputs(COUNTS[counts], K, N, way)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if a.shape[0] == 0 and way != "wgrad":
        assert _run(moe, a, b, offs, way, out_dtype=dtype).shape == (0, N)
        return
    got = _run(moe, a, b, offs, way, out_dtype=dtype, status=status)
    ref, mag = _reference(a, b, offs, way)
    n = max(COUNTS[counts]) if way == "wgrad" else K
    _check(got, ref, mag, n, f"{way} {counts} K={K} N={N}")
    assert moe.get_device_error(status) == 0


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
def test_many_experts(moe, way):
    rng = np.random.default_rng(3)
    counts = rng.multinomial(700, rng.dirichlet(np.full(256, 0.3))).tolist()
    a, b, offs = _inputs(counts, 136, 296, way)
    got = _run(moe, a, b, offs, way, out_dtype=torch.float32)
    ref, mag = _reference(a, b, offs, way)
    _check(got, ref, mag, max(counts) if way == "wgrad" else 136, way)


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("active", [(0,), (255,), (0, 255), (254, 255), (1, 2, 3, 100, 101, 250), tuple(range(7, 256, 31))])
def test_few_of_many_experts(moe, way, active):
    """Tokens in a few of 256 experts, next to each other and far apart, with several tiles each."""
    counts = [0] * 256
    for k, e in enumerate(active):
        counts[e] = 1 + 5 * k if k % 3 else 270
    a, b, offs = _inputs(counts, 72, 1288 if way != "wgrad" else 136, way)
    got = _run(moe, a, b, offs, way, out_dtype=torch.float32)
    ref, mag = _reference(a, b, offs, way)
    _check(got, ref, mag, max(counts) if way == "wgrad" else 72, way)


@pytest.mark.parametrize("way", ["fwd", "dgrad"])
def test_rows_outside_the_segments_stay(moe, way):
    a, b, offs = _inputs([5, 0, 40], 64, 136, way, lead=3, trail=70)
    out = torch.full((a.shape[0], 136), 7.0, device="cuda")
    got = _run(moe, a, b, offs, way, out=out)
    assert got is out
    ref, mag = _reference(a, b, offs, way)
    rows = slice(3, 48)
    _check(got[rows], ref[rows], mag[rows], 64, way)
    assert (got[:3] == 7).all() and (got[48:] == 7).all()


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), torch.finfo(torch.bfloat16).max])
def test_other_segments_values_stay_there(moe, way, value):
    """Infinities and NaN in one expert's rows (or weights) reach no other expert's outputs."""
    counts = [13, 21, 40, 0, 9]
    a, b, offs = _inputs(counts, 72, 136, way)
    clean, mag = _reference(a, b, offs, way)
    a[13:34] = value
    (b[13:34] if way == "wgrad" else b[1])[...] = value
    got = _run(moe, a, b, offs, way, out_dtype=torch.float32).cpu()
    n = max(counts) if way == "wgrad" else 72
    if way == "wgrad":
        keep = [0, 2, 3, 4]
        _check(got[keep], clean[keep], mag[keep], n, way)
        assert (got[3] == 0).all()
    else:
        keep = torch.cat([torch.arange(13), torch.arange(34, 83)])
        _check(got[keep], clean[keep], mag[keep], n, way)


def test_wgrad_accumulates(moe):
    counts = [20, 0, 37]
    a, g, offs = _inputs(counts, 72, 136, "wgrad")
    ref, mag = _reference(a, g, offs, "wgrad")
    start = torch.randn(3, 72, 136, generator=torch.Generator().manual_seed(9))
    out = start.cuda()
    _run(moe, a, g, offs, "wgrad", out=out, accumulate=True)
    _run(moe, a, g, offs, "wgrad", out=out, accumulate=True)
    want = start.double() + 2 * ref
    _check(out, want, 2 * mag + 3 * start.double().abs(), 40, "accumulate")


@pytest.mark.parametrize("counts,K,N", [([3, 0, 40, 17] * 24, 264, 1032), ([600, 1, 0, 555] * 5, 520, 1288)])
def test_wgrad_adds_once(moe, counts, K, N):
    """The sum is that of the gradient and what was there, rounded once, over several tiles per SM pair; empty
    segments' stay as they are, infinities and NaN too."""
    a, g, offs = _inputs(counts, K, N, "wgrad")
    start = torch.randn(len(counts), K, N, generator=torch.Generator().manual_seed(9))
    start[1, 0, :2] = torch.tensor([float("inf"), float("nan")])
    start[2, K - 1, N - 1] = float("-inf")
    start = start.cuda()
    want = start + _run(moe, a, g, offs, "wgrad")
    for _ in range(2):
        out = start.clone()
        _run(moe, a, g, offs, "wgrad", out=out, accumulate=True)
        assert torch.equal(out.nan_to_num(7.5), want.nan_to_num(7.5)) and torch.equal(out.isnan(), want.isnan())
        assert torch.equal(out[torch.tensor(counts) == 0].nan_to_num(7.5),
                           start[torch.tensor(counts) == 0].nan_to_num(7.5))


@pytest.mark.parametrize("way,M,K,N,E", [("fwd", 3, 8192, 256, 2), ("dgrad", 70, 4104, 264, 1), ("wgrad", 4099, 72, 136, 1)])
def test_split_reduction(moe, way, M, K, N, E):
    """A long reduction over few tiles is split into slices; the result is the same on every run, and
    rows outside the segments stay as they are."""
    counts = [M] if E == 1 else [1, M - 1]
    mode = {"fwd": 0, "dgrad": 1, "wgrad": 2}[way]
    assert moe.grouped_mm_workspace_size(mode, M, K, N, E) > 0
    a, b, offs = _inputs(counts, K, N, way, lead=0 if way == "wgrad" else 2, trail=0)
    scale = 1 / 64  # keeps the sums near one
    a = (a.float() * scale).bfloat16()
    ref, mag = _reference(a, b, offs, way)
    out = None if way == "wgrad" else torch.full(ref.shape, 5.0, device="cuda")
    got = _run(moe, a, b, offs, way, out=out, out_dtype=torch.float32)
    again = _run(moe, a, b, offs, way, out_dtype=torch.float32)
    lo = 0 if way == "wgrad" else 2
    n = (M if way == "wgrad" else K)
    _check(got[lo:], ref[lo:], mag[lo:], n, way)
    assert torch.equal(got[lo:], again[lo:])
    if lo:
        assert (got[:lo] == 5).all()
    one = _run(moe, a, b, offs, way, out_dtype=torch.bfloat16)
    _check(one[lo:], ref[lo:], mag[lo:], n, way)
    if way == "wgrad":
        acc = got.clone()
        _run(moe, a, b, offs, way, out=acc, accumulate=True)
        _check(acc, 2 * ref, 2 * mag, n + 2, way)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,N", [(264, 520), (904, 72), (256, 256)])
def test_wgrad_of_mostly_empty_segments(moe, K, N, dtype):
    counts = [0] * 20 + [3] + [0] * 7 + [70] + [0] * 30
    a, g, offs = _inputs(counts, K, N, "wgrad")
    out = torch.full((len(counts), K, N), 9.0, dtype=dtype, device="cuda")
    _run(moe, a, g, offs, "wgrad", out=out)
    ref, mag = _reference(a, g, offs, "wgrad")
    _check(out, ref, mag, 70, "mostly empty")


def test_wgrad_split_with_short_segments(moe):
    """Slices of a split reduction that lie past a short segment's rows are zero."""
    counts = [3, 4300]
    assert moe.grouped_mm_workspace_size(2, sum(counts), 72, 136, 2) > 0
    a, g, offs = _inputs(counts, 72, 136, "wgrad")
    a = (a.float() / 64).bfloat16()
    ref, mag = _reference(a, g, offs, "wgrad")
    for dtype in (torch.float32, torch.bfloat16):
        _check(_run(moe, a, g, offs, "wgrad", out_dtype=dtype), ref, mag, 4300, "split, short segments")


def test_bad_offsets_write_nothing_and_set_the_status(moe):
    a, b, _ = _inputs([10], 64, 64, "fwd")
    for offs in ([0, 11], [5, 3], [-1, 10]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((10, 64), 3.0, device="cuda")
        _run(moe, a, b, torch.tensor(offs, dtype=torch.int32), "fwd", out=out, status=status)
        assert moe.get_device_error(status) == moe.STATUS_BAD_OFFSETS
        assert (out == 3).all()


def test_other_stream_and_graph(moe):
    """The call runs on the stream that it is given, and replays from a graph."""
    a, b, offs = (t.cuda() for t in _inputs([40, 9, 0, 130], 136, 264, "fwd"))
    want = moe.grouped_mm(a, b, offs, out_dtype=torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = moe.grouped_mm(a, b, offs, out_dtype=torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.grouped_mm(a, b, offs, out=out)
    a.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2 * want)
