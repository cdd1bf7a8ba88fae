"""Dropout against its generator's definition, embedding and its gradient against 64 bits.

Tolerances, u = 2^-24: a dropped-out value is a product (and with a residual a sum), each rounded to fp32 (u of the
value, resp. of the sum), then to the result's type.  A row of the embedding's gradient is a sum of n rows: up to 63
one after another, or 32 of a piece and then shares of n / 128 pieces and 16 shares; and a product: (66 + n / 128) u of
the sizes' sum."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


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


def philox(key, counter, rounds=10):
    """One block of Philox4x32 in Python integers."""
    c, k, m = list(counter), list(key), 0xFFFFFFFF
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def test_the_generator_gives_the_published_vectors():
    """The known answers that the generator's authors published for ten rounds."""
    assert philox((0, 0), (0, 0, 0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert philox((f, f), (f, f, f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert philox((0xA4093822, 0x299F31D0), (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def stays(n, p, seed, offset, first=0):
    """Of the elements from ``first`` (a multiple of 8) to n - 1."""
    m = 0xFFFFFFFF
    key, off = (seed & m, seed >> 32), offset % 2 ** 64
    out = []
    for b in range(first // 8, (n + 7) // 8):
        for w in philox(key, (b & m, b >> 32, off & m, off >> 32)):
            out += [w & 0xFFFF, w >> 16]
    return torch.tensor(out[:n - first], device="cuda") >= round(p * 65536)


@pytest.mark.parametrize("n", [1, 7, 8, 9, 1000, 4096 + 5, 12345])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9999])
@pytest.mark.parametrize("seed,offset", [(0, 0), (0x123456789ABCDEF0, 77), (2 ** 64 - 1, -1)])
def test_dropout(moe, n, p, seed, offset):
    g = torch.Generator("cuda").manual_seed(n)
    keep = stays(n, p, seed, offset)
    up = 65536 / (65536 - round(p * 65536))
    for dt in (F32, BF16):
        x = torch.randn(n, generator=g, device="cuda").to(dt)
        want = torch.where(keep, x.to(D) * up, 0.0)
        got = moe.dropout(x, p, seed, offset)
        assert got.dtype is dt and (got.to(D) - want).abs().le((STEP[dt] + 2.0 ** -22) * want.abs()).all()
        for rt in (F32, BF16):
            r = torch.randn(n, generator=g, device="cuda").to(rt)
            got = moe.dropout(x, p, seed, offset, residual=r)
            total = want + r.to(D)
            assert got.dtype is rt
            assert (got.to(D) - total).abs().le(STEP[rt] * total.abs() + 2.0 ** -22 * (want.abs() + r.abs())).all()


def test_the_mask_does_not_depend_on_type_shape_alignment_or_stream(moe):
    ones = torch.ones(3 * 1111, device="cuda")
    want = moe.dropout(ones, 0.3, 5, 6).ne(0)
    assert 0.65 < want.float().mean() < 0.75  # (0.7; eight deviations of 3333 draws are 0.064)
    assert torch.equal(moe.dropout(ones.view(3, 1111), 0.3, 5, 6).ne(0).view(-1), want)
    assert torch.equal(moe.dropout(ones.bfloat16(), 0.3, 5, 6).ne(0), want)
    shifted = torch.ones(1 + ones.numel(), device="cuda").bfloat16()[1:]
    assert torch.equal(moe.dropout(shifted, 0.3, 5, 6).ne(0), want)
    at = torch.tensor([4], device="cuda")
    assert torch.equal(moe.dropout(ones, 0.3, 5, 2, offset_tensor=at).ne(0), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.dropout(ones, 0.3, 5, 6, stream=side)
    side.synchronize()
    assert torch.equal(got.ne(0), want)
    assert not torch.equal(moe.dropout(ones, 0.3, 5, 7).ne(0), want) and not torch.equal(moe.dropout(ones, 0.3, 6, 6).ne(0), want)


def test_dropped_infinities_in_place_and_empty(moe):
    x = torch.full((100,), float("inf"), device="cuda")
    x[::2] = float("nan")
    r = torch.randn(100, device="cuda")
    keep = moe.dropout(torch.ones(100, device="cuda"), 0.5, 9).ne(0)
    got = moe.dropout(x, 0.5, 9, residual=r)
    assert torch.equal(got[~keep], r[~keep]) and not got[keep].isfinite().any()
    for shift in (0, 1):  # over the residual, over x
        a, b = torch.randn(64 + shift, device="cuda")[shift:], torch.randn(64 + shift, device="cuda")[shift:]
        want = moe.dropout(a, 0.5, 9, residual=b)
        for where in (a.clone(), b.clone()):
            ops = (where, b) if torch.equal(where, a) else (a, where)
            got = moe.dropout(ops[0], 0.5, 9, residual=ops[1], out=where)
            assert got is where and torch.equal(got, want)
    assert moe.dropout(x[:0], 0.5, 1).numel() == 0


# -------------------------------------------------------------------------------------------------
EMBED = [(1, 1, 1), (1, 5, 8), (7, 3, 24), (32, 1000, 72), (33, 200, 64), (1000, 17, 33), (5000, 1, 16), (4099, 300, 264),
         (700, 5000, 1028), (65, 40, 4096), (70, 9, 8200), (20000, 100000, 8)]


def tokens(g, T, V, dtype):
    r = torch.rand(T, generator=g, device="cuda", dtype=D)
    return (r ** 4 * V).to(dtype).clamp_max_(V - 1)  # low ids often


@pytest.mark.parametrize("T,V,d", EMBED)
def test_embed(moe, T, V, d):
    g = torch.Generator("cuda").manual_seed(T + V)
    ids = tokens(g, T, V, torch.int64)
    for tt in (F32, BF16):
        table = torch.randn(V, d, generator=g, device="cuda").to(tt)
        want = 1.7 * table[ids].to(D)
        for ot in (None, F32, BF16):
            for i in (ids, ids.int()):
                got = moe.embed(i, table, 1.7, out_dtype=ot)
                assert got.dtype is (ot or tt) and got.shape == (T, d)
                assert (got.to(D) - want).abs().le((STEP[got.dtype] + 2.0 ** -22) * want.abs()).all()
    assert torch.equal(moe.embed(ids, table), table[ids])
    assert torch.equal(moe.embed(ids.view(1, T, 1), table), table[ids].view(1, T, 1, d))


@pytest.mark.parametrize("T,V,d", EMBED)
def test_embed_backward(moe, T, V, d):
    g = torch.Generator("cuda").manual_seed(T + V + 1)
    ids = tokens(g, T, V, torch.int64)
    many = torch.bincount(ids, minlength=V).to(D)[:, None]
    for dt in (F32, BF16):
        dy = torch.randn(T, d, generator=g, device="cuda").to(dt)
        want = torch.zeros(V, d, dtype=D, device="cuda").index_add_(0, ids, dy.to(D)) * 1.3
        size = torch.zeros(V, d, dtype=D, device="cuda").index_add_(0, ids, dy.to(D).abs()) * 1.3
        off = (66 + many / 128) * 2.0 ** -24 * size
        for i in (ids, ids.int()):
            got = moe.embed_backward(i, dy, V, 1.3)
            assert got.dtype is F32 and (got.to(D) - want).abs().le(off).all()
            assert torch.equal(got, moe.embed_backward(i, dy, V, 1.3))
        low = moe.embed_backward(ids, dy, V, 1.3, out_dtype=BF16)
        assert (low.to(D) - want).abs().le(2.0 ** -8 * want.abs() + off * 1.01).all()
        there = torch.randn(V, d, generator=g, device="cuda")
        out = there.clone()
        assert moe.embed_backward(ids, dy, V, 1.3, out=out, accumulate=True) is out
        total = there.to(D) + want
        assert (out.to(D) - total).abs().le(off + 2.0 ** -24 * (total.abs() + off)).all()
        assert torch.equal(out[many[:, 0] == 0], there[many[:, 0] == 0])


def test_gradient_is_the_transpose_of_the_lookup(moe):
    """sum(embed(table) dy) = sum(table dtable), in 64 bits from values that are whole numbers: equal."""
    g = torch.Generator("cuda").manual_seed(8)
    ids = tokens(g, 3000, 70, torch.int32)
    table = torch.randint(-8, 9, (70, 40), generator=g, device="cuda").float()
    dy = torch.randint(-8, 9, (3000, 40), generator=g, device="cuda").bfloat16()
    a = (moe.embed(ids, table, 2.0).to(D) * dy.to(D)).sum()
    b = (table.to(D) * moe.embed_backward(ids, dy, 70, 2.0).to(D)).sum()
    assert a == b


def test_ids_outside_the_table(moe):
    for dtype in (torch.int32, torch.int64):
        ids = torch.tensor([3, -1, 0, 10, 3, 2 ** 31 - 1, -2 ** 31, 9], device="cuda").to(dtype)
        if dtype is torch.int64:
            ids[5], ids[6] = 2 ** 40 + 3, -2 ** 50
        good = torch.tensor([0, 2, 4, 7], device="cuda")
        table, dy = torch.randn(10, 20, device="cuda"), torch.randn(8, 20, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = moe.embed(ids, table, status=status)
        assert status.item() == moe.STATUS_BAD_TOKEN
        assert torch.equal(out[good], table[ids[good].long()]) and out[[1, 3, 5, 6]].eq(0).all()
        status.zero_()
        got = moe.embed_backward(ids, dy, 10, status=status)
        assert status.item() == moe.STATUS_BAD_TOKEN
        want = moe.embed_backward(ids[good].contiguous(), dy[good].contiguous(), 10, status=status.zero_())
        assert torch.equal(got, want) and status.item() == 0
        none = torch.full((40,), -5, device="cuda", dtype=dtype)
        assert moe.embed_backward(none, torch.ones(40, 20, device="cuda"), 10).eq(0).all()
        assert moe.embed(none, table).eq(0).all()


def test_the_longest_runs_and_every_piece_border(moe):
    """One id for all tokens but a few, at all places of a piece; values that are whole numbers: exact."""
    for T in (31, 32, 33, 63, 64, 65, 97, 1025, 9000):
        for first in (0, 1, 31, 32, 33):
            ids = torch.full((T,), 5, device="cuda")
            ids[:first] = 3
            ids[T - 1] = 6
            dy = torch.randint(-4, 5, (T, 16), device="cuda").float()
            want = torch.zeros(8, 16, device="cuda").index_add_(0, ids, dy)
            assert torch.equal(moe.embed_backward(ids, dy, 8), want), (T, first)


def test_wide_vocabularies(moe):
    """More slices than blocks at a time, and a table of more than 2^31 elements."""
    V = 600_000
    ids = torch.randint(0, V, (5000,), device="cuda")
    dy = torch.randint(-4, 5, (5000, 8), device="cuda").float()
    assert torch.equal(moe.embed_backward(ids, dy, V), torch.zeros(V, 8, device="cuda").index_add_(0, ids, dy))
    V, d = 270_000, 8192
    ids = torch.tensor([0, V - 1, 262_144, 262_145, V - 1], device="cuda")
    dy = torch.randint(-4, 5, (5, d), device="cuda").bfloat16()
    got = moe.embed_backward(ids, dy, V, out_dtype=BF16)
    assert torch.equal(got[V - 1], dy[1] + dy[4]) and torch.equal(got[262_145], dy[3]) and torch.equal(got[0], dy[0])
    assert got.count_nonzero() == sum(got[i].count_nonzero() for i in (0, V - 1, 262_144, 262_145))
    assert torch.equal(moe.embed(ids, got), got[ids])


def test_graphs_other_streams_and_no_tokens(moe):
    ids, dy = torch.randint(0, 50, (500,), device="cuda"), torch.randn(500, 40, device="cuda")
    want = moe.embed_backward(ids, dy, 50)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, rows = moe.embed_backward(ids, dy, 50), moe.embed(ids, dy[:50])
    graph.replay()
    assert torch.equal(got, want) and torch.equal(rows, dy[:50][ids])
    ids.copy_(torch.randint(0, 50, (500,), device="cuda"))
    graph.replay()
    assert torch.equal(got, moe.embed_backward(ids, dy, 50))
    side = torch.cuda.Stream()
    out = torch.zeros(50, 40, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    moe.embed_backward(ids, dy, 50, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, got) and out._version > 0
    none = ids[:0]
    assert moe.embed(none, dy).shape == (0, 40)
    assert moe.embed_backward(none, dy[:0], 50).eq(0).all()
    kept = out.clone()
    moe.embed_backward(none, dy[:0], 50, out=out, accumulate=True)
    assert torch.equal(out, kept)


def test_other_types_are_refused(moe):
    ids, dy = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, 8, device="cuda")
    for dt in (torch.float16, torch.float64):
        for call in (lambda: moe.embed_backward(ids, dy.to(dt), 5), lambda: moe.embed(ids, dy.to(dt)),
                     lambda: moe.embed(ids, dy, out_dtype=dt), lambda: moe.embed_backward(ids, dy, 5, out_dtype=dt),
                     lambda: moe.dropout(dy.to(dt), 0.1, 0), lambda: moe.dropout(dy, 0.1, 0, residual=dy.to(dt)),
                     lambda: moe.layer_norm(dy.to(dt)), lambda: moe.layer_norm(dy, h=dy.to(dt)),
                     lambda: moe.route_scores(dy.to(dt), 2)):
            with pytest.raises((ValueError, TypeError)):
                call()
    with pytest.raises((ValueError, TypeError)):
        moe.embed_backward(ids.to(torch.int16), dy, 5)


def test_more_than_a_warp_lists(moe):
    """Half of many tokens with one id, in small and in wide vocabularies (whole numbers: exact in any order), and all."""
    g = torch.Generator("cuda").manual_seed(12)
    for V in (40, 190_000):
        ids = torch.randint(0, V, (70_001,), generator=g, device="cuda")
        ids[torch.rand(70_001, generator=g, device="cuda") < 0.5] = 17
        dy = torch.randint(-4, 5, (70_001, 8), generator=g, device="cuda").float()
        for i in (ids, ids.int(), torch.full_like(ids, 17)):
            want = torch.zeros(V, 8, device="cuda").index_add_(0, i, dy)
            assert torch.equal(moe.embed_backward(i, dy, V), want)
            assert torch.equal(moe.embed_backward(i, dy, V, out=want.clone(), accumulate=True), 2 * want)


@pytest.mark.parametrize("d", [2048, 2052, 2050, 2051])
def test_additions_to_more_than_the_cache_holds(moe, d):
    g = torch.Generator("cuda").manual_seed(d)
    V, T = 20_000, 25_000
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    ids[:3000] = 5
    out = torch.randint(-4, 5, (V, d), generator=g, device="cuda").float()
    for dt in (F32, BF16):
        dy = torch.randint(-4, 5, (T, d), generator=g, device="cuda").to(dt)
        want = out.clone().index_add_(0, ids, dy.float())
        assert torch.equal(moe.embed_backward(ids, dy, V, out=out.clone(), accumulate=True), want)


@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_rows_off_the_widest_loads(moe, off):
    """Tables, rows and gradients that begin at any multiple of their elements."""
    g = torch.Generator("cuda").manual_seed(off)
    ids = torch.randint(0, 30, (200,), generator=g, device="cuda")
    for dt in (F32, BF16):
        flat = torch.randint(-4, 5, (off + 200 * 64,), generator=g, device="cuda").to(dt)
        dy, table = flat[off:].view(200, 64), flat[off:off + 30 * 64].view(30, 64)
        assert torch.equal(moe.embed(ids, table), table[ids])
        want = torch.zeros(30, 64, device="cuda").index_add_(0, ids, dy.float())
        assert torch.equal(moe.embed_backward(ids, dy, 30), want)
        out = torch.zeros(off + 30 * 64, device="cuda")[off:].view(30, 64)
        assert torch.equal(moe.embed_backward(ids, dy, 30, out=out), want)
        assert torch.equal(moe.embed_backward(ids, dy, 30, out=out, accumulate=True), 2 * want)


def test_elements_beyond_32_bits(moe):
    n = 2 ** 32 + 43
    x = torch.ones(n, dtype=BF16, device="cuda")
    assert moe.dropout(x, 0.5, 3, 4, out=x) is x
    for first, last in ((0, 64), (2 ** 31 - 32, 2 ** 31 + 32), (2 ** 32 - 32, n)):
        assert torch.equal(x[first:last].ne(0), stays(last, 0.5, 3, 4, first)), first


def test_two_streams_at_once(moe):
    g = torch.Generator("cuda").manual_seed(15)
    sets = [(torch.randint(0, 3000, (5000,), generator=g, device="cuda") // (i + 1), torch.randn(5000, 264 + i, generator=g, device="cuda"))
            for i in range(2)]

    def both(ids, dy):
        d = moe.embed_backward(ids, dy, 3000)
        return [d, moe.embed(ids, d), moe.dropout(dy, 0.3, 9, residual=dy)]
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
