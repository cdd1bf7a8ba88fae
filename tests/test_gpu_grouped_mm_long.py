"""Grouped products over long reductions, against 64 bits.

Tolerances: the products of bf16 values are exact in fp32.  Within a chunk of 64-row (or 64-column) blocks each of four
additions a block truncates, by 2^-23 of a partial sum at most; the chunks' sums are added rounded to nearest,
2^-24 each; a bf16 output is rounded once more, by at most 2^-8 of its value.  A chunk is 64 blocks for a bf16
output of more than 262144 rows, all of them for one of fewer."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, D = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_fp32_gb300 import moe as m
    yield m
    torch.cuda.empty_cache()


def wgrad64(a, g, lo, hi, step=1 << 22):
    """Gradient of one segment in 64 bits, and the sum of its terms' magnitudes."""
    ref = torch.zeros(a.shape[1], g.shape[1], dtype=D, device="cuda")
    mag = torch.zeros_like(ref)
    for r in range(lo, hi, step):
        x, y = a[r:min(hi, r + step)].to(D), g[r:min(hi, r + step)].to(D)
        ref += x.T @ y
        mag += x.abs().T @ y.abs()
    return ref, mag


def check_bf16(got, ref, mag, rows, chunk_rows, what):
    chunks = -(-rows // chunk_rows)
    sums = min(rows, chunk_rows) / 16 * 2.0 ** -23 + chunks * 2.0 ** -24
    off = (got.to(D) - ref).abs()
    bound = sums * mag + 2.0 ** -8 * ref.abs() + 1e-30
    assert (off <= bound).all(), f"{what}: worst {float((off / bound).max())} of the bound"


@pytest.mark.parametrize("rows", [262144 - 3000, 262144 + 40, 300000])
def test_bf16_gradients_of_long_segments(moe, rows):
    """Positive terms, whose truncations all go one way; segments of all lengths beside the long one."""
    counts = [0, 5, rows - 2600, 700, 0, 1, 64, 1830]
    M, K, N = sum(counts), 264, 520
    offs = np.concatenate([[0], np.cumsum(counts)])
    gen = torch.Generator("cuda").manual_seed(rows)
    a = (torch.rand(M, K, generator=gen, device="cuda") + 0.5).to(BF16)
    g = (torch.rand(M, N, generator=gen, device="cuda") + 0.5).to(BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # (Without a workspace, so that the reduction is not split.)
    out = torch.full((len(counts), K, N), 7.0, dtype=BF16, device="cuda")
    L = moe.load()
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    assert L.moe_grouped_mm_wgrad(a.data_ptr(), g.data_ptr(), o.data_ptr(), M, K, N, len(counts), out.data_ptr(), 0, 0, None,
                                  0, status.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert moe.get_device_error(status) == 0
    for e, n in enumerate(counts):
        ref, mag = wgrad64(a, g, int(offs[e]), int(offs[e + 1]))
        check_bf16(out[e], ref, mag, n, 4096 if M > 262144 else 262144, f"segment of {n} rows")


def test_bf16_gradient_of_a_segment_of_seventy_million_rows(moe):
    long = (1 << 26) + (1 << 22)
    counts = [1000] * 40 + [long] + [1000] * 59  # 100 tiles: more than there are SM pairs, so never split
    M = sum(counts)
    assert moe.grouped_mm_workspace_size(2, M, 8, 8, len(counts)) == 0
    gen = torch.Generator("cuda").manual_seed(1)
    a, g = (torch.rand(M, 8, generator=gen, device="cuda").add_(0.5).to(BF16) for _ in range(2))
    offs = np.concatenate([[0], np.cumsum(counts)])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = moe.grouped_mm_wgrad(a, g, torch.tensor(offs, dtype=torch.int32, device="cuda"), out_dtype=BF16, status=status)
    assert moe.get_device_error(status) == 0
    for e, n in enumerate(counts):
        check_bf16(out[e], *wgrad64(a, g, int(offs[e]), int(offs[e + 1])), n, 4096, f"segment {e} of {n} rows")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_of_a_segment_that_takes_seconds(moe, dtype):
    """No wait inside the kernel runs out while one segment is worked on, however long it is."""
    counts = [1000] * 40 + [750_000_005] + [1000] * 59
    M = sum(counts)
    a, g = (torch.empty(M, 8, dtype=BF16, device="cuda") for _ in range(2))
    gen = torch.Generator("cuda").manual_seed(2)
    for t in (a, g):
        t.uniform_(0.5, 1.5, generator=gen)
    offs = np.concatenate([[0], np.cumsum(counts)])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out = moe.grouped_mm_wgrad(a, g, torch.tensor(offs, dtype=torch.int32, device="cuda"), out_dtype=dtype, status=status)
    end.record()
    assert moe.get_device_error(status) == 0
    print(f"{start.elapsed_time(end):.0f} ms")
    for e in (0, 39, 40, 41, 76, 99):
        n = counts[e]
        ref, mag = wgrad64(a, g, int(offs[e]), int(offs[e + 1]))
        if dtype == BF16:
            check_bf16(out[e], ref, mag, n, 4096, f"segment {e}")
        else:  # chunks of 512 rows: 32 truncations each, then the chunks' sums
            assert ((out[e].to(D) - ref).abs() <= (32 * 2.0 ** -23 + -(-n // 512) * 2.0 ** -24) * mag).all(), e


MOST = 2 ** 31 - 1025  # rows that the calls accept


@pytest.mark.parametrize("way", ["fwd", "dgrad"])
def test_as_many_rows_as_the_calls_accept(moe, way):
    """One segment of (nearly) all rows: its tile counts and positions pass 2^31 in sums."""
    gen = torch.Generator("cuda").manual_seed(3)
    a = torch.empty(MOST, 8, dtype=BF16, device="cuda").uniform_(-1, 1, generator=gen)
    b = torch.empty(2, 8, 8, dtype=BF16, device="cuda").uniform_(-1, 1, generator=gen)
    offs = torch.tensor([0, 3, MOST], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = moe.grouped_mm(a, b, offs, transpose_b=way == "dgrad", status=status)
    assert moe.get_device_error(status) == 0
    for lo in (0, 1 << 20, 1 << 30, 2139127680 - 500, MOST - 2000):
        x = a[lo:lo + 2000].to(D)
        w = (b if way == "fwd" else b.transpose(1, 2)).to(D)
        e = torch.ones(2000, dtype=torch.long, device="cuda")
        if lo == 0:
            e[:3] = 0
        ref, mag = torch.einsum("rk,rkn->rn", x, w[e]), torch.einsum("rk,rkn->rn", x.abs(), w[e].abs())
        assert ((out[lo:lo + 2000].to(D) - ref).abs() <= 2.0 ** -8 * ref.abs() + 8 * 2.0 ** -23 * mag).all(), lo


def test_gradient_of_as_many_rows_as_the_calls_accept(moe):
    gen = torch.Generator("cuda").manual_seed(4)
    a, g = (torch.empty(MOST, 8, dtype=BF16, device="cuda").uniform_(0.5, 1.5, generator=gen) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = moe.grouped_mm_wgrad(a, g, torch.tensor([0, MOST], dtype=torch.int32, device="cuda"), status=status)
    assert moe.get_device_error(status) == 0
    ref, mag = wgrad64(a, g, 0, MOST)
    slices = 16  # of the reduction: their workspace is that many gradients and more
    assert moe.grouped_mm_workspace_size(2, MOST, 8, 8, 1) > slices * 8 * 8 * 4
    assert ((out[0].to(D) - ref).abs() <= (32 * 2.0 ** -23 + (MOST // 512 // slices + 1 + slices) * 2.0 ** -24) * mag).all()


# fp32 outputs: chunks of 512 of the reduction.  Elementwise as above.  By the 2-norm, for terms of random sign: a
# chunk's partial sums grow as the root of the 32 additions' number, each loses 2^-23 at most, and the chunks' losses are
# independent: (2/3) 32^1.5 sqrt(16 / 512) 2^-23 = 21.4 * 2^-23 of the sum's norm, and 2^-24 for each chunk's addition.  Unbroken,
# n additions would lose (2/3) n of 2^-23: 341 for 8192 terms, about a third of that on average.
def check_fp32(got, ref, mag, n, what):
    chunks = -(-n // 512)
    off = (got.to(D) - ref).abs()
    assert (off <= (min(n, 512) / 16 * 2.0 ** -23 + chunks * 2.0 ** -24) * mag + 1e-30).all(), what
    rel = float(torch.linalg.norm(off) / torch.linalg.norm(ref))
    assert rel <= 21.4 * 2.0 ** -23 + chunks * 2.0 ** -24, f"{what}: off by {rel:.2e} in the 2-norm"


def unsplit(moe, way, a, b, offs, shape):
    """The C call without a workspace: the reduction is not split into slices."""
    out = torch.full(shape, 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    E, s = offs.numel() - 1, torch.cuda.current_stream().cuda_stream
    L = moe.load()
    if way == "wgrad":
        rc = L.moe_grouped_mm_wgrad(a.data_ptr(), b.data_ptr(), offs.data_ptr(), a.shape[0], a.shape[1], b.shape[1], E,
                                    out.data_ptr(), 1, 0, None, 0, status.data_ptr(), s)
    else:
        rc = L.moe_grouped_mm(a.data_ptr(), b.data_ptr(), offs.data_ptr(), a.shape[0], a.shape[1], shape[1], E,
                              int(way == "dgrad"), out.data_ptr(), 1, None, 0, status.data_ptr(), s)
    assert rc == 0 and moe.get_device_error(status) == 0
    return out


@pytest.mark.parametrize("way", ["fwd", "dgrad"])
@pytest.mark.parametrize("K", [512, 520, 1024, 1032, 1544, 2888, 8192])  # 1, 2, 2, 3, 4, 6 and 16 chunks
@pytest.mark.parametrize("counts,N", [([3], 264), ([700, 0, 1, 260, 33, 2000], 1544)])  # 2 items, and 2 for each SM pair
def test_fp32_products_in_chunks(moe, way, K, counts, N):
    gen = torch.Generator("cuda").manual_seed(K)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)
    offs = np.concatenate([[0], np.cumsum(counts)])
    a, b = r(sum(counts), K), r(len(counts), K, N) if way == "fwd" else r(len(counts), N, K)
    out = unsplit(moe, way, a, b, torch.tensor(offs, dtype=torch.int32, device="cuda"), (sum(counts), N))
    for e, n in enumerate(counts):
        if n:
            x, w = a[offs[e]:offs[e + 1]].to(D), (b[e] if way == "fwd" else b[e].T).to(D)
            check_fp32(out[offs[e]:offs[e + 1]], x @ w, x.abs() @ w.abs(), K, f"{way} of {n} rows over {K}")


@pytest.mark.parametrize("counts,K,N", [([8192, 0, 520, 1033], 264, 328), ([100, 513, 3000] * 12, 264, 520)])
def test_fp32_gradients_in_chunks(moe, counts, K, N):
    gen = torch.Generator("cuda").manual_seed(K)
    offs = np.concatenate([[0], np.cumsum(counts)])
    a, g = (torch.randn(sum(counts), w, generator=gen, device="cuda").to(BF16) for w in (K, N))
    out = unsplit(moe, "wgrad", a, g, torch.tensor(offs, dtype=torch.int32, device="cuda"), (len(counts), K, N))
    for e, n in enumerate(counts):
        if n:
            check_fp32(out[e], *wgrad64(a, g, int(offs[e]), int(offs[e + 1])), n, f"gradient of {n} rows")
        else:
            assert (out[e] == 0).all()
