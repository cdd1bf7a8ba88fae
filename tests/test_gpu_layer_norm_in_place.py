"""Layer norm over its input (y = x) and its gradient over the stream's (dx = dy), at widths whose rows begin inside an
aligned eight: a block then reads eights of which its neighbours are writing a part.  And the gradient's column sums over
many rows.

The results of a call in place are those of one that is not, bit for bit: the sums are the same, in the same order."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
D, F32, BF16 = torch.float64, torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_fp32_gb300 import moe as m
    m.load()
    return m


SHAPES = [(3, 2), (700, 33), (2000, 257), (4001, 1001), (1300, 2891), (3001, 2890), (40, 8203), (333, 9001), (5, 20001)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_over_the_stream(moe, T, d, dt):
    g = torch.Generator("cuda").manual_seed(T + d)
    x, h = torch.randn(T, d, generator=g, device="cuda").to(dt), torch.randn(T, d, generator=g, device="cuda").to(BF16)
    w = torch.randn(d, generator=g, device="cuda")
    want = moe.layer_norm(x, w, w, h=h, p=0.2, seed=4)
    for _ in range(3):
        mine = x.clone()
        y, n, stats = moe.layer_norm(mine, w, w, h=h, p=0.2, seed=4, y=mine)
        assert y is mine and torch.equal(mine, want[0]) and torch.equal(n, want[1]) and torch.equal(stats, want[2])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,d", SHAPES)
def test_gradient_over_the_streams(moe, T, d, dt):
    """Through the C call: the Python one returns new tensors."""
    g = torch.Generator("cuda").manual_seed(T + d)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dy, dn, w = randn(T, d).to(dt), randn(T, d).to(dt), randn(T, d).to(BF16), randn(d)
    stats = moe.layer_norm(x)[2]
    want = moe.layer_norm_backward(x, stats, dn, dy, w, w, True, 0.2, 4)
    lib = moe.load()
    need = lib.moe_layer_norm_backward_workspace_size(T, d)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    at = lambda t: ctypes.c_void_p(t.data_ptr())
    for _ in range(3):
        mine, dh = dy.clone(), torch.empty(T, d, dtype=BF16, device="cuda")
        dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        rc = lib.moe_layer_norm_backward(at(x), int(dt is F32), at(stats), at(dn), at(mine), at(w), T, d, 0.2, 4, 0, None,
                                         at(mine), at(dh), at(dw), at(db), at(ws), need, stream)
        assert rc == 0
        for a, name in ((mine, "x"), (dh, "h"), (dw, "weight"), (db, "bias")):
            assert torch.equal(a, want[name]), name


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,d", [(20000, 96), (16384, 1024), (16001, 2891), (8192, 4096), (4096, 16384), (3000, 65536)])
def test_column_sums_over_many_rows(moe, T, d, dt):
    """Values with a mean, so that the sums grow.  With C clusters of blocks (the workspace holds two rows of sums for
    each) a sum adds up to ceil(T / C) + 16 values one after another in a block (rows, and rows side by side), ceil(C / 16)
    and 16 more behind: as many u = 2^-24 of the sizes' sum at the most, and 4 u for a term's own roundings."""
    g = torch.Generator("cuda").manual_seed(T + d)
    x = torch.randn(T, d, generator=g, device="cuda", dtype=F32).add_(0.5).to(dt)
    dn = torch.randn(T, d, generator=g, device="cuda", dtype=BF16).add_(0.75)
    w = torch.ones(d, device="cuda")
    stats = moe.layer_norm(x)[2]
    got = moe.layer_norm_backward(x, stats, dn, None, w, w)
    sums = torch.zeros(4, d, dtype=D, device="cuda")
    for a in range(0, T, 1024):
        n = dn[a:a + 1024].to(D)
        s = stats[a:a + 1024].to(D)
        t = n * ((x[a:a + 1024].to(D) - s[:, :1]) * s[:, 1:])
        sums += torch.stack([t.sum(0), t.abs().sum(0), n.sum(0), n.abs().sum(0)])
    width = 8 * ((d + 7) // 8 + (1 if d % 8 else 0))
    C = moe.load().moe_layer_norm_backward_workspace_size(T, d) // (8 * width)
    off = (-(-T // C) + 16 + -(-C // 16) + 16 + 4) * 2.0 ** -24
    assert (got["weight"].to(D) - sums[0]).abs().le(off * sums[1]).all()
    assert (got["bias"].to(D) - sums[2]).abs().le(off * sums[3]).all()
