"""Layer norm of rows without any deviation, whose sums are not exact in fp32.

With u = 2^-24 and a row of c, the first sum over the row gives a mean m that is off by d = c - m, below 64 u |c| (and c - m
is exact, the two being within a factor of two).  The deviations' own sum is d times the row's length to within 64 u of
it, so m plus its mean is c to within 66 u d < 2^-11 u |c|, and rounds to c itself: the stats hold c, and y - c = 0, so n
is the bias.  The variance is a difference of terms of d^2, each off by at most 70 u of it: below 210 u d^2, at 1000.1
2^-32.3, which is 2^-15.7 of eps = 1e-5; half of that in 1 / std, and a few u for the root: 2^-16."""
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_fp32_gb300 import moe as m
    m.load()
    return m


@pytest.mark.parametrize("d", [1, 3, 33, 64, 96, 100, 255, 256, 264, 1000, 2891, 4096, 6091, 7168, 8200, 16384, 20001, 65536])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_constant_rows(moe, d, dt):
    values = torch.tensor([0.1, 1000.1, -7.3, 1 / 3, 999.7, 1e-3, -0.7], device="cuda").to(dt)
    x = values[:, None].expand(-1, d).contiguous().repeat(9, 1)
    c = values.repeat(9).float()
    b = torch.randn(d, device="cuda")
    for bias in (None, b):
        y, n, stats = moe.layer_norm(x, b + 1, bias)
        assert torch.equal(stats[:, 0], c)
        assert (stats[:, 1] * EPS ** 0.5 - 1).abs().max() <= 2.0 ** -16
        assert torch.equal(n, (torch.zeros(d, device="cuda") if bias is None else bias).bfloat16().expand_as(n))
    h = torch.full_like(x, 0.25, dtype=BF16)
    y, n, stats = moe.layer_norm(x, h=h)
    assert torch.equal(stats[:, 0], y[:, 0].float()) and n.eq(0).all()


def test_means_are_those_of_64_bits(moe):
    """The second sum corrects the first: what is left is the rounding of the mean itself (u of it), 64 u of what the
    first sum was off by (2^-18 of mean |y|, so 2^-36), and the corrections' own 64 u of the mean deviation."""
    g = torch.Generator("cuda").manual_seed(1)
    for d in (96, 255, 4096, 7168, 20001):
        x = torch.randn(60, d, generator=g, device="cuda") + 1000.0
        mean = moe.layer_norm(x)[2][:, 0].double()
        want = x.double().mean(1)
        off = 2.0 ** -24 * want.abs() + 2.0 ** -36 * x.double().abs().mean(1) + 2.0 ** -18 * (x.double() - want[:, None]).abs().mean(1)
        assert (mean - want).abs().le(off * 1.01).all(), d
