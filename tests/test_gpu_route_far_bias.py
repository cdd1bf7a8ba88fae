"""Groups whose biases are of very different sizes, beyond 1e30 too, against the definition in 64 bits (in which sums of
up to eight fp32 numbers do not overflow): the choice is whole numbers, so equal."""
import pytest
import torch

from test_gpu_route_nan_bias import choice

pytestmark = pytest.mark.gpu
LOW = torch.finfo(torch.float32).min


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_fp32_gb300 import moe as m
    m.load()
    return m


# Sums of one, two and more experts of a group; both lane layouts.
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept", [(10, 4, 5, 2), (24, 3, 8, 4), (64, 8, 8, 2), (256, 8, 8, 1), (160, 6, 8, 3),
                                             (256, 8, 32, 3), (40, 8, 5, 2)])
def test_sums_of_far_biases(moe, E, k, groups, kept, scoring):
    g = torch.Generator("cuda").manual_seed(E + groups)
    for round_ in range(6):
        logits = torch.randn(20, E, generator=g, device="cuda")
        noise = torch.randn(E, generator=g, device="cuda")
        power = torch.rand(E, generator=g, device="cuda") * 9 + 29.3  # up to 2e38
        lowest = torch.where(torch.rand(E, generator=g, device="cuda") < 0.7, LOW, 0.1 * noise)
        for bias in (noise * 1e30, noise.sign() * 10 ** power, -(10 ** power), noise.sign() * 10 ** (power - 30), lowest,
                     -noise.abs() * 1e31 - 1e30):
            bias = bias.clamp(LOW, -LOW)
            got = moe.route_scores(logits, k, scoring, bias, groups, kept)[0]
            want = [choice(r, bias.double().tolist(), k, scoring, groups, kept) for r in logits.double().tolist()]
            assert torch.equal(got.cpu().long(), torch.tensor(want))


def test_a_group_of_large_and_of_small_ones(moe):
    """Two kept groups of two experts: the second group's sum is -1.24e30, the third's -1.53e30."""
    bias = torch.tensor([-1.15e30, 1.59e30, -1.24e30, -1e4, -1.73e30, 1.96e29, LOW, LOW, LOW, 0.0], device="cuda")
    logits = torch.zeros(3, 10, device="cuda")
    for scoring in ("softmax", "sigmoid"):
        idx = moe.route_scores(logits, 4, scoring, bias, 5, 2)[0]
        assert idx.tolist() == [[1, 3, 0, 2]] * 3
