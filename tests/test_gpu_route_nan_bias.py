"""Routing by scores with NaN in the bias, in the logits and in both, against the definition in 64 bits: a c that is NaN
ranks below every number, NaNs by ascending id; so a group's q best are its numbers first, a group whose sum is NaN ranks
below those whose sum is a number, and the experts of a dropped group are chosen by no one.  A NaN in the bias reaches its
own expert's c alone; the scores do not depend on the bias, so the weights are held to the tolerance of the other tests
of this operator (2^-18 of the value, and 2^-126).  Choices are whole numbers: equal."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
D, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_fp32_gb300 import moe as m
    m.load()
    return m


def best(r, k):
    """Places of the k best of a list: numbers by size, then NaN, equal ones by place."""
    return sorted(range(len(r)), key=lambda e: (r[e] != r[e], -r[e] if r[e] == r[e] else 0.0, e))[:k]


def scores(row, scoring):
    if scoring == "sigmoid":
        return [NAN if v != v else 0.0 if v < -700 else 1 / (1 + math.exp(-v)) for v in row]
    top = max(row) if all(v == v for v in row) else NAN
    if top != top or top == INF:
        return [NAN] * len(row)
    e = [math.exp(v - top) if top > -INF else 0.0 for v in row]
    return [v / sum(e) if top > -INF else 0.0 for v in e]


def choice(row, bias, k, scoring, groups, kept):
    c = [s + b for s, b in zip(scores(row, scoring), bias)]
    size = len(c) // groups
    q = min(size, max(1, k // kept))
    sums = [0.0] * groups
    for g in range(groups):
        for i in best(c[g * size:(g + 1) * size], q):
            sums[g] += c[g * size + i]
    inside = sorted(g * size + i for g in best(sums, kept) for i in range(size))
    return [inside[i] for i in best([c[e] for e in inside], k)]


def weights(rows, idx, scoring):
    """Renormalised, of rows of numbers."""
    s = torch.tensor([scores(r, scoring) for r in rows], dtype=D)
    w = s.gather(1, idx)
    return w / w.sum(1, keepdim=True)


# Both lane layouts (up to 64 experts, and more), groups in fewer and more than eight lanes, more slots than numbers.
SHAPES = [(24, 3, 4, 2), (64, 8, 8, 4), (64, 6, 1, 1), (100, 5, 5, 2), (160, 6, 8, 4), (256, 8, 8, 4), (256, 8, 1, 1),
          (256, 4, 32, 3), (20, 8, 2, 2)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept", SHAPES)
def test_nan_in_the_bias(moe, E, k, groups, kept, scoring):
    g = torch.Generator("cuda").manual_seed(E + k)
    size = E // groups
    for dt in (F32, BF16):
        logits = torch.randn(37, E, generator=g, device="cuda").to(dt)
        rows = logits.to(D).tolist()
        for gone in ([0], [E - 1], [E // 2, E // 2 + 1], list(range(0, E, 2)), list(range(size)), list(range(E - k + 1)),
                     list(range(E))):
            bias = torch.randn(E, generator=g, device="cuda") * 0.1
            bias[gone] = NAN
            want = torch.tensor([choice(r, bias.to(D).tolist(), k, scoring, groups, kept) for r in rows])
            for scores_too in (False, True):
                idx, w, s = moe.route_scores(logits, k, scoring, bias, groups, kept, want_scores=scores_too)
                assert torch.equal(idx.cpu().long(), want), gone
                rw = weights(rows, want, scoring)
                assert (w.cpu().to(D) - rw).abs().le(2.0 ** -18 * rw + 2.0 ** -126).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept", SHAPES)
def test_nan_and_infinities_in_some_rows(moe, E, k, groups, kept, scoring):
    """Rows with and without them next to one another, with a bias of numbers, with NaN and with infinities."""
    g = torch.Generator("cuda").manual_seed(E + k + 1)
    logits = torch.randn(41, E, generator=g, device="cuda")
    logits[1, 3], logits[5, ::2], logits[9] = NAN, NAN, NAN
    logits[13, 5], logits[17, 1], logits[17, 7] = INF, INF, -INF
    logits[21], logits[25, 4:], logits[29, 2], logits[29, 6] = -INF, -INF, INF, NAN
    rows = logits.to(D).tolist()
    for values in ([], [(2, NAN)], [(0, NAN), (E - 1, -INF)], [(1, INF)], [(1, INF), (4, -INF), (6, NAN)]):
        bias = torch.randn(E, generator=g, device="cuda") * 0.1
        for e, v in values:
            bias[e] = v
        want = torch.tensor([choice(r, bias.to(D).tolist(), k, scoring, groups, kept) for r in rows])
        got = moe.route_scores(logits, k, scoring, bias, groups, kept)[0]
        assert torch.equal(got.cpu().long(), want), values
