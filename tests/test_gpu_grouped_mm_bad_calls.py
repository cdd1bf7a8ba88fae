"""What a grouped product whose offsets are bad, or whose wait ran out, leaves alone: everything.  The shapes
are ones whose reduction is split into slices (a second kernel joins them), and ones that are not."""
import pytest
import torch

pytestmark = pytest.mark.gpu

MODES = {"fwd": 0, "dgrad": 1, "wgrad": 2}
#         M,    K,    N,   E: split in every mode's own shape
SPLIT = {"fwd": (8, 8192, 256, 3), "dgrad": (70, 4104, 264, 3), "wgrad": (4099, 72, 136, 3)}
PLAIN = {"fwd": (8, 64, 72, 3), "dgrad": (70, 72, 64, 3), "wgrad": (90, 72, 136, 3)}


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_fp32_gb300 import moe as m
    return m


def operands(way, M, K, N, E):
    g = torch.Generator("cuda").manual_seed(M)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    return r(M, K), r(M, N) if way == "wgrad" else r(E, K, N) if way == "fwd" else r(E, N, K)


def call(moe, way, a, b, offs, **kw):
    offs = torch.tensor(offs, dtype=torch.int32, device="cuda")
    if way == "wgrad":
        return moe.grouped_mm_wgrad(a, b, offs, **kw)
    return moe.grouped_mm(a, b, offs, transpose_b=way == "dgrad", **kw)


@pytest.mark.parametrize("bad", ["falls inside", "starts below 0", "ends past the rows", "falls at the end"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("way", list(MODES))
def test_bad_offsets_leave_the_output(moe, way, split, dtype, bad):
    M, K, N, E = (SPLIT if split else PLAIN)[way]
    offs = {"falls inside": [0, M // 2 + 1, M // 2 - 1, M], "starts below 0": [-1, 1, 2, M],
            "ends past the rows": [0, 1, 2, M + 1], "falls at the end": [0, 2, M, M - 1]}[bad]
    a, b = operands(way, M, K, N, E)
    need = moe.grouped_mm_workspace_size(MODES[way], M, K, N, E)
    assert (need > 0) == split
    ws = torch.full((max(need, 16) // 4,), 5.0, device="cuda").view(torch.uint8)  # what an earlier call left there
    out = torch.full((E, K, N) if way == "wgrad" else (M, N), 3.0, dtype=dtype, device="cuda")
    for accumulate in ([False, True] if way == "wgrad" and dtype == torch.float32 else [False]):
        kw = {"accumulate": True} if accumulate else {}
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(moe, way, a, b, offs, out=out, workspace=ws, status=status, **kw)
        assert moe.get_device_error(status) == moe.STATUS_BAD_OFFSETS
        assert (out == 3).all(), f"{way}, accumulate={accumulate}"


@pytest.mark.parametrize("way", list(MODES))
def test_a_good_call_after_a_bad_one_in_the_same_workspace(moe, way):
    """The slices are joined by the call's own words, not by ones that an earlier call left in the workspace."""
    M, K, N, E = SPLIT[way]
    a, b = operands(way, M, K, N, E)
    good, bad = [0, M // 2, M // 2, M], [0, M // 2 + 1, M // 2 - 1, M]
    ws = torch.empty(moe.grouped_mm_workspace_size(MODES[way], M, K, N, E), dtype=torch.uint8, device="cuda")
    want = call(moe, way, a, b, good, out_dtype=torch.float32)
    out = torch.zeros_like(want)
    for offs in (good, bad, good, bad):
        out.fill_(3.0)
        call(moe, way, a, b, offs, out=out, workspace=ws)
        assert torch.equal(out, want) if offs is good else (out == 3).all()
