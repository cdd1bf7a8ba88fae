"""A wait inside the grouped products is made to run out (MOE_INJECT_STALL=1: the host arms the first stage of one SM
pair for 16 bytes that never arrive; nothing faults).  The kernel must give up after its limit of 1 s, report
MOE_STATUS_WAIT_TIMEOUT, free its tensor memory and return; where the reduction is split the output must be as it was; and
the next call must be right."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, D = torch.bfloat16, torch.float32, torch.float64

#         M,    K,    N,   E, type, split
CASES = {
    "fwd bf16": (600, 136, 264, 3, BF16, False),
    "fwd fp32 in chunks": (6000, 1032, 1544, 3, F32, False),
    "fwd split": (8, 8192, 256, 3, F32, True),
    "dgrad fp32": (600, 136, 264, 3, F32, False),
    "dgrad split bf16": (70, 4104, 264, 3, BF16, True),
    "wgrad bf16": (600, 264, 520, 3, BF16, False),
    "wgrad tail first": (21, 264, 520, 3, F32, False),  # each segment is one block, with rows to be zeroed
    "wgrad split": (4099, 72, 136, 3, F32, True),
}


@pytest.mark.parametrize("case", list(CASES))
def test_an_expired_wait_is_reported_and_the_next_call_is_right(monkeypatch, case):
    from mixture_experts_grouped_fp32_gb300 import moe
    way = case.split()[0]
    M, K, N, E, dtype, split = CASES[case]
    assert (moe.grouped_mm_workspace_size({"fwd": 0, "dgrad": 1, "wgrad": 2}[way], M, K, N, E) > 0) == split
    gen = torch.Generator("cuda").manual_seed(M)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)
    a, b = r(M, K), r(M, N) if way == "wgrad" else r(E, K, N) if way == "fwd" else r(E, N, K)
    host = [M * e // E for e in range(E + 1)]
    offs = torch.tensor(host, dtype=torch.int32, device="cuda")
    out = torch.full((E, K, N) if way == "wgrad" else (M, N), 3.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        if way == "wgrad":
            moe.grouped_mm_wgrad(a, b, offs, out=out, status=status)
        else:
            moe.grouped_mm(a, b, offs, transpose_b=way == "dgrad", out=out, status=status)
        torch.cuda.synchronize()

    monkeypatch.setenv("MOE_INJECT_STALL", "1")
    start = time.time()
    call()
    assert 0.5 < time.time() - start < 20
    assert moe.get_device_error(status) == moe.STATUS_WAIT_TIMEOUT
    if split:
        assert (out == 3).all()

    monkeypatch.delenv("MOE_INJECT_STALL")
    status.zero_()
    call()
    assert moe.get_device_error(status) == 0
    for e, (lo, hi) in enumerate(zip(host[:-1], host[1:])):
        x = a[lo:hi].to(D)
        if way == "wgrad":
            w, got = b[lo:hi].to(D), out[e]
            x = x.T
        else:
            w, got = (b[e] if way == "fwd" else b[e].T).to(D), out[lo:hi]
        n = hi - lo if way == "wgrad" else K
        ref, mag = x @ w, x.abs() @ w.abs()
        bound = n * 2.0 ** -23 * mag + (2.0 ** -8 * ref.abs() if dtype == BF16 else 0) + 1e-30
        assert ((got.to(D) - ref).abs() <= bound).all(), e
