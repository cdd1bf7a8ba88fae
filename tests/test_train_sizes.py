"""Sizes that do not fit the C calls' 32-bit integers are refused by name, not passed on modulo 2^32 (a call on
2^32 + 5 rows would work on 5 and return the rest as it was allocated).  Meta tensors: no memory, no GPU."""
import pytest
import torch

from mixture_experts_grouped_fp32_gb300 import moe

HUGE = 2 ** 32 + 5
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def t(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


CALLS = {
    "grouped_mm rows": lambda: moe.grouped_mm(t(HUGE, 8), t(2, 8, 8), t(3, dtype=I32)),
    "grouped_mm columns": lambda: moe.grouped_mm(t(4, 8), t(2, 8, HUGE + 3), t(3, dtype=I32)),
    "grouped_mm transposed": lambda: moe.grouped_mm(t(4, 8), t(2, HUGE + 3, 8), t(3, dtype=I32), transpose_b=True),
    "grouped_mm experts": lambda: moe.grouped_mm(t(4, 8), t(HUGE, 8, 8), t(HUGE + 1, dtype=I32)),
    "wgrad rows": lambda: moe.grouped_mm_wgrad(t(HUGE, 8), t(HUGE, 8), t(3, dtype=I32)),
    "wgrad columns": lambda: moe.grouped_mm_wgrad(t(4, 8), t(4, HUGE + 3), t(3, dtype=I32)),
    "wgrad experts": lambda: moe.grouped_mm_wgrad(t(4, 8), t(4, 8), t(HUGE + 1, dtype=I32)),
    "swiglu rows": lambda: moe.swiglu(t(HUGE, 16)),
    "swiglu columns": lambda: moe.swiglu(t(1, 2 * HUGE + 6)),
    "swiglu_backward rows": lambda: moe.swiglu_backward(t(HUGE, 16), t(HUGE, 8)),
    "block_norm rows": lambda: moe.block_norm(t(HUGE, 8), t(8, dtype=F32)),
    "block_norm columns": lambda: moe.block_norm(t(1, HUGE + 3), t(HUGE + 3, dtype=F32)),
    "block_norm_backward rows": lambda: moe.block_norm_backward(t(HUGE, 8), t(HUGE, 8)),
    "workspace size": lambda: moe.grouped_mm_workspace_size(0, HUGE, 8192, 64, 4),
    "adamw step": lambda: moe.adamw_step([t(8)], [t(8)], [t(8, dtype=F32)], [t(8, dtype=F32)], lr=1e-3, step=2 ** 32 + 1),
}


@pytest.mark.parametrize("call", list(CALLS))
def test_refused_by_size(call):
    with pytest.raises(ValueError, match=r"2\^31"):
        CALLS[call]()
