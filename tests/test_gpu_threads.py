"""The first calls of a process, made by several threads at once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys, threading
sys.path.insert(0, {root!r})
import torch
from mixture_experts_grouped_fp32_gb300 import moe
moe.load()
moe._fast = moe._fast if {fast} else None
a = torch.ones(64, 64, device="cuda", dtype=torch.bfloat16)
b = torch.ones(4, 64, 64, device="cuda", dtype=torch.bfloat16)
offs = torch.tensor([0, 16, 32, 48, 64], device="cuda", dtype=torch.int32)
torch.cuda.synchronize()
sys.setswitchinterval(1e-6)
gate, wrong = threading.Barrier(16), []

def call(i):
    s = torch.cuda.Stream()
    gate.wait()
    try:
        with torch.cuda.stream(s):
            out = moe.grouped_mm(a, b, offs, transpose_b=i % 2 == 1) if i % 3 else moe.grouped_mm_wgrad(a, a, offs)
            s.synchronize()
        if not (out == (64 if i % 3 else 16)).all():
            wrong.append("values")
    except Exception as e:
        wrong.append(repr(e))

threads = [threading.Thread(target=call, args=(i,)) for i in range(16)]
[t.start() for t in threads]
[t.join() for t in threads]
print(wrong)
sys.exit(bool(wrong))
"""


@pytest.mark.parametrize("fast", [True, False])
def test_first_calls_of_several_threads(fast):
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT, fast=fast)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
