"""The training example refuses options that nothing would read (without a GPU: before any tensor is made)."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("options", [dict(groups=4, kept=2), dict(bias_rate=1e-3), dict(balance=0.01)])
def test_router_options_need_scoring(options):
    spec = importlib.util.spec_from_file_location("train_moe", os.path.join(ROOT, "examples", "train_moe.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    with pytest.raises(ValueError, match="give scoring"):
        example.train(steps=1, **options)
