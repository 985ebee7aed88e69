"""The example that trains with the row operators runs and learns."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_distill_moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_moe.py")
    spec = importlib.util.spec_from_file_location("distill_moe", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, shares = example.main(40)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0]
    assert shares[-1] <= 1.0 and min(shares) >= 1.0 / example.EXPERTS
