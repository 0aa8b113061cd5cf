"""The point transformer example: tokens from FPS and kNN, training steps
through layer norm, rotary positions and attention, and a single query."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "point_transformer.py")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_point_transformer_learns_and_serves(dtype):
    spec = importlib.util.spec_from_file_location("point_transformer", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, model, last = ex.train(100, dtype=dtype)
    # the axes are uniform in [0.25, 1.25): guessing their mean costs 1 / 12
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) / 5 < 0.5 / 12 < losses[0]
    out = ex.serve(model, *last)
    assert out.shape == (32, 1, 96) and torch.isfinite(out).all()
