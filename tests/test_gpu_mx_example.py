"""The example that trains a layer through 4-bit products and serves it runs,
and its loss falls to the 4-bit weight's own error."""

import importlib.util
import os

import pytest
import torch

from conftest import REPO

pytestmark = pytest.mark.gpu


def test_example_trains_and_serves():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    spec = importlib.util.spec_from_file_location("microscaled_layers",
                                                  os.path.join(REPO, "examples", "microscaled_layers.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, w = example.train()
    # targets have mean square 1; 4-bit rounding of x and w leaves a few percent
    assert 0.7 < losses[0] < 1.4
    assert losses[-1] < 0.1 * losses[0], losses
    y, z = example.serve(w)
    assert y.shape == (1, w.shape[0]) and z.shape == (4, w.shape[1])
    assert y.isfinite().all() and z.isfinite().all()
