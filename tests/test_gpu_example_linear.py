"""The linear-layer operators together, as examples/train_linear_fp8.py runs
them: training in 8 bits with orthogonalised updates lowers the loss, and the
quantised network serves what it learnt, batch or single row."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location(
        "train_linear_fp8", os.path.join(ROOT, "examples", "train_linear_fp8.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_the_loss_and_serving_agrees(example):
    losses, weights, x, want = example.train(steps=40, tokens=777, width=320, hidden=500)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])
    y = example.serve(weights, x)
    served = (y.float() - want).square().mean().item()
    assert served < 0.6 * losses[0]
    # A row alone and in a batch are the same sums in another order: where their
    # last bits differ, a hidden value may round to another 8-bit value (2^-3 of
    # itself), and one of 500 carries less than 2^-2 of the row's largest result.
    one = example.serve(weights, x[5:6])
    scale = y[5].float().abs().max()
    assert (one.float() - y[5:6].float()).abs().max() <= 2.0 ** -5 * scale
