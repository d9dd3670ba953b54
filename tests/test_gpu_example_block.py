"""The operators of a pre-norm block together, as examples/train_block.py runs them:
the block's gradients against autograd of the formula in 64 bits, a few training
steps, and the block served from 8-bit integers.

Bounds, in the Frobenius norm: rounding to e4m3 is off by at most 2^-4 of an
operand, to 8-bit integers by half of a row's largest magnitude / 127 a value; the
errors of different roundings are independent, so n of them leave sqrt(n) times
one's share.  A gradient goes through eight 8-bit-float roundings at most: sqrt(8)
2^-4 = 0.18.  Served, a row of normal values has its largest below 5 times its root
mean square, so a rounding leaves 5 / 127 / sqrt(12) = 0.012 of an operand, and four
of them and the bf16 roundings (2^-8) 0.03."""
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
        "train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def formula(x, params):
    g, b, w1, w2 = params
    n = torch.nn.functional.layer_norm(x, x.shape[-1:], g, b)
    return x + torch.nn.functional.silu(n @ w1.t()) @ w2.t()


def rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("tokens,width,hidden", [(300, 320, 500), (64, 1000, 256)])
def test_gradients(example, tokens, width, hidden):
    g = torch.Generator(device="cuda").manual_seed(1)
    params = example.start(width, hidden, g)
    params[0] += 0.2 * torch.randn(width, generator=g, device="cuda")
    params[1] += 0.2 * torch.randn(width, generator=g, device="cuda")
    params = [p if p.dim() == 1 else p.bfloat16() for p in params]
    x = torch.randn((tokens, width), generator=g, device="cuda").bfloat16()
    dy = torch.randn((tokens, width), generator=g, device="cuda").bfloat16()
    ours = [t.clone().requires_grad_() for t in (x, *params)]
    exact = [t.double().requires_grad_() for t in (x, *params)]
    example.block(ours[0], ours[1:]).backward(dy)
    formula(exact[0], exact[1:]).backward(dy.double())
    for a, b in zip(ours, exact):
        assert a.grad.dtype == a.dtype
        assert rel(a.grad, b.grad) <= 0.18, (a.shape, rel(a.grad, b.grad))


def test_training_and_serving_run(example):
    log, weights, x = example.train(steps=4, tokens=200, width=320, hidden=500, max_norm=0.5)
    assert len(log) == 4 and all(v == v and n == n and n > 0 for v, n in log)
    assert all(torch.isfinite(w).all() for w in weights)
    kept = example.keep(weights)
    for rows in (x, x[:40], x[:13], x[:1]):
        got = example.serve(kept, rows).double() - rows.double()
        want = formula(rows.double(), [w.double() for w in weights]) - rows.double()
        # x + (...) is rounded to bf16: 2^-9 of its values, here of about x
        assert rel(got, want) <= 0.03 + 2.0 ** -8 * (rows.double().norm() / want.norm()).item()
