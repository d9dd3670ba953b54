"""The gradient of rows far from zero next to how little they vary, where what is read
beyond a row's end would leave fp32's range as an xhat.

A constant row c with the mean c and rstd r has xhat = 0: dx = r (g - mean(g)), dw = 0.
Bounds as in test_gpu_layer_norm.py with mean and rstd given: the sum of g is off by c u
sum|g|, c = 100 + n / 2048, and three roundings follow."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 7, 40, 64, 250, 264, 500, 520, 700, 1999, 4096, 4160, 6001, 9000, 10241, 17000])
def test_constant_rows(swz, dtype, n):
    m = 21
    value, r = 2.0 ** 110, 2.0 ** 20  # their product is beyond 2^128
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.full((m, n), value, device="cuda").to(dtype)
    x[1::3] = torch.randn((m // 3, n), generator=g, device="cuda").to(dtype)  # ordinary rows between them
    mean, rstd = torch.full((m,), value, device="cuda"), torch.full((m,), r, device="cuda")
    mean[1::3], rstd[1::3] = 0.0, 1.0
    dy = torch.randn((m, n), generator=g, device="cuda").to(dtype)
    w = (1 + 0.2 * torch.randn(n, generator=g, device="cuda"))
    for weight in (w, w.to(dtype), None):
        wd = torch.ones(n, device="cuda", dtype=torch.float64) if weight is None else weight.double()
        dx, dw, db = swz.layer_norm_backward(dy, x, weight, mean, rstd)
        gd = dy.double() * wd
        xhat = (x.double() - mean.double().unsqueeze(1)) * rstd.double().unsqueeze(1)
        m1, m2 = gd.mean(1, keepdim=True), (gd * xhat).mean(1, keepdim=True)
        want = rstd.double().unsqueeze(1) * (gd - m1 - xhat * m2)
        c = 100 + n / 2048
        bound = rstd.double().unsqueeze(1) * U * (
            c * gd.abs().mean(1, keepdim=True) + xhat.abs() * (c + 3) * (gd * xhat).abs().mean(1, keepdim=True)
            + 8 * (gd.abs() + m1.abs() + (xhat * m2).abs()))
        half = torch.finfo(dtype).eps / 2
        assert bool(((dx.double() - want).abs() <= bound + (want.abs() + bound) * half).all())
        terms = (dy.double() * xhat).abs().sum(0)
        assert bool(((dw.double() - (dy.double() * xhat).sum(0)).abs() <= (m + 130) * U * terms).all())
        assert bool(((db.double() - dy.double().sum(0)).abs() <= (m + 130) * U * dy.double().abs().sum(0)).all())
