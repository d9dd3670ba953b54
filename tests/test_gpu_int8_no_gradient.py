"""The 8-bit integer operators have no gradient, and none is lost without a word."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


@pytest.mark.parametrize("m", [1, 20, 100, 600])
def test_product_of_quantised_rows(swz, m):
    x = torch.randn((m, 64), device="cuda", requires_grad=True)
    w = torch.randn((8, 64), device="cuda", requires_grad=True)
    gain = torch.ones((), device="cuda", requires_grad=True)
    with torch.no_grad():
        kept, plain = swz.quantize_int8(w), swz.quantize_int8(x)
    q, s = swz.quantize_int8(x)
    assert torch.equal(q, plain[0]) and torch.equal(s.detach(), plain[1])
    y = swz.gemm_int8(q, s, *kept)
    assert torch.equal(y.detach(), swz.gemm_int8(*plain, *kept))
    with pytest.raises(RuntimeError, match="gemm_int8 has no gradient"):
        (y * gain).sum().backward()
    with pytest.raises(RuntimeError, match="quantize_int8 has no gradient"):
        (swz.quantize_int8(x)[1] * gain).sum().backward()
    with pytest.raises(RuntimeError, match="linear_int8 has no gradient"):
        (swz.linear_int8(x.detach(), *swz.quantize_int8(w)) * gain).sum().backward()


def test_nothing_asked_for(swz):
    """Without a gradient to lose the results are plain tensors."""
    x = torch.randn((4, 64), device="cuda", requires_grad=True)
    for get in (lambda: swz.quantize_int8(x.detach()), torch.no_grad()(lambda: swz.quantize_int8(x))):
        q, s = get()
        assert not s.requires_grad and not swz.gemm_int8(q, s, q, s).requires_grad
