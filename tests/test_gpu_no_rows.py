"""Matrices without rows, in whatever strides torch gives them (their columns are nowhere):
accepted by the operators of and around linear layers, with results that have no rows."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


@pytest.mark.parametrize("strides", [(128, 1), (1, 7), (0, 128), (5, 3)])
def test_no_rows(swz, strides):
    def none(dtype, n=128):
        return torch.empty_strided((0, n), strides, dtype=dtype, device="cuda")
    w = torch.randn((64, 128), device="cuda").bfloat16()
    x = none(torch.bfloat16)
    q, s = swz.quantize_fp8(x)
    assert q.shape == (0, 128) and s.shape == (1, 0)
    qw, sw = swz.quantize_fp8(w, "square")
    assert swz.gemm_fp8(q, s, qw, sw).shape == (0, 64)
    assert swz.gemm_fp8(none(torch.float8_e4m3fn), s, qw, sw).shape == (0, 64)
    assert swz.linear_fp8(x, qw, sw).shape == (0, 64)
    q, s = swz.quantize_int8(x)
    assert q.shape == (0, 128) and s.shape == (0,)
    qw, sw = swz.quantize_int8(w)
    assert swz.gemm_int8(q, s, qw, sw).shape == (0, 64)
    assert swz.gemm_int8(none(torch.int8), s, qw, sw, out=none(torch.float32, 64)).shape == (0, 64)
    assert swz.linear_int8(x, qw, sw).shape == (0, 64)
    y, mean, rstd = swz.layer_norm_forward(x)
    assert y.shape == (0, 128) and mean.shape == rstd.shape == (0,)
    dx, dw, db = swz.layer_norm_backward(none(torch.bfloat16), x, None, mean, rstd)
    assert dx.shape == (0, 128) and not dw.any() and not db.any()
    torch.cuda.synchronize()
