"""fp8_linear on the inputs a layer meets: any leading dimensions, any layout,
each type, nothing at all.  What a layout gives is what its contiguous copy
gives, bit for bit; each type against 64-bit sums of the 8-bit values, with the
tolerances of test_gpu_fp8.py."""
import pytest
import torch

from gpu_util import require_gpu
from test_gpu_fp8 import check_product, rand, ref_quant, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


def layer(swz, x, w, dy):
    x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
    y = swz.fp8_linear(x, w)
    y.backward(dy)
    return y.detach(), x.grad, w.grad


KINDS = ["rows of a wider one", "transposed", "every other column", "one row for all",
         "one column for all", "one vector", "one row", "three dimensions", "permuted",
         "last dimension outer", "four dimensions"]


def layouts(K):
    wide = rand((200, 2 * K), torch.bfloat16, 1).cuda()
    deep = rand((6, 5 * K), torch.bfloat16, 2).cuda().view(6, 5, K)
    return dict(zip(KINDS, (
        wide[3:90, 5:5 + K], rand((K, 70), torch.bfloat16, 3).cuda().t(), wide[:40, ::2],
        wide[:1, :K].expand(30, K), wide[:30, :1].expand(30, K), wide[0, :K], wide[:1, :K], deep,
        deep.transpose(0, 1), deep.permute(2, 0, 1).contiguous().permute(1, 2, 0),
        deep.view(2, 3, 5, K))))


@pytest.mark.parametrize("kind", KINDS)
def test_layouts_of_x(swz, kind):
    K, N = 300, 140
    x = layouts(K)[kind]
    w = rand((N, K), torch.bfloat16, 4).cuda()
    dy = rand((x.numel() // K, N), torch.bfloat16, 5).cuda().view(*x.shape[:-1], N)
    got = layer(swz, x, w, dy)
    swz.check_status()
    want = layer(swz, x.contiguous().view(-1, K), w, dy.reshape(-1, N))
    assert got[0].shape == (*x.shape[:-1], N) and got[1].shape == x.shape
    assert torch.equal(got[0].reshape(-1, N), want[0])
    assert torch.equal(got[1].reshape(-1, K), want[1]) and torch.equal(got[2], want[2])


def test_layouts_of_w_and_of_the_gradient(swz):
    x = rand((90, 200), torch.bfloat16, 1).cuda()
    wide = rand((150, 400), torch.bfloat16, 2).cuda()
    dy = rand((90, 150), torch.bfloat16, 3).cuda()
    for w in (rand((200, 150), torch.bfloat16, 4).cuda().t(), wide[:, ::2], wide[:, 7:207],
              wide[:1, :200].expand(150, 200)):
        for d in (dy, dy.t().contiguous().t(), dy[:1].expand(90, 150), dy[:, :1].expand(90, 150)):
            for got, want in zip(layer(swz, x, w, d), layer(swz, x, w.contiguous(), d.contiguous())):
                assert torch.equal(got, want)
    swz.check_status()


@pytest.mark.parametrize("xt", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wt", [torch.float16, torch.bfloat16, torch.float32])
def test_types(swz, xt, wt):
    x, w = rand((3, 50, 200), xt, 1, False), rand((130, 200), wt, 2)
    dy = rand((150, 130), xt, 3)
    y, dx, dw = layer(swz, x.cuda(), w.cuda(), dy.cuda().view(3, 50, 130))
    swz.check_status()
    assert (y.dtype, dx.dtype, dw.dtype) == (xt, xt, wt)
    v = lambda t, b: values(*ref_quant(t, b, "e4m3"), b)  # noqa: E731
    x = x.view(150, 200)
    check_product(y.view(150, 130), v(x, "row"), v(w, "square"))
    check_product(dx.view(150, 200), v(dy, "row"), v(w, "square").t())
    check_product(dw, v(dy.t(), "row"), v(x.t(), "row"))


@pytest.mark.parametrize("shape,N", [((0, 40), 30), ((2, 0, 40), 30), ((5, 0), 30), ((2, 3, 0), 30),
                                     ((5, 40), 0)])
def test_nothing(swz, shape, N):
    x = torch.ones(shape, device="cuda")
    w = torch.ones((N, shape[-1]), device="cuda")
    dy = torch.ones((*shape[:-1], N), device="cuda")
    y, dx, dw = layer(swz, x, w, dy)
    swz.check_status()
    assert y.shape == dy.shape and dx.shape == x.shape and dw.shape == w.shape
    assert (y == 0).all() and (dx == 0).all() and (dw == 0).all()


def test_one_gradient_alone(swz):
    x, w = rand((90, 200), torch.bfloat16, 1).cuda(), rand((150, 200), torch.bfloat16, 2).cuda()
    dy = rand((90, 150), torch.bfloat16, 3).cuda()
    _, dx, dw = layer(swz, x, w, dy)
    a = x.clone().requires_grad_()
    swz.fp8_linear(a, w).backward(dy)
    assert torch.equal(a.grad, dx)
    b = w.clone().requires_grad_()
    swz.fp8_linear(x, b).backward(dy)
    assert torch.equal(b.grad, dw)
    with torch.no_grad():
        assert not swz.fp8_linear(a, b).requires_grad
