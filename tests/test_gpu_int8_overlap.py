"""The layer in 8-bit integers with its result over x, bit for bit what it is elsewhere."""
import pytest
import torch

from gpu_util import capture_graph, require_gpu

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
ROWS = [1, 2, 3, 20, 100, 600]


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weights(swz, n, k):
    return swz.quantize_int8(torch.randn((n, k), generator=gen(n + k), device="cuda"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("k", [77, 1000, 4096])
def test_in_place(swz, dtype, m, k):
    w = weights(swz, k, k)
    for seed in range(4):
        x = torch.randn((m, k), generator=gen(seed), device="cuda").to(dtype)
        want = swz.linear_int8(x, *w)
        y = x.clone()
        assert swz.linear_int8(y, *w, out=y) is y
        assert torch.equal(y, want)


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,shift", [(4000, 1), (300, -7), (4000, 2500), (5000, -8)])
def test_across(swz, m, n, shift):
    """x and the result begin at different places of the same memory."""
    k = 4096
    w = weights(swz, n, k)
    for seed in range(4):
        x = torch.randn((m, k), generator=gen(seed), device="cuda").half()
        want = swz.linear_int8(x, *w)
        flat = torch.zeros(m * (k + n) + 64, dtype=torch.float16, device="cuda")
        xv = flat[16:16 + m * k].view(m, k)
        xv.copy_(x)
        out = flat[16 + shift:16 + shift + m * n].view(m, n)
        assert torch.equal(swz.linear_int8(xv, *w, out=out), want)


@pytest.mark.parametrize("m", ROWS)
def test_other_type(swz, m):
    """32-bit results over 16-bit values of x."""
    k = n = 2048
    w = weights(swz, n, k)
    x = torch.randn((m, k), generator=gen(m), device="cuda").bfloat16()
    want = swz.linear_int8(x, *w, out_dtype=torch.float32)
    out = torch.zeros((m, n), device="cuda")
    xv = out.flatten().view(torch.bfloat16)[:m * k].view(m, k)
    xv.copy_(x)
    assert torch.equal(swz.linear_int8(xv, *w, out=out), want)


@pytest.mark.parametrize("m", ROWS)
def test_beside(swz, m):
    """Columns of one buffer: x in some, the result in others; x and the rest stay."""
    k, n = 1000, 520
    w = weights(swz, n, k)
    buf = torch.randn((m, k + n + 30), generator=gen(m), device="cuda").bfloat16()
    before = buf.clone()
    want = swz.linear_int8(buf[:, :k], *w)
    swz.linear_int8(buf[:, :k], *w, out=buf[:, k + 10:k + 10 + n])
    assert torch.equal(buf[:, k + 10:k + 10 + n], want)
    buf[:, k + 10:k + 10 + n] = before[:, k + 10:k + 10 + n]
    assert torch.equal(buf, before)


@pytest.mark.parametrize("m", [1, 2, 20])
def test_captured(swz, m):
    k = 4096
    w = weights(swz, k, k)
    y = torch.zeros((m, k), device="cuda").bfloat16()
    g = capture_graph(lambda: swz.linear_int8(y, *w, out=y))
    for seed in range(4):
        x = torch.randn((m, k), generator=gen(seed), device="cuda").bfloat16()
        y.copy_(x)
        g.replay()
        assert torch.equal(y, swz.linear_int8(x, *w))


@pytest.mark.parametrize("m", [1, 5, 40, 600])
def test_products_over_operands_are_refused(swz, m):
    k, n = 256, 64
    qw, sw = weights(swz, 1000, k)
    qx, sx = swz.quantize_int8(torch.randn((m, k), generator=gen(m), device="cuda"))
    kept = [t.clone() for t in (qx, sx, qw, sw)]
    over = qx.view(torch.float16)[:, 64:64 + n]  # the right half of x's bytes
    with pytest.raises(swz.SwzError):
        swz.gemm_int8(qx, sx, qw[:n], sw[:n], out=over)
    over = qw.view(torch.float16)[:m, :n]  # the left half of W's
    with pytest.raises(swz.SwzError):
        swz.gemm_int8(qx, sx, qw[:n], sw[:n], out=over)
    with pytest.raises(swz.SwzError):
        swz.linear_int8(torch.zeros((m, k), device="cuda"), qw[:n], sw[:n], out=over)
    assert all(torch.equal(a, b) for a, b in zip(kept, (qx, sx, qw, sw)))
    # rows of W that the call does not read, and bytes of x beyond its columns, are not in the way
    if m <= 900:
        want = swz.gemm_int8(qx, sx, qw[:n], sw[:n], out_dtype=torch.float16)
        got = swz.gemm_int8(qx, sx, qw[:n], sw[:n], out=qw.view(torch.float16)[n:n + m, :n])
        assert torch.equal(got, want)
