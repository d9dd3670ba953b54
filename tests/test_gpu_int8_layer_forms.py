"""Every way that linear_int8 goes by the size of x, bit for bit: x quantised in the
kernel of one or two rows or before it, by K; and both operands widened, K of several
blocks."""
import pytest
import torch

from gpu_util import capture_graph, require_gpu

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def exact(x, qw, sw, dtype):
    """The definition, every rounding where it stands."""
    ac = x.float().abs().amax(1).clamp_min(2.0 ** -96)
    top = torch.full_like(ac, 127.0)
    q = torch.round(x.double() * (top / ac).double().unsqueeze(1))
    return ((q @ qw.double().t()).float() * ((ac / top).unsqueeze(1) * sw)).to(dtype)


def operands(swz, m, n, k, dtype):
    x = torch.randn((m, k), generator=gen(k), device="cuda").to(dtype)
    return (x, *swz.quantize_int8(torch.randn((n, k), generator=gen(n), device="cuda")))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [
    (2, 3, 5), (2, 1000, 4099), (2, 130, 16383), (2, 33, 16384), (1, 77, 32768),  # x in the kernel
    (1, 300, 32769), (2, 300, 16385), (2, 301, 40001), (1, 64, 131071), (2, 5000, 20000),  # before it
    (513, 1111, 1999), (600, 300, 2000), (1000, 130, 4099)])  # both operands widened
def test_forms(swz, dtype, m, n, k):
    x, qw, sw = operands(swz, m, n, k, dtype)
    want = exact(x, qw, sw, dtype)
    assert torch.equal(swz.linear_int8(x, qw, sw), want)
    # rows that start anywhere, what lies beside them NaN
    flat = torch.full((m * (k + 3) + 64,), float("nan"), dtype=dtype, device="cuda")
    v = flat[1:1 + m * (k + 3)].view(m, k + 3)[:, :k]
    v.copy_(x)
    assert torch.equal(swz.linear_int8(v, qw, sw), want)
    out = torch.full((m, n + 3), 7.0, dtype=torch.float32, device="cuda")
    swz.linear_int8(x, qw, sw, out=out[:, :n])
    assert torch.equal(out[:, :n], exact(x, qw, sw, torch.float32)) and (out[:, n:] == 7.0).all()
    swz.check_status()


@pytest.mark.parametrize("m,k", [(2, 4099), (1, 40001), (2, 40001), (600, 2000)])
def test_bad_rows(swz, m, k):
    """A NaN in one row makes that row NaN and no other."""
    x, qw, sw = operands(swz, m, 70, k, torch.float32)
    want = swz.linear_int8(x, qw, sw)
    x[m - 1, k - 1] = float("nan")
    y = swz.linear_int8(x, qw, sw)
    assert torch.isnan(y[m - 1]).all() and torch.equal(y[:m - 1], want[:m - 1])


@pytest.mark.parametrize("m,k", [(1, 40001), (2, 40001), (600, 2000)])
def test_graphs_and_streams(swz, m, k):
    """Two graphs and two streams, each call with its own workspace."""
    n = 640
    x, qw, sw = operands(swz, m, n, k, torch.bfloat16)
    out = {}

    def call():
        out["y"] = swz.linear_int8(x, qw, sw)
    g1 = capture_graph(call)
    first = out["y"]
    g2 = capture_graph(call)
    for seed in (1, 2):
        x.copy_(torch.randn((m, k), generator=gen(seed), device="cuda"))
        want = exact(x, qw, sw, torch.bfloat16)
        g1.replay()
        g2.replay()
        assert torch.equal(first, want) and torch.equal(out["y"], want)
    other = x.flip(0).contiguous() * 2
    wants = [want, exact(other, qw, sw, torch.bfloat16)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for i, (s, v) in enumerate(zip(streams, (x, other))):
            with torch.cuda.stream(s):
                got.append((i, swz.linear_int8(v, qw, sw)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, wants[i]) for i, y in got)
    swz.check_status()
