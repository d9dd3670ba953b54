"""8-bit integer operators on the GPU at the ends of the sizes they take."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


@pytest.mark.parametrize("k", [2 ** 31 - 8, 2 ** 31 - 7, 2 ** 31 - 1])
def test_quantize_longest_rows(swz, k):
    """Rows whose number of values, rounded up to eight, does not fit 32 bits: a few
    values among zeros, at both ends."""
    x = torch.zeros((1, k), dtype=torch.bfloat16, device="cuda")
    values = {0: 1.0, 5: -2.0, k // 2: 0.5, k - 9: 0.25, k - 1: -1.5}
    for at, v in values.items():
        x[0, at] = v
    q, s = swz.quantize_int8(x)
    # amax 2: r = 127 / 2 exactly, so q = 63.5 v to even
    for at, v in values.items():
        assert q[0, at].item() == round(63.5 * v), at
    assert s.item() == (torch.tensor(2.0) / torch.tensor(127.0)).item()
    part = 1 << 28
    assert sum(int(torch.count_nonzero(q[0, i:i + part])) for i in range(0, k, part)) == len(values)


def rows_and_scales(swz, m, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = swz.int8_empty(m, k)
    flat = q if q.is_contiguous() else torch.as_strided(q, (m, q.stride(0)), q.stride())
    part = 1 << 24
    for i in range(0, m, part):  # what lies beyond the columns as well
        flat[i:i + part].random_(-128, 128, generator=g)
    return q, torch.rand(m, generator=g, device="cuda") + 0.5


def check(c, a, sa, b, sb):
    """Whole sums below 2^24, rounded products of the scales, one rounding of the result."""
    part = 1 << 24
    for i in range(0, b.shape[0], part):
        s = a.float() @ b[i:i + part].float().t()
        want = (s * (sa.unsqueeze(1) * sb[i:i + part])).to(c.dtype)
        assert torch.equal(c[:, i:i + part], want), i


@pytest.mark.parametrize("k", [16, 32, 45, 100])
@pytest.mark.parametrize("m", [1, 2])
def test_many_channels(swz, m, k):
    """More rows of B a CTA than it has partial sums for: several turns."""
    a, sa = rows_and_scales(swz, m, k, 1)
    b, sb = rows_and_scales(swz, 700001, k, 2)
    check(swz.gemm_int8(a, sa, b, sb, out_dtype=torch.float32), a, sa, b, sb)
    x = torch.randn((m, k), device="cuda")
    q, s = swz.quantize_int8(x)
    check(swz.linear_int8(x, b, sb), q, s, b, sb)


@pytest.mark.parametrize("m", [1, 2])
def test_most_channels(swz, m):
    """As many rows of B as the sizes can say, the last ones' numbers next to 2^31."""
    a, sa = rows_and_scales(swz, m, 16, 3)
    b, sb = rows_and_scales(swz, 2 ** 31 - 1, 16, 4)
    check(swz.gemm_int8(a, sa, b, sb), a, sa, b, sb)
