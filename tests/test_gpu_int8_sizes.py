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
