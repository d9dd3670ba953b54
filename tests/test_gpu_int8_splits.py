"""The product in 8-bit integers with the kernel chosen by itself and a split of K that
the caller asks for: done by whichever kernel has that split."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


@pytest.mark.parametrize("k", [1000, 2048, 4096, 8192, 16384])
@pytest.mark.parametrize("m", [3, 32, 33, 40, 100, 250, 256, 300, 512, 513])
def test_own_split(swz, m, k):
    g = torch.Generator(device="cuda").manual_seed(m * k)
    n = 130
    a, sa = swz.quantize_int8(torch.randn((m, k), generator=g, device="cuda"))
    b, sb = swz.quantize_int8(torch.randn((n, k), generator=g, device="cuda"))
    # exact sums, rounded to fp32 and multiplied by the rounded product of the scales
    want = (a.double() @ b.double().t()).float() * (sa.unsqueeze(1) * sb)
    for split in (0, 1, 2, 4, 8):
        got = swz.gemm_int8(a, sa, b, sb, split_k=split, out_dtype=torch.float32)
        assert torch.equal(got, want), split
    swz.check_status()


def test_more_parts_than_blocks(swz):
    for m in (20, 100, 600):
        a, sa = swz.quantize_int8(torch.randn((m, 200), device="cuda"))
        b, sb = swz.quantize_int8(torch.randn((70, 200), device="cuda"))
        with pytest.raises(swz.SwzError) as e:
            swz.gemm_int8(a, sa, b, sb, split_k=4)
        assert e.value.code == swz.SWZ_EUNSUPPORTED
