"""Calls of the linear-layer operators that follow one another in a stream with
nothing of another library between them, so that each starts while the one
before still runs."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


@pytest.mark.parametrize("split", [1, 2])
@pytest.mark.parametrize("rows", [5, 20])
def test_the_bound_of_few_rows_does_not_count_the_kernel_before(swz, rows, split):
    # one CTA takes 6 ms for the large product; the other SMs have room for the
    # small one, whose waits are bounded by 1 ms of its own work
    a = swz.quantize_fp8(torch.randn(4096, 2048, device="cuda"))
    b = swz.quantize_fp8(torch.randn(4096, 2048, device="cuda"), "square")
    few = swz.quantize_fp8(torch.randn(rows, 2048, device="cuda"))
    want = swz.gemm_fp8(*few, *b, split_k=split)
    out, large = torch.empty_like(want), torch.empty(4096, 4096, device="cuda")
    swz.check_status()
    swz.gemm_fp8(*a, *b, out=large, tile=128, num_programs=1)
    swz.gemm_fp8(*few, *b, out=out, split_k=split, timeout_ms=1)
    swz.check_status()
    assert torch.equal(out, want)
