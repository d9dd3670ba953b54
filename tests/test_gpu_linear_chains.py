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


@pytest.mark.parametrize("M,N,K", [(300, 520, 640), (2048, 1024, 512), (17, 512, 384)])
def test_what_a_kernel_reads_is_what_the_one_before_wrote(swz, M, N, K):
    # A product into the same buffer again and again, each time quantised and, as a
    # gradient is, orthogonalised and quantised; every other pass has other operands.
    ops = []
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        a = torch.randn(M, K, generator=g, device="cuda")
        b = torch.randn(N, K, generator=g, device="cuda")
        ops.append((*swz.quantize_fp8(a), *swz.quantize_fp8(b, "square")))
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    D = torch.empty(M, N, dtype=torch.float32, device="cuda")
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def chain(qa, sa, qb, sb, between):
        out = []
        swz.gemm_fp8(qa, sa, qb, sb, out=C)
        between()
        out += swz.quantize_fp8(C, "row", transposed=True)
        between()
        swz.gemm_fp8(qa, sa, qb, sb, out=D)
        between()
        swz.newton_schulz(D, out=Y)
        between()
        out += swz.quantize_fp8(Y, "square")
        between()
        return out
    want = [chain(*o, torch.cuda.synchronize) for o in ops]
    got = [chain(*ops[i % 2], lambda: None) for i in range(40)]
    torch.cuda.synchronize()
    swz.check_status()
    for i, results in enumerate(got):
        for x, w in zip(results, want[i % 2]):
            assert torch.equal(x.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8)), i


def test_operands_freed_while_another_stream_works_on_them(swz):
    # the side stream is busy when the calls are made; what they read is freed and
    # asked for again before it gets there
    side = torch.cuda.Stream()
    x, w = torch.randn(256, 512, device="cuda").bfloat16(), torch.randn(384, 512, device="cuda")
    want = swz.linear_fp8(x, *swz.quantize_fp8(w, "square"))
    update = swz.newton_schulz(w)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    qw, sw = swz.quantize_fp8(w, "square")
    one = x + 0
    two = w + 0
    side.wait_stream(torch.cuda.current_stream())
    y = swz.linear_fp8(one, qw, sw, stream=side)
    z = swz.newton_schulz(two, stream=side)
    del one, two, qw, sw
    for _ in range(4):  # what would take the memory over
        junk = [torch.full_like(x, 7.0), torch.full_like(w, 7.0),
                torch.full(w.shape, 7, dtype=torch.uint8, device="cuda")]
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(z, update) and len(junk) == 3
