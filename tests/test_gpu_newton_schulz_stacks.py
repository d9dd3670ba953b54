"""newton_schulz of stacks: each matrix's result is its own, wherever the others
lie, and whatever memory the result shares with what it is made of.  Tolerance
against the iteration in 64 bits as in test_gpu_newton_schulz.py."""
import pytest
import torch

from gpu_util import require_gpu
from test_gpu_newton_schulz import check, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("shape", [(64, 64, 64), (40, 100, 300), (24, 700, 90), (6, 256, 320),
                                   (5, 200, 130), (300, 512), (100, 60), (512, 192)])
def test_a_result_of_other_size_over_its_input(swz, shape, steps):
    # fp32 G and bf16 Y from the same address: a matrix's Y is over another's G
    G = normal(shape, torch.float32, sum(shape))
    buf = G.cuda()
    Y = buf.flatten().view(torch.bfloat16)[:G.numel()].view(shape)
    swz.newton_schulz(buf, steps, out=Y)
    swz.check_status()
    check(Y, G, steps)
    # and bf16 G with an fp32 Y
    buf = torch.empty(G.shape, dtype=torch.float32, device="cuda")
    G = G.bfloat16()
    over = buf.flatten().view(torch.bfloat16)[:G.numel()].view(shape)
    over.copy_(G)
    swz.newton_schulz(over, steps, out=buf)
    swz.check_status()
    check(buf, G, steps)


@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("shape", [(60, 64, 64), (30, 90, 300), (7, 256, 320)])
def test_a_result_shifted_over_its_input(swz, shape, steps):
    batch, m, n = shape
    G = normal((batch + 1, m, n), torch.float32, 3)
    for src, dst in ((slice(0, batch), slice(1, batch + 1)), (slice(1, batch + 1), slice(0, batch))):
        buf = G.cuda()
        swz.newton_schulz(buf[src], steps, out=buf[dst])
        swz.check_status()
        check(buf[dst], G[src], steps)
    # by some rows, and by some columns
    buf = normal((m + 5, n + 16), torch.float32, 4).cuda()
    for dr, dc in ((5, 0), (0, 8), (3, 2)):
        one = buf.clone()
        swz.newton_schulz(one[:m, :n], steps, out=one[dr:dr + m, dc:dc + n])
        swz.check_status()
        check(one[dr:dr + m, dc:dc + n], buf[:m, :n].cpu(), steps)


@pytest.mark.parametrize("shape", [(20, 64, 64), (9, 100, 300), (3, 256, 320)])
def test_results_beside_their_input(swz, shape):
    # columns of the same rows: no value is shared, and the result is that of
    # buffers of their own
    batch, m, n = shape
    for steps in (1, 5):
        buf = normal((batch, m, 2 * n + 8), torch.float32, 5).cuda()
        G = buf[:, :, :n].clone()
        want = swz.newton_schulz(G, steps, out_dtype=torch.float32)
        left = buf.clone()
        swz.newton_schulz(left[:, :, :n], steps, out=left[:, :, n + 8:])
        swz.check_status()
        assert torch.equal(left[:, :, n + 8:], want)
        assert torch.equal(left[:, :, :n + 8], buf[:, :, :n + 8])
