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


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("shape", [(3, 130, 200), (5, 200, 64), (9, 33, 33), (4, 520, 300),
                                   (2, 300, 640)])
def test_a_stack_is_its_matrices(swz, shape, tile):
    # sizes of magnitudes apart, so that a neighbour's scale would show
    G = normal(shape, torch.float32, 2) * torch.logspace(-6, 6, shape[0]).reshape(-1, 1, 1)
    G = G.cuda()
    Y = swz.newton_schulz(G, out_dtype=torch.float32, tile=tile)
    swz.check_status()
    for i in range(shape[0]):
        assert torch.equal(Y[i], swz.newton_schulz(G[i], out_dtype=torch.float32, tile=tile)), i


@pytest.mark.parametrize("shape", [(7, 64, 64), (5, 100, 333), (6, 300, 90), (5, 256, 320),
                                   (40, 100, 1030), (4, 1300, 200)])
def test_a_stack_in_another_order(swz, shape):
    G = normal(shape, torch.bfloat16, 2) * torch.logspace(-6, 6, shape[0]).reshape(-1, 1, 1)
    G = G.bfloat16().cuda()
    order = torch.randperm(shape[0], generator=torch.Generator().manual_seed(1)).cuda()
    Y = swz.newton_schulz(G)
    assert torch.equal(swz.newton_schulz(G[order]), Y[order])
    swz.check_status()


@pytest.mark.parametrize("tile", [0, 128, 256])
@pytest.mark.parametrize("shape", [(64, 64), (100, 333), (333, 100), (128, 1100), (256, 512),
                                   (301, 203), (3, 70, 150)])
def test_half_precision_in_and_out(swz, shape, tile):
    G = normal(shape, torch.float16, sum(shape))
    for out in (torch.float16, torch.float32):
        Y = swz.newton_schulz(G.cuda(), out_dtype=out, tile=tile)
        swz.check_status()
        check(Y, G)
    G = normal(shape, torch.float32, sum(shape))
    check(swz.newton_schulz(G.cuda(), out_dtype=torch.float16, tile=tile), G)


# more tiles than CTA pairs: of the update (81 for 76), and of every product (84 and 144)
@pytest.mark.parametrize("shape", [(2300, 2310), (4, 1300, 1290)])
def test_pairs_take_more_than_one_tile(swz, shape):
    G = normal(shape, torch.float32, 7)
    Y = swz.newton_schulz(G.cuda(), out_dtype=torch.float32, tile=256)
    swz.check_status()
    check(Y, G)
    assert torch.equal(Y, swz.newton_schulz(G.cuda(), out_dtype=torch.float32, tile=256))
