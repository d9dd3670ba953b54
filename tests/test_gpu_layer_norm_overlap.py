"""Where the results of a layer norm may lie: the columns beside its input, not across it."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


@pytest.mark.parametrize("m", [1, 2, 70])
@pytest.mark.parametrize("n", [40, 1000, 1999, 4096, 17000])
def test_beside_and_across(swz, m, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    buf = torch.randn((m, 2 * n + 24), generator=g, device="cuda").bfloat16()
    w = torch.randn(n, generator=g, device="cuda")
    before, x, out = buf.clone(), buf[:, :n], buf[:, n + 8:2 * n + 8]
    want = swz.layer_norm_forward(x.clone(), w)[0]
    swz.layer_norm_forward(x, w, out=out)
    assert torch.equal(out, want)
    out.copy_(before[:, n + 8:2 * n + 8])
    assert torch.equal(buf, before)
    for over in (buf[:, 1:n + 1], buf[:, n - 1:2 * n - 1], buf.view(torch.float16)[:, :n]):
        with pytest.raises(swz.SwzError):
            swz.layer_norm_forward(x, w, out=over)
    if m > 2:  # one row further on (of two rows it is another one)
        with pytest.raises(swz.SwzError):
            swz.layer_norm_forward(buf[:-1, :n], w, out=buf[1:, :n])
    assert torch.equal(buf, before)
