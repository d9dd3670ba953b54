"""newton_schulz against the iteration in 64 bits.

Tolerance, relative in the Frobenius norm: a step rounds X, A and B once each
to fp16, relative error at most 2^-11 of an entry (2^-11 / sqrt(3) in the root
mean square); the 3 * steps roundings are taken to add up linearly and, by the
choice of where X is kept in fp32, not to grow on the way:
3 * steps * 2^-11 / sqrt(3) (4.2e-3 for five steps), plus the result's own
rounding (2^-8 / sqrt(3) for bf16)."""
import math

import pytest
import torch

from gpu_util import capture_graph, require_gpu

pytestmark = pytest.mark.gpu
COEF = (3.4445, -4.7750, 2.0315)
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


def reference(G, steps=5, coef=COEF, eps=1e-7):
    a, b, c = coef
    x = G.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    for _ in range(steps):
        p = x @ x.mT
        x = a * x + (b * p + c * p @ p) @ x
    return x.mT if tall else x


def check(Y, G, steps=5, coef=COEF, eps=1e-7):
    want = reference(G.cpu(), steps, coef, eps)
    tol = (3 * steps * 2.0 ** -11 + ROUND[Y.dtype]) / math.sqrt(3)
    y = Y.cpu().double()
    for got, w in zip(y.reshape(-1, *y.shape[-2:]), want.reshape(-1, *y.shape[-2:])):
        err = (got - w).norm() / w.norm()
        assert err <= tol, (err.item(), tol)


def normal(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("tile", [0, 128, 256])
@pytest.mark.parametrize("shape", [(1, 1), (1, 300), (17, 5), (100, 333), (333, 100), (128, 128),
                                   (129, 130), (256, 512), (640, 300), (513, 515)])
def test_shapes(swz, shape, tile):
    for dtype, out in ((torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16)):
        G = normal(shape, dtype, sum(shape))
        Y = swz.newton_schulz(G.cuda(), out_dtype=out, tile=tile)
        swz.check_status()
        check(Y, G)


# the one-kernel form's ranges: 1 to 8 ranks, 64 to 256 columns each, both ways round
@pytest.mark.parametrize("shape", [(128, 64), (40, 129), (128, 257), (300, 128), (64, 513), (1024, 33),
                                   (100, 1025), (128, 2048), (2048, 128), (5, 1999), (128, 2049),
                                   (3, 90, 700), (2, 700, 90)])
def test_one_kernel_shapes(swz, shape):
    G = normal(shape, torch.float32, sum(shape))
    Y = swz.newton_schulz(G.cuda(), out_dtype=torch.float32)
    swz.check_status()
    check(Y, G)
    other = swz.newton_schulz(G.cuda(), out_dtype=torch.float32, tile=128)
    check(other, G)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 10])
@pytest.mark.parametrize("shape", [(60, 200), (200, 60)])
def test_steps(swz, shape, steps):
    G = normal(shape, torch.float32, steps)
    check(swz.newton_schulz(G.cuda(), steps, out_dtype=torch.float32), G, steps)


@pytest.mark.parametrize("coef", [(1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5),
                                  (1.0, 0.0, 0.0)])
def test_coefficients(swz, coef):
    G = normal((90, 140), torch.float32, 1)
    check(swz.newton_schulz(G.cuda(), 5, coef, out_dtype=torch.float32), G, 5, coef)


@pytest.mark.parametrize("shape", [(3, 130, 200), (5, 200, 64), (1, 64, 64), (9, 33, 33)])
def test_batch_equals_single(swz, shape):
    G = normal(shape, torch.bfloat16, 2) * torch.logspace(-6, 6, shape[0]).reshape(-1, 1, 1)
    G = G.bfloat16().cuda()
    Y = swz.newton_schulz(G, out_dtype=torch.float32)
    check(Y, G, eps=1e-7)
    for i in range(shape[0]):
        assert torch.equal(swz.newton_schulz(G[i], out_dtype=torch.float32, tile=128),
                           swz.newton_schulz(G[i:i + 1], out_dtype=torch.float32, tile=128)[0])


@pytest.mark.parametrize("kind", ["decay", "low rank", "identity", "one entry"])
def test_spectra(swz, kind):
    g = torch.Generator().manual_seed(3)
    m, n = 256, 384
    if kind == "decay":
        u = torch.linalg.qr(torch.randn(m, m, generator=g))[0]
        v = torch.linalg.qr(torch.randn(n, m, generator=g))[0]
        G = u @ torch.diag(torch.logspace(0, -4, m)) @ v.t()
    elif kind == "low rank":
        G = torch.randn(m, 8, generator=g) @ torch.randn(8, n, generator=g)
        G += 1e-2 * torch.randn(m, n, generator=g)
    elif kind == "identity":
        G = torch.eye(m, n)
    else:
        G = torch.zeros(m, n)
        G[200, 301] = -5.0
    check(swz.newton_schulz(G.cuda(), out_dtype=torch.float32), G)


@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e-12, 1e12, 1e25, 1e37])
def test_scales(swz, scale):
    G = normal((70, 90), torch.float32, 4) * scale
    check(swz.newton_schulz(G.cuda(), out_dtype=torch.float32), G)
    if scale < 1:  # without eps the scale drops out
        check(swz.newton_schulz(G.cuda(), eps=0.0, out_dtype=torch.float32), G, eps=0.0)


def test_zero_and_not_finite(swz):
    Z = torch.zeros((3, 40, 50), device="cuda")
    Z[1] = torch.randn(40, 50, device="cuda")
    for eps in (1e-7, 0.0):
        Y = swz.newton_schulz(Z, eps=eps)
        assert (Y[0] == 0).all() and (Y[2] == 0).all() and Y[1].isfinite().all()
    for bad in (float("nan"), float("inf")):
        B = Z.clone()
        B[0, 3, 4] = bad
        Y = swz.newton_schulz(B)
        assert not Y[0].isfinite().all() and Y[1].isfinite().all() and (Y[2] == 0).all()


def test_strides_in_place_and_out(swz):
    big = normal((4, 150, 300), torch.bfloat16, 6).cuda()
    for G in (big[0, 3:103, 5:205], big[:, 3:103, 5:205], big[::2, 1::2, :77], big[1, :1, 9:200]):
        want = swz.newton_schulz(G.contiguous())
        assert torch.equal(swz.newton_schulz(G), want)
        out = torch.full(big.shape, 9.0, dtype=torch.bfloat16, device="cuda")
        view = out[0, 3:103, 5:205] if G.dim() == 2 and G.shape[0] == 100 else None
        if view is not None:
            swz.newton_schulz(G, out=view)
            assert torch.equal(view, want)
            out[0, 3:103, 5:205] = 9.0
            assert (out == 9.0).all()
        for steps in (1, 5):
            same = G.clone()
            want = swz.newton_schulz(same, steps)
            swz.newton_schulz(same, steps, out=same)
            assert torch.equal(same, want)


@pytest.mark.parametrize("shape", [(0, 5), (5, 0), (0, 4, 4)])
def test_empty(swz, shape):
    assert swz.newton_schulz(torch.zeros(shape, device="cuda")).shape == shape


def test_stream_and_graph(swz):
    G = normal((300, 200), torch.float32, 8).cuda()
    want = swz.newton_schulz(G)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [swz.newton_schulz(G, stream=side) for _ in range(10)]
    side.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    Gs, out = G.clone(), torch.empty_like(want)
    g = capture_graph(lambda: swz.newton_schulz(Gs, out=out))
    G2 = normal((300, 200), torch.float32, 9).cuda()
    Gs.copy_(G2)
    g.replay()
    assert torch.equal(out, swz.newton_schulz(G2))


@pytest.mark.parametrize("tile,shape", [(128, (300, 200)), (256, (300, 200)), (0, (100, 60)),
                                        (0, (100, 600))])
def test_timeout_is_reported(swz, tile, shape):
    G = normal(shape, torch.float32, 8).cuda()
    want = swz.newton_schulz(G)
    swz.newton_schulz(G, tile=tile, debug_flags=swz.SWZ_DEBUG_SKIP_FIRST_LOAD, timeout_ms=20)
    with pytest.raises(swz.SwzError) as e:
        swz.check_status()
    assert e.value.code == swz.SWZ_ETIMEOUT
    swz.check_status()
    assert torch.equal(swz.newton_schulz(G), want)


def test_refusals(swz):
    G = torch.zeros((8, 8), device="cuda")
    with pytest.raises(ValueError):
        swz.newton_schulz(G[0])
    with pytest.raises(TypeError):
        swz.newton_schulz(G.double())
    with pytest.raises(ValueError):
        swz.newton_schulz(torch.zeros((8, 4), device="cuda").t())
    with pytest.raises(ValueError):
        swz.newton_schulz(G, out=torch.zeros((8, 9), device="cuda"))
    for kw in (dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=float("nan")),
               dict(coefficients=(float("inf"), 0.0, 0.0))):
        with pytest.raises(swz.SwzError) as e:
            swz.newton_schulz(G, **kw)
        assert e.value.code == swz.SWZ_EINVAL
    for kw in (dict(tile=64), dict(coefficients=(1e9, 0.0, 0.0), steps=4)):
        with pytest.raises(swz.SwzError) as e:
            swz.newton_schulz(G, **kw)
        assert e.value.code == swz.SWZ_EUNSUPPORTED


# stacks around what one wave of the one-kernel form holds, and well above it
@pytest.mark.parametrize("shape", [(14, 128, 1100), (40, 100, 1030), (153, 64, 64), (700, 33, 40),
                                   (80, 200, 120)])
def test_stacks_of_small_matrices(swz, shape):
    G = normal(shape, torch.float32, shape[0])
    Y = swz.newton_schulz(G.cuda(), out_dtype=torch.float32)
    swz.check_status()
    check(Y, G)


@pytest.mark.parametrize("shape", [(100, 60), (300, 200), (200, 520), (600, 520)])
def test_far_rows(swz, shape):
    """Rows of G and of the result further apart than 32 bits reach."""
    G = normal(shape, torch.bfloat16, 1).cuda()
    want = swz.newton_schulz(G)
    m, n = shape
    stride = -(-(2 ** 31 + 1000) // ((m - 1) * 64)) * 64
    views = []
    for _ in range(2):
        flat = torch.empty((m - 1) * stride + n, dtype=torch.bfloat16, device="cuda")
        views.append(flat.as_strided((m, n), (stride, 1)))
    views[0].copy_(G)
    swz.newton_schulz(views[0], out=views[1])
    swz.check_status()
    assert torch.equal(views[1], want)


@pytest.mark.parametrize("tile", [0, 128, 256])
@pytest.mark.parametrize("shape", [(33, 2000), (64, 2048), (77, 2246), (2246, 77), (5, 64, 2050),
                                   (150, 150), (256, 300)])
def test_short_sides_in_bf16(swz, shape, tile):
    """A bf16 result is no more than 1.5 times as far off as the exact one
    rounded once: what comes before the rounding stays below it."""
    G = normal(shape, torch.bfloat16, 3)
    Y = swz.newton_schulz(G.cuda(), tile=tile)
    swz.check_status()
    want = reference(G)
    got = Y.cpu().double()
    for y, w in zip(got.reshape(-1, *got.shape[-2:]), want.reshape(-1, *want.shape[-2:])):
        assert (y - w).norm() <= 1.5 * (w.bfloat16().double() - w).norm()


# few tiles and a long K, also where it does not divide evenly
@pytest.mark.parametrize("tile", [0, 128])
@pytest.mark.parametrize("shape", [(130, 1024), (130, 1153), (200, 3000), (3000, 200), (150, 2049),
                                   (3, 140, 2200), (600, 4000)])
def test_long_k(swz, shape, tile):
    G = normal(shape, torch.float32, 5)
    Y = swz.newton_schulz(G.cuda(), out_dtype=torch.float32, tile=tile)
    swz.check_status()
    check(Y, G)
    assert torch.equal(Y, swz.newton_schulz(G.cuda(), out_dtype=torch.float32, tile=tile))
