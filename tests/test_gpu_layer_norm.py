"""The layer norm and its gradient on the GPU against the formula in 64 bits.

Bounds, elementwise, with u = 2^-24 and c the longest chain of fp32 additions of a
sum over a row (a thread's values, a warp's exchange, the warps of a CTA: below 100
for a row in registers, and a turn of the loop for each 4096 values of longer
ones):
  mean    c u mean|x| =: dm
  x - mean  dm + u |x - mean|
  rstd    relative: half of var's, which is 2 dm / s + (c + 3) u with s = sqrt(var + eps),
          and 3 u of its own =: dr
  xhat    dm / s + |xhat| (u + dr + u) =: E
  y       |w| E + 3 u (|xhat w| + |b|) and the rounding to y's type
  dx      rstd (c u mean|g| + |xhat| ((c + 3) u mean|g xhat| + mean(|g| E))
          + E |mean(g xhat)| + 5 u (|g| + |mean g| + |xhat mean(g xhat)|)) + dr |dx|
  dw, db  with c' additions over rows: sum |dy| E + c' u sum |dy xhat|, c' u sum |dy|
A rounding to a type is half of its eps relative (and half of the smallest step of
fp16 absolute)."""
import pytest
import torch

from gpu_util import capture_graph, require_gpu

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, want, bound):
    """|got - want| within bound and the rounding to got's type."""
    step = torch.finfo(got.dtype)
    least = step.tiny * step.eps  # the smallest step of the type
    allowed = bound + (want.abs() + bound) * step.eps / 2 + least
    off = (got.double() - want).abs()
    assert bool((off <= allowed).all()), ((off / allowed).max().item(), off.max().item())


def formula(x, w, b, eps, dy=None):
    """y, mean, rstd (and dx, dw, db) in 64 bits, each with its bound."""
    n, m = x.shape[1], x.shape[0]
    x = x.double()
    w = torch.ones(n, device="cuda", dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(n, device="cuda", dtype=torch.float64) if b is None else b.double()
    c = 100 + n / 4096 * 2
    mean = x.mean(1, keepdim=True)
    d = x - mean
    s = (d.square().mean(1, keepdim=True) + eps).sqrt()
    xhat = d / s
    dm = c * U * x.abs().mean(1, keepdim=True)
    dr = dm / s + (c + 3) / 2 * U + 3 * U
    E = dm / s + xhat.abs() * (2 * U + dr)
    out = {"y": (xhat * w + b, w.abs() * E + 3 * U * ((xhat * w).abs() + b.abs())),
           "mean": (mean.squeeze(1), dm.squeeze(1)), "rstd": ((1 / s).squeeze(1), (dr / s).squeeze(1))}
    if dy is None:
        return out
    dy = dy.double()
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = (g - m1 - xhat * m2) / s
    bound = (c * U * g.abs().mean(1, keepdim=True)
             + xhat.abs() * ((c + 3) * U * (g * xhat).abs().mean(1, keepdim=True)
                             + (g.abs() * E).mean(1, keepdim=True))
             + E * m2.abs() + 5 * U * (g.abs() + m1.abs() + (xhat * m2).abs())) / s + dr * dx.abs()
    c2 = m / 64 + 128
    out["dx"] = dx, bound
    out["dw"] = (dy * xhat).sum(0), (dy.abs() * E).sum(0) + c2 * U * (dy * xhat).abs().sum(0)
    out["db"] = dy.sum(0), c2 * U * dy.abs().sum(0)
    return out


def spaced(x, extra, offset):
    """x in rows `extra` elements longer that start `offset` elements into their memory."""
    m, n = x.shape
    flat = torch.full((offset + m * (n + extra) + 64,), float("nan"), dtype=x.dtype, device="cuda")
    v = flat[offset:offset + m * (n + extra)].view(m, n + extra)[:, :n]
    v.copy_(x)
    return v


def inputs(m, n, dtype, wtype, seed=0, shift=0.0):
    g = gen(seed + m * 131 + n)
    x = (torch.randn((m, n), generator=g, device="cuda") * 2 + shift).to(dtype)
    w = (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(wtype)
    b = torch.randn(n, generator=g, device="cuda").to(wtype)
    dy = torch.randn((m, n), generator=g, device="cuda").to(dtype)
    return x, w, b, dy


SHAPES = [(1, 1), (3, 2), (1, 8), (9, 255), (17, 256), (5, 257), (33, 600), (1, 1024), (10, 1025),
          (12, 1999), (7, 2048), (3, 2049), (1, 4096), (20, 4096), (3, 5001), (2, 8192), (4, 10240),
          (2, 16384), (3, 16385), (2, 40003), (2000, 64), (5000, 33), (1001, 600), (700, 1999), (900, 4096)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", SHAPES)
def test_forward_and_backward(swz, dtype, m, n):
    x, w, b, dy = inputs(m, n, dtype, torch.float32 if m % 2 else dtype)
    want = formula(x, w, b, 1e-5, dy)
    for extra, offset in ((0, 0), (3, 1)):
        xv, dv = (spaced(x, extra, offset), spaced(dy, extra + 2, offset)) if extra else (x, dy)
        y, mean, rstd = swz.layer_norm_forward(xv, w, b, 1e-5)
        assert y.dtype == dtype and mean.dtype == rstd.dtype == torch.float32
        dx, dw, db = swz.layer_norm_backward(dv, xv, w, mean, rstd)
        assert dx.dtype == dtype and dw.dtype == db.dtype == torch.float32
        for name, got in (("y", y), ("mean", mean), ("rstd", rstd), ("dx", dx), ("dw", dw), ("db", db)):
            within(got, *want[name])
        again = swz.layer_norm_backward(dv, xv, w, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", [(5, 300), (6, 1999), (3, 4100), (2, 17000)])
def test_types_and_options(swz, dtype, m, n):
    for wtype in TYPES:
        x, w, b, _ = inputs(m, n, dtype, wtype)
        for out_dtype in TYPES:
            for wv, bv in ((w, b), (None, b), (w, None), (None, None)):
                y, mean, rstd = swz.layer_norm_forward(x, wv, bv, 0.1, out_dtype=out_dtype)
                assert y.dtype == out_dtype
                within(y, *formula(x, wv, bv, 0.1)["y"])
            dy = torch.randn((m, n), generator=gen(3), device="cuda").to(out_dtype)
            want = formula(x, w, None, 0.1, dy)
            dx, dw, db = swz.layer_norm_backward(dy, x, w, mean, rstd, dx_dtype=out_dtype, dw_dtype=wtype)
            assert dx.dtype == out_dtype and dw.dtype == db.dtype == wtype
            for name, got in (("dx", dx), ("dw", dw), ("db", db)):
                within(got, *want[name])
            for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (0, 0, 0)):
                some = swz.layer_norm_backward(dy, x, w, mean, rstd, need_dx=need[0], need_dw=need[1],
                                               need_db=need[2], dx_dtype=out_dtype, dw_dtype=wtype)
                for got, full, asked in zip(some, (dx, dw, db), need):
                    assert torch.equal(got, full) if asked else got is None


@pytest.mark.parametrize("n", [40, 700, 1999, 9000, 20000])
def test_far_from_zero_and_constant_rows(swz, n):
    """The variance of rows far from zero, of constant rows, and of tiny values."""
    x, w, b, dy = inputs(6, n, torch.float32, torch.float32, shift=1000.0)
    x[2] = 3.25
    x[3] = 0.0
    x[4] *= 1e-20
    want = formula(x, w, b, 1e-5, dy)
    y, mean, rstd = swz.layer_norm_forward(x, w, b, 1e-5)
    dx, dw, db = swz.layer_norm_backward(dy, x, w, mean, rstd)
    for name, got in (("y", y), ("dx", dx), ("dw", dw), ("db", db)):
        within(got, *want[name])
    assert torch.equal(y[3], b) and torch.isfinite(rstd).all()


def test_bad_rows_stay_alone(swz):
    for n in (50, 1500, 5000, 17000):
        x, w, b, dy = inputs(9, n, torch.float32, torch.float32)
        good = swz.layer_norm_forward(x, w, b)
        gx = swz.layer_norm_backward(dy, x, w, *good[1:])[0]
        x[1, n - 1], x[4, 0] = float("nan"), float("inf")
        y, mean, rstd = swz.layer_norm_forward(x, w, b)
        dx, dw, _ = swz.layer_norm_backward(dy, x, w, mean, rstd)
        assert torch.isnan(y[[1, 4]]).all() and torch.isnan(dx[[1, 4]]).all()
        keep = [0, 2, 3, 5, 6, 7, 8]
        assert torch.equal(y[keep], good[0][keep]) and torch.equal(dx[keep], gx[keep])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [63, 1000, 1999, 4096, 16500])
def test_out(swz, dtype, n):
    """Results in rows that start anywhere and over x itself; what lies beside stays."""
    m = 11
    x, w, b, _ = inputs(m, n, dtype, dtype)
    want = swz.layer_norm_forward(x, w, b)[0]
    for extra, offset in ((0, 0), (5, 3), (8 - n % 8, 0), (1, 8)):
        flat = torch.full((offset + m * (n + extra) + 40,), 7.0, dtype=dtype, device="cuda")
        out = flat[offset:offset + m * (n + extra)].view(m, n + extra)[:, :n]
        assert swz.layer_norm_forward(x, w, b, out=out)[0] is out
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert (flat == 7.0).all()
    for v in (x.clone(), spaced(x, 3, 1)):
        swz.layer_norm_forward(v, w, b, out=v)
        assert torch.equal(v, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [300, 1000, 1999, 4096, 9000, 17000])
def test_gradient_over_its_inputs(swz, dtype, n):
    """dx over x or over dy (C entry point): the same bits, dw and db among them."""
    m = 70
    x, w, _, dy = inputs(m, n, dtype, torch.float32)
    code = {torch.bfloat16: swz.SWZ_BF16, torch.float16: swz.SWZ_F16, torch.float32: swz.SWZ_F32}[dtype]
    _, mean, rstd = swz.layer_norm_forward(x, w)
    want = swz.layer_norm_backward(dy, x, w, mean, rstd)
    rc, need = swz.swz_layer_norm_backward_workspace_size(m, n)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for over in (0, 1):
        a, b = x.clone(), dy.clone()
        to = (a, b)[over]
        dw, db = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        assert swz.swz_layer_norm_backward(
            b.data_ptr(), code, n, a.data_ptr(), code, n, w.data_ptr(), swz.SWZ_F32, mean.data_ptr(),
            rstd.data_ptr(), to.data_ptr(), code, n, dw.data_ptr(), db.data_ptr(), swz.SWZ_F32, m, n,
            ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == swz.SWZ_OK
        for got, exact in zip((to, dw, db), want):
            assert torch.equal(got, exact)


def test_empty(swz):
    w = torch.ones(16, device="cuda")
    y, mean, rstd = swz.layer_norm_forward(torch.empty((0, 16), device="cuda"), w)
    assert y.shape == (0, 16) and mean.shape == rstd.shape == (0,)
    dx, dw, db = swz.layer_norm_backward(y, y, w, mean, rstd)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()
    y, mean, rstd = swz.layer_norm_forward(torch.empty((4, 0), device="cuda"))
    assert y.shape == (4, 0)
    x = torch.empty((0, 16), device="cuda", requires_grad=True)
    swz.layer_norm(x, w).sum().backward()
    assert x.grad.shape == (0, 16)


@pytest.mark.parametrize("dtype", TYPES)
def test_autograd(swz, dtype):
    """The form with a gradient against autograd of the formula in 64 bits, for inputs of
    more dimensions, transposed ones, and an expanded gradient."""
    g = gen(5)
    base = torch.randn((3, 200, 7), generator=g, device="cuda").to(dtype)
    w = (1 + 0.1 * torch.randn(200, generator=g, device="cuda")).requires_grad_()
    b = torch.randn(200, generator=g, device="cuda").to(dtype).requires_grad_()
    for dy in (torch.randn((3, 7, 200), generator=g, device="cuda").to(dtype),
               torch.ones((), device="cuda", dtype=dtype).expand(3, 7, 200)):
        x = base.clone().requires_grad_()
        w.grad = b.grad = None
        y = swz.layer_norm(x.transpose(1, 2), w, b, 1e-3)
        y.backward(dy)
        want = formula(base.transpose(1, 2).reshape(21, 200), w.detach(), b.detach(), 1e-3,
                       dy.reshape(21, 200))
        within(y.detach().reshape(21, 200), *want["y"])
        within(x.grad.transpose(1, 2).reshape(21, 200), *want["dx"])
        within(w.grad, *want["dw"])
        within(b.grad, *want["db"])
        assert w.grad.dtype == torch.float32 and b.grad.dtype == dtype
    x = base.clone().requires_grad_()  # over the last dimension, 7, without weight and bias
    swz.layer_norm(x).backward(torch.ones_like(base))
    within(x.grad.reshape(600, 7), *formula(base.reshape(600, 7), None, None, 1e-5,
                                            torch.ones_like(base).reshape(600, 7))["dx"])


def test_gradient_against_differences(swz):
    """Central differences of the formula in 64 bits along random directions: step 1e-4
    leaves 1e-8 of truncation and 1e-12 of rounding, the kernel 100 u, relative to the
    norms of the parts."""
    m, n = 6, 777
    x, w, b, dy = inputs(m, n, torch.float32, torch.float32)
    y, mean, rstd = swz.layer_norm_forward(x, w, b, 1e-5)
    grads = swz.layer_norm_backward(dy, x, w, mean, rstd)

    def loss(xd, wd, bd):
        return (formula(xd, wd, bd, 1e-5)["y"][0] * dy.double()).sum().item()
    args = [t.double() for t in (x, w, b)]
    for i, grad in enumerate(grads):
        v = torch.randn(args[i].shape, generator=gen(i), device="cuda", dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-4 * v, args[i] - 1e-4 * v
        diff = (loss(*up) - loss(*down)) / 2e-4
        along = (grad.double() * v).sum().item()
        assert abs(diff - along) <= 2e-5 * (grad.double() * v).abs().sum().item() + 1e-6


def test_second_derivative_raises(swz):
    x = torch.randn((4, 32), device="cuda", requires_grad=True)
    (gx,) = torch.autograd.grad(swz.layer_norm(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()


@pytest.mark.parametrize("m,n", [(1, 4096), (300, 1000), (64, 20000)])
def test_graph_and_streams(swz, m, n):
    x, w, b, dy = inputs(m, n, torch.bfloat16, torch.float32)
    out = {}

    def call():
        y, mean, rstd = swz.layer_norm_forward(x, w, b)
        out["all"] = (y, *swz.layer_norm_backward(dy, x, w, mean, rstd))
    g1 = capture_graph(call)
    first = out["all"]
    g2 = capture_graph(call)
    x2, _, _, dy2 = inputs(m, n, torch.bfloat16, torch.float32, seed=9)
    x.copy_(x2)
    dy.copy_(dy2)
    y, mean, rstd = swz.layer_norm_forward(x2, w, b)
    want = (y, *swz.layer_norm_backward(dy2, x2, w, mean, rstd))
    g1.replay()
    g2.replay()
    for got in (first, out["all"]):
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = swz.layer_norm_forward(x, w, b, stream=side)
    got = (y, *swz.layer_norm_backward(dy, x, w, mean, rstd, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
