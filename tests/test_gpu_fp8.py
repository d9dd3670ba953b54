"""8-bit linear layers: the block quantiser bit for bit, the products against
64-bit sums of the same 8-bit values, the layer's gradient against the formula
and against differences, and what the entry points refuse.

Tolerances of the products, from the arithmetic: the products of 8-bit values
are exact in fp32; a block of 128 is summed in four steps of 32 and scaled
(two roundings), the blocks are added in turn.  Each of these (KB + 16)
roundings is at most 2^-23 of the sum of magnitudes S = sum |a| |b|, and the
result is rounded once to its type (2^-8 for bf16, 2^-11 for fp16)."""
import numpy as np
import pytest
import torch

from gpu_util import capture_graph, require_gpu

pytestmark = pytest.mark.gpu

F_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
F_TYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


def rand(shape, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x *= torch.exp(torch.randn((shape[0], 1), generator=g))
    return x.to(dtype)


def ref_quant(x, block, fmt):
    """The rule on the CPU, block by block: (q as fp32 values, scales)."""
    x = x.float().cpu()
    M, K = x.shape
    F = torch.tensor(F_MAX[fmt])
    kb, mb = -(-K // 128), -(-M // 128)
    q = torch.zeros_like(x)
    s = torch.zeros((mb, kb) if block == "square" else (kb, M))
    for j in range(kb):
        c = slice(128 * j, min(K, 128 * j + 128))
        for i in range(mb if block == "square" else 1):
            r = slice(128 * i, min(M, 128 * i + 128)) if block == "square" else slice(0, M)
            a = x[r, c].abs()
            ac = (a.max().reshape(1, 1) if block == "square" else a.amax(1, keepdim=True))
            ac = torch.maximum(ac, torch.tensor(2.0 ** -96))
            q[r, c] = (x[r, c] * (F / ac)).clamp(-F, F).to(F_TYPE[fmt]).float()
            if block == "square":
                s[i, j] = (ac / F)[0, 0]
            else:
                s[j] = (ac / F)[:, 0]
    return q, s


def values(q, s, block):
    """64-bit values of an 8-bit matrix."""
    q, s = q.cpu().double(), s.cpu().double()
    M, K = q.shape
    if block == "row":
        return q * s.t().repeat_interleave(128, 1)[:, :K]
    return q * s.repeat_interleave(128, 0).repeat_interleave(128, 1)[:M, :K]


def check_product(C, A, B):
    want = (A @ B.t()).numpy()
    S = (A.abs() @ B.abs().t()).numpy()
    kb = -(-A.shape[1] // 128)
    tol = (kb + 16) * 2.0 ** -23 * S + ROUND[C.dtype] * np.abs(want) * 1.01
    if C.dtype == torch.float16:
        tol = tol + 2.0 ** -24  # subnormal results
    err = np.abs(C.cpu().double().numpy() - want)
    assert (err <= tol).all(), (err.max(), (err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (128, 128), (129, 127), (77, 1000), (300, 16),
                                   (256, 640), (1, 4099)])
def test_quantize_bit_exact(swz, shape, dtype, block, fmt):
    x = rand(shape, dtype, sum(shape))
    q, s, qt, st = swz.quantize_fp8(x.cuda(), block, fmt, True)
    for got, gs, src in ((q, s, x), (qt, st, x.t())):
        wq, ws = ref_quant(src, block, fmt)
        assert torch.equal(gs.cpu(), ws)
        assert torch.equal(got.float().cpu(), wq)
    q2, s2 = swz.quantize_fp8(x.cuda(), block, fmt)
    assert torch.equal(q2.float(), q.float()) and torch.equal(s2, s)


@pytest.mark.parametrize("block", ["row", "square"])
def test_quantize_strided_and_odd_alignment(swz, block):
    big = rand((200, 1000), torch.bfloat16, 3).cuda()
    for x in (big[3:150, 7:560], big[:, :512], big[::2, 8:300], big[5:6, 1:900]):
        q, s, qt, st = swz.quantize_fp8(x, block, "e4m3", True)
        wq, ws = ref_quant(x, block, "e4m3")
        wqt, wst = ref_quant(x.t(), block, "e4m3")
        assert torch.equal(q.float().cpu(), wq) and torch.equal(s.cpu(), ws)
        assert torch.equal(qt.float().cpu(), wqt) and torch.equal(st.cpu(), wst)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_zeros_tiny_and_not_finite(swz, dtype):
    x = torch.zeros((4, 512), dtype=dtype)
    x[0, 130] = 1e-30           # below 2^-96: the bound's scale
    x[1, 5], x[1, 6] = float("inf"), 1.0
    x[2, 300], x[2, 301] = float("nan"), 2.0
    x[3, 400] = -torch.finfo(dtype).max
    q, s = swz.quantize_fp8(x.cuda(), "row")
    back = values(q.float(), s, "row")
    wq, ws = ref_quant(x, "row", "e4m3")
    assert torch.equal(s.cpu().isnan(), ws.isnan())
    assert torch.equal(s.cpu().nan_to_num(nan=-1.0), ws.nan_to_num(nan=-1.0))
    assert torch.equal(q.float().cpu().isnan(), wq.isnan())
    assert (back[0, :128] == 0).all() and (s[0] > 0).all()
    assert not back[1, 5].isfinite() and back[2, 256:384].isnan().all()
    assert back[3, 400] == -torch.finfo(dtype).max or abs(
        back[3, 400] / -torch.finfo(dtype).max - 1) < 1e-6
    assert back[2, :256].isfinite().all()


# tile and split variants, forms, types, ragged edges
@pytest.mark.parametrize("b_block", ["square", "row"])
@pytest.mark.parametrize("M,N,K,cfg", [
    (1, 1, 1, {}), (128, 128, 128, dict(tile=128)), (256, 256, 512, dict(tile=256)),
    (130, 257, 1000, dict(tile=128)), (300, 520, 1999, dict(tile=256)),
    (77, 200, 2048, dict(tile=128, split_k=8)), (200, 140, 1100, dict(tile=128, split_k=4)),
    (129, 300, 333, dict(tile=128, split_k=2)), (513, 1111, 600, {}),
    (700, 900, 384, dict(tile=256, num_programs=4)), (700, 900, 384, dict(tile=128, num_programs=5)),
    (1, 300, 200, {}), (16, 129, 2000, {}), (17, 1000, 1100, {}), (33, 500, 5000, {}), (64, 257, 640, {}),
    (5, 200, 1100, dict(split_k=8)), (40, 4100, 300, dict(split_k=1)), (64, 64, 3000, dict(split_k=4)),
])
def test_gemm_fp8(swz, M, N, K, cfg, b_block):
    a, b = rand((M, K), torch.float32, M + K).cuda(), rand((N, K), torch.float32, N + 7).cuda()
    qa, sa = swz.quantize_fp8(a, "row")
    qb, sb = swz.quantize_fp8(b, b_block)
    A, B = values(qa.float(), sa, "row"), values(qb.float(), sb, b_block)
    for dtype in (torch.float32, torch.bfloat16):
        C = swz.gemm_fp8(qa, sa, qb, sb, b_block=b_block, out_dtype=dtype, **cfg)
        swz.check_status()
        check_product(C, A, B)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("tile", [128, 256])
def test_gemm_fp8_formats(swz, fa, fb, tile):
    a, b = rand((200, 700), torch.float32, 1).cuda(), rand((300, 700), torch.float32, 2).cuda()
    (qa, sa), (qb, sb) = swz.quantize_fp8(a, "row", fa), swz.quantize_fp8(b, "square", fb)
    C = swz.gemm_fp8(qa, sa, qb, sb, out_dtype=torch.float32, tile=tile)
    swz.check_status()
    check_product(C, values(qa.float(), sa, "row"), values(qb.float(), sb, "square"))


@pytest.mark.parametrize("order,group", [("row", 1), ("col", 1), ("panel", 3), ("serpentine", 2),
                                         ("morton", 1), ("xor", 1)])
def test_gemm_fp8_orders_agree(swz, order, group):
    a, b = rand((1024, 512), torch.float32, 1).cuda(), rand((1024, 512), torch.float32, 2).cuda()
    (qa, sa), (qb, sb) = swz.quantize_fp8(a), swz.quantize_fp8(b, "square")
    want = swz.gemm_fp8(qa, sa, qb, sb, out_dtype=torch.float32, tile=128, split_k=1)
    got = swz.gemm_fp8(qa, sa, qb, sb, out_dtype=torch.float32, tile=128, split_k=1, order=order,
                       group=group)
    assert torch.equal(got, want)


@pytest.mark.parametrize("ld,off", [(264, 0), (257, 0), (272, 4), (300, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cfg", [dict(tile=256), dict(tile=128), dict(tile=128, split_k=2)])
def test_gemm_fp8_output_strides(swz, ld, off, dtype, cfg):
    M, N, K = 140, 250, 300
    a, b = rand((M, K), torch.float32, 5).cuda(), rand((N, K), torch.float32, 6).cuda()
    (qa, sa), (qb, sb) = swz.quantize_fp8(a), swz.quantize_fp8(b, "square")
    buf = torch.full((M + 1, ld), 7.0, dtype=dtype, device="cuda")
    out = buf[:M, off:off + N]
    swz.gemm_fp8(qa, sa, qb, sb, out=out, **cfg)
    swz.check_status()
    want = swz.gemm_fp8(qa, sa, qb, sb, out_dtype=dtype, **cfg)
    assert torch.equal(out, want)
    buf[:M, off:off + N] = 7.0
    assert (buf == 7.0).all()


def test_gemm_fp8_not_finite_stays_in_its_row(swz):
    a, b = rand((150, 300), torch.float32, 5), rand((140, 300), torch.float32, 6)
    a[20, 10], a[30, 200] = float("inf"), float("nan")
    (qa, sa), (qb, sb) = swz.quantize_fp8(a.cuda()), swz.quantize_fp8(b.cuda(), "square")
    for cfg in (dict(tile=128), dict(tile=256), dict(split_k=2)):
        C = swz.gemm_fp8(qa, sa, qb, sb, out_dtype=torch.float32, **cfg).cpu()
        bad = ~C.isfinite()
        assert bad[20].all() and bad[30].all() and bad.sum() == 2 * 140


def test_gemm_fp8_padding_is_not_read(swz):
    # bytes beyond K in the rows' padding hold NaN
    qa, sa = swz.quantize_fp8(rand((40, 100), torch.float32, 1).cuda())
    qb, sb = swz.quantize_fp8(rand((50, 100), torch.float32, 2).cuda(), "square")
    want = swz.gemm_fp8(qa, sa, qb, sb, out_dtype=torch.float32)
    pa = torch.full((40, 112), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    pb = torch.full((50, 112), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    pa[:, :100], pb[:, :100] = qa, qb
    got = swz.gemm_fp8(pa[:, :100], sa, pb[:, :100], sb, out_dtype=torch.float32)
    assert torch.equal(got, want)
    x = rand((3, 100), torch.bfloat16, 4).cuda()
    assert torch.equal(swz.linear_fp8(x, pb[:, :100], sb), swz.linear_fp8(x, qb, sb))


@pytest.mark.parametrize("w_block,fmt", [("square", "e4m3"), ("row", "e4m3"), ("square", "e5m2")])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 128), (1, 4096, 4096), (3, 100, 77),
                                   (8, 1000, 1999), (9, 130, 5000), (16, 515, 640), (17, 515, 640),
                                   (100, 300, 1000), (2, 700, 9000), (16, 40, 14000), (5, 5000, 300)])
def test_linear_fp8(swz, M, N, K, w_block, fmt):
    for dtype, out in ((torch.bfloat16, None), (torch.float16, torch.float32),
                       (torch.float32, torch.bfloat16)):
        x = rand((M, K), dtype, M + N)
        qw, sw = swz.quantize_fp8(rand((N, K), torch.float32, K).cuda(), w_block, fmt)
        y = swz.linear_fp8(x.cuda(), qw, sw, w_block=w_block, out_dtype=out)
        swz.check_status()
        qx, sx = ref_quant(x, "row", "e4m3")
        check_product(y, values(qx, sx, "row"), values(qw.float(), sw, w_block))


def test_linear_fp8_strided(swz):
    big = rand((40, 700), torch.bfloat16, 9).cuda()
    qw, sw = swz.quantize_fp8(rand((200, 333), torch.float32, 1).cuda(), "square")
    for x in (big[:9, 5:338], big[:30, 8:341], big[1:20:3, :333]):
        assert torch.equal(swz.linear_fp8(x, qw, sw), swz.linear_fp8(x.contiguous(), qw, sw))


@pytest.mark.parametrize("M,N,K", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (40, 7, 0)])
def test_empty(swz, M, N, K):
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((N, K), dtype=torch.bfloat16, device="cuda")
    qx, sx, _, _ = swz.quantize_fp8(x, transposed=True)
    qw, sw = swz.quantize_fp8(w, "square")
    for y in (swz.gemm_fp8(qx, sx, qw, sw), swz.linear_fp8(x, qw, sw)):
        assert y.shape == (M, N) and (y == 0).all()


@pytest.mark.parametrize("M,N,K", [(200, 300, 260), (1, 128, 64), (129, 65, 130)])
def test_layer_gradient_formula(swz, M, N, K):
    x, w, dy = (rand((M, K), torch.bfloat16, 1), rand((N, K), torch.bfloat16, 2),
                rand((M, N), torch.bfloat16, 3))
    xg, wg = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = swz.fp8_linear(xg, wg)
    y.backward(dy.cuda())
    v = lambda t, b: values(*ref_quant(t, b, "e4m3"), b)  # noqa: E731
    check_product(y.detach(), v(x, "row"), v(w, "square"))
    check_product(xg.grad, v(dy, "row"), v(w, "square").t())
    check_product(wg.grad, v(dy.t(), "row"), v(x.t(), "row"))
    _, saved = swz.linear_fp8_forward(x.cuda(), w.cuda())
    dx, dw = swz.linear_fp8_backward(dy.cuda(), saved)
    assert dw.dtype == torch.float32 and torch.equal(dx, xg.grad)
    assert torch.equal(dw.to(torch.bfloat16), wg.grad)
    assert swz.linear_fp8_backward(dy.cuda(), saved, need_dx=False)[0] is None


def test_layer_gradient_differences(swz):
    # On values that 8 bits hold exactly (small integers, a power-of-two
    # largest magnitude times 1.75 = 448 / 256 in every block) quantisation is
    # the identity, the layer is linear, and differences give its gradient.
    g = torch.Generator().manual_seed(0)

    def exact(shape):
        t = torch.randint(-3, 4, shape, generator=g).float()
        t[::1, ::128] = 7.0
        t[::128, :] = 7.0
        return t
    M, N, K = 160, 140, 150
    x, w, dy = exact((M, K)), exact((N, K)), exact((M, N))
    y, saved = swz.linear_fp8_forward(x.cuda(), w.cuda(), out_dtype=torch.float32)
    dx, dw = swz.linear_fp8_backward(dy.cuda(), saved, dx_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), x.double() @ w.double().t())
    loss = lambda a, b: ((a.double() @ b.double().t()) * dy.double()).sum().item()  # noqa: E731
    for i, j in ((0, 0), (17, 130), (159, 149)):
        e = torch.zeros_like(x)
        e[i, j] = 1.0
        assert dx[i, j].item() == (loss(x + e, w) - loss(x - e, w)) / 2
    for i, j in ((0, 0), (139, 149), (65, 3)):
        e = torch.zeros_like(w)
        e[i, j] = 1.0
        assert dw[i, j].item() == (loss(x, w + e) - loss(x, w - e)) / 2


def test_streams_graph_and_repeat(swz):
    x = rand((300, 512), torch.bfloat16, 1).cuda()
    w = rand((400, 512), torch.bfloat16, 2).cuda()
    qw, sw = swz.quantize_fp8(w, "square")
    want = swz.linear_fp8(x, qw, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [swz.linear_fp8(x, qw, sw, stream=side) for _ in range(20)]
    side.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.empty_like(want)
    xs = x.clone()
    g = capture_graph(lambda: swz.linear_fp8(xs, qw, sw, out=out))
    x2 = rand((300, 512), torch.bfloat16, 5).cuda()
    xs.copy_(x2)
    g.replay()
    assert torch.equal(out, swz.linear_fp8(x2, qw, sw))


def test_timeout_is_reported(swz):
    (qa, sa) = swz.quantize_fp8(rand((300, 512), torch.bfloat16, 1).cuda())
    (qb, sb) = swz.quantize_fp8(rand((300, 512), torch.bfloat16, 2).cuda(), "square")
    want = swz.gemm_fp8(qa, sa, qb, sb)
    few = swz.quantize_fp8(rand((9, 512), torch.bfloat16, 3).cuda())
    for split in (1, 2):
        want_few = swz.gemm_fp8(*few, qb, sb, split_k=split)
        swz.gemm_fp8(*few, qb, sb, split_k=split, debug_flags=swz.SWZ_DEBUG_SKIP_FIRST_LOAD,
                     timeout_ms=50)
        with pytest.raises(swz.SwzError) as e:
            swz.check_status()
        assert e.value.code == swz.SWZ_ETIMEOUT
        assert torch.equal(swz.gemm_fp8(*few, qb, sb, split_k=split), want_few)
    for cfg in (dict(tile=128), dict(tile=256), dict(tile=128, split_k=2)):
        swz.gemm_fp8(qa, sa, qb, sb, debug_flags=swz.SWZ_DEBUG_SKIP_FIRST_LOAD, timeout_ms=50, **cfg)
        with pytest.raises(swz.SwzError) as e:
            swz.check_status()
        assert e.value.code == swz.SWZ_ETIMEOUT
        swz.check_status()
        assert torch.equal(swz.gemm_fp8(qa, sa, qb, sb), want)


def test_refusals(swz):
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    q, s = swz.quantize_fp8(x)
    qs, ss = swz.quantize_fp8(x, "square")
    with pytest.raises(TypeError):
        swz.quantize_fp8(x.int())
    with pytest.raises(ValueError):
        swz.quantize_fp8(x.t())
    with pytest.raises(ValueError):
        swz.quantize_fp8(x, "column")
    with pytest.raises(ValueError):
        swz.quantize_fp8(x, fmt="e3m4")
    with pytest.raises(ValueError):
        swz.quantize_fp8(x.cpu())
    with pytest.raises(ValueError):
        swz.gemm_fp8(q, s, qs, s)                      # scales of the wrong shape
    with pytest.raises(TypeError):
        swz.gemm_fp8(x, s, qs, ss)
    with pytest.raises(ValueError):
        swz.gemm_fp8(q, s, *swz.quantize_fp8(x[:, :64].contiguous(), "square"))
    with pytest.raises(ValueError):
        swz.gemm_fp8(q, s, qs, ss, out=torch.empty((4, 5), device="cuda"))
    with pytest.raises(TypeError):
        swz.gemm_fp8(q, s, qs, ss, out_dtype=torch.int32)
    odd = torch.zeros((4, 200), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        swz.gemm_fp8(odd[:, 1:129], s, qs, ss)         # rows not on 16 bytes
    for kw in (dict(tile=64), dict(split_k=3), dict(tile=256, split_k=2), dict(split_k=4)):
        with pytest.raises(swz.SwzError) as e:
            swz.gemm_fp8(q, s, qs, ss, **kw)
        assert e.value.code == swz.SWZ_EUNSUPPORTED
    with pytest.raises(swz.SwzError) as e:
        swz.gemm_fp8(q, s, qs, ss, order="panel", group=0)
    assert e.value.code == swz.SWZ_EINVAL
    y, saved = swz.linear_fp8_forward(x, x)
    with pytest.raises(ValueError):
        swz.linear_fp8_backward(x, saved)


def test_second_derivative_is_refused(swz):
    """The gradient is made of the library's calls, which torch cannot differentiate."""
    x = torch.randn(40, 64, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(48, 64, device="cuda").bfloat16().requires_grad_()
    dx, = torch.autograd.grad(swz.fp8_linear(x, w).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.float().sum().backward()


def test_layer_checks_its_operands(swz):
    x = torch.randn(40, 64, device="cuda").bfloat16()
    w = torch.randn(48, 64, device="cuda").bfloat16()
    with pytest.raises(ValueError):
        swz.linear_fp8_forward(x, w[:, :48].contiguous())
    with pytest.raises(TypeError):
        swz.linear_fp8_forward(x, w, out_dtype=torch.float64)
    y, saved = swz.linear_fp8_forward(x, w)
    with pytest.raises(ValueError):
        swz.linear_fp8_backward(y[:, :40].contiguous(), saved)
    qxt, sxt, qwt, swt = saved
    with pytest.raises(ValueError):
        swz.linear_fp8_backward(y, (qxt, sxt[:, :63], qwt, swt))


def far(rows, cols, dtype, elements):
    """Uninitialised (rows, cols) view whose last row starts `elements` into its buffer."""
    stride = -(-elements // ((rows - 1) * 64)) * 64
    flat = torch.empty((rows - 1) * stride + cols, dtype=dtype, device="cuda")
    return flat.as_strided((rows, cols), (stride, 1))


@pytest.mark.parametrize("block", ["row", "square"])
def test_quantize_far_rows(swz, block):
    """Rows further apart than 32 bits reach, in elements as in bytes."""
    x = torch.randn(150, 300, device="cuda").bfloat16()
    v = far(150, 300, x.dtype, 2 ** 32 + 1000)
    v.copy_(x)
    for got, want in zip(swz.quantize_fp8(v, block, transposed=True),
                         swz.quantize_fp8(x, block, transposed=True)):
        assert torch.equal(got.view(torch.uint8) if got.element_size() == 1 else got,
                           want.view(torch.uint8) if want.element_size() == 1 else want)


@pytest.mark.parametrize("M,cfg", [(300, dict(tile=256)), (300, dict(tile=128)),
                                   (300, dict(tile=128, split_k=2)), (17, dict()),
                                   (17, dict(split_k=2))])
def test_gemm_fp8_far_rows(swz, M, cfg):
    qa, sa = swz.quantize_fp8(torch.randn(M, 500, device="cuda"))
    qb, sb = swz.quantize_fp8(torch.randn(260, 500, device="cuda"), "square")
    want = swz.gemm_fp8(qa, sa, qb, sb, **cfg)
    a = far(M, 500, torch.uint8, 2 ** 32 + 1000).view(qa.dtype)
    a.view(torch.uint8).copy_(qa.view(torch.uint8))
    out = far(M, 260, torch.bfloat16, 2 ** 31 + 1000)
    swz.gemm_fp8(a, sa, qb, sb, out=out, **cfg)
    swz.check_status()
    assert torch.equal(out, want)
