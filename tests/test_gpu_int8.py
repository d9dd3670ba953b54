"""8-bit integer operators on the GPU against their definition in 64 bits.

Everything but the result's last rounding is exact or a stated sequence of fp32
roundings, so the comparisons are of bits: q = the exact product x r rounded to
the nearest whole number; C = fl(fl32(S) * fl32(sa sb)) rounded to C's type, with
the whole number S from a product in 64 bits (|S| < 2^53)."""
import pytest
import torch

from gpu_util import capture_graph, require_gpu

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def swz():
    return require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def bits(a, b):
    """Whether a and b are the same, NaN included."""
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(
        torch.nan_to_num(a.float(), nan=12345.0), torch.nan_to_num(b.float(), nan=12345.0))


def rows_of(x, swz_ld=0, offset=0):
    """x in rows of `swz_ld` elements that start `offset` elements into their memory."""
    m, k = x.shape
    ld = swz_ld or k
    flat = torch.full((offset + m * ld + 64,), float("nan"), dtype=x.dtype, device="cuda")
    v = flat[offset:offset + m * ld].view(m, ld)[:, :k]
    v.copy_(x)
    return v


def exact_q(x):
    ac = x.float().abs().amax(1).clamp_min(2.0 ** -96) if x.shape[1] else torch.full(
        (x.shape[0],), 2.0 ** -96, device="cuda")
    bad = ~torch.isfinite(ac)
    top = torch.full_like(ac, 127.0)
    q = torch.round(x.double() * (top / ac).double().unsqueeze(1))
    q = torch.where(bad.unsqueeze(1), torch.zeros_like(q), q).to(torch.int8)
    return q, torch.where(bad, torch.full_like(ac, float("nan")), ac / top)


def int8_rows(swz, m, k, seed, low=-128):
    q = swz.int8_empty(m, k)
    q.copy_(torch.randint(low, 128, (m, k), generator=gen(seed), device="cuda", dtype=torch.int32))
    s = torch.exp(torch.randn(m, generator=gen(seed + 1), device="cuda") - 4)
    return q, s


def exact_c(a, sa, b, sb, dtype):
    s = a.double() @ b.double().t()
    return (s.float() * (sa.unsqueeze(1) * sb.unsqueeze(0))).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (1, 8), (9, 255), (2, 257), (77, 1000), (8, 1024),
                                 (5, 1025), (4, 4096), (3, 4099), (2, 16384), (2, 16387), (1, 40001),
                                 (300, 129)])
def test_quantize(swz, dtype, m, k):
    x = torch.randn((m, k), generator=gen(m * k), device="cuda").to(dtype)
    for v in (x, rows_of(x, k + 3, 1), rows_of(x, (k + 15) // 8 * 8, 0)):
        q, s = swz.quantize_int8(v)
        want, ws = exact_q(x)
        assert q.dtype == torch.int8 and q.data_ptr() % 16 == 0
        assert torch.equal(q, want) and bits(s, ws)


@pytest.mark.parametrize("k", [1, 7, 8, 13, 250, 1029, 4099, 16390])
def test_quantize_leaves_what_is_beside(swz, k):
    m, ld = 3, (k + 15) // 16 * 16 + 16
    x = torch.randn((m, k), generator=gen(k), device="cuda")
    q = torch.full((m, ld), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(m, device="cuda")
    assert swz.swz_quantize_int8(x.data_ptr(), swz.SWZ_F32, k, m, k, q.data_ptr(), ld, s.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream) == swz.SWZ_OK
    assert torch.equal(q[:, :k], exact_q(x)[0]) and (q[:, k:] == 99).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_values(swz, dtype):
    """Ties, the largest and smallest magnitudes, zeros, infinities and NaN."""
    k = 254
    x = torch.zeros((10, k), dtype=torch.float64, device="cuda")
    x[0] = torch.arange(k, device="cuda") / 2 - 63.5  # ties at every second value: amax 63.5, r = 2
    x[1, 5] = torch.finfo(dtype).max
    x[2, 7] = -torch.finfo(dtype).tiny
    x[3] = 1.0
    x[5, 3], x[5, 4] = float("inf"), 1.0
    x[6, 200] = float("nan")
    x[7, 0], x[7, 1] = float("-inf"), float("nan")
    x[8] = -0.0
    x[9] = torch.linspace(-1, 1, k, device="cuda", dtype=torch.float64) * 2.0 ** -100
    x = x.to(dtype)
    q, s = swz.quantize_int8(x)
    want, ws = exact_q(x)
    assert torch.equal(q, want) and bits(s, ws)
    assert torch.isnan(s[5:8]).all() and not q[5:8].any()
    assert torch.isnan(swz.gemm_int8(q, s, q[3:4], s[3:4], out_dtype=torch.float32)[5:8]).all()


SHAPES = [(1, 1, 1), (1, 1, 0), (1, 5, 16), (2, 130, 17), (7, 300, 100), (13, 1000, 4096), (32, 257, 1024),
          (33, 64, 1025), (64, 4096, 2048), (65, 129, 3000), (100, 1, 500), (128, 128, 64), (129, 255, 2047),
          (256, 256, 8192), (333, 1111, 1999), (1000, 520, 5000), (2048, 2048, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm(swz, m, n, k):
    a, sa = int8_rows(swz, m, k, 1)
    b, sb = int8_rows(swz, n, k, 7)
    for dtype in TYPES:
        assert bits(swz.gemm_int8(a, sa, b, sb, out_dtype=dtype), exact_c(a, sa, b, sb, dtype)), dtype
    swz.check_status()


@pytest.mark.parametrize("tile,split", [(128, 1), (128, 2), (128, 4), (128, 8), (256, 0)])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1100), (130, 260, 2500), (300, 513, 4096), (700, 900, 1030)])
def test_gemm_tiles(swz, tile, split, m, n, k):
    a, sa = int8_rows(swz, m, k, 3)
    b, sb = int8_rows(swz, n, k, 4)
    for order, group in (("serpentine", 8), ("row", 1), ("panel", 2)):
        c = swz.gemm_int8(a, sa, b, sb, tile=tile, split_k=split, order=order, group=group)
        assert bits(c, exact_c(a, sa, b, sb, torch.bfloat16))
    swz.check_status()


@pytest.mark.parametrize("split", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1100), (1, 4096, 4096), (8, 1000, 1024), (9, 3, 20000), (16, 10240, 1500),
                                   (17, 2000, 4100), (33, 6000, 1111), (64, 129, 8192), (64, 50000, 1030),
                                   (2, 100000, 1200), (30, 90001, 1024)])
def test_few_rows(swz, m, n, k, split):
    """Tiles that one or several CTAs share, several of them a CTA, and ragged ones."""
    a, sa = int8_rows(swz, m, k, 3)
    b, sb = int8_rows(swz, n, k, 4)
    want = exact_c(a, sa, b, sb, torch.bfloat16)
    # of tile 64 the sums of each 1024 of K have columns of their own for each row (whole
    # sixteens of them), 256 in all; a part of K has one block of 128 at least
    rows, blocks, parts = (m + 15) // 16 * 16, (k + 127) // 128, split or 8
    for tile, refused in ((32, m > 32 or split > blocks),
                          (64, -(-(-(-blocks // parts)) // 8) * rows > 256 or split > blocks)):
        if refused:
            with pytest.raises(swz.SwzError):
                swz.gemm_int8(a, sa, b, sb, tile=tile, split_k=split)
        else:
            assert bits(swz.gemm_int8(a, sa, b, sb, tile=tile, split_k=split), want), tile
    assert bits(swz.gemm_int8(a, sa, b, sb), want)
    swz.check_status()


@pytest.mark.parametrize("m", [65, 100, 128, 129, 250, 256, 257, 300, 600])
@pytest.mark.parametrize("n,k", [(130, 1024), (1000, 2500), (4096, 300)])
def test_batches(swz, m, n, k):
    a, sa = int8_rows(swz, m, k, 5)
    b, sb = int8_rows(swz, n, k, 6)
    want = exact_c(a, sa, b, sb, torch.float16)
    for kw in (dict(), dict(tile=64), dict(tile=64, split_k=4 if k > 1000 else 2), dict(tile=128), dict(tile=256)):
        assert bits(swz.gemm_int8(a, sa, b, sb, out_dtype=torch.float16, **kw), want), kw
    swz.check_status()


@pytest.mark.parametrize("m", [1, 40, 300])
def test_gemm_extreme_sums(swz, m):
    """The largest sums: every product 2^14 over the longest K, and all of one sign."""
    n, k = 70, 131071
    a, b = swz.int8_empty(m, k), swz.int8_empty(n, k)
    a.fill_(-128)
    b.fill_(-128)
    b[1::2] = 127
    one = lambda r: torch.ones(r, device="cuda")  # noqa: E731
    c = swz.gemm_int8(a, one(m), b, one(n), out_dtype=torch.float32)
    want = torch.tensor([16384.0 * k, -16256.0 * k], dtype=torch.float64, device="cuda").float()
    assert torch.equal(c, want.repeat(35).expand(m, n))
    # sums whose last bits fp32 accumulation over all of K would lose
    a, sa = int8_rows(swz, m, 20000, 5, low=100)
    b, sb = int8_rows(swz, n, 20000, 6, low=100)
    assert bits(swz.gemm_int8(a, sa, b, sb, out_dtype=torch.float32),
                exact_c(a, sa, b, sb, torch.float32))


@pytest.mark.parametrize("m", [1, 5, 33, 200])
@pytest.mark.parametrize("dtype", TYPES)
def test_out_rows(swz, m, dtype):
    """Results in rows that start anywhere; what lies beside them stays."""
    n, k = 203, 1200
    a, sa = int8_rows(swz, m, k, 8)
    b, sb = int8_rows(swz, n, k, 9)
    want = exact_c(a, sa, b, sb, dtype)
    for ld, offset in ((n, 0), (n + 5, 3), (256, 0), (208, 8)):
        flat = torch.full((offset + m * ld + 32,), 7.0, dtype=dtype, device="cuda")
        out = flat[offset:offset + m * ld].view(m, ld)[:, :n]
        assert swz.gemm_int8(a, sa, b, sb, out=out) is out
        assert bits(out, want)
        out.fill_(7.0)
        assert (flat == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (1, 3, 5), (5, 100, 333), (32, 1000, 2000),
                                   (50, 640, 1999), (333, 1111, 1999), (600, 300, 64)])
def test_linear(swz, dtype, m, n, k):
    x = torch.randn((m, k), generator=gen(k), device="cuda").to(dtype)
    qw, sw = swz.quantize_int8(torch.randn((n, k), generator=gen(n), device="cuda"))
    q, s = exact_q(x)
    want = exact_c(q, s, qw, sw, dtype)
    assert bits(swz.linear_int8(x, qw, sw), want)
    assert bits(swz.linear_int8(rows_of(x, k + 1, 1), qw, sw), want)
    assert bits(swz.linear_int8(x, qw, sw, out_dtype=torch.float32),
                exact_c(q, s, qw, sw, torch.float32))


def test_linear_bad_rows(swz):
    """A NaN or an infinity in one row makes that row NaN and no other."""
    for m in (6, 100):
        x = torch.randn((m, 300), generator=gen(2), device="cuda")
        qw, sw = swz.quantize_int8(torch.randn((40, 300), generator=gen(3), device="cuda"))
        good = swz.linear_int8(x, qw, sw)
        x[1, 7], x[4, 299] = float("nan"), float("-inf")
        y = swz.linear_int8(x, qw, sw)
        assert torch.isnan(y[[1, 4]]).all()
        keep = [i for i in range(m) if i not in (1, 4)]
        assert torch.equal(y[keep], good[keep])


def test_empty(swz):
    qw, sw = swz.quantize_int8(torch.randn((8, 64), device="cuda"))
    assert swz.linear_int8(torch.empty((0, 64), device="cuda"), qw, sw).shape == (0, 8)
    q, s = swz.quantize_int8(torch.empty((0, 64), device="cuda"))
    assert swz.gemm_int8(q, s, qw, sw).shape == (0, 8)
    q, s = swz.quantize_int8(torch.empty((3, 0), device="cuda"))
    q2, s2 = swz.quantize_int8(torch.empty((4, 0), device="cuda"))
    assert not swz.gemm_int8(q, s, q2, s2).any()
    assert not swz.linear_int8(torch.empty((3, 0), device="cuda"), q2, s2).any()


@pytest.mark.parametrize("m", [1, 20, 500])
def test_graph_and_streams(swz, m):
    n, k = 640, 1500
    x = torch.zeros((m, k), device="cuda").bfloat16()
    qw, sw = swz.quantize_int8(torch.randn((n, k), generator=gen(3), device="cuda"))
    out = {}

    def call():
        out["y"] = swz.linear_int8(x, qw, sw)
        q, s = swz.quantize_int8(x)
        out["c"] = swz.gemm_int8(q, s, qw, sw)
    g1 = capture_graph(call)
    kept = dict(out)
    g2 = capture_graph(call)  # a second graph of the same calls, with its own workspaces
    for seed in (1, 2):
        x.copy_(torch.randn((m, k), generator=gen(seed), device="cuda"))
        q, s = exact_q(x)
        want = exact_c(q, s, qw, sw, torch.bfloat16)
        g1.replay()
        g2.replay()
        for o in (kept, out):
            assert bits(o["y"], want) and bits(o["c"], want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = swz.linear_int8(x, qw, sw, stream=side)
    with torch.cuda.stream(side):
        z = swz.linear_int8(x, qw, sw)
    torch.cuda.current_stream().wait_stream(side)
    assert bits(y, want) and bits(z, want)


def test_no_gradient(swz):
    x = torch.randn((4, 64), device="cuda", requires_grad=True)
    qw, sw = swz.quantize_int8(torch.randn((8, 64), device="cuda"))
    with pytest.raises(RuntimeError, match="no gradient"):
        swz.linear_int8(x, qw, sw).sum().backward()


def test_timeout_is_reported(swz):
    """A load that never arrives: the waits run out, the call ends, the status says so."""
    for m, n, kw in ((300, 300, dict(tile=256)), (300, 300, dict(tile=128)), (300, 300, dict(tile=128, split_k=4)),
                     (20, 300, dict()), (20, 90000, dict()), (3, 300, dict(tile=64, split_k=4)), (3, 300, dict(tile=32, split_k=4)), (3, 90000, dict(tile=32)), (200, 300, dict(tile=64))):
        a, sa = int8_rows(swz, m, 4096, 1)
        b, sb = int8_rows(swz, n, 4096, 2)
        swz.gemm_int8(a, sa, b, sb, debug_flags=swz.SWZ_DEBUG_SKIP_FIRST_LOAD, timeout_ms=50, **kw)
        with pytest.raises(swz.SwzError):
            swz.check_status()
        assert bits(swz.gemm_int8(a, sa, b, sb, **kw), exact_c(a, sa, b, sb, torch.bfloat16))
        swz.check_status()


def test_two_streams_at_once(swz):
    """Calls of every form under way on two streams together, each with its own workspace."""
    n, k = 1000, 1500
    qw, sw = swz.quantize_int8(torch.randn((n, k), generator=gen(1), device="cuda"))
    xs = [torch.randn((m, k), generator=gen(m), device="cuda").bfloat16() for m in (1, 2, 20, 60, 200, 700)]
    want = [exact_c(*exact_q(x), qw, sw, torch.bfloat16) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(len(xs)):
            for j, s in enumerate(streams):
                at = (i + 3 * j) % len(xs)  # different forms on the two
                with torch.cuda.stream(s):
                    got[j].append((at, swz.linear_int8(xs[at], qw, sw)))
    torch.cuda.synchronize()
    swz.check_status()
    for results in got:
        assert all(bits(y, want[at]) for at, y in results)


@pytest.mark.parametrize("m,n,k", [(3, 40, 5000), (1300, 9, 2048), (7, 5, 131071), (2000, 3000, 4100)])
def test_wide_form(swz, m, n, k):
    """Rows of several parts, of one value more than whole ones, and more rows than warps."""
    a, sa = int8_rows(swz, m, k, 11)
    b, sb = int8_rows(swz, n, k, 12)
    want = exact_c(a, sa, b, sb, torch.float32)
    for tile in (128, 256):
        assert bits(swz.gemm_int8(a, sa, b, sb, tile=tile, out_dtype=torch.float32), want)
