"""The norm and clipping of gradients on the GPU against 64 bits.

Bounds, with u = 2^-24: a thread's squares are added in fp32, 64 at most, so their
sum is off by 65 u relative (all terms have one sign), everything above in 64 bits;
half of that and a rounding is the norm's: 34 u.  The factor adds an addition and
a division: 36 u; a result the product's and the type's rounding: 37 u + eps / 2."""
import math

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


def exact_norm(grads):
    top = max((g.double().abs().max().item() for g in grads if g.numel()), default=0.0)
    if top == 0 or not math.isfinite(top):
        return top
    return top * math.sqrt(math.fsum((g.double() / top).square().sum().item() for g in grads))


def check(swz, grads, max_norm, out=None, eps=1e-6):
    before = [g.clone() for g in grads]
    want = exact_norm(before)
    norm = swz.clip_grad_norm(grads, max_norm, eps, out=out)
    assert norm.shape == () and norm.dtype == torch.float32
    # fp32 holds the norm down to its smallest step, and up to its largest number: 5900
    # normal values of size 1e37 have the norm 1e37 sqrt(5900) = 7.7e38, above 3.4e38
    if want > torch.finfo(torch.float32).max:
        assert norm.item() == float("inf")
    else:
        assert abs(norm.item() - want) <= 34 * U * want + 2.0 ** -149, (norm.item(), want)
    assert swz.grad_norm(before).item() == norm.item()
    f = min(1.0, max_norm / (want + eps)) if want + eps else 1.0
    for o, b in zip(grads if out is None else out, before):
        exact = b.double() * f
        step = torch.finfo(o.dtype)
        allowed = exact.abs() * (37 * U + step.eps / 2) + step.tiny * step.eps
        assert bool(((o.double() - exact).abs() <= allowed).all())
        if f == 1.0 and o.dtype == b.dtype:
            assert torch.equal(o, b)
    if out is not None:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    return norm


SHAPES = [[(1,)], [(7,), (300, 5), (2, 3, 4)], [(16384,), (16385,), (16383,), ()],
          [(1000, 999)], [(64, 64)] * 33, [(0, 4), (5,), (0,)], [(2048, 2049), (3,), (513, 1023)]]


@pytest.mark.parametrize("shapes", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip(swz, shapes, dtype, max_norm):
    make = lambda: [torch.randn(s, generator=gen(i), device="cuda").to(dtype)  # noqa: E731
                    for i, s in enumerate(shapes)]
    check(swz, make(), max_norm)
    for out_dtype in TYPES:
        out = [torch.full(s, 7.0, dtype=out_dtype, device="cuda") for s in shapes]
        check(swz, make(), max_norm, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out_dtype", TYPES)
def test_any_alignment(swz, dtype, out_dtype):
    """Tensors one after another in one piece of memory, at every offset; what lies between
    and around stays."""
    sizes = [1, 2, 3, 5, 8, 13, 250, 2047, 20001, 40000, 7]
    gaps = [0, 1, 0, 2, 0, 0, 1, 0, 3, 1, 0]
    total = sum(sizes) + sum(gaps) + 64
    a = torch.randn(total, generator=gen(1), device="cuda").to(dtype)
    b = torch.full((total + 3,), 7.0, dtype=out_dtype, device="cuda")
    grads, out, at = [], [], 0
    for n, gap in zip(sizes, gaps):
        at += gap
        grads.append(a[at:at + n])
        out.append(b[at + 3:at + 3 + n])
        at += n
    check(swz, grads, 0.25, out)
    for o in out:
        o.fill_(7.0)
    assert (b == 7.0).all()
    whole = a.clone()
    swz.clip_grad_norm(grads, 0.25)
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    at = 0
    for n, gap in zip(sizes, gaps):
        inside[at + gap:at + gap + n] = True
        at += gap + n
    assert torch.equal(a[~inside], whole[~inside]) and not torch.equal(a[inside], whole[inside])


def test_mixed_types_and_layouts(swz):
    g = gen(3)
    grads = [torch.randn((100, 50), generator=g, device="cuda").bfloat16().t(),
             torch.randn((3, 4, 5), generator=g, device="cuda").permute(2, 0, 1),
             torch.randn(999, generator=g, device="cuda").half(),
             torch.randn((1, 6), generator=g, device="cuda")]
    check(swz, grads, 2.0)
    out = [torch.empty_strided(t.shape, t.stride(), dtype=torch.float32, device="cuda") for t in grads]
    check(swz, grads, 1.0, out)


@pytest.mark.parametrize("size", [1e-30, 1e-25, 1e-12, 1e15, 1e17, 1e25, 1e37])
def test_squares_outside_fp32(swz, size):
    grads = [torch.randn(5000, generator=gen(1), device="cuda") * size,
             torch.randn((30, 30), generator=gen(2), device="cuda") * size]
    check(swz, grads, size, eps=0.0)
    grads.append(torch.full((20000,), 1e-3, device="cuda"))
    check(swz, grads, size, eps=0.0)


def test_zeros(swz):
    grads = [torch.zeros(100, device="cuda"), torch.zeros((3, 3), device="cuda").half()]
    assert check(swz, grads, 1.0).item() == 0
    assert check(swz, grads, 0.0, eps=0.0).item() == 0
    assert swz.clip_grad_norm([torch.empty(0, device="cuda")], 1.0).item() == 0
    g = torch.randn(100, generator=gen(1), device="cuda")
    swz.clip_grad_norm([g], 0.0)
    assert not g.any()


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan(swz, dtype):
    a = torch.randn(5000, generator=gen(1), device="cuda").to(dtype)
    b = torch.randn(50, generator=gen(2), device="cuda").to(dtype)
    b[7] = float("-inf")
    out = [torch.empty_like(a), torch.empty_like(b)]
    assert swz.clip_grad_norm([a, b], 1.0, out=out).item() == float("inf")
    assert not out[0].any() and torch.isnan(out[1][7]) and not out[1][:7].any()
    b[8] = float("nan")
    assert math.isnan(swz.clip_grad_norm([a, b], 1.0, out=out).item())
    assert torch.isnan(out[0]).all() and torch.isnan(out[1]).all()
    assert math.isnan(swz.grad_norm([b, a]).item())


@pytest.mark.parametrize("count", [32, 33, 1000, 1001, 2500])
def test_many_tensors(swz, count):
    sizes = [1 + (i * 37) % 400 for i in range(count)]
    flat = torch.randn(sum(sizes), generator=gen(count), device="cuda")
    check(swz, list(flat.split(sizes)), 1.0)


def test_one_large_tensor(swz):
    """Offsets past 2^31 bytes and elements: the first, the last and every 2^20-th value."""
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[::1 << 20] = 2.0
    g[-1] = 4.0
    want = math.sqrt(g[::1 << 20].numel() * 4.0 + 16.0)
    norm = swz.clip_grad_norm([g], want / 2, eps=0.0)
    assert abs(norm.item() - want) <= 34 * U * want
    assert g[-1].item() == 2.0 and (g[::1 << 20] == 1.0).all() and not g[1:1 << 20].any()


def test_repeated_calls_are_the_same(swz):
    grads = [torch.randn((1000, 1001), generator=gen(i), device="cuda").bfloat16() for i in range(3)]
    out = [torch.empty_like(g, dtype=torch.float32) for g in grads]
    norms, results = [], []
    for _ in range(3):
        norms.append(swz.clip_grad_norm(grads, 1.0, out=out).item())
        results.append([o.clone() for o in out])
    assert len(set(norms)) == 1
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(results[0], r))


def test_graph_and_streams(swz):
    grads = [torch.zeros((300, 301), device="cuda"), torch.zeros(77, device="cuda").half()]
    out = [torch.zeros_like(g, dtype=torch.float32) for g in grads]
    box = {}

    def call():
        box["norm"] = swz.clip_grad_norm(grads, 1.0, out=out)
    g1 = capture_graph(call)
    norm1 = box["norm"]
    g2 = capture_graph(call)
    for seed in (1, 2):
        for i, g in enumerate(grads):
            g.copy_(torch.randn(g.shape, generator=gen(seed * 10 + i), device="cuda"))
        want = swz.grad_norm(grads).item()
        g1.replay()
        first = [o.clone() for o in out]
        g2.replay()
        assert norm1.item() == box["norm"].item() == want
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = swz.clip_grad_norm(grads, 1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert norm.item() == want and torch.equal(grads[0], out[0])


def test_overlaps_are_refused(swz):
    a = torch.randn(100, device="cuda")
    before = a.clone()
    for grads, out in (([a, a], None), ([a[:60], a[50:]], None), ([a[:40], a[40:]], [a[40:80], a[:60]]),
                       ([a[:50]], [a[1:51]]), ([a[:10], a[20:30]], [a[50:60], a[55:65]])):
        with pytest.raises(swz.SwzError):
            swz.clip_grad_norm(grads, 0.1, out=out)
    half = a.half()
    with pytest.raises(swz.SwzError):
        swz.clip_grad_norm([a[:50]], 0.1, out=[a[:25].view(torch.float16)])
    assert torch.equal(a, before) and half.numel() == 100
    b = torch.empty(200, device="cuda")  # a tensor may be read twice
    check(swz, [a, a], 0.1, [b[:100], b[100:]])
