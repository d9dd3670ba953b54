"""What the linear-layer operators refuse or do with their operands before any
CUDA call (CPU only: tensors are stand-ins, the library's launches are not
reached)."""
import pytest
import torch


@pytest.fixture(scope="module")
def swz():
    from thread_block_smem_gb300 import build
    build.build()
    import thread_block_smem_gb300 as m
    m.lib()
    return m


@pytest.fixture(autouse=True)
def current_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)


class Operand:
    """A row-major CUDA tensor as the entry points see one, without memory."""

    def __init__(self, shape, dtype=torch.bfloat16, device=0, stride=None):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device = torch.device("cuda", device)
        self.is_cuda, self.requires_grad = True, False
        self._stride = stride or tuple(
            int(torch.Size(shape[i + 1:]).numel()) for i in range(len(shape)))

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 4096

    def narrow(self, dim, at, n):
        return Operand([n if i == dim else v for i, v in enumerate(self.shape)], self.dtype, 0,
                       self._stride)


BIG = 2 ** 32 + 8  # an int would hold 8


def test_sizes_past_an_int_are_refused_by_the_mirrors(swz):
    E = swz.SWZ_EINVAL
    for at in range(3):
        sizes = [8, 5, 200]
        sizes[at] = BIG
        assert swz.swz_linear_fp8_workspace_size(*sizes)[0] == E
        sizes = [2, 5, 200]
        sizes[at] = BIG
        assert swz.swz_newton_schulz_workspace_size(*sizes)[0] == E
    # the calls below are no-ops (a size of zero) unless a size is refused
    quantize = [256, 1, 64, 0, 64, 0, 0, 4096, 64, 8192, 8, 0, 0, 0, 0]
    assert swz.swz_quantize_fp8(*quantize) == swz.SWZ_OK
    for at in (1, 3, 4, 5, 6):  # dtype, M, K, block, fmt
        a = list(quantize)
        a[at] += 2 ** 32
        assert swz.swz_quantize_fp8(*a) == E, at
    mat = swz.swz_fp8_matrix(4096, 64, 256, 8, 0, 0)
    gemm = [mat, mat, 4096, 8, 3, 0, 8, 64]
    assert swz.swz_gemm_fp8(*gemm) == swz.SWZ_OK
    for at in (4, 5, 6, 7):
        a = list(gemm)
        a[at] += 2 ** 32
        assert swz.swz_gemm_fp8(*a) == E, at
    linear = [256, 1, 64, mat, 4096, 8, 1, 0, 8, 64, 65536, 1 << 20]
    assert swz.swz_linear_fp8(*linear) == swz.SWZ_OK
    for at in (1, 6, 7, 8, 9):
        a = list(linear)
        a[at] += 2 ** 32
        assert swz.swz_linear_fp8(*a) == E, at
    update = [256, 3, 64, 0, 4096, 1, 64, 0, 0, 8, 64, 5, 3.4, -4.8, 2.0, 1e-7, None, 65536, 1 << 30]
    assert swz.swz_newton_schulz(*update) == swz.SWZ_OK
    for at in (1, 5, 8, 9, 10, 11):
        a = list(update)
        a[at] += 2 ** 32
        assert swz.swz_newton_schulz(*a) == E, at


@pytest.mark.parametrize("shape", [(1, BIG), (BIG, 1), (3, 2 ** 31)])
def test_sizes_past_an_int_are_refused(swz, shape):
    x = Operand(shape)
    f8 = Operand(shape, torch.float8_e4m3fn)
    s = Operand((1, 1), torch.float32)
    other = Operand((4, 128), torch.float8_e4m3fn)
    other_s = Operand((1, 1), torch.float32)
    with pytest.raises(ValueError, match="2\\^31"):
        swz.quantize_fp8(x)
    with pytest.raises(ValueError, match="2\\^31"):
        swz.gemm_fp8(f8, s, other, other_s)
    with pytest.raises(ValueError, match="2\\^31"):
        swz.linear_fp8(x, other, other_s)
    with pytest.raises(ValueError, match="2\\^31"):
        swz.linear_fp8_forward(x, x)
    with pytest.raises(ValueError, match="2\\^31"):
        swz.newton_schulz(x, out=x)
    with pytest.raises(ValueError, match="2\\^31"):
        swz.newton_schulz(Operand((BIG, 2, 2)), out=Operand((BIG, 2, 2)))


def test_options_past_their_type_are_refused(swz):
    q, s = Operand((4, 128), torch.float8_e4m3fn), Operand((1, 4), torch.float32)
    qb, sb = q, Operand((1, 1), torch.float32)
    out = Operand((4, 4))
    for kw in (dict(order=2 ** 32 + 5), dict(group=BIG), dict(tile=2 ** 32 + 128), dict(split_k=2 ** 32),
               dict(num_programs=-2 ** 32), dict(timeout_ms=2 ** 32), dict(debug_flags=2 ** 32)):
        with pytest.raises(ValueError, match="range"):
            swz.gemm_fp8(q, s, qb, sb, out=out, **kw)
    for kw in (dict(steps=2 ** 32 + 5), dict(tile=2 ** 32), dict(timeout_ms=2 ** 32)):
        with pytest.raises(ValueError, match="range"):
            swz.newton_schulz(Operand((8, 8)), out=Operand((8, 8)), **kw)


def calls(swz, at):
    """Each operator on operands of which the one named by the key is on device `at[key]`, else 0."""
    d = lambda name: at.get(name, 0)  # noqa: E731
    f8, f32 = torch.float8_e4m3fn, torch.float32
    x = Operand((4, 128), device=d("x"))
    q, s = Operand((4, 128), f8, d("q")), Operand((1, 4), f32, d("s"))
    w, sw = Operand((4, 128), f8, d("w")), Operand((1, 1), f32, d("sw"))
    out = Operand((4, 4), device=d("out"))
    dy = Operand((4, 4), device=d("dy"))
    saved = (Operand((128, 4), f8, d("qxt"), (16, 1)), Operand((1, 128), f32, d("sxt")),
             Operand((128, 4), f8, d("qwt"), (16, 1)), Operand((1, 1), f32, d("swt")))
    return {
        "quantize_fp8": (("x",), lambda: swz.quantize_fp8(x)),
        "gemm_fp8": (("q", "s", "w", "sw", "out"), lambda: swz.gemm_fp8(q, s, w, sw, out=out)),
        "linear_fp8": (("x", "w", "sw", "out"), lambda: swz.linear_fp8(x, w, sw, out=out)),
        "forward": (("x", "x2"), lambda: swz.linear_fp8_forward(
            x, Operand((4, 128), device=d("x2")))),
        "backward": (("dy", "qxt", "sxt", "qwt", "swt"),
                     lambda: swz.linear_fp8_backward(dy, saved)),
        "newton_schulz": (("x", "g"), lambda: swz.newton_schulz(
            x, out=Operand((4, 128), device=d("g")))),
    }


OPERATORS = ["quantize_fp8", "gemm_fp8", "linear_fp8", "forward", "backward", "newton_schulz"]


@pytest.mark.parametrize("operator", OPERATORS)
def test_operands_on_different_devices_are_refused(swz, operator):
    names = calls(swz, {})[operator][0]
    for name in names[1:]:
        with pytest.raises(ValueError, match="device"):
            calls(swz, {name: 1})[operator][1]()


@pytest.mark.parametrize("operator", OPERATORS)
def test_a_device_that_is_not_current_is_refused(swz, operator):
    with pytest.raises(ValueError, match="current device"):
        calls(swz, {name: 1 for name in calls(swz, {})[operator][0]})[operator][1]()


class Launches:
    """Stands in for the library: every call succeeds and is counted."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append(name)
            return 0
        return call


class Kept(Operand):
    """An operand that notes the streams it is used on."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)

    def unsqueeze(self, _):
        return Kept((1, *self.shape), self.dtype, 0, (0, *self._stride))


@pytest.fixture
def launches(swz, monkeypatch):
    linear = swz.linear
    swz.linear._init()
    fake = Launches()
    monkeypatch.setattr(linear, "_L", fake)
    monkeypatch.setattr(linear, "_empty", lambda shape, dtype, x, stream: Operand(
        shape if isinstance(shape, tuple) else tuple(shape) if hasattr(shape, "__len__") else (shape,),
        dtype))
    monkeypatch.setattr(linear, "_handle", lambda stream, x: 0)
    return fake


def test_operands_are_kept_for_the_stream_that_uses_them(swz, launches, monkeypatch):
    class Stream:
        cuda_stream = 0

    class ExternalStream(Stream):
        pass
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", ExternalStream)
    side = Stream()
    f8, f32 = torch.float8_e4m3fn, torch.float32

    def operands(*specs):
        return [Kept(*s) for s in specs]

    def check(tensors):
        assert launches.calls and all(t.streams == [side] for t in tensors), [t.streams for t in tensors]
        launches.calls.clear()
    x, = operands(((4, 128),))
    swz.quantize_fp8(x, stream=side)
    check([x])
    used = operands(((4, 128), f8), ((1, 4), f32), ((4, 128), f8), ((1, 1), f32))
    out, = operands(((4, 4),))
    swz.gemm_fp8(*used, out=out, stream=side)
    check(used + [out])
    used = operands(((4, 128),), ((4, 128), f8), ((1, 1), f32))
    out, = operands(((4, 4),))
    swz.linear_fp8(*used, out=out, stream=side)
    check(used + [out])
    used = operands(((4, 128),), ((4, 128),))
    swz.linear_fp8_forward(*used, stream=side)
    check(used)
    used = operands(((4, 4),), ((128, 4), f8, 0, (16, 1)), ((1, 128), f32),
                    ((128, 4), f8, 0, (16, 1)), ((1, 1), f32))
    swz.linear_fp8_backward(used[0], used[1:], stream=side)
    check(used)
    used = operands(((8, 8),), ((8, 8),))
    swz.newton_schulz(used[0], out=used[1], stream=side)
    check(used)
    # the current stream, and streams that the caller made and may destroy, keep nothing
    for stream in (None, 0, ExternalStream()):
        x, = operands(((4, 128),))
        swz.quantize_fp8(x, stream=stream)
        assert x.streams == []


class OnDevice(torch.Tensor):
    """A host tensor that the entry points take for one on the device."""
    is_cuda = True

    def get_device(self):
        return 0


def on_device(*shape, dtype=torch.float32, grad=False):
    t = torch.zeros(shape).to(dtype).as_subclass(OnDevice)
    return t.requires_grad_() if grad else t


def test_a_lost_gradient_is_an_error_in_the_backward(swz, launches, monkeypatch):
    # linear_fp8, gemm_fp8 and newton_schulz have no gradient; a backward through
    # them says so instead of leaving their inputs without one
    monkeypatch.setattr(swz.linear, "_empty",
                        lambda shape, dtype, x, stream: torch.zeros(shape, dtype=dtype))
    f8 = torch.float8_e4m3fn
    q, s = on_device(4, 128, dtype=f8), on_device(1, 4)
    w, sw = on_device(4, 128, dtype=f8), on_device(1, 1)
    x, sx = on_device(4, 128, grad=True), on_device(1, 4, grad=True)
    for call in (lambda: swz.linear_fp8(x, w, sw), lambda: swz.newton_schulz(x),
                 lambda: swz.gemm_fp8(q, sx, w, sw)):
        y = call()
        assert y.requires_grad
        with pytest.raises(RuntimeError, match="no gradient"):
            y.float().sum().backward()
        with torch.no_grad():
            assert not call().requires_grad
    # where nothing asks for one, and into a buffer of the caller's, as before
    assert not swz.gemm_fp8(q, s, w, sw).requires_grad
    assert not swz.linear_fp8(x.detach(), w, sw).requires_grad
    out = torch.zeros(4, 4).as_subclass(OnDevice)
    assert swz.linear_fp8(x, w, sw, out=out) is out and not out.requires_grad
