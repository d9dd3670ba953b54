"""Host side of the 8-bit integer operators, the layer norm and the gradients' norm
(CPU only): argument checks of the C entry points before any CUDA call, workspace
sizes, what the tensor-level calls refuse, and the ranges that
perf/more_operators.py draws from."""
import importlib.util
import os
import random

import pytest
import torch

from conftest import ROOT
from test_linear_operands import BIG, Operand


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


def refused(call, good, changes, code):
    for at in changes:
        a = list(good)
        for k, v in at.items():
            a[k] = v
        assert call(*a) == code, at


def test_quantize_checks(swz):
    E = swz.SWZ_EINVAL
    # x, dtype, ldx, M, K, q, ldq, scales
    good = [256, 1, 64, 8, 64, 4096, 64, 8192]
    refused(swz.swz_quantize_int8, good,
            ({0: 0}, {0: 257}, {1: 2}, {1: 7}, {2: 63}, {3: -1}, {4: -1}, {5: 0}, {5: 4104}, {6: 72}, {6: 48},
             {7: 0}, {7: 8193}, {1: 2 ** 32 + 1}, {3: 2 ** 32 + 8}, {4: 2 ** 32 + 64}), E)
    assert swz.swz_quantize_int8(*good[:3], 0, *good[4:]) == swz.SWZ_OK


def test_gemm_checks(swz):
    E, U = swz.SWZ_EINVAL, swz.SWZ_EUNSUPPORTED
    # A, lda, sa, B, ldb, sb, C, ldc, c_dtype, M, N, K, opts, ws, bytes
    good = [4096, 64, 256, 4096, 64, 256, 8192, 100, 3, 100, 100, 64, None, 65536, 1 << 20]
    refused(swz.swz_gemm_int8, good,
            ({0: 0}, {0: 4097}, {1: 48}, {1: 72}, {2: 0}, {2: 258}, {3: 0}, {3: 4104}, {4: 63}, {5: 0}, {5: 257},
             {6: 0}, {6: 8194}, {7: 99}, {8: 2}, {8: 9}, {9: -1}, {10: -1}, {11: -1}, {11: 131072, 1: 131072, 4: 131072},
             {13: 0}, {13: 65537}, {14: 16}, {9: 2 ** 32 + 100}, {11: 2 ** 32 + 64}), E)
    opts = lambda **kw: swz.swz_gemm_int8_opts(**dict(dict(order=5, group=8), **kw))  # noqa: E731
    refused(swz.swz_gemm_int8, good, ({12: opts(order=9)}, {12: opts(order=2, group=0)}), E)
    refused(swz.swz_gemm_int8, good, ({12: opts(tile=16)}, {12: opts(split_k=3)}, {12: opts(tile=256, split_k=2)}), U)
    for at in (9, 10):
        a = list(good)
        a[at] = 0
        assert swz.swz_gemm_int8(*a) == swz.SWZ_OK
    assert swz.swz_gemm_int8_workspace_size(0, 5, 64) == (0, 0)
    for bad in ((-1, 5, 64), (5, -1, 64), (5, 5, -1), (5, 5, 131072), (2 ** 32 + 5, 5, 64)):
        assert swz.swz_gemm_int8_workspace_size(*bad)[0] == E
        assert swz.swz_linear_int8_workspace_size(*bad)[0] == E
    # by rows of A: nothing, A as fp16 in rows of whole lines, both operands
    for m, need in ((1, 0), (2, 0), (3, 0), (32, 0), (33, 33), (512, 512), (513, 513 + 300)):
        assert swz.swz_gemm_int8_workspace_size(m, 300, 70) == (0, need * 128 * 2), m
    assert swz.swz_gemm_int8_workspace_size(500, 300, 70, 128) == (0, 800 * 128 * 2)


def test_linear_checks(swz):
    E = swz.SWZ_EINVAL
    # x, dtype, ldx, W, ldw, sw, y, ldy, y_dtype, M, N, K, ws, bytes
    good = [256, 1, 64, 4096, 64, 256, 8192, 100, 1, 100, 100, 64, 65536, 1 << 20]
    refused(swz.swz_linear_int8, good,
            ({0: 0}, {0: 257}, {1: 2}, {2: 63}, {3: 0}, {3: 4097}, {4: 48}, {5: 0}, {5: 258}, {6: 0}, {6: 8193},
             {7: 99}, {8: 2}, {9: -1}, {10: -1}, {11: -1}, {11: 131072, 2: 131072, 4: 131072}, {12: 0}, {12: 65537},
             {13: 16}, {1: 2 ** 32 + 1}, {9: 2 ** 32 + 100}), E)
    for at in (9, 10):
        a = list(good)
        a[at] = 0
        assert swz.swz_linear_int8(*a) == swz.SWZ_OK


def test_layer_norm_checks(swz):
    E = swz.SWZ_EINVAL
    # x, dtype, ldx, w, w_dtype, b, b_dtype, eps, y, y_dtype, ldy, mean, rstd, M, N
    good = [256, 1, 64, 512, 1, 512, 1, 1e-5, 4096, 1, 64, 8192, 8192, 8, 64]
    refused(swz.swz_layer_norm, good,
            ({0: 0}, {0: 257}, {1: 2}, {2: 63}, {3: 513}, {4: 2}, {5: 513}, {6: 5}, {7: -1.0}, {7: float("nan")},
             {7: float("inf")}, {8: 0}, {8: 4097}, {9: 2}, {10: 63}, {11: 0}, {11: 8194}, {12: 0}, {12: 8193}, {13: -1},
             {14: -1}, {13: 2 ** 32 + 8}), E)
    for at in (13, 14):
        a = list(good)
        a[at] = 0
        assert swz.swz_layer_norm(*a) == swz.SWZ_OK
    # dy, dtype, ld, x, dtype, ld, w, dtype, mean, rstd, dx, dtype, ld, dw, db, dtype, M, N, ws, bytes
    good = [256, 1, 64, 256, 1, 64, 512, 1, 8192, 8192, 4096, 1, 64, 1024, 2048, 3, 8, 64, 65536, 1 << 20]
    refused(swz.swz_layer_norm_backward, good,
            ({0: 0}, {0: 257}, {1: 2}, {2: 63}, {3: 0}, {4: 2}, {5: 63}, {6: 513}, {7: 2}, {8: 0}, {8: 8193}, {9: 0},
             {10: 4097}, {11: 2}, {12: 63}, {13: 1026}, {14: 2049}, {15: 2}, {16: -1}, {17: -1}, {18: 0}, {18: 65537},
             {19: 16}, {10: 0, 13: 0, 14: 0}, {16: 2 ** 32 + 8}), E)
    a = list(good)
    a[17] = 0
    assert swz.swz_layer_norm_backward(*a) == swz.SWZ_OK
    assert swz.swz_layer_norm_backward_workspace_size(3, 50) == (0, 3 * 2 * 56 * 4)
    assert swz.swz_layer_norm_backward_workspace_size(-1, 50)[0] == E


def test_grad_norm_checks(swz):
    E = swz.SWZ_EINVAL
    good = dict(in_=4096, out=65536, n=100, dtype=1, out_dtype=3)

    def call(*records, count=None, max_norm=1.0, eps=0.0, norm=256, ws=512, size=1 << 20, clip=True):
        a = (swz.swz_grad * max(len(records), 1))(*[swz.swz_grad(**dict(good, **r)) for r in records])
        count = len(records) if count is None else count
        if not clip:
            return swz.swz_grad_norm(a, count, norm, ws, size)
        return swz.swz_clip_grad_norm(a, count, max_norm, eps, norm, ws, size)
    for r in (dict(in_=0), dict(in_=4097), dict(n=-1), dict(n=1 << 45), dict(dtype=2)):
        assert call(r) == E and call(r, clip=False) == E, r
    for r in (dict(out=0), dict(out=65538), dict(out_dtype=2), dict(out=4096), dict(out=4196, out_dtype=1)):
        assert call(r) == E, r
    for kw in (dict(norm=0), dict(norm=258), dict(ws=0), dict(ws=520 + 1), dict(size=8), dict(count=-1),
               dict(count=2 ** 32 + 1)):
        assert call({}, **kw) == E and call({}, clip=False, **kw) == E, kw
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0), dict(eps=float("nan"))):
        assert call({}, **kw) == E, kw
    # results over one another, over another's values, and over their own in another place
    assert call({}, dict(in_=8192)) == E
    assert call({}, dict(in_=65536, out=131072)) == E
    assert call({}, dict(in_=8192, out=4292)) == E
    assert call(dict(out=4198, out_dtype=1, in_=4198 - 2)) == E
    rc, need = swz.swz_grad_norm_workspace_size(1)
    assert rc == 0 and need > 0 and swz.swz_grad_norm_workspace_size(1001)[1] == 2 * need
    assert swz.swz_grad_norm_workspace_size(0) == (0, 0) and swz.swz_grad_norm_workspace_size(-1)[0] == E


def test_int8_calls_refuse(swz):
    i8, f32 = torch.int8, torch.float32
    q, s = Operand((4, 128), i8), Operand((4,), f32)
    x, out = Operand((4, 128)), Operand((4, 4))
    for bad in (Operand((4, 128), torch.uint8), Operand((4, 128), torch.float8_e4m3fn)):
        with pytest.raises(TypeError, match="int8"):
            swz.gemm_int8(bad, s, q, s, out=out)
        with pytest.raises(TypeError, match="int8"):
            swz.linear_int8(x, bad, s, out=out)
    for bad, why in ((Operand((4,), torch.float16), "fp32"), (Operand((5,), f32), "shape"),
                     (Operand((4, 1), f32), "shape"), (Operand((4,), f32, stride=(2,)), "contiguous")):
        with pytest.raises((TypeError, ValueError), match=why):
            swz.gemm_int8(q, bad, q, s, out=out)
        with pytest.raises((TypeError, ValueError), match=why):
            swz.gemm_int8(q, s, q, bad, out=out)
    for bad, why in ((Operand((4, 128), i8, stride=(136, 1)), "16 bytes"), (Operand((4, 64), i8), "inner"),
                     (Operand((4, 128), i8, stride=(1, 128)), "contiguous rows"),
                     (Operand((1, 131072), i8), "131071"), (Operand((4, 128, 1), i8), "2-D")):
        with pytest.raises(ValueError, match=why):
            swz.gemm_int8(q, s, bad, Operand((bad.shape[0],), f32), out=out)
    for kw in (dict(order=2 ** 32 + 5), dict(group=BIG), dict(tile=2 ** 32 + 128), dict(split_k=2 ** 32),
               dict(timeout_ms=2 ** 32), dict(debug_flags=2 ** 32)):
        with pytest.raises(ValueError, match="range"):
            swz.gemm_int8(q, s, q, s, out=out, **kw)
    with pytest.raises(ValueError, match="2\\^31"):
        swz.quantize_int8(Operand((1, BIG)))
    with pytest.raises(TypeError, match="fp16, bf16 or fp32"):
        swz.quantize_int8(Operand((4, 128), torch.float64))
    with pytest.raises(ValueError, match="shape"):
        swz.gemm_int8(q, s, q, s, out=Operand((4, 5)))


def test_norm_calls_refuse(swz):
    x, w, s = Operand((4, 128)), Operand((128,)), Operand((4,), torch.float32)
    for bad, why in ((Operand((127,)), "shape"), (Operand((1, 128)), "shape"),
                     (Operand((128,), stride=(2,)), "contiguous"), (Operand((128,), torch.float64), "fp16")):
        for kw in (dict(weight=bad), dict(bias=bad)):
            with pytest.raises((TypeError, ValueError), match=why):
                swz.layer_norm_forward(x, out=x, **kw)
        with pytest.raises((TypeError, ValueError), match=why):
            swz.layer_norm_backward(x, x, bad, s, s)
    for bad in (Operand((5,), torch.float32), Operand((4, 1), torch.float32), Operand((4,), torch.float16)):
        with pytest.raises((TypeError, ValueError)):
            swz.layer_norm_backward(x, x, w, bad, s)
        with pytest.raises((TypeError, ValueError)):
            swz.layer_norm_backward(x, x, w, s, bad)
    with pytest.raises(ValueError, match="shape of x"):
        swz.layer_norm_backward(Operand((4, 120)), x, w, s, s)
    with pytest.raises(ValueError, match="2-D"):
        swz.layer_norm_forward(Operand((4, 4, 4)), out=x)
    with pytest.raises(ValueError, match="2\\^31"):
        swz.layer_norm_forward(Operand((BIG, 2)), out=x)


class Grad(Operand):
    def is_contiguous(self):
        return Operand(self.shape)._stride == self._stride

    def numel(self):
        return self.shape.numel()


def test_clip_calls_refuse(swz):
    g = Grad((4, 8))
    with pytest.raises(ValueError, match="one tensor at least"):
        swz.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="one tensor for each"):
        swz.clip_grad_norm([g], 1.0, out=[])
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError, match="at least 0"):
            swz.clip_grad_norm([g], bad)
        with pytest.raises(ValueError, match="at least 0"):
            swz.clip_grad_norm([g], 1.0, bad)
    for grads, out, why in (([Grad((4, 8), torch.float64)], None, "fp16"), ([g, Grad((4, 8), device=1)], None, "different"),
                            ([Grad((4, 8), device=1)], None, "not the current"),
                            ([Grad((4, 8), stride=(9, 1))], None, "one piece"),
                            ([Grad((4, 8), stride=(0, 1))], None, "one piece"),
                            ([g], [Grad((8, 4))], "shape"), ([g], [Grad((4, 8), stride=(1, 4))], "strides"),
                            ([g], [Grad((4, 8), device=1)], "different")):
        with pytest.raises((TypeError, ValueError), match=why):
            swz.clip_grad_norm(grads, 1.0, out=out)
    g.requires_grad = True
    with pytest.raises(ValueError, match="no gradient"):
        swz.clip_grad_norm([g], 1.0)


@pytest.mark.parametrize("name", ["quantize", "gemm", "linear", "forward", "backward", "clip"])
def test_devices(swz, name):
    """Operands on another device than the current one, or on two, are refused."""
    i8, f32 = torch.int8, torch.float32

    def call(at):
        d = lambda n: at.get(n, 0)  # noqa: E731
        x, out = Operand((4, 128), device=d("x")), Operand((4, 4), device=d("out"))
        q, s = Operand((4, 128), i8, d("q")), Operand((4,), f32, d("s"))
        w, t = Operand((128,), device=d("w")), Operand((4,), f32, d("t"))
        y = Operand((4, 128), device=d("y"))
        if name == "quantize":
            return ["x"], lambda: swz.quantize_int8(x)
        if name == "gemm":
            return ["q", "s", "out"], lambda: swz.gemm_int8(q, s, Operand((4, 128), i8), Operand((4,), f32), out=out)
        if name == "linear":
            return ["x", "q", "s", "out"], lambda: swz.linear_int8(x, q, s, out=out)
        if name == "forward":
            return ["x", "w", "y"], lambda: swz.layer_norm_forward(x, w, Operand((128,)), out=y)
        if name == "backward":
            return ["x", "w", "s", "t", "y"], lambda: swz.layer_norm_backward(y, x, w, s, t)
        g, o = Grad((4, 8), device=d("x")), Grad((4, 8), f32, device=d("out"))
        return ["x", "out"], lambda: swz.clip_grad_norm([g], 1.0, out=[o])
    names, _ = call({})
    for n in names:
        with pytest.raises(ValueError, match="device"):
            call({n: 1})[1]()


def test_performance_cases_are_well_formed():
    spec = importlib.util.spec_from_file_location(
        "more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cases = m.listed()
    names = [c["name"] for c in cases]
    assert len(set(names)) == len(names)
    rng = random.Random(1)
    for c in cases + [m.draw(rng) for _ in range(200)]:
        w = m.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0
