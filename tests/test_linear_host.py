"""Host side of the linear-layer operators (CPU only): argument checks of the C
entry points before any CUDA call, workspace sizes, and the ranges that
perf/operators.py draws from."""
import importlib.util
import os
import random

import pytest

from conftest import ROOT


@pytest.fixture(scope="module")
def swz():
    from thread_block_smem_gb300 import build
    build.build()
    import thread_block_smem_gb300 as m
    m.lib()
    return m


def test_quantize_checks(swz):
    E, ok = swz.SWZ_EINVAL, swz.SWZ_OK
    # x, dtype, ldx, M, K, block, fmt, q, ldq, s, lds, qt, ldqt, st, ldst
    good = [256, 1, 64, 8, 64, 0, 0, 4096, 64, 8192, 8, 0, 0, 0, 0]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return swz.swz_quantize_fp8(*a)
    for at in (dict(_0=0), dict(_0=257), dict(_1=2), dict(_1=7), dict(_2=63), dict(_3=-1),
               dict(_4=-1), dict(_5=2), dict(_6=2), dict(_7=4097), dict(_8=72), dict(_8=48),
               dict(_9=0), dict(_9=8193), dict(_10=7), dict(_7=0), dict(_11=4096, _12=16),
               dict(_11=4096, _12=8, _13=8192, _14=64), dict(_11=4096, _12=16, _13=8192, _14=63)):
        assert call(**at) == E, at
    assert call(_3=0) == ok and call(_4=0) == ok


def test_gemm_checks(swz):
    E, U = swz.SWZ_EINVAL, swz.SWZ_EUNSUPPORTED
    mat = lambda rows=8, **kw: swz.swz_fp8_matrix(**dict(  # noqa: E731
        data=4096, ld=64, scales=256, ld_scales=rows, fmt=0, block=0, **kw))

    def call(A=None, B=None, C=4096, ldc=8, dtype=3, M=8, N=8, K=64, opts=None):
        return swz.swz_gemm_fp8(A or mat(), B or mat(), C, ldc, dtype, M, N, K, opts)

    def with_(field, value):
        m = mat()
        setattr(m, field, value)
        return m
    for field, value in (("data", 0), ("data", 4097), ("ld", 48), ("ld", 72), ("scales", None),
                         ("scales", 258), ("ld_scales", 7), ("fmt", 2), ("block", 2)):
        assert call(A=with_(field, value)) == E, field
        assert call(B=with_(field, value)) == E, field
    assert call(A=with_("block", 1)) == U                     # A by rows only
    for kw in (dict(C=0), dict(C=4098), dict(ldc=7), dict(dtype=2), dict(M=-1), dict(N=-1),
               dict(K=-1)):
        assert call(**kw) == E, kw
    assert call(M=0) == swz.SWZ_OK and call(N=0) == swz.SWZ_OK
    opts = lambda **kw: swz.swz_gemm_fp8_opts(**dict(dict(order=5, group=8), **kw))  # noqa: E731
    for kw in (dict(order=9), dict(order=2, group=0), dict(num_programs=-1),
               dict(num_programs=4)):
        assert call(opts=opts(**kw)) == E, kw
    for kw in (dict(tile=64), dict(split_k=3), dict(tile=256, split_k=2)):
        assert call(opts=opts(**kw)) == U, kw


def test_linear_checks_and_workspace(swz):
    E = swz.SWZ_EINVAL
    W = swz.swz_fp8_matrix(4096, 64, 256, 8, 0, 0)
    good = [256, 1, 64, W, 4096, 8, 1, 8, 8, 64, 65536, 1 << 20]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return swz.swz_linear_fp8(*a)
    for at in (dict(_0=0), dict(_0=257), dict(_1=2), dict(_2=63), dict(_4=0), dict(_5=7),
               dict(_6=2), dict(_7=-1), dict(_8=-1), dict(_9=-1), dict(_10=0), dict(_10=65537),
               dict(_11=16)):
        assert call(**at) == E, at
    assert call(_7=0) == swz.SWZ_OK
    # x in 8 bits in rows of a multiple of 16 bytes, then a scale for 128 of them
    assert swz.swz_linear_fp8_workspace_size(3, 5, 200) == (0, 768 + 2 * 3 * 4)
    assert swz.swz_linear_fp8_workspace_size(0, 5, 200) == (0, 0)
    assert swz.swz_linear_fp8_workspace_size(1, 1, -1)[0] == E


def test_newton_schulz_checks_and_workspace(swz):
    E, U = swz.SWZ_EINVAL, swz.SWZ_EUNSUPPORTED
    # G, dtype, ldg, bsg, Y, dtype, ldy, bsy, batch, m, n, steps, a, b, c, eps, opts, ws, bytes
    good = [256, 3, 64, 0, 4096, 1, 64, 0, 1, 8, 64, 5, 3.4, -4.8, 2.0, 1e-7, None, 65536, 1 << 30]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return swz.swz_newton_schulz(*a)
    for at in (dict(_0=0), dict(_0=258), dict(_1=2), dict(_2=63), dict(_4=0), dict(_4=4097),
               dict(_6=63), dict(_8=-1), dict(_8=65536), dict(_8=2), dict(_9=1 << 20, _10=1 << 20),
               dict(_11=0), dict(_11=65), dict(_12=float("nan")), dict(_15=-1.0),
               dict(_15=float("inf")), dict(_17=0), dict(_17=65537), dict(_18=100)):
        assert call(**at) == E, at
    assert call(_12=1e9, _11=3) == U
    assert call(_16=swz.swz_newton_schulz_opts(tile=64)) == U
    assert call(_8=0) == swz.SWZ_OK and call(_9=0) == swz.SWZ_OK
    rc, small = swz.swz_newton_schulz_workspace_size(1, 8, 64)
    rc2, large = swz.swz_newton_schulz_workspace_size(4, 300, 200)
    # two fp16 X and an fp32 one, A and B, of rows of a multiple of 16
    assert rc == rc2 == 0 and large >= 4 * (300 * 208 * 8 + 2 * 200 * 208 * 2) > small
    assert swz.swz_newton_schulz_workspace_size(-1, 8, 8)[0] == E


def test_performance_cases_are_well_formed():
    spec = importlib.util.spec_from_file_location(
        "operators", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cases = m.listed()
    names = [c["name"] for c in cases]
    assert len(set(names)) == len(names)
    rng = random.Random(1)
    for c in cases + [m.draw(rng) for _ in range(200)]:
        w = m.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0
        assert all(v != 3072 for v in c.values())
