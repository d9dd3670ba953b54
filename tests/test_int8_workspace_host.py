"""Workspace sizes of the 8-bit integer product by its options (CPU only)."""
import pytest


@pytest.fixture(scope="module")
def swz():
    from thread_block_smem_gb300 import build
    build.build()
    import thread_block_smem_gb300 as m
    m.lib()
    return m


def size(swz, m, n, k, **kw):
    return swz.swz_gemm_int8_workspace_size_ex(m, n, k, swz.swz_gemm_int8_opts(order=5, group=8, **kw))


def test_sizes_by_options(swz):
    n = 300
    for m in (0, 1, 2, 3, 32, 33, 256, 512, 513, 2000):
        for k in (0, 15, 70, 4096, 16384):
            plain = swz.swz_gemm_int8_workspace_size(m, n, k)
            assert size(swz, m, n, k) == swz.swz_gemm_int8_workspace_size_ex(m, n, k) == plain
            for tile in (64, 128, 256):
                assert size(swz, m, n, k, tile=tile) == swz.swz_gemm_int8_workspace_size(m, n, k, tile)
    # K = 4096 are four sums of 256 columns each, of 512: two parts have room, one has not, and
    # the kernel that widens both operands takes it
    a, both = 256 * 4096 * 2, (256 + n) * 4096 * 2
    assert size(swz, 256, n, 4096, split_k=2) == (0, a)
    assert size(swz, 256, n, 4096, split_k=1) == (0, both)
    assert size(swz, 256, n, 4096, split_k=1, tile=64) == (0, a)
    for bad in ((-1, 5, 64), (5, -1, 64), (5, 5, -1), (5, 5, 131072), (2 ** 32 + 5, 5, 64)):
        assert size(swz, *bad)[0] == swz.SWZ_EINVAL
