"""What the 8-bit integer products and the layer norm refuse of results over operands (CPU
only: every call here is refused before any CUDA call), and the test of two sets of rows
in memory behind it against all of their bytes."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <set>
#include "common.h"

int main() {
  using swz::RowsInMemory;
  std::srand(1);
  long met = 0, total = 200000;
  for (long t = 0; t < total; ++t) {
    RowsInMemory r[2];
    const bool same_ld = std::rand() % 2;
    for (int i = 0; i < 2; ++i) {
      r[i].rows = std::rand() % 6;
      r[i].width = std::rand() % 8;
      r[i].ld = r[i].width + std::rand() % 9;
      r[i].p = reinterpret_cast<const void*>(1000 + std::rand() % 80);
    }
    if (same_ld) r[0].ld = r[1].ld = std::max(r[0].ld, r[1].ld);
    std::set<long> bytes;
    for (long j = 0; j < r[0].rows; ++j)
      for (long k = 0; k < r[0].width; ++k) bytes.insert(long(r[0].p) + j * r[0].ld + k);
    bool meet = false;
    for (long j = 0; j < r[1].rows; ++j)
      for (long k = 0; k < r[1].width; ++k) meet |= bytes.count(long(r[1].p) + j * r[1].ld + k) > 0;
    if (swz::rows_meet(r[0], r[1]) != meet || swz::rows_meet(r[1], r[0]) != meet) {
      for (auto& x : r) std::printf("%ld %ld %ld %ld\n", long(x.p), x.rows, x.ld, x.width);
      return 1;
    }
    met += meet;
  }
  std::printf("%ld of %ld\n", met, total);
  return met > total / 10 && met < total * 9 / 10 ? 0 : 2;
}
"""


@pytest.fixture(scope="module")
def swz():
    from thread_block_smem_gb300 import build
    build.build()
    import thread_block_smem_gb300 as m
    m.lib()
    return m


def test_rows_meet(tmp_path):
    cc, cuda = shutil.which("g++"), "/usr/local/cuda/include"
    if cc is None or not os.path.isdir(cuda):
        pytest.skip("no host compiler or CUDA headers")
    (tmp_path / "meet.cc").write_text("#include <algorithm>\n" + PROGRAM)
    r = subprocess.run([cc, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I", cuda, "-I",
                        os.path.join(ROOT, "thread_block_smem_gb300", "csrc"), "meet.cc", "-o", "meet"],
                       cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([tmp_path / "meet"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


MB = 1 << 20


@pytest.mark.parametrize("m", [1, 2, 3, 20, 100, 600])
def test_gemm_over_its_operands(swz, m):
    k, n = 64, 100
    # A, lda, sa, B, ldb, sb, C, ldc, c_dtype, M, N, K, opts, ws, bytes
    good = [MB, k, 2 * MB, 3 * MB, k, 4 * MB, 5 * MB, n, swz.SWZ_BF16, m, n, k, None, 6 * MB, 1 << 30]
    bytes_c = m * n * 2
    for at, size in ((0, m * k), (2, m * 4), (3, n * k), (5, n * 4)):
        for to in (good[at], good[at] + size - 4, good[at] - bytes_c + 2):
            a = list(good)
            a[6] = to
            assert swz.swz_gemm_int8(*a) == swz.SWZ_EINVAL, (at, to)


@pytest.mark.parametrize("m", [1, 2, 3, 20, 100, 600])
def test_linear_over_its_operands(swz, m):
    k, n = 64, 100
    # x, dtype, ldx, W, ldw, sw, y, ldy, y_dtype, M, N, K, ws, bytes
    good = [MB, swz.SWZ_BF16, k, 3 * MB, k, 4 * MB, 5 * MB, n, swz.SWZ_BF16, m, n, k, 6 * MB, 1 << 30]
    bytes_y = m * n * 2
    for at, size in ((3, n * k), (5, n * 4)):
        for to in (good[at], good[at] + size - 4, good[at] - bytes_y + 2):
            a = list(good)
            a[6] = to
            assert swz.swz_linear_int8(*a) == swz.SWZ_EINVAL, (at, to)
    # over x: one or two rows need a workspace that they otherwise do not
    if m <= 2:
        assert swz.swz_linear_int8_workspace_size(m, n, k) == (0, 0)
        for to in (good[0], good[0] + m * k * 2 - 2, good[0] - bytes_y + 2):
            a = list(good)
            a[6] = to
            for ws, size in ((6 * MB, 256 + m * k - 1), (0, 0)):
                a[12:] = [ws, size]
                assert swz.swz_linear_int8(*a) == swz.SWZ_EINVAL, to


def test_layer_norm_over_its_operands(swz):
    m, n, bf16 = 8, 64, swz.SWZ_BF16
    size = m * n * 2
    # x, dtype, ldx, w, w_dtype, b, b_dtype, eps, y, y_dtype, ldy, mean, rstd, M, N
    good = [MB, bf16, n, 2 * MB, bf16, 3 * MB, 3, 1e-5, 4 * MB, bf16, n, 5 * MB, 6 * MB, m, n]
    changes = [{8: MB + 2}, {8: MB + size - 2}, {8: MB - size + 2}, {8: MB, 9: swz.SWZ_F16}, {8: MB, 9: 3},
               {8: MB, 10: n + 8}, {8: MB, 2: n + 8}, {8: 2 * MB}, {8: 2 * MB + 2 * n - 2}, {8: 3 * MB},
               {8: 3 * MB + 4 * n - 2}, {8: 3 * MB - size + 2}]
    for at in changes:
        a = list(good)
        for k, v in at.items():
            a[k] = v
        assert swz.swz_layer_norm(*a) == swz.SWZ_EINVAL, at
    # dy, dtype, ld, x, dtype, ld, w, dtype, mean, rstd, dx, dtype, ld, dw, db, dtype, M, N, ws, bytes
    good = [MB, bf16, n, 2 * MB, bf16, n, 3 * MB, bf16, 4 * MB, 5 * MB, 6 * MB, bf16, n, 7 * MB, 8 * MB, 3, m, n,
            9 * MB, 1 << 30]
    changes = [{10: MB + 2}, {10: MB - size + 2}, {10: MB, 11: 3}, {10: MB, 12: n + 8}, {10: 2 * MB + size - 2},
               {10: 2 * MB, 11: swz.SWZ_F16}, {10: 2 * MB, 5: n + 2}, {10: 3 * MB}, {10: 3 * MB + 2 * n - 2},
               {10: 4 * MB}, {10: 4 * MB + 4 * m - 2}, {10: 5 * MB}, {10: 5 * MB - size + 2}]
    for at in changes:
        a = list(good)
        for k, v in at.items():
            a[k] = v
        assert swz.swz_layer_norm_backward(*a) == swz.SWZ_EINVAL, at


def test_quantize_over_its_input(swz):
    m, k = 8, 64
    # x, dtype, ldx, M, K, q, ldq, scales
    good = [MB, swz.SWZ_BF16, k, m, k, 2 * MB, k, 3 * MB]
    for at in ({5: MB}, {5: MB + 2 * m * k - 16}, {5: MB - m * k + 16}, {7: MB}, {7: MB + 2 * m * k - 4},
               {7: MB - 4 * m + 4}, {5: MB + k, 6: 2 * k, 2: k + 8}):
        a = list(good)
        for i, v in at.items():
            a[i] = v
        assert swz.swz_quantize_int8(*a) == swz.SWZ_EINVAL, at
