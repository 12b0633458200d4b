"""What the adapters' kernel reads of B, walked on the host over whole calls (CPU only: the header is compiled with g++).

A buffer load is bounded by its lane's own offset alone: every offset must name eight values of the adapter that the call
needs, or lie past the buffer's end, also where the last columns are no whole step and waves have no column at all.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

from bit_weight_only_tq_amd import build

SOURCE = r"""
#include "tq_lora_index.h"
#include <vector>
// 0, or the number of the rule that a read breaks.  seen[n]: how many lanes took column n's ranks 0 .. 7.
extern "C" uint32_t offset(int r, int n, int i16, int g, int t, int st) { return tq::lora_b_lane(r, i16, g, t, st) + tq::lora_b_step(r, n); }
extern "C" int walk(int N, int r, int RT, int W, int cols, int* seen) {
    const int kKs = (RT + 1) / 2;
    const uint32_t bytes = (uint32_t)N * (uint32_t)r * 2u;
    for (int n_lo = 0; n_lo < N; n_lo += cols) {
        const int n_hi = n_lo + cols < N ? n_lo + cols : N;
        for (int wave = 0; wave < W; ++wave)
            for (int i = 0; tq::lora_step(n_lo, cols, W, wave, i) < n_hi; ++i) {
                const int n = tq::lora_step(n_lo, cols, W, wave, i);
                for (int lane = 0; lane < 64; ++lane)
                    for (int t = 0; t < 2; ++t)
                        for (int st = 0; st < kKs; ++st) {
                            const int g = lane >> 4, i16 = lane & 15, row = n + 8 * (i16 >> 2) + 4 * t + (i16 & 3);
                            const uint32_t off = offset(r, n, i16, g, t, st);
                            const bool wanted = row < N && 32 * st + 8 * g < r;
                            if (wanted && off != ((uint32_t)row * r + 32 * st + 8 * g) * 2u) return 1;
                            if (wanted && off + 16 > bytes) return 2;
                            if (!wanted && off < bytes) return 3;
                            if (wanted && st == 0 && g == 0) ++seen[row];
                        }
            }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    folder = tmp_path_factory.mktemp("lora_index")
    source, lib = folder / "walk.cpp", folder / "walk.so"
    source.write_text(SOURCE)
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, str(source), "-o", str(lib)], check=True)
    loaded = ctypes.CDLL(str(lib))
    loaded.offset.restype = ctypes.c_uint32
    return loaded


@pytest.mark.parametrize("RT, W, ranks", [(1, 16, (8, 16)), (1, 8, (8, 16)), (2, 8, (24, 32)), (4, 8, (40, 48, 64)), (8, 8, (72, 128)),
                                          (16, 8, (136, 256))])
@pytest.mark.parametrize("N", [1, 7, 8, 31, 33, 100, 513, 1025, 4096, 4101])
def test_reads_of_b(library, RT, W, ranks, N):
    for r in ranks:
        for passes in (1, 2, 3, 9):
            seen = (ctypes.c_int * N)()
            assert library.walk(N, r, RT, W, 32 * W * passes, seen) == 0
            assert all(s == 1 for s in seen)  # each column by one lane


def test_the_kernel_reads_b_through_it():
    """No scalar offset on the loads of B: that is not part of the bounds check."""
    text = open(os.path.join(build.CSRC, "lora.hip")).read()
    assert text.count("raw_buffer_load_b128(bbuf") == 1
    assert "raw_buffer_load_b128(bbuf, b_lane[t][st] + lora_b_step(a.r, n), 0, 0)" in text
    assert "b_lane[t][st] = lora_b_lane(a.r, i16, g, t, st)" in text


def test_the_largest_matrix(library):
    """2^29 values: the last row is read, rows and ranks that are not there lie past the end, without wrapping."""
    end = 1 << 30
    for r, N in ((128, 1 << 22), (256, 1 << 21)):
        for n in range(N - 32, N + 512, 32):
            for i16 in range(16):
                for t in (0, 1):
                    row = n + 8 * (i16 >> 2) + 4 * t + (i16 & 3)
                    off = library.offset(r, n, i16, 3, t, r // 32 - 1)
                    assert off == (row * r + r - 8) * 2 and (off < end) == (row < N)
        assert all(library.offset(r - 8, n, 15, 3, 1, r // 32 - 1) >= end for n in (0, N - 32, N + 480))
