"""The cut into workgroups that an expert product takes, and that the GPU tests reach every one of them (CPU only).

Off the GPU the compute-unit count is that of the MI355X, 256.
"""
import os
import re

import bit_weight_only_tq_amd as tq
from test_gpu_29_experts_cuts import CASES, cut_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUTS = int(re.search(r"#define TQ_MOE_CUTS (\d+)", open(os.path.join(ROOT, "include", "tq.h")).read()).group(1))


def test_the_cases_take_their_cuts():
    for (fmt, cut), sizes in CASES.items():
        assert cut_of(fmt, *sizes) == cut, (fmt, cut)


def test_no_cut_is_left_out():
    """W4A16 has no kernels of the first cut: it is not asked for."""
    want = {("ternary", i) for i in range(CUTS)} | {(f, i) for f in ("w4", "w4z") for i in range(1, CUTS)}
    assert set(CASES) == want


def test_w4a16_never_takes_the_first_cut():
    for zeros in (False, True):
        for P in (1, 2, 7, 48, 333, 4096):
            for E in (1, 8, 64, 128):
                for N in (1, 34, 4096, 28672):
                    for K in (128, 1408, 4096, 14336):
                        assert 1 <= tq.tq_moe_select_cut("w4a16", P, E, N, K, zeros) < CUTS


def test_refused_sizes():
    sel = tq.tq_moe_select_cut
    assert sel("ternary", 4, 2, 32, 64) >= 0 and sel("w4a16", 4, 2, 32, 128) >= 1
    for bad in (("ternary", 0, 2, 32, 64), ("ternary", 4, 0, 32, 64), ("ternary", 4, 65537, 32, 64), ("ternary", 4, 2, 0, 64),
                ("ternary", 4, 2, 32, 96), ("w4a16", 4, 2, 32, 64), ("ternary", 1 << 31, 2, 32, 64),
                ("ternary", 4, 2, 1 << 22, 2048), ("ternary", 4, 2, 32, 64, True)):
        assert sel(*bad) == -1, bad
