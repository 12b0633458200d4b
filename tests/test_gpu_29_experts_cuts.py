"""Every compiled kernel of the experts' products: each cut of a call, format, type, gated and plain, against the fp64 oracle.

test_experts_cuts.py asserts on the host that the cases below take the cuts they stand for and leave none out.
"""
import pytest

import bit_weight_only_tq_amd as tq
from gpu_common import log
from test_gpu_23_experts import check
from test_gpu_25_moe_layer import uneven

pytestmark = pytest.mark.gpu

# (format, cut): experts, rows of each in the mean, weight rows, columns
CASES = {
    ("ternary", 0): (2, 1, 17772, 832), ("ternary", 1): (35, 1, 520, 2048), ("ternary", 2): (3, 1, 34, 4160),
    ("ternary", 3): (40, 3, 2080, 320), ("ternary", 4): (2, 1, 34, 320), ("ternary", 5): (6, 9, 1032, 576),
    ("ternary", 6): (12, 700, 34, 128), ("ternary", 7): (8, 700, 528, 320), ("ternary", 8): (8, 2500, 142, 320),
    ("w4", 1): (35, 1, 520, 1408), ("w4", 2): (3, 1, 34, 4224), ("w4", 3): (40, 3, 2080, 384), ("w4", 4): (2, 1, 8200, 384),
    ("w4", 5): (6, 9, 1032, 640), ("w4", 6): (12, 700, 34, 128), ("w4", 7): (7, 2773, 386, 256), ("w4", 8): (12, 2540, 142, 896),
    ("w4z", 1): (12, 1, 2080, 512), ("w4z", 2): (3, 1, 34, 4224), ("w4z", 3): (8, 1, 2080, 128), ("w4z", 4): (12, 1, 2080, 256),
    ("w4z", 5): (2, 20, 34, 512), ("w4z", 6): (24, 700, 34, 128), ("w4z", 7): (3, 2500, 530, 256), ("w4z", 8): (7, 2773, 386, 128),
}


def cut_of(fmt, E, rows, N, K):
    return tq.tq_moe_select_cut("ternary" if fmt == "ternary" else "w4a16", E * rows, E, N, K, zeros=fmt == "w4z")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt, cut", CASES)
def test_every_kernel(fmt, cut, gated, dt):
    E, rows, N, K = CASES[fmt, cut]
    log(f"experts {fmt} cut {cut} E={E} rows={rows} N={N} K={K} gated={gated} {dt}")
    assert cut_of(fmt, E, rows, N, K) == cut
    check(fmt, E, N, K, uneven(E, rows, N), dt, seed=cut, fan=int(gated), bias=True, gated=gated)
