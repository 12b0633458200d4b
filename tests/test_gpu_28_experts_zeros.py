"""Zero points of every 8-bit value in w4a16_moe_gemm: a weight is (q - zero) * scale in both types, exactly."""
import numpy as np
import pytest

from gpu_common import log
from moe_common import to_dev
from test_gpu_23_experts import call, compare, make, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E, N, K, counts", [(3, 40, 128, [2, 0, 1]), (2, 272, 640, [1, 2]), (2, 130, 17408, [2, 1]), (3, 96, 1408, [20, 9, 13]),
                                             (2, 528, 512, [33, 40]), (2, 272, 512, [300, 513])])
def test_zero_points_of_every_value(E, N, K, counts, gated, dt):
    import torch
    log(f"experts zero points E={E} N={N} K={K} counts={counts} gated={gated} {dt}")
    d, h = make("w4z", E, N, K, counts, dt, 21)
    scale = values(d["packed"]["scale"])[..., None]
    old = d["packed"]["zeros"].cpu().numpy().astype(np.float64)[..., None]
    new = np.random.default_rng(22).integers(0, 256, old.shape[:-1]).astype(np.uint8)
    new.reshape(-1)[:256] = np.arange(256)[:new.size]
    q = np.rint(h["W"].reshape(*old.shape[:-1], 128) / scale) + old
    assert q.min() == 0 and q.max() == 15
    h["W"] = ((q - new.astype(np.float64)[..., None]) * scale).reshape(E, N, K)
    d["packed"]["zeros"] = to_dev(new, d["A"].device)
    out = torch.full((h["P"], N // 2 if gated else N), 123.0, dtype=d["A"].dtype, device=d["A"].device)
    A = d["A"] * 0.125
    call(A, d["packed"], d["off"], gated=gated, out=out)
    torch.cuda.synchronize()
    h["A"] = values(A)
    compare(values(out), h, K, dt, gated, "zero points")
