"""Sampling of long rows with min-p whose first part holds no logit above -inf, or only masks of the type's lowest
value: the list begun in the first pass over the row must not lose the tokens behind (fp64 oracle, tokens equal)."""
import numpy as np
import pytest
import torch

from gpu_common import log
from test_gpu_12_sample import DT, _check, _logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("mask", [float("-inf"), float("nan"), "lowest"])
@pytest.mark.parametrize("V", [65537, 70001, 150001])
def test_first_part_masked(V, mask, dt):
    """32768 masked logits, then: few, or thousands, of the type's lowest value; ordinary ones; one token."""
    t = getattr(torch, DT[dt])
    low = torch.finfo(t).min
    log(f"masked first part V={V} {dt} {mask}")
    x = torch.full((5, V), float("-inf"), dtype=t)
    x[0, 32768:] = low
    x[1, 32768:33000] = low
    x[2, 32768:] = _logits(1, V - 32768, dt)[0]
    x[3, V - 1] = low
    x[4, 40000] = 3.0
    x[:, :32768] = low if mask == "lowest" else mask
    u = np.array([0.3, 0.7, 0.5, 0.9, 0.0], dtype=np.float32)
    for T, k, p, m in ((1.0, None, None, 0.05), (0.7, 40, 0.9, 0.3), (1.0, None, 0.8, 1e-4), (1.0, 3000, None, 1.0)):
        _check(x, u, T, k, p, m)
