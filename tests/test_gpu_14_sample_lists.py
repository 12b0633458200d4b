"""Sampling where the candidates' list is short, long, begun early, full of ties or overflowing, against the fp64 oracle
(tokens equal, log probabilities within the rounding derived in test_gpu_12_sample)."""
import numpy as np
import pytest

from gpu_common import log
from test_gpu_12_sample import DT, _check, _logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [513, 2206, 4096, 4097, 9001, 70001])
@pytest.mark.parametrize("k", [2, 63, 64, 65, 300, 512, 513, 1000, 1024, 1025])
def test_list_lengths(V, k, dt):
    """Lists around the lengths at which their handling changes, in 16 bits with ties at the cut."""
    log(f"sample V={V} k={k} {dt}")
    u = np.random.default_rng(k).random(3).astype(np.float32)
    _check(_logits(3, V, dt, k), u, 0.9, k)
    _check(_logits(3, V, dt, k + 1), u, 1.3, k, 0.9)
    _check(_logits(3, V, dt, k + 2), u, 0.8, k, 0.95, 0.001)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("min_p", [1e-6, 1e-3, 0.02, 0.3, 1.0])
def test_list_begun_in_the_first_pass(min_p, dt):
    """Long rows with min-p, the best token in the first part of the row, in the last, and everywhere."""
    V = 140001 if dt == "f32" else 150001
    for where in (0, 70000, V - 1):
        log(f"sample V={V} {dt} min_p={min_p} best at {where}")
        x = _logits(2, V, dt, 4)
        x[0, where] = 30.0
        u = np.random.default_rng(5).random(2).astype(np.float32)
        _check(x, u, 0.7, None, None, min_p)
        _check(x, u, 1.0, 40, 0.9, min_p)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_lists_that_overflow(dt):
    """Rows in which thousands of tokens pass every bound: flat, rising, and of two values."""
    import torch
    V = 70001
    rise = torch.linspace(0, 3, V)
    x = torch.stack([torch.zeros(V), rise, rise.flip(0), (torch.arange(V) % 7 == 0).float()]).to(getattr(torch, DT[dt]))
    u = np.array([0.1, 0.5, 0.9, 0.3], dtype=np.float32)
    log(f"overflow {dt}")
    for T, k, p, m in ((1.0, 1000, None, None), (1.0, 1000, 0.5, 0.1), (0.8, None, 0.5, None), (2.0, None, 0.9, 0.05),
                       (1.0, 30000, None, None), (1.0, 30000, 0.7, 0.2), (0.5, None, None, 0.4), (20.0, None, 0.6, None)):
        _check(x, u, T, k, p, m)


def test_tokens_of_hardly_any_weight():
    """u = 0 takes the first kept token however small, and small ones do not disturb the others."""
    import torch
    log("tiny weights")
    x = torch.full((3, 5000), -30.0)
    x[:, 2500] = 10.0
    x[1, 4000], x[2, 10] = 9.0, -700.0
    for T in (0.06, 0.5, 1.0):
        _check(x, [0.0, 0.3, 0.999999], T, 50)
        _check(x, [0.0, 0.0, 0.0], T, 50, 0.99)
        _check(x, [0.0, 0.0, 0.5], T)


def test_peaks_in_one_thread_s_share():
    """The best tokens side by side: a bound taken from the threads' maxima still holds k tokens."""
    import torch
    log("side by side")
    for dt in ("f32", "f16"):
        x = _logits(2, 32000, dt, 1)
        x[0, 1000:1064] = torch.arange(64).to(x.dtype) / 8 + 20
        x[1, 31990:] = 25.0
        for k in (3, 10, 50, 64, 200):
            _check(x, [0.35, 0.7], 5.0, k)
            _check(x, [0.35, 0.7], 5.0, k, 0.8)
