"""Routing, weighted sums and adapters of more rows than one launch takes, against torch.

Values are small whole numbers and weights powers of two, so every result is exact.
"""
import pytest

from gpu_common import log, require_gpu

pytestmark = pytest.mark.gpu


def test_route():
    """Chunks of many passes: the largest two of five distinct logits, and the stable order of the pairs."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    T, E, k = (1 << 22) + 5, 5, 2
    log(f"route {T} tokens")
    x = torch.argsort(torch.rand((T, E), device=dev), dim=1).to(torch.bfloat16)
    x[::7, 1:] = float("-inf")  # one expert alone
    r = tq.tq_moe_route(x, k)
    order = torch.argsort(x.float(), dim=1, descending=True, stable=True)[:, :k].int()
    order[::7, 1] = -1
    assert torch.equal(r.experts, order)
    one = (order[:, 1] < 0).float()
    first = 1.0 / (1.0 + torch.exp(torch.tensor(-1.0, device=dev)))
    want = torch.stack([one + (1 - one) * first, (1 - one) * (1 - first)], 1)
    assert bool(((r.weights - want).abs() <= 8 * 2.0 ** -24).all())
    flat = torch.where(order < 0, E, order).reshape(-1)
    rows = torch.argsort(flat, stable=True)
    assert torch.equal(r.rows, rows.int())
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    assert r.offsets.tolist() == [0] + torch.cumsum(counts, 0).tolist()
    places = torch.empty_like(rows)
    places[rows] = torch.arange(T * k, device=dev)
    assert torch.equal(r.places, torch.where(order < 0, -1, places.view(T, k)).int())


@pytest.mark.parametrize("N", [8192, 8187])
def test_combine(N):
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    T, P = (1 << 20) + 2050, 40
    log(f"combine {T} x {N}")
    y = torch.randint(-8, 9, (P, N), device=dev).half()
    places = torch.randint(0, P, (T, 2), device=dev, dtype=torch.int32)
    weights = torch.tensor([0.5, -2.0], device=dev).expand(T, 2).contiguous()
    out = tq.tq_moe_combine(y, places, weights)
    for t in range(0, T, 1 << 16):
        p = places[t:t + (1 << 16)].long()
        assert torch.equal(out[t:t + (1 << 16)], y[p[:, 0]] * 0.5 - y[p[:, 1]] * 2.0), t


@pytest.mark.parametrize("N, r", [(8, 8), (9, 8), (16, 32), (11, 72), (8, 136)])
def test_lora(N, r):
    """Through LDS, and by direct loads where rows or ranks ask for them; a tail of few rows in a launch of its own."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    T, K, L = (1 << 20) + 19, 64, 3
    log(f"lora {T} rows N={N} r={r}")
    x = torch.randint(-2, 3, (T, K), device=dev).half()
    base = torch.randint(-8, 9, (T, N), device=dev).half()
    A, B = torch.zeros((L, r, K), device=dev), torch.zeros((L, N, r), device=dev)
    for l in range(L):  # one column of x a rank, two ranks a column
        A[l, torch.arange(r), torch.randint(0, K, (r,))] = 1.0
        for n in range(N):
            B[l, n, torch.randperm(r)[:2]] = torch.tensor([1.0, -2.0], device=dev)
    ids = (torch.arange(T, device=dev) // 1000 % (L + 1) - 1).int()
    out = tq.tq_lora(x, base, A.half(), B.half(), ids, scale=torch.tensor([1.0, 0.5, 2.0], device=dev))
    both = torch.cat([torch.zeros((1, N, K), device=dev), torch.bmm(B, A) * torch.tensor([1.0, 0.5, 2.0], device=dev)[:, None, None]])
    for t in range(0, T, 1 << 17):
        at = slice(t, t + (1 << 17))
        want = base[at].float()
        for l in range(L + 1):
            m = ids[at] == l - 1
            want[m] += x[at][m].float() @ both[l].t().contiguous()
        assert torch.equal(out[at].float(), want), t
