"""Appends and samplings of more tokens and rows than one launch has workgroups for, against torch."""
import pytest
import torch

from gpu_common import log, require_gpu

pytestmark = pytest.mark.gpu

MANY = (1 << 22) + 5


@pytest.mark.parametrize("D,rot", [(1, 0), (8, 0), (2, 2), (8, 8)])
def test_append(D, rot):
    """Element and 16-byte form, with and without rotation (by a quarter turn, which is exact)."""
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log(f"append {MANY} tokens D={D} rot={rot}")
    x = torch.randint(-100, 100, (MANY, 4, D), device=dev).half()
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    pages = -(-MANY // 16)
    kc, vc = [torch.zeros((pages, 1, 16, D), dtype=torch.float16, device=dev) for _ in range(2)]
    slots = torch.arange(MANY, device=dev).flip(0).contiguous()
    more = {}
    if rot:
        more = dict(positions=(torch.arange(MANY, device=dev) % 2).int(), interleaved=True,
                    rope=torch.tensor([[1.0] * (rot // 2) + [0.0] * (rot // 2), [0.0] * (rot // 2) + [1.0] * (rot // 2)], device=dev))
    out = tq.tq_kv_append(q, k, v, kc, vc, slots, **more)

    def turned(t):
        if not rot:
            return t
        y = torch.stack([-t[..., 1::2], t[..., ::2]], -1).flatten(-2)
        return torch.where((torch.arange(MANY, device=dev) % 2 == 1)[:, None, None], y, t)

    assert torch.equal(out, turned(q))
    for cache, new in ((kc, turned(k)), (vc, v)):
        assert torch.equal(cache.reshape(-1, D)[:MANY], new[:, 0].flip(0))


def test_sample():
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log(f"sample {MANY} rows")
    x = torch.zeros((MANY, 4), dtype=torch.bfloat16, device=dev)
    at = torch.randint(0, 4, (MANY,), device=dev)
    x.scatter_(1, at[:, None], 5.0)
    u = ((torch.arange(MANY, device=dev) % 8) / 8).float()
    tokens, logprobs = tq.tq_sample(x, u, top_k=torch.ones(MANY, dtype=torch.int32, device=dev))
    assert torch.equal(tokens.long(), at) and not logprobs.any()
    tokens, logprobs = tq.tq_sample(torch.zeros_like(x), u)  # four tokens of one weight
    assert torch.equal(tokens, (u * 4).int()) and bool((logprobs + 1.3862944 < 1e-6).all())
