"""One token or one head in a tensor whose stride over it is no multiple of a vector: such strides lead nowhere."""
import pytest
import torch

from gpu_common import log, require_gpu
from test_gpu_11_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (1, 1)])
@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
def test_attention_of_one_token(dt, D, Hq, Hkv):
    log(f"one token {dt} D={D} Hq={Hq}")
    c = Case([1], [200], Hq, Hkv, D, 16, dt)
    q = torch.empty_strided((1, Hq, D), (Hq * D + 3, D, 1), dtype=c.dt, device=require_gpu())
    q.copy_(c.q)
    assert q.stride(0) % 8 and torch.equal(c.run(q=q)[0], c.run()[0])
    c.check(c.run(q=q))


def test_attention_of_one_head():
    log("one head")
    c = Case([3, 40], [60, 70], 1, 1, 64, 16, "f16")
    q = torch.empty_strided((43, 1, 64), (64, 65, 1), dtype=c.dt, device=require_gpu())
    q.copy_(c.q)
    assert torch.equal(c.run(q=q)[0], c.run()[0])
    c.check(c.run(q=q))


@pytest.mark.parametrize("rot", [0, 64])
def test_append_of_one_token(rot):
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log(f"append one token rot={rot}")
    x = torch.empty_strided((1, 4, 64), (4 * 64 + 5, 64, 1), dtype=torch.float16, device=dev)
    x.normal_()
    q, k, v = x.split([2, 1, 1], 1)
    slots = torch.tensor([21], device=dev)
    more = dict(positions=torch.tensor([3], dtype=torch.int32, device=dev), rope=torch.rand((9, 64), device=dev)) if rot else {}
    got = [torch.zeros((2, 1, 16, 64), dtype=torch.float16, device=dev) for _ in range(4)]
    a = tq.tq_kv_append(q, k, v, got[0], got[1], slots, **more)
    b = tq.tq_kv_append(q.contiguous(), k.contiguous(), v.contiguous(), got[2], got[3], slots, **more)
    assert torch.equal(a, b) and torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
    assert torch.equal(got[1][1, 0, 5], v[0, 0])
