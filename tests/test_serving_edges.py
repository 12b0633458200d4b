"""Host checks of the serving calls at their edges: what is allowed is not refused (CPU only)."""
import pytest

from bit_weight_only_tq_amd import _lib
from test_serving_checks import ATTN, PLAN, V, call


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_attention_of_no_tokens(lib):
    """A step in which every request rests has no new tokens, and none as the most of a request."""
    assert call(lib, "tq_paged_attention", ATTN, T=0, max_q=0) == "TQ_OK"
    assert call(lib, "tq_paged_attention", ATTN, T=0, max_q=0, max_kv=0, q=None) == "TQ_OK"
    assert call(lib, "tq_paged_attention", ATTN, T=0, max_q=-1) == "TQ_ERR_SHAPE"
    assert call(lib, "tq_paged_attention", ATTN, T=1, max_q=0) == "TQ_ERR_SHAPE"


OUTPUTS = {"cu": 5 * 4, "kv": 4 * 4, "pos": 7 * 4, "slots": 7 * 8, "state": 2 * 4}  # bytes for B = 4, T = 7
INPUTS = {"ctx": 4 * 4, "new": 4 * 4, "table": (3 * 8 + 8) * 4, "free": 10 * 4, "head": 4}


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("other", [*INPUTS, *OUTPUTS])
def test_plan_refuses_outputs_over_its_inputs(lib, out, other):
    """Workgroups read the lengths, the table and the free list while others write: what is written lies by itself."""
    if out == other:
        return
    apart = {n: V(0x100000 * (i + 1)) for i, n in enumerate([*INPUTS, *OUTPUTS])}
    size = {**INPUTS, **OUTPUTS}
    for at in (apart[other].value, apart[other].value + size[other] - 4, apart[other].value - size[out] + 8):
        if out == "slots" and at % 8:
            at -= 4
        assert call(lib, "tq_paged_plan", PLAN, **dict(apart, **{out: V(at)})) == "TQ_ERR_VALUE"


def test_plan_outputs_side_by_side(lib):
    """Outputs may touch each other and the inputs: the checks pass, and without a device the launch is what fails."""
    at, where = 0x100000, {}
    for name, size in (*INPUTS.items(), ("slots", 56), ("cu", 20), ("kv", 16), ("pos", 28), ("state", 8)):
        at = -(-at // 8) * 8 if name == "slots" else at
        where[name] = V(at)
        at += size
    import torch
    if not torch.cuda.is_available():
        assert call(lib, "tq_paged_plan", PLAN, **where) == "TQ_ERR_HIP"


@pytest.mark.parametrize("change", [
    dict(B=1 << 24, T=1), dict(B=1 << 30, T=3), dict(T=1 << 30, B=1), dict(T=(1 << 31) - 1, Hq=64, Hkv=1),
])
def test_attention_of_more_workgroups_than_a_launch_takes(lib, change):
    """Refused on the host, where a launch of 2^32 threads would be the runtime's to judge."""
    assert call(lib, "tq_paged_attention", ATTN, **change) == "TQ_ERR_SHAPE"
