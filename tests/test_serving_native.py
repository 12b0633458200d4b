"""The native entry of the serving calls: what is not a tensor or a number is refused before any device call (CPU only)."""
import pytest
import torch

import bit_weight_only_tq_amd as tq

I = torch.zeros(3, dtype=torch.int32)  # noqa: E741
H = torch.zeros((3, 1, 64), dtype=torch.float16)
C = torch.zeros((4, 1, 16, 64), dtype=torch.float16)


@pytest.mark.parametrize("call", [
    lambda: tq.tq_paged_plan([1, 2], I, I.view(3, 1), I, I[:1], 3),
    lambda: tq.tq_paged_plan(I, I, I.view(3, 1), I, I[:1], 3.5),
    lambda: tq.tq_paged_plan(I, I, I.view(3, 1), I, I[:1], 3, out=[I] * 5),
    lambda: tq.tq_kv_append(H, None, H, C, C, torch.zeros(3, dtype=torch.int64)),
    lambda: tq.tq_kv_append(3, H, H, C, C, torch.zeros(3, dtype=torch.int64)),
    lambda: tq.tq_paged_attention(H, C, C, I.view(1, 3), I[:2], I[:1], "3", 40),
    lambda: tq.tq_paged_attention(H, C, C, I.view(1, 3), I[:2], I[:1], 3, 40, scale="x"),
    lambda: tq.tq_paged_attention(H, C, C, I.view(1, 3), I[:2], I[:1], 3, 40, workspace=5),
    lambda: tq.tq_sample(None, torch.zeros(2)),
    lambda: tq.tq_sample(torch.zeros((2, 9)), torch.zeros(2), out=(I,)),
])
def test_not_a_tensor_or_a_number(call):
    with pytest.raises(TypeError):
        call()


def test_numbers_past_64_bits():
    with pytest.raises(ValueError, match="64 bits"):
        tq.tq_paged_plan(I, I, I.view(3, 1), I, I[:1], 1 << 70)


def test_messages_name_the_argument():
    with pytest.raises(TypeError, match="new_lens must be a 1-D"):
        tq.tq_paged_plan(I, I.long(), I.view(3, 1), I, I[:1], 3)
    with pytest.raises(ValueError, match="u must have 2 entries, got 3"):
        tq.tq_sample(torch.zeros((2, 9)), torch.zeros(3))
    with pytest.raises(ValueError, match="k and v must have the cache's 1 heads, got 2 and 1"):
        tq.tq_kv_append(None, H.expand(3, 2, 64).contiguous(), H, C, C, torch.zeros(3, dtype=torch.int64))


def test_every_source_is_built():
    """Each kernel and API file of csrc is one of the library's sources."""
    import os
    from bit_weight_only_tq_amd import build
    names = {f for f in os.listdir(build.CSRC) if f.endswith(".hip") or f.startswith("api")}
    assert names == set(build.SOURCES)
