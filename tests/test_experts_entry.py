"""What the Python entry of the experts and adapters refuses beside test_experts_checks.py (CPU only)."""
import pytest
import torch

import bit_weight_only_tq_amd as tq

H = lambda *s: torch.zeros(s, dtype=torch.float16)   # noqa: E731
I = lambda *s: torch.zeros(s, dtype=torch.int32)     # noqa: E731, E741
U = lambda *s: torch.zeros(s, dtype=torch.uint8)     # noqa: E731


def test_weights_of_the_other_format():
    """A product takes the weights of its own format: the other's are neither read as its own nor multiplied as theirs."""
    with pytest.raises(TypeError, match="codes must be a 3-D uint8 tensor"):
        tq.tq_moe_gemm(H(4, 128), I(2, 8, 16), H(2, 8, 1), I(3))
    with pytest.raises(TypeError, match="qweight must be a 3-D int32 tensor"):
        tq.w4a16_moe_gemm(H(4, 128), U(2, 8, 32), H(2, 8), I(3))
    with pytest.raises(TypeError, match="qweight must be a 3-D int32 tensor"):
        tq.w4a16_moe_gemm(H(4, 128), U(2, 8, 32), H(2, 8), I(3), zeros=U(2, 8, 1))
