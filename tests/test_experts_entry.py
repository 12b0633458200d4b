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


@pytest.mark.parametrize("i, name", [(0, "x"), (1, "base"), (2, "A"), (3, "B"), (5, "scale"), (6, "out")])
def test_adapters_that_want_a_gradient(i, name):
    """No gradient is lost in silence; without gradients the same tensors go on to the next check."""
    args = [H(4, 64), H(4, 32), H(3, 16, 64), H(3, 32, 16), I(4), torch.zeros(3), H(4, 32)]
    args[i].requires_grad_(True)
    call = lambda: tq.tq_lora(*args[:5], scale=args[5], out=args[6])  # noqa: E731
    with pytest.raises(ValueError, match=f"{name} requires a gradient"):
        call()
    for off in (torch.no_grad, torch.inference_mode):
        with off(), pytest.raises(ValueError, match="device tensors"):
            call()
