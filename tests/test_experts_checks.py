"""Refusals of the experts' and adapters' calls, by the C ABI and by the Python entry (CPU only: nothing is launched)."""
import ctypes

import pytest
import torch

import bit_weight_only_tq_amd as tq
from bit_weight_only_tq_amd import _lib

V = ctypes.c_void_p
NAME = _lib.STATUS_NAMES


def P(i):
    """Addresses 2^32 apart, never dereferenced: every call below fails a host check."""
    return V((i + 1) << 36)


def _route(**c):
    a = dict(logits=P(0), dt=0, T=9, E=8, stride=8, k=2, renorm=1, experts=P(1), weights=P(2), offsets=P(3), rows=P(4),
             places=P(5), ws=None, bytes=0, stream=None)
    a.update(c)
    return NAME[_lib.load().tq_moe_route(*a.values())]


@pytest.mark.parametrize("change, want", [
    (dict(logits=None), "TQ_ERR_NULL"), (dict(experts=None), "TQ_ERR_NULL"), (dict(weights=None), "TQ_ERR_NULL"),
    (dict(offsets=None), "TQ_ERR_NULL"), (dict(rows=None), "TQ_ERR_NULL"), (dict(places=None), "TQ_ERR_NULL"),
    (dict(dt=3), "TQ_ERR_DTYPE"), (dict(T=0), "TQ_ERR_SHAPE"), (dict(T=-1), "TQ_ERR_SHAPE"), (dict(E=0), "TQ_ERR_SHAPE"),
    (dict(E=1025, stride=1025), "TQ_ERR_SHAPE"), (dict(k=0), "TQ_ERR_SHAPE"), (dict(k=9), "TQ_ERR_SHAPE"),
    (dict(E=100, stride=100, k=65), "TQ_ERR_SHAPE"), (dict(T=1 << 30, k=2), "TQ_ERR_SHAPE"), (dict(stride=7), "TQ_ERR_VALUE"),
    (dict(experts=V(0x10002)), "TQ_ERR_ALIGN"), (dict(logits=V(0x10001)), "TQ_ERR_ALIGN"), (dict(dt=2, logits=V(0x10002)), "TQ_ERR_ALIGN"),
    (dict(T=65), "TQ_ERR_SHAPE"), (dict(T=65, ws=P(6), bytes=63), "TQ_ERR_SHAPE"),
    (dict(rows=P(4), places=V((5 << 36) + 68)), "TQ_ERR_VALUE"), (dict(experts=P(0)), "TQ_ERR_VALUE"),
    (dict(T=65, ws=P(4), bytes=64), "TQ_ERR_VALUE"),
])
def test_route(change, want):
    assert _route(**change) == want


def test_route_workspace_query():
    wb = tq.tq_moe_route_workspace_bytes
    assert wb(1, 8, 2) == wb(64, 1024, 64) == 0
    assert wb(65, 8, 2) == 2 * 8 * 4 and wb(16383, 128, 8) == 256 * 128 * 4  # chunks of 64 tokens
    assert wb(16385, 128, 8) == 129 * 128 * 4                                 # at most 256 chunks, of whole 64s
    assert wb(10, 8, 9) == wb(0, 8, 2) == wb(10, 2000, 2) == 0


def _gemm(w4=False, **c):
    a = dict(A=P(0), dt=0, T=6, P=12, E=4, N=32, K=128, w=P(1), scale=P(2))
    if w4:
        a.update(zeros=None, group=128)
    a.update(offsets=P(3), rows=P(4), bias=None, gated=0, C=P(5), stream=None)
    a.update(c)
    return NAME[(_lib.load().w4a16_moe_gemm if w4 else _lib.load().tq_moe_gemm)(*a.values())]


@pytest.mark.parametrize("w4", [False, True])
@pytest.mark.parametrize("change, want", [
    (dict(A=None), "TQ_ERR_NULL"), (dict(w=None), "TQ_ERR_NULL"), (dict(scale=None), "TQ_ERR_NULL"),
    (dict(offsets=None), "TQ_ERR_NULL"), (dict(C=None), "TQ_ERR_NULL"), (dict(dt=2), "TQ_ERR_DTYPE"),
    (dict(P=13), "TQ_ERR_SHAPE"), (dict(rows=None), "TQ_ERR_SHAPE"), (dict(T=0), "TQ_ERR_SHAPE"), (dict(T=-1), "TQ_ERR_SHAPE"),
    (dict(P=-12), "TQ_ERR_SHAPE"), (dict(E=0), "TQ_ERR_SHAPE"), (dict(E=65537), "TQ_ERR_SHAPE"), (dict(N=0), "TQ_ERR_SHAPE"),
    (dict(K=96), "TQ_ERR_SHAPE"), (dict(K=0), "TQ_ERR_SHAPE"), (dict(K=(1 << 22) + 128), "TQ_ERR_SHAPE"),
    (dict(N=33, gated=1), "TQ_ERR_SHAPE"), (dict(A=V(0x10008)), "TQ_ERR_ALIGN"), (dict(w=V(0x10008)), "TQ_ERR_ALIGN"),
    (dict(scale=V(0x10001)), "TQ_ERR_ALIGN"), (dict(offsets=V(0x10002)), "TQ_ERR_ALIGN"), (dict(rows=V(0x10002)), "TQ_ERR_ALIGN"),
    (dict(bias=V(0x10001)), "TQ_ERR_ALIGN"), (dict(C=V(0x10001)), "TQ_ERR_ALIGN"),
])
def test_products(w4, change, want):
    assert _gemm(w4, **change) == want


@pytest.mark.parametrize("w4", [False, True])
def test_products_over_their_inputs(w4):
    last = dict(A=6 * 128 * 2 - 2, w=4 * 32 * 128 // (2 if w4 else 4) - 2, scale=4 * 32 * 2 - 2, offsets=5 * 4 - 2, rows=12 * 4 - 2,
                bias=4 * 32 * 2 - 2)
    for name, at in last.items():
        assert _gemm(w4, **{name: P(7), "C": V((8 << 36) + at)}) == "TQ_ERR_VALUE", name
    first = V((8 << 36) - 12 * 32 * 2 + 2)
    assert _gemm(w4, A=P(7), C=first) == "TQ_ERR_VALUE" and _gemm(w4, rows=P(7), C=first) == "TQ_ERR_VALUE"
    if w4:
        assert _gemm(True, zeros=P(7), C=V((8 << 36) + 4 * 32 - 2)) == "TQ_ERR_VALUE"


def test_products_nothing_to_do():
    assert _gemm(T=0, P=0) == "TQ_OK" and _gemm(True, T=0, P=0, rows=None, A=None, C=None) == "TQ_OK"
    assert _gemm(True, group=64) == "TQ_ERR_GROUP" and _gemm(True, K=192) == "TQ_ERR_SHAPE"


def _combine(**c):
    a = dict(y=P(0), dt=1, T=5, P=10, N=16, k=2, places=P(1), weights=P(2), add=None, add_stride=0, out=P(3), stream=None)
    a.update(c)
    return NAME[_lib.load().tq_moe_combine(*a.values())]


@pytest.mark.parametrize("change, want", [
    (dict(y=None), "TQ_ERR_NULL"), (dict(places=None), "TQ_ERR_NULL"), (dict(weights=None), "TQ_ERR_NULL"),
    (dict(out=None), "TQ_ERR_NULL"), (dict(dt=2), "TQ_ERR_DTYPE"), (dict(T=-1), "TQ_ERR_SHAPE"), (dict(P=-1), "TQ_ERR_SHAPE"),
    (dict(N=0), "TQ_ERR_SHAPE"), (dict(k=0), "TQ_ERR_SHAPE"), (dict(add=P(4), add_stride=15), "TQ_ERR_VALUE"),
    (dict(out=P(0)), "TQ_ERR_VALUE"), (dict(out=P(2)), "TQ_ERR_VALUE"), (dict(add=P(3), add_stride=17), "TQ_ERR_VALUE"),
    (dict(add=V((4 << 36) + 2), add_stride=16), "TQ_ERR_VALUE"), (dict(y=V(0x10001)), "TQ_ERR_ALIGN"),
    (dict(weights=V(0x10002)), "TQ_ERR_ALIGN"), (dict(T=0), "TQ_OK"),
])
def test_combine(change, want):
    assert _combine(**change) == want


def _lora(**c):
    a = dict(x=P(0), xs=64, base=P(1), bs=32, dt=0, T=5, K=64, N=32, L=3, r=16, A=P(2), B=P(3), ids=P(4), scale=None,
             out=P(5), os=32, stream=None)
    a.update(c)
    return NAME[_lib.load().tq_lora(*a.values())]


@pytest.mark.parametrize("change, want", [
    (dict(x=None), "TQ_ERR_NULL"), (dict(base=None), "TQ_ERR_NULL"), (dict(A=None), "TQ_ERR_NULL"), (dict(B=None), "TQ_ERR_NULL"),
    (dict(ids=None), "TQ_ERR_NULL"), (dict(out=None), "TQ_ERR_NULL"), (dict(dt=2), "TQ_ERR_DTYPE"), (dict(T=-1), "TQ_ERR_SHAPE"),
    (dict(K=60, xs=64), "TQ_ERR_SHAPE"), (dict(K=0), "TQ_ERR_SHAPE"), (dict(N=0), "TQ_ERR_SHAPE"), (dict(L=0), "TQ_ERR_SHAPE"),
    (dict(r=0), "TQ_ERR_SHAPE"), (dict(r=12), "TQ_ERR_SHAPE"), (dict(r=264), "TQ_ERR_SHAPE"), (dict(xs=56), "TQ_ERR_VALUE"),
    (dict(bs=31), "TQ_ERR_VALUE"), (dict(os=31), "TQ_ERR_VALUE"), (dict(xs=68), "TQ_ERR_ALIGN"), (dict(x=V(0x10008)), "TQ_ERR_ALIGN"),
    (dict(A=V(0x10008)), "TQ_ERR_ALIGN"), (dict(B=V(0x10008)), "TQ_ERR_ALIGN"), (dict(out=V(0x10001)), "TQ_ERR_ALIGN"),
    (dict(out=P(0)), "TQ_ERR_VALUE"), (dict(out=P(2)), "TQ_ERR_VALUE"), (dict(out=V((2 << 36) + 64)), "TQ_ERR_VALUE"),
    (dict(out=P(1), os=40), "TQ_ERR_VALUE"), (dict(T=0), "TQ_OK"), (dict(xs=(1 << 25) + 8), "TQ_ERR_VALUE"),
    (dict(os=(1 << 25) + 1), "TQ_ERR_VALUE"), (dict(K=1 << 22, xs=1 << 22, r=136), "TQ_ERR_SHAPE"),
    (dict(N=1 << 22, bs=1 << 22, os=1 << 22, r=256), "TQ_ERR_SHAPE"),
])
def test_lora(change, want):
    assert _lora(**change) == want


H = lambda *s: torch.zeros(s, dtype=torch.float16)   # noqa: E731
F = lambda *s: torch.zeros(s)                        # noqa: E731
I = lambda *s: torch.zeros(s, dtype=torch.int32)     # noqa: E731, E741
U = lambda *s: torch.zeros(s, dtype=torch.uint8)     # noqa: E731


@pytest.mark.parametrize("call, error, match", [
    (lambda: tq.tq_moe_route(3, 2), TypeError, "logits must be a tensor"),
    (lambda: tq.tq_moe_route(F(4), 2), TypeError, "2-D"),
    (lambda: tq.tq_moe_route(F(4, 8).double(), 2), TypeError, "float16, bfloat16 or float32"),
    (lambda: tq.tq_moe_route(F(8, 4).t(), 2), ValueError, "rows of logits must be contiguous"),
    (lambda: tq.tq_moe_route(F(1, 8).expand(4, 8), 2), ValueError, "must not overlap"),
    (lambda: tq.tq_moe_route(F(4, 8), 2.5), TypeError, "integer"),
    (lambda: tq.tq_moe_route(F(4, 8), 9), tq.TQError, "TQ_ERR_SHAPE"),
    (lambda: tq.tq_moe_route(F(0, 8), 2), tq.TQError, "TQ_ERR_SHAPE"),
    (lambda: tq.tq_moe_route(F(4, 8), 2), ValueError, "device tensors"),
    (lambda: tq.tq_moe_gemm(H(4), U(2, 8, 16), H(2, 8), I(3)), TypeError, "A must be 2-D"),
    (lambda: tq.tq_moe_gemm(F(4, 64), U(2, 8, 16), H(2, 8), I(3)), TypeError, "float16 or bfloat16"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(8, 16), H(2, 8), I(3)), TypeError, "3-D uint8"),
    (lambda: tq.tq_moe_gemm(H(4, 96), U(2, 8, 24), H(2, 8), I(3)), ValueError, "multiple of 64"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 8, 15), H(2, 8), I(3)), ValueError, "codes must be"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 8, 16), H(2, 7), I(3)), ValueError, "scale must be"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 8, 16), H(2, 8), I(2)), ValueError, "offsets must have 3 entries"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 8, 16), H(2, 8), I(3), rows=I(7)), ValueError, "multiple of A's 4 rows"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 8, 16), H(2, 8), I(3), rows=I(8).long()), TypeError, "rows must be a 1-D"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 7, 16), H(2, 7), I(3), gated=True), ValueError, "even number"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 8, 16), H(2, 8), I(3), bias=H(8)), TypeError, "bias must be a 2-D"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 8, 16), H(2, 8), I(3), out=H(4, 9)), ValueError, "out must be"),
    (lambda: tq.tq_moe_gemm(H(4, 64), U(2, 8, 16), H(2, 8), I(3)), ValueError, "device tensors"),
    (lambda: tq.w4a16_moe_gemm(H(4, 64), I(2, 8, 8), H(2, 8, 1), I(3)), ValueError, "multiple of 128"),
    (lambda: tq.w4a16_moe_gemm(H(4, 128), I(2, 8, 16), H(2, 8, 2), I(3)), ValueError, "scales must be"),
    (lambda: tq.w4a16_moe_gemm(H(4, 128), I(2, 8, 16), H(2, 8, 1), I(3), zeros=U(2, 8)), TypeError, "zeros must be a 3-D"),
    (lambda: tq.w4a16_moe_gemm(H(4, 128), I(2, 8, 16), H(2, 8, 1), I(3), group_size=64), tq.TQError, "TQ_ERR_GROUP"),
    (lambda: tq.tq_moe_combine(H(8), I(4, 2), F(4, 2)), TypeError, "y must be 2-D"),
    (lambda: tq.tq_moe_combine(H(8, 16), I(4, 2), F(4, 3)), ValueError, "weights must be"),
    (lambda: tq.tq_moe_combine(H(8, 16), I(4, 2), F(4, 2), add=H(4, 15)), ValueError, "add must be"),
    (lambda: tq.tq_moe_combine(H(8, 16), I(8), F(4, 2)), TypeError, "places must be a 2-D"),
    (lambda: tq.tq_moe_combine(H(8, 16), I(4, 2), F(4, 2)), ValueError, "device tensors"),
    (lambda: tq.tq_lora(H(4, 64), H(4, 32), H(3, 16, 64), H(3, 32, 8), I(4)), ValueError, "B must be"),
    (lambda: tq.tq_lora(H(4, 64), H(4, 32), H(3, 16, 56), H(3, 32, 16), I(4)), ValueError, "A must be"),
    (lambda: tq.tq_lora(H(4, 64), H(5, 32), H(3, 16, 64), H(3, 32, 16), I(4)), ValueError, "base must be"),
    (lambda: tq.tq_lora(H(4, 64), H(4, 32).bfloat16(), H(3, 16, 64), H(3, 32, 16), I(4)), TypeError, "base must be"),
    (lambda: tq.tq_lora(H(4, 64), H(4, 32), H(3, 16, 64), H(3, 32, 16), I(5)), ValueError, "ids must have 4"),
    (lambda: tq.tq_lora(H(4, 64), H(4, 32), H(3, 16, 64), H(3, 32, 16), I(4), scale=F(2)), ValueError, "scale must have 3"),
    (lambda: tq.tq_lora(H(4, 64), H(4, 32), H(3, 16, 64), H(3, 32, 16), I(4)), ValueError, "device tensors"),
])
def test_python_entry(call, error, match):
    with pytest.raises(error, match=match):
        call()
