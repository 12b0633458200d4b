"""Experts and adapters beside the packed linear layers.

A mixture of experts whose experts are packed layers of this library: routing,
the products grouped by expert, the weighted sum; and low-rank adapters of many
requests beside a shared projection.  Like the calls of serving.py these go
through _serving.so (csrc/binding.cpp), which checks tensors' types, shapes,
strides and devices, allocates what is not given and calls the entry points of
the same names in include/tq.h: TypeError and ValueError come from its checks,
TQError from the library's.  There is no CPU fallback, and no backward pass:
results carry no gradient.

    r = tq_moe_route(logits, top_k)
    h = w4a16_moe_gemm(x, w13, s13, r.offsets, rows=r.rows, gated=True)
    y = w4a16_moe_gemm(h, w2, s2, r.offsets)
    out = tq_moe_combine(y, r.places, r.weights, add=residual)

Experts are packed as one matrix of E * N rows and viewed by expert:
``codes.view(E, N, -1)``.
"""

from typing import NamedTuple

from . import _lib
from .serving import _entry, _result


class MoeRoute(NamedTuple):
    """The experts of a batch of tokens (device tensors): see tq_moe_route."""
    experts: object  # int32 [T, k] experts, largest logit first, -1 without one
    weights: object  # fp32 [T, k]
    offsets: object  # int32 [E + 1] first place of each expert
    rows: object     # int32 [T * k] pair (t * k + j) at each place
    places: object   # int32 [T, k] place of each pair, -1 without an expert


def tq_moe_route_workspace_bytes(T: int, E: int, top_k: int) -> int:
    """Bytes of workspace tq_moe_route needs (0: none)."""
    return int(_lib.load().tq_moe_route_workspace_bytes(T, E, top_k))


def tq_moe_route(logits, top_k: int, renormalize: bool = True, out: MoeRoute = None, workspace="auto") -> MoeRoute:
    """The top_k experts of each token, their weights, and the pairs sorted by expert.

    logits [T, E] fp16, bf16 or fp32 (rows may be strided), T >= 1, E <= 1024, top_k <= 64;
    weights: softmax over the chosen experts, or over all with renormalize=False.
    out: a MoeRoute to write into.  workspace: "auto", or a contiguous device
    tensor of tq_moe_route_workspace_bytes bytes, of any contents (None where
    that is 0)."""
    r = _result("tq_moe_route", _entry().moe_route(logits, top_k, renormalize, out, workspace))
    return r if out is not None else MoeRoute(*r)


def tq_moe_gemm(A, codes, scale, offsets, rows=None, bias=None, gated: bool = False, out=None):
    """C[p] = A[row(p)] @ dequant(codes[e], scale[e])^T (+ bias[e]) for offsets[e] <= p < offsets[e + 1].

    A [T, K] fp16/bf16; codes uint8 [E, N, K / 4], scale fp16 [E, N]; offsets
    int32 [E + 1].  rows int32 [P], P a multiple of T: row(p) is rows[p] // (P / T);
    None: row(p) is p.  bias [E, N].  gated: the first N / 2 weight rows are the
    gate g, the others u, and C[p] = g / (1 + exp(-g)) * u, [P, N / 2].  Rows
    behind offsets[E] are not written."""
    return _result("tq_moe_gemm", _entry().moe_gemm(A, codes, scale, None, offsets, rows, bias, gated, out, False))


def w4a16_moe_gemm(A, qweight, scales, offsets, rows=None, zeros=None, bias=None, group_size: int = 128,
                   gated: bool = False, out=None):
    """tq_moe_gemm with W4A16 experts: qweight int32 [E, N, K / 8], scales fp16 [E, N, K / 128], zeros uint8
    [E, N, K / 128] (any values) or None for 8."""
    if group_size != 128:
        _lib._check("w4a16_moe_gemm", 5)  # TQ_ERR_GROUP
    return _result("w4a16_moe_gemm", _entry().moe_gemm(A, qweight, scales, zeros, offsets, rows, bias, gated, out, True))


def tq_moe_select_cut(fmt: str, P: int, E: int, N: int, K: int, zeros: bool = False) -> int:
    """Which of the library's cuts into workgroups a product of these sizes takes ("ternary", "w4a16"); -1: refused."""
    return int(_lib.load().tq_moe_select_cut({"ternary": 0, "w4a16": 1}[fmt], int(zeros), P, E, N, K))


def tq_moe_combine(y, places, weights, add=None, out=None):
    """out[t] = add[t] + sum over j of weights[t, j] * y[places[t, j]]; -> [T, N].

    y [P, N] fp16/bf16; places int32 [T, k] (outside [0, P): adds nothing), weights
    fp32 [T, k]; add [T, N] (rows may be strided).  out may be add."""
    return _result("tq_moe_combine", _entry().moe_combine(y, places, weights, add, out))


def tq_lora(x, base, A, B, ids, scale=None, out=None):
    """base[t] + scale[l] * (x[t] @ A[l]^T) @ B[l]^T, l = ids[t]; base[t] where ids[t] is outside [0, L).

    x [T, K] and base [T, N] fp16/bf16 (rows may be strided); A [L, r, K], B
    [L, N, r], r a multiple of 8 up to 256; ids int32 [T]; scale fp32 [L].  out may
    be base: the update is then made in place.  Forward only: a tensor that requires
    a gradient is refused, unless gradients are off (torch.no_grad())."""
    return _result("tq_lora", _entry().lora(x, base, A, B, ids, scale, out))
