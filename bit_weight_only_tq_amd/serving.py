"""The serving operators of libtq.so.

The step of a served model that uses the packed linear layers also plans its
paged cache, appends keys and values to it, attends over its pages and samples
its next tokens.  The calls go through _serving.so (csrc/binding.cpp), which
checks tensors' types, shapes, strides and devices, allocates what is not given
and calls the entry points of the same names in include/tq.h: TypeError and
ValueError come from its checks, TQError from the library's.  As in _lib.py
there is no CPU fallback.
"""

from typing import NamedTuple

from . import _lib

_native = None


def _entry():
    """The module _serving, behind libtq.so and torch (whose libraries it needs)."""
    global _native
    if _native is None:
        _lib.load()
        try:
            from . import _serving
        except ImportError as e:
            raise RuntimeError(f"_serving.so not built or not loadable ({e}): run `python -m bit_weight_only_tq_amd.build`") from e
        _native = _serving
    return _native


def _result(fn, r):
    """What a call returned; a status instead raises TQError."""
    if type(r) is int:
        _lib._check(fn, r)
    return r


# --------------------------------------------------------------------- plan

class PagedPlan(NamedTuple):
    """One step's plan (device tensors): see tq_paged_plan."""
    cu_q: object       # int32 [B + 1] offsets of the requests' new tokens
    kv_lens: object    # int32 [B] lengths after the step
    positions: object  # int32 [T] position of each new token
    slots: object      # int64 [T] slot of each new token, -1 without one
    state: object      # int32 [2] free-list head after the step, tokens without a slot


def tq_paged_plan(ctx_lens, new_lens, page_table, free_pages, free_head, tokens: int, page_size: int = 16,
                  out: PagedPlan = None) -> PagedPlan:
    """Page tables, offsets, positions and slots of a step, from its requests' lengths.

    ctx_lens, new_lens: int32 [B]; page_table: int32 [B, width], updated in
    place (rows may be strided); free_pages: int32 [n]; free_head: int32 [1],
    read only: the head after the step is state[0]; tokens: entries of
    positions and slots, at least new_lens' sum (a larger number pads with
    slot -1).  out: a plan to write into, for steps replayed from a graph; none
    of it may lie over the inputs (kv_lens is not ctx_lens, state not free_head)."""
    r = _result("tq_paged_plan", _entry().paged_plan(ctx_lens, new_lens, page_table, free_pages, free_head, tokens, page_size,
                                                     out))
    return r if out is not None else PagedPlan(*r)


# ------------------------------------------------------------------- append

def tq_kv_append(q, k, v, k_cache, v_cache, slots, positions=None, rope=None, interleaved: bool = False, out=None):
    """Rotates q and k by their positions and stores k and v in their slots; -> rotated q.

    q [T, Hq, D] (or None), k and v [T, Hkv, D]: fp16/bf16, any token and head
    strides; k_cache, v_cache [pages, Hkv, page_size, D]; slots int64 [T];
    positions int32 [T] and rope fp32 [rows, rot] (rot / 2 cosines, then
    rot / 2 sines) together, or neither: then nothing is rotated and the
    result is a copy of q.  out: where the rotated queries go, contiguous."""
    return _result("tq_kv_append", _entry().kv_append(q, k, v, k_cache, v_cache, slots, positions, rope, interleaved, out))


# ---------------------------------------------------------------- attention

def tq_paged_attention_workspace_bytes(tokens: int, Hq: int, Hkv: int, D: int, B: int, max_q: int, max_kv: int,
                                       window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace tq_paged_attention uses for its fastest schedule (0: none)."""
    return int(_lib.load().tq_paged_attention_workspace_bytes(tokens, Hq, Hkv, D, B, max_q, max_kv, window, sinks))


def tq_paged_attention(q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q: int, max_kv: int, scale: float = None,
                       window: int = 0, sinks: int = 0, return_lse: bool = False, out=None, workspace="auto"):
    """Attention of each request's new tokens over its pages; -> out [T, Hq, D], or (out, lse [T, Hq] fp32).

    q [T, Hq, D] fp16/bf16 (token and head strides free, multiples of 8);
    k_cache, v_cache [pages, Hkv, page_size, D] holding the new tokens already;
    page_table int32 [B, width]; cu_q int32 [B + 1]; kv_lens int32 [B];
    max_q, max_kv: the largest numbers of new tokens and of keys of a request;
    scale: 1 / sqrt(D) by default; window, sinks: a token sees its last
    `window` keys (0: all) and the first `sinks`.  Causal in each request.
    workspace: as for tq_gemm ("auto", None or a contiguous device tensor);
    "auto" allocates and clears one in every call, so a program that makes many
    keeps one (new_workspace of tq_paged_attention_workspace_bytes)."""
    return _result("tq_paged_attention", _entry().paged_attention(q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q, max_kv,
                                                                  scale, window, sinks, return_lse, out, workspace))


# ----------------------------------------------------------------- sampling

def tq_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None):
    """One token per row: -> (tokens int32 [B], logprobs fp32 [B]).

    logits [B, V] fp16, bf16 or fp32 (rows may be strided); u fp32 [B] in
    [0, 1).  temperature, top_p, min_p fp32 [B] and top_k int32 [B], or None
    for 1, 1, 0 and 0 (no cut); temperature 0 takes the best token.  A row
    without a logit above -inf gives token -1.  out: (tokens, logprobs) to
    write into."""
    return _result("tq_sample", _entry().sample(logits, u, temperature, top_k, top_p, min_p, out))
