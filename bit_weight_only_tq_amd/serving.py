"""ctypes binding of the serving operators of libtq.so: argument marshalling only.

The step of a served model that uses the packed linear layers also plans its
paged cache, appends keys and values to it, attends over its pages and samples
its next tokens; these calls forward to the entry points of the same names in
include/tq.h.  As in _lib.py, shapes, types and strides are checked before any
call (the C ABI takes bare pointers), and there is no CPU fallback.
"""

from typing import NamedTuple

from . import _lib
from ._lib import TQ_BF16, TQ_F16, TQ_F32, _check, _dtype_enum, _ptr, _stream

_LOGITS = {"torch.float16": TQ_F16, "torch.bfloat16": TQ_BF16, "torch.float32": TQ_F32}


def _tensor(name, t, dtype, dim, shape=None):
    if t.dtype != dtype or t.dim() != dim:
        raise TypeError(f"{name} must be a {dim}-D {dtype} tensor, got {t.dim()}-D {t.dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _on_device(*ts):
    """All tensors are device tensors of one device."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be device tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors must live on one device, got {dev} and {t.device}")
    return dev


def _contiguous(**ts):
    for name, t in ts.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _table_stride(page_table):
    """Elements between the rows of a page table (rows contiguous, not overlapping)."""
    B, width = page_table.shape
    if width > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table rows must be contiguous")
    stride = page_table.stride(0) if B > 1 else width
    if stride < width:
        raise ValueError("page_table rows must not overlap")
    return stride


def _cache(k_cache, v_cache):
    """Checks the caches [pages, Hkv, page_size, D]; -> elements between pages."""
    import torch
    if k_cache.dim() != 4 or k_cache.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("k_cache must be a 4-D float16 or bfloat16 tensor [pages, heads, page_size, D]")
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype or v_cache.stride() != k_cache.stride():
        raise ValueError("k_cache and v_cache must be alike in shape, type and strides")
    pages, H, page, D = k_cache.shape
    if not k_cache[:1].is_contiguous():
        raise ValueError("the pages of a cache must be contiguous")
    stride = k_cache.stride(0) if pages > 1 else H * page * D
    if stride < H * page * D:
        raise ValueError("the pages of a cache must not overlap")
    return stride


def _heads(name, t, dtype, T, D):
    """Checks a [T, heads, D] tensor whose last dimension is contiguous; -> (heads, token stride, head stride)."""
    if t.dim() != 3 or t.dtype != dtype:
        raise TypeError(f"{name} must be a 3-D {dtype} tensor, got {t.dim()}-D {t.dtype}")
    if t.shape[0] != T or t.shape[2] != D:
        raise ValueError(f"{name} must be [{T}, heads, {D}], got {tuple(t.shape)}")
    if D > 1 and t.stride(2) != 1:
        raise ValueError(f"the heads of {name} must be contiguous")
    return t.shape[1], t.stride(0), t.stride(1)


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
    slot -1).  out: a plan to write into, for steps replayed from a graph."""
    import torch
    i32 = torch.int32
    _tensor("ctx_lens", ctx_lens, i32, 1)
    B = ctx_lens.shape[0]
    _tensor("new_lens", new_lens, i32, 1, (B,))
    _tensor("page_table", page_table, i32, 2)
    _tensor("free_pages", free_pages, i32, 1)
    _tensor("free_head", free_head, i32, 1, (1,))
    if page_table.shape[0] != B:
        raise ValueError(f"page_table must have {B} rows, got {page_table.shape[0]}")
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    stride = _table_stride(page_table)
    _contiguous(ctx_lens=ctx_lens, new_lens=new_lens, free_pages=free_pages)
    if out is not None:
        _tensor("out.cu_q", out.cu_q, i32, 1, (B + 1,))
        _tensor("out.kv_lens", out.kv_lens, i32, 1, (B,))
        _tensor("out.positions", out.positions, i32, 1, (tokens,))
        _tensor("out.slots", out.slots, torch.int64, 1, (tokens,))
        _tensor("out.state", out.state, i32, 1, (2,))
        _contiguous(cu_q=out.cu_q, kv_lens=out.kv_lens, positions=out.positions, slots=out.slots, state=out.state)
    dev = _on_device(ctx_lens, new_lens, page_table, free_pages, free_head, *(out or ()))
    if out is None:
        new = ctx_lens.new_empty
        out = PagedPlan(new((B + 1,)), new((B,)), new((tokens,)), new((tokens,), dtype=torch.int64), new((2,)))
    _check("tq_paged_plan", _lib.load().tq_paged_plan(
        _ptr(ctx_lens), _ptr(new_lens), _ptr(page_table), stride, _ptr(free_pages), _ptr(free_head), B,
        page_table.shape[1], free_pages.shape[0], tokens, page_size, _ptr(out.cu_q), _ptr(out.kv_lens),
        _ptr(out.positions), _ptr(out.slots), _ptr(out.state), _stream(dev)))
    return out


# ------------------------------------------------------------------- append

def tq_kv_append(q, k, v, k_cache, v_cache, slots, positions=None, rope=None, interleaved: bool = False, out=None):
    """Rotates q and k by their positions and stores k and v in their slots; -> rotated q.

    q [T, Hq, D] (or None), k and v [T, Hkv, D]: fp16/bf16, any token and head
    strides; k_cache, v_cache [pages, Hkv, page_size, D]; slots int64 [T];
    positions int32 [T] and rope fp32 [rows, rot] (rot / 2 cosines, then
    rot / 2 sines) together, or neither: then nothing is rotated and the
    result is a copy of q.  out: where the rotated queries go, contiguous."""
    import torch
    stride = _cache(k_cache, v_cache)
    pages, Hkv, page, D = k_cache.shape
    dt = k_cache.dtype
    if k.dim() != 3:
        raise TypeError(f"k must be 3-D [T, {Hkv}, {D}], got {k.dim()}-D")
    T = k.shape[0]
    kh, k_tok, k_head = _heads("k", k, dt, T, D)
    vh, v_tok, v_head = _heads("v", v, dt, T, D)
    if kh != Hkv or vh != Hkv:
        raise ValueError(f"k and v must have the cache's {Hkv} heads, got {kh} and {vh}")
    Hq = q_tok = q_head = 0
    if q is not None:
        Hq, q_tok, q_head = _heads("q", q, dt, T, D)
    _tensor("slots", slots, torch.int64, 1, (T,))
    if (rope is None) != (positions is None):
        raise ValueError("rope and positions come together")
    rot = rows = 0
    if rope is not None:
        _tensor("rope", rope, torch.float32, 2)
        _tensor("positions", positions, torch.int32, 1, (T,))
        rows, rot = rope.shape
        if rot > D or rot % 2:
            raise ValueError(f"rope must have an even number of columns, at most {D}, got {rot}")
    if out is not None:
        if q is None:
            raise ValueError("out needs q")
        _tensor("out", out, dt, 3, (T, Hq, D))
    _contiguous(slots=slots, positions=positions, rope=rope, out=out)
    dev = _on_device(q, k, v, k_cache, v_cache, slots, positions, rope, out)
    if out is None and q is not None:
        out = q.new_empty((T, Hq, D))
    _check("tq_kv_append", _lib.load().tq_kv_append(
        _ptr(q), q_tok, q_head, _ptr(k), k_tok, k_head, _ptr(v), v_tok, v_head, _dtype_enum(k_cache), T, Hq, Hkv, D,
        _ptr(k_cache), _ptr(v_cache), pages, page, stride, _ptr(slots), _ptr(positions), _ptr(rope), rows, rot,
        1 if interleaved else 0, _ptr(out), _stream(dev)))
    return out


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
    workspace: as for tq_gemm ("auto", None or a contiguous device tensor)."""
    import torch
    stride = _cache(k_cache, v_cache)
    pages, Hkv, page, D = k_cache.shape
    if q.dim() != 3:
        raise TypeError(f"q must be 3-D [T, heads, {D}], got {q.dim()}-D")
    T = q.shape[0]
    Hq, q_tok, q_head = _heads("q", q, k_cache.dtype, T, D)
    i32 = torch.int32
    _tensor("page_table", page_table, i32, 2)
    B, width = page_table.shape
    _tensor("cu_q", cu_q, i32, 1, (B + 1,))
    _tensor("kv_lens", kv_lens, i32, 1, (B,))
    tab = _table_stride(page_table)
    if out is not None:
        _tensor("out", out, q.dtype, 3, (T, Hq, D))
    _contiguous(cu_q=cu_q, kv_lens=kv_lens, out=out)
    dev = _on_device(q, k_cache, v_cache, page_table, cu_q, kv_lens, out)
    lib = _lib.load()
    if out is None:
        out = q.new_empty((T, Hq, D))
    lse = q.new_empty((T, Hq), dtype=torch.float32) if return_lse else None
    if isinstance(workspace, str):
        workspace = _lib.new_workspace(lib.tq_paged_attention_workspace_bytes(T, Hq, Hkv, D, B, max_q, max_kv, window,
                                                                              sinks), dev)
    nbytes = 0
    if workspace is not None:
        _on_device(q, workspace)
        _contiguous(workspace=workspace)
        nbytes = workspace.numel() * workspace.element_size()
    _check("tq_paged_attention", lib.tq_paged_attention(
        _ptr(q), q_tok, q_head if Hq > 1 else 0, _dtype_enum(q), T, Hq, Hkv, D, _ptr(k_cache), _ptr(v_cache), pages, page, stride,
        _ptr(page_table), tab, width, _ptr(cu_q), _ptr(kv_lens), B, max_q, max_kv,
        D ** -0.5 if scale is None else scale, window, sinks, _ptr(out), _ptr(lse), _ptr(workspace), nbytes,
        _stream(dev)))
    return (out, lse) if return_lse else out


# ----------------------------------------------------------------- sampling

def tq_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None):
    """One token per row: -> (tokens int32 [B], logprobs fp32 [B]).

    logits [B, V] fp16, bf16 or fp32 (rows may be strided); u fp32 [B] in
    [0, 1).  temperature, top_p, min_p fp32 [B] and top_k int32 [B], or None
    for 1, 1, 0 and 0 (no cut); temperature 0 takes the best token.  A row
    without a logit above -inf gives token -1.  out: (tokens, logprobs) to
    write into."""
    import torch
    f32 = torch.float32
    if logits.dim() != 2:
        raise TypeError(f"logits must be 2-D [B, V], got {logits.dim()}-D")
    dt = _LOGITS.get(str(logits.dtype))
    if dt is None:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {logits.dtype}")
    B, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("the rows of logits must be contiguous")
    stride = logits.stride(0) if B > 1 else V
    if stride < V:
        raise ValueError("the rows of logits must not overlap")
    _tensor("u", u, f32, 1, (B,))
    for name, t, want in (("temperature", temperature, f32), ("top_k", top_k, torch.int32), ("top_p", top_p, f32),
                          ("min_p", min_p, f32)):
        if t is not None:
            _tensor(name, t, want, 1, (B,))
    if out is not None:
        _tensor("tokens", out[0], torch.int32, 1, (B,))
        _tensor("logprobs", out[1], f32, 1, (B,))
        _contiguous(tokens=out[0], logprobs=out[1])
    _contiguous(u=u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    dev = _on_device(logits, u, temperature, top_k, top_p, min_p, *(out or ()))
    tokens, logprobs = out or (u.new_empty((B,), dtype=torch.int32), u.new_empty((B,)))
    _check("tq_sample", _lib.load().tq_sample(
        _ptr(logits), dt, B, V, stride, _ptr(u), _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
        _ptr(tokens), _ptr(logprobs), _stream(dev)))
    return tokens, logprobs
