"""ctypes binding of the serving operators of libtq.so: argument marshalling only.

The step of a served model that uses the packed linear layers also plans its
paged cache, appends keys and values to it, attends over its pages and samples
its next tokens; these calls forward to the entry points of the same names in
include/tq.h.  As in _lib.py, shapes, types and strides are checked before any
call (the C ABI takes bare pointers), and there is no CPU fallback.
"""

from typing import NamedTuple

from . import _lib
from ._lib import TQ_BF16, TQ_F16, TQ_F32, _check

# A serving step calls these once a layer, often on a few rows: what a call
# costs is then the host's time, so a check is a comparison or two, pointers
# are passed as the integers they are, and only a failed check pays for words.


class _Torch:
    """torch's types and its current stream, looked up at the first call."""

    def __init__(self):
        import torch
        self.i32, self.i64, self.f32 = torch.int32, torch.int64, torch.float32
        self.cache = {torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}
        self.logits = {**self.cache, torch.float32: TQ_F32}
        # the stream's handle without a Stream object around it (2 us less), where torch has it
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)


_torch = None


def _types():
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _tensor(name, t, dtype, dim, shape=None):
    if t.dtype is not dtype or t.dim() != dim:
        raise TypeError(f"{name} must be a {dim}-D {dtype} tensor, got {t.dim()}-D {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _vector(name, t, dtype, n=None):
    """A contiguous vector (of n entries); -> its address."""
    if t.dtype is not dtype or t.dim() != 1:
        raise TypeError(f"{name} must be a 1-D {dtype} tensor, got {t.dim()}-D {t.dtype}")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on_device(*ts):
    """All tensors are device tensors of one device; -> its index."""
    index = None
    for t in ts:
        if t is None:
            continue
        i = t.get_device()  # -1: host memory
        if i < 0:
            raise ValueError("tensors must be device tensors")
        if i != index:
            if index is not None:
                raise ValueError(f"tensors must live on one device, got {index} and {i}")
            index = i
    return index


def _contiguous(name, t):
    if not t.is_contiguous():
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
    """Checks the caches [pages, Hkv, page_size, D]; -> (tq_dtype, elements between pages)."""
    dt = _types().cache.get(k_cache.dtype)
    if k_cache.dim() != 4 or dt is None:
        raise TypeError("k_cache must be a 4-D float16 or bfloat16 tensor [pages, heads, page_size, D]")
    if v_cache.shape != k_cache.shape or v_cache.dtype is not k_cache.dtype or v_cache.stride() != k_cache.stride():
        raise ValueError("k_cache and v_cache must be alike in shape, type and strides")
    pages, H, page, D = k_cache.shape
    if k_cache.is_contiguous():
        return dt, H * page * D
    if not k_cache[:1].is_contiguous():
        raise ValueError("the pages of a cache must be contiguous")
    stride = k_cache.stride(0) if pages > 1 else H * page * D
    if stride < H * page * D:
        raise ValueError("the pages of a cache must not overlap")
    return dt, stride


def _heads(name, t, dtype, T, D):
    """Checks a [T, heads, D] tensor whose last dimension is contiguous; -> (heads, token stride, head stride)."""
    if t.dim() != 3 or t.dtype is not dtype:
        raise TypeError(f"{name} must be a 3-D {dtype} tensor, got {t.dim()}-D {t.dtype}")
    n, heads, d = t.shape
    if n != T or d != D:
        raise ValueError(f"{name} must be [{T}, heads, {D}], got {tuple(t.shape)}")
    token, head, one = t.stride()
    if one != 1 and D > 1:
        raise ValueError(f"the heads of {name} must be contiguous")
    return heads, token, head


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
    ty = _types()
    i32 = ty.i32
    ctx = _vector("ctx_lens", ctx_lens, i32)
    B = ctx_lens.shape[0]
    new = _vector("new_lens", new_lens, i32, B)
    _tensor("page_table", page_table, i32, 2)
    free = _vector("free_pages", free_pages, i32)
    head = _vector("free_head", free_head, i32, 1)
    if page_table.shape[0] != B:
        raise ValueError(f"page_table must have {B} rows, got {page_table.shape[0]}")
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    stride = _table_stride(page_table)
    if out is not None:
        _vector("out.cu_q", out.cu_q, i32, B + 1)
        _vector("out.kv_lens", out.kv_lens, i32, B)
        _vector("out.positions", out.positions, i32, tokens)
        _vector("out.slots", out.slots, ty.i64, tokens)
        _vector("out.state", out.state, i32, 2)
    dev = _on_device(ctx_lens, new_lens, page_table, free_pages, free_head, *(out or ()))
    if out is None:  # one allocation, the slots first: they are 8 bytes each
        slots, cu_q, kv_lens, positions, state = ctx_lens.new_empty((2 * B + 3 * tokens + 3,)).split_with_sizes(
            (2 * tokens, B + 1, B, tokens, 2))
        out = PagedPlan(cu_q, kv_lens, positions, slots.view(ty.i64), state)
    cu_q, kv_lens, positions, slots, state = out
    status = _lib.load().tq_paged_plan(
        ctx, new, page_table.data_ptr(), stride, free, head, B, page_table.shape[1], free_pages.shape[0], tokens, page_size,
        cu_q.data_ptr(), kv_lens.data_ptr(), positions.data_ptr(), slots.data_ptr(), state.data_ptr(), ty.stream(dev))
    if status:
        _check("tq_paged_plan", status)
    return out


# ------------------------------------------------------------------- append

def tq_kv_append(q, k, v, k_cache, v_cache, slots, positions=None, rope=None, interleaved: bool = False, out=None):
    """Rotates q and k by their positions and stores k and v in their slots; -> rotated q.

    q [T, Hq, D] (or None), k and v [T, Hkv, D]: fp16/bf16, any token and head
    strides; k_cache, v_cache [pages, Hkv, page_size, D]; slots int64 [T];
    positions int32 [T] and rope fp32 [rows, rot] (rot / 2 cosines, then
    rot / 2 sines) together, or neither: then nothing is rotated and the
    result is a copy of q.  out: where the rotated queries go, contiguous."""
    ty = _types()
    dt, stride = _cache(k_cache, v_cache)
    pages, Hkv, page, D = k_cache.shape
    dtype = k_cache.dtype
    if k.dim() != 3:
        raise TypeError(f"k must be 3-D [T, {Hkv}, {D}], got {k.dim()}-D")
    T = k.shape[0]
    kh, k_tok, k_head = _heads("k", k, dtype, T, D)
    vh, v_tok, v_head = _heads("v", v, dtype, T, D)
    if kh != Hkv or vh != Hkv:
        raise ValueError(f"k and v must have the cache's {Hkv} heads, got {kh} and {vh}")
    Hq = q_tok = q_head = 0
    if q is not None:
        Hq, q_tok, q_head = _heads("q", q, dtype, T, D)
    at = _vector("slots", slots, ty.i64, T)
    if (rope is None) != (positions is None):
        raise ValueError("rope and positions come together")
    rot = rows = pos = angles = None
    if rope is not None:
        _tensor("rope", rope, ty.f32, 2)
        _contiguous("rope", rope)
        pos = _vector("positions", positions, ty.i32, T)
        angles = rope.data_ptr()
        rows, rot = rope.shape
        if rot > D or rot % 2:
            raise ValueError(f"rope must have an even number of columns, at most {D}, got {rot}")
    if out is not None:
        if q is None:
            raise ValueError("out needs q")
        _tensor("out", out, dtype, 3, (T, Hq, D))
        _contiguous("out", out)
    dev = _on_device(q, k, v, k_cache, v_cache, slots, positions, rope, out)
    if out is None and q is not None:
        out = q.new_empty((T, Hq, D))
    status = _lib.load().tq_kv_append(
        None if q is None else q.data_ptr(), q_tok, q_head, k.data_ptr(), k_tok, k_head, v.data_ptr(), v_tok, v_head, dt, T,
        Hq, Hkv, D, k_cache.data_ptr(), v_cache.data_ptr(), pages, page, stride, at, pos, angles, rows or 0, rot or 0,
        1 if interleaved else 0, None if out is None else out.data_ptr(), ty.stream(dev))
    if status:
        _check("tq_kv_append", status)
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
    ty = _types()
    dt, stride = _cache(k_cache, v_cache)
    pages, Hkv, page, D = k_cache.shape
    if q.dim() != 3:
        raise TypeError(f"q must be 3-D [T, heads, {D}], got {q.dim()}-D")
    T = q.shape[0]
    Hq, q_tok, q_head = _heads("q", q, k_cache.dtype, T, D)
    i32 = ty.i32
    _tensor("page_table", page_table, i32, 2)
    B, width = page_table.shape
    cu = _vector("cu_q", cu_q, i32, B + 1)
    kv = _vector("kv_lens", kv_lens, i32, B)
    tab = _table_stride(page_table)
    if out is not None:
        _tensor("out", out, q.dtype, 3, (T, Hq, D))
        _contiguous("out", out)
    dev = _on_device(q, k_cache, v_cache, page_table, cu_q, kv_lens, out)
    lib = _lib.load()
    if out is None:
        out = q.new_empty((T, Hq, D))
    lse = q.new_empty((T, Hq), dtype=ty.f32) if return_lse else None
    if isinstance(workspace, str):
        workspace = _lib.new_workspace(lib.tq_paged_attention_workspace_bytes(T, Hq, Hkv, D, B, max_q, max_kv, window,
                                                                              sinks), q.device)
    room = nbytes = 0
    if workspace is not None:
        _on_device(q, workspace)
        _contiguous("workspace", workspace)
        room, nbytes = workspace.data_ptr(), workspace.nbytes
    status = lib.tq_paged_attention(
        q.data_ptr(), q_tok, q_head if Hq > 1 else 0, dt, T, Hq, Hkv, D, k_cache.data_ptr(), v_cache.data_ptr(), pages, page,
        stride, page_table.data_ptr(), tab, width, cu, kv, B, max_q, max_kv, D ** -0.5 if scale is None else scale, window,
        sinks, out.data_ptr(), None if lse is None else lse.data_ptr(), room, nbytes, ty.stream(dev))
    if status:
        _check("tq_paged_attention", status)
    return (out, lse) if return_lse else out


# ----------------------------------------------------------------- sampling

def tq_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None):
    """One token per row: -> (tokens int32 [B], logprobs fp32 [B]).

    logits [B, V] fp16, bf16 or fp32 (rows may be strided); u fp32 [B] in
    [0, 1).  temperature, top_p, min_p fp32 [B] and top_k int32 [B], or None
    for 1, 1, 0 and 0 (no cut); temperature 0 takes the best token.  A row
    without a logit above -inf gives token -1.  out: (tokens, logprobs) to
    write into."""
    ty = _types()
    f32 = ty.f32
    if logits.dim() != 2:
        raise TypeError(f"logits must be 2-D [B, V], got {logits.dim()}-D")
    dt = ty.logits.get(logits.dtype)
    if dt is None:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {logits.dtype}")
    B, V = logits.shape
    stride, one = logits.stride()
    if one != 1 and V > 1:
        raise ValueError("the rows of logits must be contiguous")
    if B <= 1:
        stride = V
    if stride < V:
        raise ValueError("the rows of logits must not overlap")
    at = _vector("u", u, f32, B)
    t = None if temperature is None else _vector("temperature", temperature, f32, B)
    k = None if top_k is None else _vector("top_k", top_k, ty.i32, B)
    p = None if top_p is None else _vector("top_p", top_p, f32, B)
    m = None if min_p is None else _vector("min_p", min_p, f32, B)
    if out is not None:
        _vector("tokens", out[0], ty.i32, B)
        _vector("logprobs", out[1], f32, B)
    dev = _on_device(logits, u, temperature, top_k, top_p, min_p, *(out or ()))
    tokens, logprobs = out or (u.new_empty((B,), dtype=ty.i32), u.new_empty((B,)))
    status = _lib.load().tq_sample(logits.data_ptr(), dt, B, V, stride, at, t, k, p, m, tokens.data_ptr(),
                                   logprobs.data_ptr(), ty.stream(dev))
    if status:
        _check("tq_sample", status)
    return tokens, logprobs
