"""The serving calls refuse what they cannot run, on the host, before any device call.

The C ABI checks sizes, types and pointers; the binding checks tensors'
shapes, types and strides (the ABI takes bare pointers).  CPU only: a
well-formed call with CPU tensors gets as far as the device check.
"""
import ctypes

import pytest
import torch

import bit_weight_only_tq_amd as tq
from bit_weight_only_tq_amd import _lib

V = ctypes.c_void_p
FAKE, ODD = V(0x10000), V(0x10001)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def call(lib, name, good, **change):
    args = dict(good, **change)
    return _lib.STATUS_NAMES[getattr(lib, name)(*args.values())]


# --------------------------------------------------------------------- plan

PLAN = dict(ctx=FAKE, new=FAKE, table=FAKE, stride=8, free=FAKE, head=FAKE, B=4, width=8, n_free=10, T=7, page=16,
            cu=FAKE, kv=FAKE, pos=FAKE, slots=FAKE, state=FAKE, stream=None)


@pytest.mark.parametrize("change, want", [
    *[({n: None}, "TQ_ERR_NULL") for n in ("ctx", "new", "table", "free", "head", "cu", "kv", "pos", "slots", "state")],
    *[({n: ODD}, "TQ_ERR_ALIGN") for n in ("ctx", "new", "table", "free", "head", "cu", "kv", "pos", "slots", "state")],
    ({"slots": V(0x10004)}, "TQ_ERR_ALIGN"),
    ({"B": 0}, "TQ_ERR_SHAPE"), ({"B": 16385}, "TQ_ERR_SHAPE"), ({"width": 0}, "TQ_ERR_SHAPE"),
    ({"n_free": -1}, "TQ_ERR_SHAPE"), ({"T": -1}, "TQ_ERR_SHAPE"), ({"T": 1 << 31}, "TQ_ERR_SHAPE"),
    ({"stride": 7}, "TQ_ERR_VALUE"),
    *[({"page": p}, "TQ_ERR_VALUE") for p in (0, -16, 8, 24, 2048)],
])
def test_plan_host_checks(lib, change, want):
    assert call(lib, "tq_paged_plan", PLAN, **change) == want


def _plan_args(B=3, width=4, tokens=5):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(ctx_lens=i(B), new_lens=i(B), page_table=i(B, width), free_pages=i(9), free_head=i(1), tokens=tokens)


def test_plan_well_formed_cpu_tensors_reach_device_check():
    with pytest.raises(ValueError, match="device tensors"):
        tq.tq_paged_plan(**_plan_args())


@pytest.mark.parametrize("change", [
    dict(ctx_lens=torch.zeros(3, dtype=torch.int64)), dict(new_lens=torch.zeros(4, dtype=torch.int32)),
    dict(page_table=torch.zeros((2, 4), dtype=torch.int32)), dict(page_table=torch.zeros((4, 3), dtype=torch.int32).T),
    dict(page_table=torch.zeros((1, 4), dtype=torch.int32).expand(3, 4)),
    dict(free_pages=torch.zeros(18, dtype=torch.int32)[::2]), dict(free_head=torch.zeros(2, dtype=torch.int32)),
    dict(tokens=-1),
    dict(out=tq.PagedPlan(torch.zeros(3, dtype=torch.int32), *[torch.zeros(5, dtype=torch.int32)] * 4)),
])
def test_plan_rejects(change):
    with pytest.raises((ValueError, TypeError)) as e:
        tq.tq_paged_plan(**dict(_plan_args(), **change))
    assert "device tensors" not in str(e.value)


# ------------------------------------------------------------------- append

APPEND = dict(q=FAKE, qs=128, qh=64, k=FAKE, ks=64, kh=64, v=FAKE, vs=64, vh=64, dt=0, T=3, Hq=2, Hkv=1, D=64,
              kc=FAKE, vc=FAKE, pages=4, page=16, stride=1024, slots=FAKE, pos=FAKE, rope=FAKE, rows=10, rot=64,
              inter=0, out=FAKE, stream=None)


@pytest.mark.parametrize("change, want", [
    *[({n: None}, "TQ_ERR_NULL") for n in ("q", "k", "v", "kc", "vc", "slots", "pos", "rope", "out")],
    *[({n: ODD}, "TQ_ERR_ALIGN") for n in ("q", "k", "v", "kc", "vc", "slots", "pos", "rope", "out")],
    ({"dt": 2}, "TQ_ERR_DTYPE"), ({"dt": 7}, "TQ_ERR_DTYPE"),
    ({"T": -1}, "TQ_ERR_SHAPE"), ({"Hkv": 0}, "TQ_ERR_SHAPE"), ({"Hq": -1}, "TQ_ERR_SHAPE"), ({"D": 0}, "TQ_ERR_SHAPE"),
    ({"pages": 0}, "TQ_ERR_SHAPE"), ({"rot": 63}, "TQ_ERR_SHAPE"), ({"rot": 66}, "TQ_ERR_SHAPE"),
    ({"rows": 0}, "TQ_ERR_SHAPE"),
    ({"page": 20}, "TQ_ERR_VALUE"), ({"stride": 1023}, "TQ_ERR_VALUE"),
    ({"T": 0, "k": None}, "TQ_OK"),
])
def test_append_host_checks(lib, change, want):
    assert call(lib, "tq_kv_append", APPEND, **change) == want


def _append_args(T=3, Hq=2, Hkv=1, D=64, page=16, pages=4):
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    return dict(q=h(T, Hq, D), k=h(T, Hkv, D), v=h(T, Hkv, D), k_cache=h(pages, Hkv, page, D),
                v_cache=h(pages, Hkv, page, D), slots=torch.zeros(T, dtype=torch.int64),
                positions=torch.zeros(T, dtype=torch.int32), rope=torch.zeros(10, D))


def test_append_well_formed_cpu_tensors_reach_device_check():
    a = _append_args()
    with pytest.raises(ValueError, match="device tensors"):
        tq.tq_kv_append(**a)
    fused = torch.zeros((3, 4 * 64), dtype=torch.float16)  # parts of one projection's output
    q, k, v = fused.split([128, 64, 64], 1)
    with pytest.raises(ValueError, match="device tensors"):
        tq.tq_kv_append(**dict(a, q=q.unflatten(1, (2, 64)), k=k.unflatten(1, (1, 64)), v=v.unflatten(1, (1, 64))))


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros((3, 2, 64))), dict(q=torch.zeros((4, 2, 64), dtype=torch.float16)),
    dict(k=torch.zeros((3, 64), dtype=torch.float16)), dict(k=torch.zeros((3, 2, 64), dtype=torch.float16)),
    dict(v=torch.zeros((3, 1, 64), dtype=torch.bfloat16)),
    dict(q=torch.zeros((3, 64, 2), dtype=torch.float16).transpose(1, 2)),
    dict(k_cache=torch.zeros((4, 1, 16, 64))), dict(v_cache=torch.zeros((5, 1, 16, 64), dtype=torch.float16)),
    dict(k_cache=torch.zeros((4, 16, 1, 64), dtype=torch.float16).transpose(1, 2).expand(4, 1, 16, 64)[:, :, :, :32]),
    dict(slots=torch.zeros(3, dtype=torch.int32)), dict(positions=None), dict(rope=None),
    dict(rope=torch.zeros(10, 63)), dict(rope=torch.zeros(10, 66)), dict(rope=torch.zeros(10, 64, dtype=torch.float16)),
    dict(out=torch.zeros((3, 2, 64), dtype=torch.bfloat16)), dict(q=None, out=torch.zeros((3, 2, 64), dtype=torch.float16)),
])
def test_append_rejects(change):
    with pytest.raises((ValueError, TypeError)) as e:
        tq.tq_kv_append(**dict(_append_args(), **change))
    assert "device tensors" not in str(e.value)


# ---------------------------------------------------------------- attention

ATTN = dict(q=FAKE, qs=128, qh=64, dt=0, T=3, Hq=2, Hkv=1, D=64, kc=FAKE, vc=FAKE, pages=4, page=16, stride=1024,
            table=FAKE, tstride=4, width=4, cu=FAKE, kv=FAKE, B=1, max_q=3, max_kv=40, scale=0.125, window=0, sinks=0,
            out=FAKE, lse=FAKE, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change, want", [
    *[({n: None}, "TQ_ERR_NULL") for n in ("q", "kc", "vc", "table", "cu", "kv", "out")],
    *[({n: V(0x10008)}, "TQ_ERR_ALIGN") for n in ("q", "kc", "vc", "out", "ws")],
    *[({n: ODD}, "TQ_ERR_ALIGN") for n in ("table", "cu", "kv", "lse")],
    ({"qs": 132}, "TQ_ERR_ALIGN"), ({"qh": 65}, "TQ_ERR_ALIGN"), ({"stride": 1028}, "TQ_ERR_ALIGN"),
    ({"dt": 2}, "TQ_ERR_DTYPE"), ({"dt": -1}, "TQ_ERR_DTYPE"),
    *[({n: -1}, "TQ_ERR_SHAPE") for n in ("T", "Hq", "Hkv", "D", "pages", "width", "B", "max_q", "max_kv")],
    *[({n: 0}, "TQ_ERR_SHAPE") for n in ("Hq", "Hkv", "D", "pages", "width", "B", "max_q")],
    ({"Hq": 3, "Hkv": 2, "stride": 4096}, "TQ_ERR_SHAPE"), ({"D": 96}, "TQ_ERR_SHAPE"), ({"D": 256}, "TQ_ERR_SHAPE"),
    *[({"page": p}, "TQ_ERR_VALUE") for p in (0, 8, 48, 2048)],
    ({"stride": 1016}, "TQ_ERR_VALUE"), ({"tstride": 3}, "TQ_ERR_VALUE"),
    *[({"scale": x}, "TQ_ERR_VALUE") for x in (0.0, -1.0, float("nan"), float("inf"))],
    ({"window": -1}, "TQ_ERR_VALUE"), ({"sinks": -1}, "TQ_ERR_VALUE"), ({"window": 1 << 31}, "TQ_ERR_VALUE"),
    ({"T": 0, "q": None}, "TQ_OK"),
])
def test_attention_host_checks(lib, change, want):
    assert call(lib, "tq_paged_attention", ATTN, **change) == want


def test_attention_workspace_query():
    """Nothing for invalid sizes or where there is nothing to split; the counters and the partials otherwise."""
    wb = tq.tq_paged_attention_workspace_bytes
    assert wb(1, 32, 8, 128, 1, 1, 64) == 0           # two key blocks
    assert wb(1, 32, 8, 96, 1, 1, 9999) == 0 and wb(1, 31, 8, 128, 1, 1, 9999) == 0 and wb(0, 32, 8, 128, 1, 1, 9999) == 0
    long = wb(2, 32, 8, 128, 2, 1, 131071)
    assert long > tq.TQ_WORKSPACE_FLAG_BYTES and (long - tq.TQ_WORKSPACE_FLAG_BYTES) % (2 * 8 * 4 * 130 * 4) == 0
    assert wb(2, 32, 8, 128, 2, 1, 131071, 64) == 0   # a window of 64 keys
    assert wb(4096, 32, 8, 128, 1024, 4, 4096) == 0   # more tiles than counters


def _attn_args(T=3, Hq=2, Hkv=1, D=64, page=16, pages=4):
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(q=h(T, Hq, D), k_cache=h(pages, Hkv, page, D), v_cache=h(pages, Hkv, page, D), page_table=i(1, 4),
                cu_q=i(2), kv_lens=i(1), max_q=3, max_kv=40)


def test_attention_well_formed_cpu_tensors_reach_device_check():
    with pytest.raises(ValueError, match="device tensors"):
        tq.tq_paged_attention(**_attn_args())


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros((3, 128), dtype=torch.float16)), dict(q=torch.zeros((3, 2, 64), dtype=torch.bfloat16)),
    dict(q=torch.zeros((3, 2, 32), dtype=torch.float16)), dict(q=torch.zeros((3, 64, 2), dtype=torch.float16).transpose(1, 2)),
    dict(v_cache=torch.zeros((4, 1, 16, 64), dtype=torch.bfloat16)), dict(k_cache=torch.zeros((4, 1, 16, 64))),
    dict(page_table=torch.zeros((1, 4), dtype=torch.int64)), dict(page_table=torch.zeros(4, dtype=torch.int32)),
    dict(cu_q=torch.zeros(3, dtype=torch.int32)), dict(kv_lens=torch.zeros(1, dtype=torch.int64)),
    dict(cu_q=torch.zeros(4, dtype=torch.int32)[::2]), dict(out=torch.zeros((3, 2, 64))),
    dict(out=torch.zeros((3, 4, 64), dtype=torch.float16)[:, ::2]),
])
def test_attention_rejects(change):
    with pytest.raises((ValueError, TypeError)) as e:
        tq.tq_paged_attention(**dict(_attn_args(), **change))
    assert "device tensors" not in str(e.value)


# ----------------------------------------------------------------- sampling

SAMPLE = dict(logits=FAKE, dt=2, B=2, V=100, stride=100, u=FAKE, temperature=FAKE, top_k=FAKE, top_p=FAKE, min_p=FAKE,
              tokens=FAKE, logprobs=FAKE, stream=None)


@pytest.mark.parametrize("change, want", [
    *[({n: None}, "TQ_ERR_NULL") for n in ("logits", "u", "tokens")],
    *[({n: ODD}, "TQ_ERR_ALIGN") for n in ("logits", "u", "temperature", "top_k", "top_p", "min_p", "tokens", "logprobs")],
    ({"logits": V(0x10002)}, "TQ_ERR_ALIGN"), ({"logits": V(0x10001), "dt": 0}, "TQ_ERR_ALIGN"),
    ({"dt": 3}, "TQ_ERR_DTYPE"), ({"B": -1}, "TQ_ERR_SHAPE"), ({"V": 0}, "TQ_ERR_SHAPE"),
    ({"V": (1 << 20) + 1, "stride": 1 << 21}, "TQ_ERR_SHAPE"), ({"stride": 99}, "TQ_ERR_VALUE"),
    ({"B": 0, "logits": None}, "TQ_OK"),
])
def test_sample_host_checks(lib, change, want):
    assert call(lib, "tq_sample", SAMPLE, **change) == want


def test_sample_well_formed_cpu_tensors_reach_device_check():
    with pytest.raises(ValueError, match="device tensors"):
        tq.tq_sample(torch.zeros((2, 100)), torch.zeros(2))


@pytest.mark.parametrize("change", [
    dict(logits=torch.zeros(100)), dict(logits=torch.zeros((2, 100), dtype=torch.float64)),
    dict(logits=torch.zeros((100, 2)).T), dict(logits=torch.zeros((1, 100)).expand(2, 100)),
    dict(u=torch.zeros(3)), dict(u=torch.zeros(2, dtype=torch.float64)), dict(temperature=torch.zeros(1)),
    dict(top_k=torch.zeros(2)), dict(top_p=torch.zeros((2, 1))), dict(min_p=torch.zeros(4)[::2]),
    dict(out=(torch.zeros(2, dtype=torch.int64), torch.zeros(2))),
])
def test_sample_rejects(change):
    with pytest.raises((ValueError, TypeError)) as e:
        tq.tq_sample(**dict(dict(logits=torch.zeros((2, 100)), u=torch.zeros(2)), **change))
    assert "device tensors" not in str(e.value)
