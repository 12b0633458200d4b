"""The example that serves a layer from the paged cache, against the same layer in fp64 with its error carried along.

Every tensor is a pair of its fp64 value and a bound of the path's error: products are sums in fp32 of fp16 values
(2e-3 of sum |a w| + 1e-3, the library's own bound for its products, holds the rounding of the output), a rotation or a
sum rounds to fp16 once (half a step, 2^-11 of the value), and a softmax whose scores are off by e has weights off by at
most exp(2 e) - 1, rounded to fp16 before the product (2^-11).
"""
import os
import sys

import numpy as np
import pytest

from gpu_common import log, require_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -11


def _example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_step
    return serve_step


def _product(x, e, w):
    mag = np.abs(x) @ np.abs(w).T
    return x @ w.T, e @ np.abs(w).T + 2e-3 * (mag + e @ np.abs(w).T) + 1e-3


def _rotate(x, e, pos, D):
    a = pos[:, None, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
    c, s = np.cos(a), np.sin(a)
    h = D // 2
    x0, x1, e0, e1 = x[..., :h], x[..., h:], e[..., :h], e[..., h:]
    y = np.concatenate([x0 * c - x1 * s, x1 * c + x0 * s], -1)
    ey = np.concatenate([e0 * np.abs(c) + e1 * np.abs(s), e1 * np.abs(c) + e0 * np.abs(s)], -1)
    # the table is fp32: angles' cosines off by 2^-24
    mag = np.concatenate([np.abs(x0) + np.abs(x1)] * 2, -1)
    return y, ey + U * (np.abs(y) + ey) + 2.0 ** -22 * mag + 2.0 ** -25


def _reference(model, weights, tokens):
    """Logits of the last token of one request, and their error bound."""
    D, Hq, Hkv = model.D, model.Hq, model.Hkv
    x = model.embed.double().cpu().numpy()[tokens]
    e = np.zeros_like(x)
    h, eh = _product(x, e, weights["qkv"])
    h, eh = h.reshape(len(tokens), -1, D), eh.reshape(len(tokens), -1, D)
    pos = np.arange(len(tokens), dtype=np.float64)
    q, eq = _rotate(h[:, :Hq], eh[:, :Hq], pos, D)
    k, ek = _rotate(h[:, Hq:Hq + Hkv], eh[:, Hq:Hq + Hkv], pos, D)
    v, ev = h[:, Hq + Hkv:], eh[:, Hq + Hkv:]
    o, eo = np.zeros((Hq, D)), np.zeros((Hq, D))
    for a in range(Hq):  # of the last token
        b = a * Hkv // Hq
        s = k[:, b] @ q[-1, a] * D ** -0.5
        es = (np.abs(k[:, b]) @ eq[-1, a] + ek[:, b] @ (np.abs(q[-1, a]) + eq[-1, a])) * D ** -0.5
        es = es.max() + 2.0 ** -16 * (1 + np.abs(s).max())
        p = np.exp(s - s.max())
        p /= p.sum()
        rel = np.exp(2 * es) - 1 + 2 * U
        o[a] = p @ v[:, b]
        eo[a] = (1 + rel) * (p @ ev[:, b]) + rel * (p @ np.abs(v[:, b]))
        eo[a] += U * (np.abs(o[a]) + eo[a]) + 2.0 ** -20
    y, ey = _product(o.reshape(1, -1), eo.reshape(1, -1), weights["out"])
    y, ey = y + x[-1:], ey
    ey = ey + U * (np.abs(y) + ey)
    return [z[0] for z in _product(y, ey, weights["head"])]


def _unpacked(model):
    import bit_weight_only_tq_amd as tq
    sizes = {"qkv": ((model.Hq + 2 * model.Hkv) * model.D, model.embed.shape[1]),
             "out": (model.embed.shape[1], model.Hq * model.D), "head": (model.embed.shape[0], model.embed.shape[1])}
    out = {}
    for name, (n, k) in sizes.items():
        codes, scale = getattr(model, name)
        t, _ = tq.tq_unpack(codes, scale, k)
        out[name] = t.cpu().double().numpy() * scale.cpu().double().numpy()[:, None]
    return out


def test_served_logits():
    """Prompts in chunks beside decoding requests: every step's logits within the error carried through the layer."""
    import torch
    require_gpu()
    log("serve")
    ex = _example()
    model = ex.random_model(seed=3)
    weights = _unpacked(model)
    server = ex.Server(model)
    g = torch.Generator().manual_seed(2)
    texts = [torch.randint(0, 1024, (n,), generator=g).tolist() for n in (9, 47, 30, 80)]
    done = [0, 0, 0, 0]
    for step in ((5, 0, 30, 33), (1, 40, 0, 30), (1, 6, 0, 16), (1, 1, 0, 1), (1, 0, 0, 0)):
        feed = [t[d:d + n] for t, d, n in zip(texts, done, step)]
        got = server.logits(feed).double().cpu().numpy()
        done = [d + n for d, n in zip(done, step)]
        assert server.ctx.tolist() == done
        for b, n in enumerate(step):
            if n:
                want, tol = _reference(model, weights, np.array(texts[b][:done[b]]))
                err = np.abs(got[b] - want) / tol
                assert err.max() <= 1, f"request {b}: {err.max()} of the bound"
    assert int(server.head) == sum(-(-d // 16) for d in done)


def test_example_runs(capsys):
    require_gpu()
    _example().main()
    assert "pages in use" in capsys.readouterr().out


@pytest.mark.parametrize("mode", ["inference_mode", "no_grad", "enable_grad"])
def test_outputs_are_ordinary_tensors(mode):
    """A plan's outputs share one allocation: each can be changed in place, viewed, copied and outlive the others."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log(f"outputs {mode}")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    with getattr(torch, mode)():
        plan = tq.tq_paged_plan(i32([3, 0, 16]), i32([2, 1, 4]), torch.full((3, 4), -1, dtype=torch.int32, device=dev),
                                i32([9, 8, 7, 6]), i32([0]), 8)
        assert plan.cu_q.tolist() == [0, 2, 3, 7] and plan.kv_lens.tolist() == [5, 1, 20]
        assert all(t.is_contiguous() and not t.requires_grad and t.device == dev for t in plan)
        slots, state = plan.slots, plan.state
        plan.positions.add_(100)
        plan.cu_q.mul_(0)
        plan.kv_lens.view(3, 1).fill_(7)
        assert plan.positions.tolist() == [103, 104, 100, 116, 117, 118, 119, 100] and plan.kv_lens.tolist() == [7] * 3
        assert slots.dtype == torch.int64 and slots[2].item() == 9 * 16 and slots[7].item() == -1
        del plan
        torch.empty(1 << 20, device=dev).fill_(1.0)
        assert state.clone().tolist() == [2, 2] and slots[3:7].cpu().tolist() == [128, 129, 130, 131]
        tokens, logprobs = tq.tq_sample(torch.zeros((2, 8), device=dev), torch.tensor([0.0, 0.99], device=dev))
        assert tokens.add_(0).tolist() == [0, 7] and torch.allclose(logprobs.exp(), torch.full((2,), 0.125, device=dev))
