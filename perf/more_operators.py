"""Experts and adapters beside the packed linear layers, as measured cases.

A model whose projections are this library's packed layers may have a set of
experts in place of one MLP, and may be served with low-rank adapters:

  route    the top_k experts of each token, their weights, and the pairs
           (token, expert) sorted by expert (tq_moe_route)
  experts  each pair's row times its expert's packed weights, ternary or W4A16,
           optionally with the gated activation of a fused gate and up
           projection (tq_moe_gemm, w4a16_moe_gemm)
  combine  the weighted sum of each token's rows (tq_moe_combine)
  lora     the low-rank updates of many requests' adapters, added to what the
           shared projection gave (tq_lora)

Each case is run in a plain form (elementary torch operations in 32 bits) or,
with ``own`` set, by the library's calls.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
NEG_INF = float("-inf")
GROUP = 128  # columns that share a W4A16 scale

# the largest listed products: what a drawn case may take
MAX_FLOPS = 2 * 8192 * 28672 * 4096
MAX_WEIGHTS = 8 * 28672 * 4096


# -------------------------------------------------------------------- cases

def listed():
    return [
        # One token of one user among eight experts: a launch's latency.
        dict(name="route_one_token", op="route", dt="f32", T=1, E=8, k=2, renorm=True),
        # A full prompt batch of a model with many small experts.
        dict(name="route_prompt_16383", op="route", dt="bf16", T=16383, E=128, k=8, renorm=True),
        # One token's gate and up projections, two of eight ternary experts of the 8B MLP's size: the read of the weights.
        dict(name="experts_one_token", op="experts", fmt="ternary", dt="f16", T=1, E=8, k=2, K=4096, N=28672, gated=True,
             gather=True, zeros=False, skew=0.0),
        # A decode step of 48 requests over 64 small experts, a few rows each.
        dict(name="experts_decode_48", op="experts", fmt="w4", dt="bf16", T=48, E=64, k=6, K=2048, N=2816, gated=True,
             gather=True, zeros=False, skew=0.0),
        # The down projection of a short prompt's chunk: about forty rows an expert, a K of eleven groups, zero points.
        dict(name="experts_chunk_down", op="experts", fmt="w4", dt="f16", T=333, E=16, k=2, K=1408, N=4096, gated=False,
             gather=False, zeros=True, skew=0.3),
        # A prompt's gate and up projections, experts of the 8B MLP's size.
        dict(name="experts_prompt_4096", op="experts", fmt="w4", dt="bf16", T=4096, E=8, k=2, K=4096, N=28672, gated=True,
             gather=True, zeros=False, skew=0.3),
        # The down projection of a shorter prompt, ternary, unevenly loaded experts.
        dict(name="experts_prompt_down", op="experts", fmt="ternary", dt="f16", T=2047, E=8, k=2, K=14336, N=4096, gated=False,
             gather=False, zeros=False, skew=0.6),
        # One token's two rows, with the residual stream.
        dict(name="combine_one_token", op="combine", dt="f16", T=1, k=2, N=4096, add=True),
        # A prompt batch, six rows a token.
        dict(name="combine_prompt_8191", op="combine", dt="bf16", T=8191, k=6, N=2048, add=False),
        # One token of one request: the latency of two thin products.
        dict(name="lora_one_token", op="lora", dt="bf16", T=1, L=8, r=16, K=4096, N=4096, prompts=0, without=0.0),
        # A decode step of 64 requests with 32 adapters beside the fused qkv projection; some requests have none.
        dict(name="lora_decode_64", op="lora", dt="f16", T=64, L=32, r=16, K=4096, N=6144, prompts=0, without=0.2),
        # Several requests' prompts in one batch, larger rank.
        dict(name="lora_prompt_8191", op="lora", dt="bf16", T=8191, L=6, r=64, K=4096, N=4096, prompts=5, without=0.1),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "experts", "combine", "lora", "lora"])
    dt = rng.choice(["f16", "bf16"])
    if op == "route":
        E = _log(rng, 4, 256)
        return dict(op="route", dt=rng.choice(["f16", "bf16", "f32"]), T=_log(rng, 1, 16383), E=E,
                    k=min(E, rng.choice([1, 2, 2, 4, 6, 8])), renorm=rng.random() < 0.7)
    if op == "combine":
        T = _log(rng, 1, 8191)
        return dict(op="combine", dt=dt, T=T, k=rng.choice([1, 2, 2, 4, 6]), N=_log(rng, 256, 2048 if T > 2048 else 8192),
                    add=rng.random() < 0.5)
    if op == "lora":
        T = _log(rng, 1, 8191)
        L = _log(rng, 1, 64)
        return dict(op="lora", dt=dt, T=T, L=L, r=rng.choice([8, 16, 16, 32, 64]), K=64 * _log(rng, 8, 64),
                    N=_log(rng, 256, 4096 if T > 2048 else 14336), prompts=0 if T <= 256 and rng.random() < 0.7 else rng.randint(1, 12),
                    without=rng.choice([0.0, 0.0, 0.1, 0.5]))
    fmt = rng.choice(["ternary", "w4"])
    step = 64 if fmt == "ternary" else GROUP
    while True:
        E = _log(rng, 2, 128)
        k = min(E, rng.choice([1, 2, 2, 4, 6, 8]))
        K = step * _log(rng, 512 // step, 14336 // step)
        N = 2 * _log(rng, 256, 14336) if rng.random() < 0.7 else _log(rng, 512, 28672)
        T = _log(rng, 1, 4096)
        if E * K * N <= MAX_WEIGHTS and 2 * T * k * K * N <= MAX_FLOPS:
            break
    gated = N % 2 == 0 and rng.random() < 0.5
    return dict(op="experts", fmt=fmt, dt=dt, T=T, E=E, k=k, K=K, N=N, gated=gated, gather=gated or rng.random() < 0.3,
                zeros=fmt == "w4" and rng.random() < 0.4, skew=rng.choice([0.0, 0.3, 0.6]) if T * k >= 8 * E else 0.0)


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"route": _prepare_route, "experts": _prepare_experts, "combine": _prepare_combine,
            "lora": _prepare_lora}[case["op"]](case, g)


def _routing(T, E, k, skew, g):
    """Distinct experts of each token, more often the ones that the skew favours: [T, k]."""
    favour = torch.linspace(-1.0, 1.0, E, device=DEV) * skew * 2
    score = torch.randn((T, E), generator=g, device=DEV) + favour[torch.randperm(E, generator=g, device=DEV)]
    return score.topk(k, dim=1).indices


def _grouped(ids, E):
    """Pairs sorted by expert: (offsets [E + 1], rows [P], places [P])."""
    flat = ids.reshape(-1)
    rows = torch.argsort(flat, stable=True)
    places = torch.empty_like(rows)
    places[rows] = torch.arange(rows.numel(), device=DEV)
    offsets = torch.searchsorted(flat[rows].contiguous(), torch.arange(E + 1, device=DEV))
    return offsets.to(torch.int32), rows.to(torch.int32), places.to(torch.int32)


def _prepare_route(c, g):
    x = torch.randn((c["T"], c["E"]), generator=g, device=DEV) * 1.5
    x = x + torch.randn((c["E"],), generator=g, device=DEV) * 0.5  # some experts are liked by most tokens
    return {"op": "route", "logits": x.to(DTYPES[c["dt"]]), "k": c["k"], "renorm": c["renorm"]}


def _prepare_experts(c, g):
    T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
    offsets, rows, _ = _grouped(_routing(T, E, k, c["skew"], g), E)
    s = {"op": "experts", "fmt": c["fmt"], "gated": c["gated"], "offsets": offsets, "rows": rows if c["gather"] else None,
         "counts": (offsets[1:] - offsets[:-1]).tolist(), "k": k, "zeros": None}
    s["A"] = torch.randn((T if c["gather"] else T * k, K), generator=g, device=DEV, dtype=DTYPES[c["dt"]])
    if c["fmt"] == "ternary":
        s["scale"] = (torch.rand((E, N), generator=g, device=DEV) * 0.02 + 0.01).half()
        codes = torch.zeros((E, N, K // 4), dtype=torch.uint8, device=DEV)
        for f in range(4):  # a third of the weights each of -1, 0 and +1
            codes |= torch.randint(0, 3, codes.shape, generator=g, device=DEV, dtype=torch.uint8) << (2 * f)
        s["w"] = codes
    else:
        s["scale"] = (torch.rand((E, N, K // GROUP), generator=g, device=DEV) * 0.004 + 0.002).half()
        s["w"] = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), generator=g, device=DEV, dtype=torch.int32)
        if c["zeros"]:
            s["zeros"] = torch.randint(4, 12, (E, N, K // GROUP), generator=g, device=DEV, dtype=torch.uint8)
    return s


def _prepare_combine(c, g):
    T, k, N = c["T"], c["k"], c["N"]
    dt = DTYPES[c["dt"]]
    E = max(8, 4 * k)
    _, _, places = _grouped(_routing(T, E, k, 0.3, g), E)
    w = torch.rand((T, k), generator=g, device=DEV) + 0.1
    return {"op": "combine", "y": torch.randn((T * k, N), generator=g, device=DEV, dtype=dt), "places": places.reshape(T, k),
            "weights": w / w.sum(1, keepdim=True),
            "add": torch.randn((T, N), generator=g, device=DEV, dtype=dt) if c["add"] else None}


def _prepare_lora(c, g):
    T, L, r, K, N = c["T"], c["L"], c["r"], c["K"], c["N"]
    dt = DTYPES[c["dt"]]
    h = torch.Generator()
    h.manual_seed(int(torch.randint(0, 2 ** 31, (1,), generator=g, device=DEV)))
    n = c["prompts"] or T  # requests: a token each, or prompts of ragged lengths
    who = torch.randint(0, L, (n,), generator=h)
    who[torch.rand(n, generator=h) < c["without"]] = -1
    if c["prompts"]:
        cuts = torch.sort(torch.randint(0, T + 1, (n - 1,), generator=h)).values.tolist()
        ids = who.repeat_interleave(torch.tensor([b - a for a, b in zip([0] + cuts, cuts + [T])]))
    else:
        ids = who
    idn = ids.tolist()
    return {"op": "lora", "x": torch.randn((T, K), generator=g, device=DEV, dtype=dt),
            "base": torch.randn((T, N), generator=g, device=DEV, dtype=dt),
            "A": torch.randn((L, r, K), generator=g, device=DEV, dtype=dt) / math.sqrt(K),
            "B": torch.randn((L, N, r), generator=g, device=DEV, dtype=dt) / math.sqrt(r),
            "scale": torch.rand((L,), generator=g, device=DEV) + 0.5, "ids": ids.to(torch.int32).to(DEV),
            "counts": [idn.count(l) for l in range(-1, L)]}


# ---------------------------------------------------------------------- run

def run(state):
    op = state["op"]
    if own:
        return _own(state, op)
    return {"route": _plain_route, "experts": _plain_experts, "combine": _plain_combine, "lora": _plain_lora}[op](state)


def _own(s, op):
    import bit_weight_only_tq_amd as tq
    if op == "route":
        r = tq.tq_moe_route(s["logits"], s["k"], renormalize=s["renorm"])
        return {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "places": r.places}
    if op == "experts":
        if s["fmt"] == "ternary":
            return tq.tq_moe_gemm(s["A"], s["w"], s["scale"], s["offsets"], rows=s["rows"], gated=s["gated"])
        return tq.w4a16_moe_gemm(s["A"], s["w"], s["scale"], s["offsets"], rows=s["rows"], zeros=s["zeros"], gated=s["gated"])
    if op == "combine":
        return tq.tq_moe_combine(s["y"], s["places"], s["weights"], add=s["add"])
    return tq.tq_lora(s["x"], s["base"], s["A"], s["B"], s["ids"], scale=s["scale"])


def _plain_route(s):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), NEG_INF, x)
    T, E = x.shape
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)  # ties: lowest index first
    w = torch.exp(val - val[:, :1])
    k = s["k"]
    weights = w[:, :k] / (w[:, :k] if s["renorm"] else w).sum(1, keepdim=True)
    chosen = val[:, :k] > NEG_INF
    weights = torch.where(chosen, weights, 0.0)
    experts = torch.where(chosen, idx[:, :k], -1)
    flat = experts.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    rows = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[rows].contiguous(), torch.arange(E + 1, device=x.device))
    places = torch.empty_like(rows)
    places[rows] = torch.arange(T * k, device=x.device)
    places = torch.where(flat < 0, -1, places).reshape(T, k)
    return {"experts": experts.to(torch.int32), "weights": weights, "offsets": offsets.to(torch.int32),
            "rows": rows.to(torch.int32), "places": places.to(torch.int32)}


def _plain_experts(s):
    A, k = s["A"], s["k"]
    src = s["rows"].long() // k if s["rows"] is not None else None
    P = A.shape[0] * k if src is not None else A.shape[0]
    N = s["w"].shape[1]
    out = torch.empty((P, N // 2 if s["gated"] else N), dtype=A.dtype, device=A.device)
    p = 0
    for e, n in enumerate(s["counts"]):
        if not n:
            continue
        x = (A[src[p:p + n]] if src is not None else A[p:p + n]).float()
        y = torch.matmul(x, _plain_weights(s, e).t())
        if s["gated"]:
            gate, up = y.chunk(2, 1)
            y = gate / (1.0 + torch.exp(-gate)) * up
        out[p:p + n] = y.to(A.dtype)
        p += n
    return out


def _plain_weights(s, e):
    """Expert e's weights in 32 bits, [N, K]."""
    w = s["w"][e]
    if s["fmt"] == "ternary":
        t = torch.stack([(w >> (2 * f)) & 3 for f in range(4)], -1).flatten(1)
        return (t.float() - 1.0) * s["scale"][e].float()[:, None]
    q = torch.stack([(w >> (4 * f)) & 15 for f in range(8)], -1).flatten(1)
    z = s["zeros"][e].float()[:, :, None] if s["zeros"] is not None else 8.0
    q = q.unflatten(1, (-1, GROUP)).float()
    return ((q - z) * s["scale"][e].float()[:, :, None]).flatten(1)


def _plain_combine(s):
    y = s["y"][s["places"].long()].float()
    out = (s["weights"][:, :, None] * y).sum(1)
    if s["add"] is not None:
        out = out + s["add"].float()
    return out.to(s["y"].dtype)


def _plain_lora(s):
    out = s["base"].float()
    order = torch.argsort(s["ids"], stable=True)
    p = s["counts"][0]  # rows without an adapter come first
    for l, n in enumerate(s["counts"][1:]):
        if not n:
            continue
        rows = order[p:p + n]
        h = torch.matmul(s["x"][rows].float(), s["A"][l].float().t())
        out[rows] += s["scale"][l] * torch.matmul(h, s["B"][l].float().t())
        p += n
    return out.to(s["base"].dtype)


# ------------------------------------------------------- work and exactness

def work(case):
    c = case
    T = c["T"]
    if c["op"] == "route":
        size = 4 if c["dt"] == "f32" else 2
        return {"bytes": T * c["E"] * size + 16 * T * c["k"] + 4 * (c["E"] + 1), "flops": 4 * T * c["E"]}
    if c["op"] == "experts":
        E, k, K, N = c["E"], c["k"], c["K"], c["N"]
        P = T * k
        used = E * (1.0 - (1.0 - k / E) ** T)  # experts with a row, where all are as likely
        row = N * K // 4 + 2 * N if c["fmt"] == "ternary" else N * K // 2 + N * (K // GROUP) * (3 if c["zeros"] else 2)
        return {"bytes": used * row + 2 * (T if c["gather"] else P) * K + 2 * P * (N // 2 if c["gated"] else N)
                + (4 * P if c["gather"] else 0), "flops": 2 * P * K * N}
    if c["op"] == "combine":
        k, N = c["k"], c["N"]
        return {"bytes": T * (k + 1 + (1 if c["add"] else 0)) * N * 2 + 8 * T * k, "flops": 2 * T * k * N}
    L, r, K, N = c["L"], c["r"], c["K"], c["N"]
    n = c["prompts"] or T
    share = 1.0 - c["without"]
    used = L * (1.0 - (1.0 - share / L) ** n)
    return {"bytes": used * r * (K + N) * 2 + T * share * K * 2 + 2 * T * N * 2 + 4 * T, "flops": 2 * T * share * r * (K + N)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "combine": _exact_combine, "lora": _exact_lora}[s["op"]](s)


def _exact_route(s):
    import numpy as np
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    k = s["k"]
    experts = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    of = [[] for _ in range(E + 1)]
    for t in range(T):
        order = np.lexsort((np.arange(E), -x[t]))
        w = np.exp(x[t][order] - x[t][order[0]])
        total = w[:k].sum() if s["renorm"] else w.sum()
        for j in range(k):
            e = int(order[j])
            if x[t, e] > NEG_INF:
                experts[t, j], weights[t, j] = e, w[j] / total
                of[e].append(t * k + j)
            else:
                of[E].append(t * k + j)
    rows = np.concatenate([np.asarray(v, np.int32) for v in of])
    places = np.full(T * k, -1, np.int32)
    n = T * k - len(of[E])
    places[rows[:n]] = np.arange(n)
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in of[:E]])]).astype(np.int32)
    f = torch.from_numpy
    return {"experts": f(experts), "weights": f(weights), "offsets": f(offsets), "rows": f(rows), "places": f(places.reshape(T, k))}


def _exact_experts(s):
    A = s["A"].double()
    off = s["offsets"].tolist()
    E, N = s["w"].shape[0], s["w"].shape[1]
    K = A.shape[1]
    col = torch.arange(K, device=A.device)
    P = off[-1]
    out = torch.zeros((P, N // 2 if s["gated"] else N), dtype=torch.float64, device=A.device)
    token = torch.arange(P, device=A.device)
    if s["rows"] is not None:
        token = torch.div(s["rows"].long(), s["k"], rounding_mode="floor")
    for e in range(E):
        at = slice(off[e], off[e + 1])
        if off[e + 1] == off[e]:
            continue
        y = torch.empty((off[e + 1] - off[e], N), dtype=torch.float64, device=A.device)
        for n0 in range(0, N, 4096):
            n1 = min(N, n0 + 4096)
            word = s["w"][e, n0:n1]
            if s["fmt"] == "ternary":
                code = (word[:, col // 4].int() >> (2 * (col % 4)).int()) & 3
                w = (code - 1).double() * s["scale"][e, n0:n1, None].double()
            else:
                code = (word[:, col // 8] >> (4 * (col % 8)).int()) & 15
                zero = 8 if s["zeros"] is None else s["zeros"][e, n0:n1].int()[:, col // GROUP]
                w = (code - zero).double() * s["scale"][e, n0:n1].double()[:, col // GROUP]
            y[:, n0:n1] = A[token[at]] @ w.T.contiguous()
        out[at] = torch.sigmoid(y[:, :N // 2]) * y[:, :N // 2] * y[:, N // 2:] if s["gated"] else y
    return out


def _exact_combine(s):
    T, k = s["places"].shape
    out = torch.zeros((T, s["y"].shape[1]), dtype=torch.float64, device=s["y"].device)
    if s["add"] is not None:
        out += s["add"].double()
    for j in range(k):
        out += s["weights"][:, j:j + 1].double() * s["y"][s["places"][:, j].long()].double()
    return out


def _exact_lora(s):
    out = s["base"].double()
    ids = s["ids"].cpu().numpy()
    for l in sorted(set(ids.tolist())):
        if l < 0:
            continue
        at = torch.from_numpy((ids == l).nonzero()[0]).to(out.device)
        both = s["B"][l].double() @ s["A"][l].double()  # [N, K]
        out[at] += float(s["scale"][l]) * (s["x"][at].double() @ both.T.contiguous())
    return out
