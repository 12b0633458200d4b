"""The serving operators around the quantized linear layers, as measured cases.

A decoding or prefilling step of a model whose projections are the packed
linear layers of this repository also needs, between the products:

  plan    page tables, slot map, positions and offsets of a step, made on the
          device from the requests' lengths (tq_paged_plan)
  append  rotary positions applied to the new queries and keys, keys and values
          written to their slots of the paged cache (tq_kv_append)
  attend  attention of each request's new tokens over its pages, causal, with
          an optional sliding window and first tokens that stay visible
          (tq_paged_attention)
  sample  one token per row from its logits with temperature, top-k, min-p and
          top-p, from a given random number (tq_sample)

Each case is run in a plain form (elementary torch operations in 32 bits, 64
where a sum decides a border) or, with ``own`` set, by the library's calls.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
NEG_INF = float("-inf")


# -------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step's plan at a small batch: a launch's latency.
        dict(name="plan_decode_8", op="plan", B=8, page=16, width=512, ctx_lo=1, ctx_hi=8000, decode=8, new_hi=1),
        # A scheduler's largest step: thousands of decoding requests beside long prompt chunks.
        dict(name="plan_mixed_2048", op="plan", B=2048, page=16, width=2048, ctx_lo=0, ctx_hi=30000, decode=1920,
             new_hi=1023),
        # One new token of one request, 8B heads (32 query, 8 KV heads of 128).
        dict(name="append_one_token", op="append", dt="bf16", T=1, Hq=32, Hkv=8, D=128, page=16, rot=128,
             interleaved=False, pages=512, P=8192),
        # A full prompt batch, 70B heads (64 query, 8 KV heads of 128).
        dict(name="append_prompt_16383", op="append", dt="f16", T=16383, Hq=64, Hkv=8, D=128, page=64, rot=128,
             interleaved=False, pages=512, P=131072),
        # A single user's short conversation: the smallest decode call.
        dict(name="attend_decode_short", op="attend", dt="bf16", B=1, Hq=32, Hkv=8, D=128, page=16, kv_lo=777,
             kv_hi=777, q_lo=1, q_hi=1, chunks=0, window=0, sinks=0),
        # Two users with very long contexts: few rows, a long axis to split.
        dict(name="attend_decode_long", op="attend", dt="bf16", B=2, Hq=32, Hkv=8, D=128, page=64, kv_lo=100001,
             kv_hi=131071, q_lo=1, q_hi=1, chunks=0, window=0, sinks=0),
        # A busy server's decode step, 70B heads, ragged lengths.
        dict(name="attend_decode_64", op="attend", dt="f16", B=64, Hq=64, Hkv=8, D=128, page=16, kv_lo=33,
             kv_hi=8191, q_lo=1, q_hi=1, chunks=0, window=0, sinks=0),
        # A long prompt's second chunk over what its first left in the cache.
        dict(name="attend_chunk_8192", op="attend", dt="bf16", B=1, Hq=32, Hkv=8, D=128, page=16, kv_lo=12288,
             kv_hi=12288, q_lo=8192, q_hi=8192, chunks=1, window=0, sinks=0),
        # A mixed step of a sliding-window model with smaller heads: decoding
        # requests and ragged prompt chunks together.
        dict(name="attend_mixed_window", op="attend", dt="f16", B=33, Hq=24, Hkv=8, D=64, page=32, kv_lo=100,
             kv_hi=9001, q_lo=65, q_hi=1501, chunks=9, window=2047, sinks=4),
        # One row of a small vocabulary: latency.
        dict(name="sample_one_row", op="sample", dt="f32", B=1, V=32000, k=50, p=0.95, minp=0.0, T=0.8),
        # A decode step's rows, 16-bit logits, top-k and top-p together.
        dict(name="sample_64_topk", op="sample", dt="bf16", B=64, V=128000, k=200, p=0.9, minp=0.0, T=1.0),
        # A large batch without top-k on an odd vocabulary: the nucleus alone, with min-p.
        dict(name="sample_256_topp", op="sample", dt="f32", B=256, V=129281, k=0, p=0.92, minp=0.02, T=0.7),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "sample", "sample"])
    if op == "plan":
        B = _log(rng, 1, 2048)
        width = _log(rng, 64, 2048)
        page = rng.choice([16, 32, 64, 128])
        decode = rng.randint(0, B)
        room = width * page
        ctx_hi = _log(rng, 16, room - room // 4)
        return dict(op="plan", B=B, page=page, width=width, ctx_lo=0, ctx_hi=ctx_hi, decode=decode,
                    new_hi=max(1, min(room - ctx_hi, 131072 // max(B - decode, 1))))
    if op == "append":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
        T = _log(rng, 1, 16383)
        page = rng.choice([16, 32, 64, 128])
        return dict(op="append", dt=rng.choice(["f16", "bf16"]), T=T, Hq=Hq, Hkv=Hkv, D=D, page=page,
                    rot=rng.choice([D, D, D // 2, 0]), interleaved=rng.random() < 0.3,
                    pages=-(-T // page) + rng.randint(1, 64), P=_log(rng, 20000, 131072))
    if op == "attend":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
        dt = rng.choice(["f16", "bf16"])
        page = rng.choice([16, 32, 64, 128])
        window, sinks = (0, 0) if rng.random() < 0.6 else (_log(rng, 16, 4096), rng.choice([0, 1, 4, 17]))
        kind = rng.choice(["decode", "chunk", "mixed"])
        if kind == "decode":
            B = _log(rng, 1, 64)
            hi = _log(rng, 16, min(131072, 262144 // B))
            return dict(op="attend", dt=dt, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, kv_lo=max(1, hi // 4), kv_hi=hi,
                        q_lo=1, q_hi=rng.choice([1, 1, 1, 2, 5]), chunks=0, window=window, sinks=sinks)
        if kind == "chunk":
            q = _log(rng, 2, 8192)
            kv = q + _log(rng, 1, 4096)
            return dict(op="attend", dt=dt, B=1, Hq=min(Hq, 32), Hkv=Hkv if Hq <= 32 else 4, D=D, page=page, kv_lo=kv,
                        kv_hi=kv, q_lo=q, q_hi=q, chunks=1, window=window, sinks=sinks)
        B = _log(rng, 2, 48)
        q_hi = _log(rng, 16, 1024)
        return dict(op="attend", dt=dt, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, kv_lo=8, kv_hi=q_hi + _log(rng, 64, 4096),
                    q_lo=max(1, q_hi // 8), q_hi=q_hi, chunks=rng.randint(1, B), window=window, sinks=sinks)
    dt = rng.choice(["f16", "bf16", "f32"])
    V = _log(rng, 2000, 200000)
    return dict(op="sample", dt=dt, B=max(1, min(_log(rng, 1, 256), 256 * 129281 // V)), V=V,
                k=rng.choice([0, 1, 20, 50, 1000]), p=rng.choice([1.0, 0.95, 0.8, 0.5]),
                minp=rng.choice([0.0, 0.0, 0.05, 0.3]), T=rng.choice([0.0, 0.6, 1.0, 1.3]))


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    return {"plan": _prepare_plan, "append": _prepare_append, "attend": _prepare_attend,
            "sample": _prepare_sample}[case["op"]](case, g, h)


def _spread(h, lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], in an order of the seed's: their sum is the case's own."""
    v = torch.linspace(lo, hi, n, dtype=torch.float64) if n > 1 else torch.tensor([hi], dtype=torch.float64)
    return v.round().to(torch.int32)[torch.randperm(n, generator=h)]


def _prepare_plan(c, g, h):
    B, page, width = c["B"], c["page"], c["width"]
    ctx = _spread(h, c["ctx_lo"], c["ctx_hi"], B)
    new = torch.ones(B, dtype=torch.int32)  # decoding requests bring one token, the others a chunk
    who = torch.randperm(B, generator=h)[:B - c["decode"]]
    new[who] = _spread(h, 1, c["new_hi"], len(who))
    held = (ctx + page - 1) // page
    total = int(held.sum())
    need = int(((ctx + new + page - 1) // page - held).sum())
    ids = torch.randperm(total + need + 64, generator=g, device=DEV, dtype=torch.int32)
    cols = torch.arange(width, dtype=torch.int32)[None, :].expand(B, width)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[(cols < held[:, None]).to(DEV)] = ids[:total]
    return {"op": "plan", "ctx": ctx.to(DEV), "new": new.to(DEV), "table": table, "free": ids[total:].contiguous(),
            "head": torch.full((1,), 5, dtype=torch.int32, device=DEV), "tokens": int(new.sum()), "page": page}


def _prepare_append(c, g, h):
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    dt = DTYPES[c["dt"]]
    # the fused projection's output: queries, keys and values of a token side by side
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV, dtype=dt)
    shape = (c["pages"], Hkv, c["page"], D)
    kc = torch.randn(shape, generator=g, device=DEV, dtype=dt)
    vc = torch.randn(shape, generator=g, device=DEV, dtype=dt)
    slots = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:T].contiguous()
    start = int(torch.randint(0, c["P"] - T + 1, (1,), generator=h))
    pos = torch.arange(start, start + T, dtype=torch.int32, device=DEV)
    rope = None
    if c["rot"]:
        inv = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
        ang = torch.arange(c["P"], dtype=torch.float64, device=DEV)[:, None] * inv
        rope = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    return {"op": "append", "q": q.unflatten(1, (Hq, D)), "k": k.unflatten(1, (Hkv, D)), "v": v.unflatten(1, (Hkv, D)),
            "kc": kc, "vc": vc, "slots": slots, "pos": pos, "rope": rope, "interleaved": c["interleaved"]}


def _prepare_attend(c, g, h):
    B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    dt = DTYPES[c["dt"]]
    kv = _spread(h, c["kv_lo"], c["kv_hi"], B)
    if c["chunks"]:
        qn = torch.ones(B, dtype=torch.int32)
        who = torch.randperm(B, generator=h)[:c["chunks"]]
        qn[who] = _spread(h, c["q_lo"], c["q_hi"], len(who))
    else:
        qn = _spread(h, c["q_lo"], c["q_hi"], B)
    kv = torch.maximum(kv, qn)  # a request's new tokens are in the cache already
    blocks = (kv + page - 1) // page
    width = int(blocks.max())
    pages = int(blocks.sum()) + 8
    ids = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
    cols = torch.arange(width, dtype=torch.int32)[None, :].expand(B, width)
    table = torch.zeros((B, width), dtype=torch.int32, device=DEV)
    table[(cols < blocks[:, None]).to(DEV)] = ids[:int(blocks.sum())]
    kc = torch.randn((pages, Hkv, page, D), generator=g, device=DEV, dtype=dt)
    vc = torch.randn((pages, Hkv, page, D), generator=g, device=DEV, dtype=dt)
    T = int(qn.sum())
    q = torch.randn((T, Hq, D), generator=g, device=DEV, dtype=dt) * 2
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = qn.cumsum(0)
    s = {"op": "attend", "q": q, "kc": kc, "vc": vc, "table": table, "cu": cu.to(DEV), "kv": kv.to(DEV),
         "qn": qn.tolist(), "kvn": kv.tolist(), "window": c["window"], "sinks": c["sinks"], "page": page}
    if own:
        import bit_weight_only_tq_amd as tq
        s["ws"] = tq.new_workspace(tq.tq_paged_attention_workspace_bytes(
            T, Hq, Hkv, D, B, max(s["qn"]), max(s["kvn"]), c["window"], c["sinks"]), torch.device(DEV, 0))
    return s


def _prepare_sample(c, g, h):
    B, V = c["B"], c["V"]
    # a broad body of unlikely tokens and a few dozen likely ones in each row
    x = torch.randn((B, V), generator=g, device=DEV) * 2.0
    n = 64
    at = torch.randint(0, V, (B, n), generator=g, device=DEV)
    x.scatter_add_(1, at, torch.rand((B, n), generator=g, device=DEV) ** 2 * 14)
    f = lambda v, dtype=torch.float32: torch.full((B,), v, dtype=dtype, device=DEV)  # noqa: E731
    return {"op": "sample", "logits": x.to(DTYPES[c["dt"]]), "u": torch.rand((B,), generator=g, device=DEV),
            "T": f(c["T"]), "k": f(c["k"], torch.int32), "p": f(c["p"]), "minp": f(c["minp"])}


# ---------------------------------------------------------------------- run

def run(state):
    op = state["op"]
    if own:
        return _own(state, op)
    return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[op](state)


def _own(s, op):
    import bit_weight_only_tq_amd as tq
    if op == "plan":
        r = tq.tq_paged_plan(s["ctx"], s["new"], s["table"], s["free"], s["head"], s["tokens"], page_size=s["page"])
        return {"table": s["table"], "cu_q": r.cu_q, "kv_lens": r.kv_lens, "positions": r.positions, "slots": r.slots,
                "state": r.state}
    if op == "append":
        q = tq.tq_kv_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], rope=s["rope"],
                            positions=None if s["rope"] is None else s["pos"], interleaved=s["interleaved"])
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    if op == "attend":
        out, lse = tq.tq_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], max(s["qn"]),
                                         max(s["kvn"]), window=s["window"], sinks=s["sinks"], return_lse=True,
                                         workspace=s["ws"])
        return {"out": out, "lse": lse}
    tokens, logprobs = tq.tq_sample(s["logits"], s["u"], temperature=s["T"], top_k=s["k"], top_p=s["p"],
                                    min_p=s["minp"])
    return {"tokens": tokens, "logprobs": logprobs}


def _plain_plan(s):
    ctx, new, table, page = s["ctx"], s["new"], s["table"], s["page"]
    B, width = table.shape
    T = s["tokens"]
    cu = torch.zeros(B + 1, dtype=torch.int32, device=ctx.device)
    cu[1:] = torch.cumsum(new, 0)
    kv = ctx + new
    held = torch.clamp((ctx + page - 1) // page, max=width)
    need = torch.clamp((kv + page - 1) // page, max=width)
    take = torch.cumsum(need - held, 0) - (need - held)  # pages taken by the requests before
    cols = torch.arange(width, device=ctx.device)[None, :]
    fresh = (cols >= held[:, None]) & (cols < need[:, None])
    at = s["head"] + take[:, None] + cols - held[:, None]
    ok = fresh & (at < s["free"].numel())
    got = torch.where(ok, s["free"][torch.clamp(at, 0, s["free"].numel() - 1)], -1)
    table.copy_(torch.where(fresh, got.to(torch.int32), table))
    t = torch.arange(T, device=ctx.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = ctx[b] + (t - cu[b])
    blk = pos // page
    pg = torch.where(blk < width, table[b, torch.clamp(blk, max=width - 1)], -1)
    slots = torch.where(pg >= 0, pg.long() * page + pos % page, -1)
    head = torch.clamp(s["head"] + (need - held).sum(), max=s["free"].numel())
    return {"table": table, "cu_q": cu, "kv_lens": kv, "positions": pos.to(torch.int32), "slots": slots,
            "state": torch.cat([head, (slots < 0).sum().reshape(1)]).to(torch.int32)}


def _rotate(x, rope, pos, interleaved):
    x = x.float()
    if rope is None:
        return x
    cos, sin = rope[pos.long()].chunk(2, 1)
    cos, sin = cos[:, None], sin[:, None]
    rot = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    q, k, kc, vc, slots = s["q"], s["k"], s["kc"], s["vc"], s["slots"]
    page = kc.shape[2]
    pg, off = slots // page, slots % page
    kc[pg, :, off] = _rotate(k, s["rope"], s["pos"], s["interleaved"]).to(k.dtype)
    vc[pg, :, off] = s["v"]
    return {"q": _rotate(q, s["rope"], s["pos"], s["interleaved"]).to(q.dtype), "k_cache": kc, "v_cache": vc}


def _plain_attend(s):
    q, kc, vc, page = s["q"], s["kc"], s["vc"], s["page"]
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D)
    out = torch.empty_like(q)
    lse = torch.empty((T, Hq), device=q.device)
    t0 = 0
    for b, (n, kv) in enumerate(zip(s["qn"], s["kvn"])):
        ids = s["table"][b, :-(-kv // page)].long()
        k = kc[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :kv].float()
        v = vc[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :kv].float()
        j = torch.arange(kv, device=q.device)[None, :]
        rows = max(1, (1 << 28) // (kv * Hq))
        for r0 in range(0, n, rows):
            r1 = min(n, r0 + rows)
            i = torch.arange(kv - n + r0, kv - n + r1, device=q.device)[:, None]
            see = j <= i
            if s["window"]:
                see = see & ((i - j < s["window"]) | (j < s["sinks"]))
            x = q[t0 + r0:t0 + r1].float().reshape(r1 - r0, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
            w = torch.matmul(x, k.transpose(1, 2).contiguous()).mul_(scale).reshape(Hkv, G, r1 - r0, kv)
            w = w.masked_fill_(~see, NEG_INF)
            m = w.amax(-1, keepdim=True)
            w = w.sub_(m).exp_()
            z = w.sum(-1, keepdim=True)
            o = torch.matmul(w.reshape(Hkv, -1, kv), v).reshape(Hkv, G, r1 - r0, D) / z
            out[t0 + r0:t0 + r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, Hq, D).to(q.dtype)
            lse[t0 + r0:t0 + r1] = (m + z.log())[..., 0].permute(2, 0, 1).reshape(r1 - r0, Hq)
        t0 += n
    return {"out": out, "lse": lse}


def _plain_sample(s):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), NEG_INF, x)
    B, V = x.shape
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)  # ties: lowest index first
    temp = s["T"].double()[:, None]
    greedy = temp <= 0
    w = torch.exp((val.double() - val[:, :1].double()) / torch.where(greedy, 1.0, temp))
    rank = torch.arange(V, device=x.device)[None, :]
    k = s["k"].long()[:, None]
    k = torch.where((k <= 0) | (k > V), V, k)
    k = torch.where(greedy, 1, k)
    keep = (rank < k) & (w >= s["minp"].double()[:, None])
    w = torch.where(keep, w, 0.0)
    before = torch.cumsum(w, 1) - w
    p = s["p"].double()[:, None]
    keep = keep & ((before < p * w.sum(1, keepdim=True)) | (p >= 1) | (rank == 0))
    w = torch.where(keep, w, 0.0)
    flat = torch.zeros((B, V), dtype=torch.float64, device=x.device).scatter_(1, idx, w)
    total = flat.sum(1, keepdim=True)
    past = torch.cumsum(flat, 1) > s["u"].double()[:, None] * total
    tok = torch.argmax((past & (flat > 0)).to(torch.int8), 1)
    lp = torch.log(flat.gather(1, tok[:, None]) / total)[:, 0]
    return {"tokens": tok.to(torch.int32), "logprobs": lp.float()}


# ------------------------------------------------------- work and exactness

def _attend_counts(c):
    """Expected keys read, query tokens and (query, key) pairs of one head of an attend case."""
    B, w, s = c["B"], c["window"], c["sinks"]
    kv = (c["kv_lo"] + c["kv_hi"]) / 2 if B > 1 else c["kv_hi"]
    n = c["chunks"] or B
    q = (c["q_lo"] + c["q_hi"]) / 2 if n > 1 else c["q_hi"]
    kinds = [(n, q), (B - n, 1.0)]
    keys = tokens = pairs = 0.0
    for n, q in kinds:
        q = min(q, kv)
        read, seen = kv, kv - (q - 1) / 2
        if w:
            read, seen = min(kv, w + s + q - 1), min(seen, w + s)
        keys, tokens, pairs = keys + n * read, tokens + n * q, pairs + n * q * seen
    return keys, tokens, pairs


def work(case):
    c = case
    if c["op"] == "plan":
        tokens = c["decode"] + (c["B"] - c["decode"]) * (1 + c["new_hi"]) / 2
        # lengths read, offsets and lengths written; per token its position and slot; a page id read and written per
        # new page, and the id of a page already held where a token lands in one
        pages = tokens / c["page"]
        return {"bytes": 16 * c["B"] + 12 * tokens + 8 * pages + 4 * c["B"], "flops": 0}
    if c["op"] == "append":
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": c["T"] * (2 * heads * c["D"] * 2 + 4 * c["rot"] + 12),
                "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "attend":
        keys, tokens, pairs = _attend_counts(c)
        return {"bytes": 2 * 2 * keys * c["Hkv"] * c["D"] + 2 * 2 * tokens * c["Hq"] * c["D"] + 4 * tokens * c["Hq"]
                + 4 * keys / c["page"], "flops": 4 * pairs * c["Hq"] * c["D"]}
    size = 4 if c["dt"] == "f32" else 2
    return {"bytes": c["B"] * (c["V"] * size + 28), "flops": 2 * c["B"] * c["V"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[s["op"]](s)


def _exact_plan(s):
    ctx, new, free = s["ctx"].tolist(), s["new"].tolist(), s["free"].tolist()
    table, page = s["table"].cpu().numpy().copy(), s["page"]
    width = table.shape[1]
    head, cu, positions, slots = int(s["head"]), [0], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        for blk in range(min(width, -(-c // page)), min(width, -(-(c + n) // page))):
            table[b, blk] = free[head] if head < len(free) else -1
            head = min(head + 1, len(free))
        row = table[b].tolist()
        for i in range(c, c + n):
            pg = row[i // page] if i // page < width else -1
            positions.append(i)
            slots.append(pg * page + i % page if pg >= 0 else -1)
        cu.append(cu[-1] + n)
    t = lambda v, d=torch.int32: torch.tensor(v, dtype=d)  # noqa: E731
    return {"table": torch.from_numpy(table), "cu_q": t(cu), "kv_lens": t([c + n for c, n in zip(ctx, new)]),
            "positions": t(positions), "slots": t(slots, torch.int64), "state": t([head, sum(x < 0 for x in slots)])}


def _exact_append(s):
    kc, vc = s["kc"].double(), s["vc"].double()
    Pn, Hkv, page, D = kc.shape

    def turn(x):
        x = x.double()
        if s["rope"] is None:
            return x
        r = s["rope"].double()[s["pos"].long()]
        h = r.shape[1] // 2
        first = torch.arange(h, device=x.device)
        first, second = (2 * first, 2 * first + 1) if s["interleaved"] else (first, first + h)
        y = x.clone()
        for a in range(x.shape[1]):
            u, v = x[:, a][:, first], x[:, a][:, second]
            y[:, a, first] = u * r[:, :h] - v * r[:, h:]
            y[:, a, second] = v * r[:, :h] + u * r[:, h:]
        return y

    for cache, new in ((kc, turn(s["k"])), (vc, s["v"].double())):
        by_token = cache.transpose(1, 2).reshape(Pn * page, Hkv, D).clone()
        by_token[s["slots"]] = new
        cache.copy_(by_token.reshape(Pn, page, Hkv, D).transpose(1, 2))
    return {"q": turn(s["q"]), "k_cache": kc, "v_cache": vc}


def _exact_attend(s):
    q = s["q"].double()
    T, Hq, D = q.shape
    Hkv = s["kc"].shape[1]
    out, lse = torch.zeros_like(q), torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    t0 = 0
    for b, n in enumerate(s["qn"]):
        kv = s["kvn"][b]
        where = torch.arange(kv, device=q.device)
        ids, off = s["table"][b].long()[where // s["page"]], where % s["page"]
        for a in range(Hkv):
            k, v = s["kc"][ids, a, off].double(), s["vc"][ids, a, off].double()
            for hq in range(a * Hq // Hkv, (a + 1) * Hq // Hkv):
                z = q[t0:t0 + n, hq] @ k.T.contiguous() / math.sqrt(D)
                at = (kv - n + torch.arange(n, device=q.device))[:, None]
                hide = where[None, :] > at
                if s["window"]:
                    hide |= (at - where[None, :] >= s["window"]) & (where[None, :] >= s["sinks"])
                z[hide] = NEG_INF
                l = torch.logsumexp(z, 1)
                lse[t0:t0 + n, hq] = l
                out[t0:t0 + n, hq] = torch.exp(z - l[:, None]) @ v
        t0 += n
    return {"out": out, "lse": lse}


def _exact_sample(s):
    import numpy as np
    x = s["logits"].double().cpu().numpy()
    T, k, p, minp, u = (s[n].cpu().numpy() for n in ("T", "k", "p", "minp", "u"))
    tok, lp = [], []
    for b in range(x.shape[0]):
        row = x[b]
        V = row.size
        order = np.lexsort((np.arange(V), -row))
        if T[b] <= 0:
            tok.append(int(order[0]))
            lp.append(0.0)
            continue
        w = np.exp((row[order] - row[order[0]]) / float(T[b]))
        n = V if k[b] <= 0 else min(V, int(k[b]))
        n = min(n, int(np.count_nonzero(w >= float(minp[b]))))
        order, w = order[:n], w[:n]
        if p[b] < 1:
            run_sum = np.concatenate([[0.0], np.cumsum(w)[:-1]])
            n = max(1, int(np.count_nonzero(run_sum < float(p[b]) * w.sum())))
            order, w = order[:n], w[:n]
        by_index = np.argsort(order)
        c = np.cumsum(w[by_index])
        i = min(int(np.searchsorted(c, float(u[b]) * c[-1], side="right")), n - 1)
        tok.append(int(order[by_index[i]]))
        lp.append(float(np.log(w[by_index[i]] / c[-1])))
    return {"tokens": torch.tensor(tok, dtype=torch.int32), "logprobs": torch.tensor(lp, dtype=torch.float64)}
