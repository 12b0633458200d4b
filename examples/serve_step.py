"""A decoder layer served from a paged cache: the quantized linear layers and the serving operators together.

A small random model (one attention layer with ternary projections, a ternary
output layer) answers a few prompts: every step plans its pages on the device
(tq_paged_plan), projects the new tokens (tq_gemm), rotates and appends them
(tq_kv_append), attends over the pages (tq_paged_attention) and samples one
token a request (tq_sample).  Prompts come in as chunks beside requests that
already decode.  Needs a GPU and the built library:

    python examples/serve_step.py
"""

import math
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_only_tq_amd as tq  # noqa: E402


class Model(NamedTuple):
    """Weights of the layer: fp16 embedding, packed (codes, scale) projections."""
    embed: torch.Tensor   # [V, width]
    qkv: tuple            # [(Hq + 2 Hkv) D, width]
    out: tuple            # [width, Hq D]
    head: tuple           # [V, width]
    rope: torch.Tensor    # [positions, D]
    Hq: int
    Hkv: int
    D: int


def random_model(seed=0, V=1024, width=256, Hq=8, Hkv=2, D=64, positions=4096, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    pack = lambda n, k: tq.tq_pack((torch.randn((n, k), generator=g) * k ** -0.5).to(device))  # noqa: E731
    embed = torch.randn((V, width), generator=g).to(device).half()
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2).double() / D)
    rope = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
    return Model(embed, pack((Hq + 2 * Hkv) * D, width), pack(width, Hq * D), pack(V, width), rope, Hq, Hkv, D)


class Server:
    """Requests in a fixed number of slots over one paged cache."""

    def __init__(self, model, requests=4, pages=64, page_size=16, width=32):
        self.m, self.page = model, page_size
        dev = model.embed.device
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
        self.ctx, self.table = i32(requests), torch.full((requests, width), -1, dtype=torch.int32, device=dev)
        self.free, self.head = torch.arange(pages, dtype=torch.int32, device=dev), i32(1)
        shape = (pages, model.Hkv, page_size, model.D)
        self.k, self.v = (torch.zeros(shape, dtype=torch.float16, device=dev) for _ in range(2))

    def logits(self, tokens):
        """One step: tokens[b] are request b's new tokens (none, one, or a chunk of its prompt); -> logits [B, V] of
        each request's last token (of its last one before, for a request that rests: not used)."""
        m, dev = self.m, self.m.embed.device
        n = [len(t) for t in tokens]
        new = torch.tensor(n, dtype=torch.int32).to(dev)
        T = sum(n)
        plan = tq.tq_paged_plan(self.ctx, new, self.table, self.free, self.head, T, page_size=self.page)
        x = m.embed[torch.tensor([t for r in tokens for t in r], device=dev)]
        heads = tq.tq_gemm(x, *m.qkv).unflatten(1, (m.Hq + 2 * m.Hkv, m.D))
        q, k, v = heads.split([m.Hq, m.Hkv, m.Hkv], 1)
        q = tq.tq_kv_append(q, k, v, self.k, self.v, plan.slots, positions=plan.positions, rope=m.rope)
        a = tq.tq_paged_attention(q, self.k, self.v, self.table, plan.cu_q, plan.kv_lens, max(n),
                                  self.table.shape[1] * self.page)
        x = x + tq.tq_gemm(a.flatten(1), *m.out)
        last = (plan.cu_q[1:].long() - 1).clamp(min=0)
        self.ctx, self.head = plan.kv_lens, plan.state[:1].clone()
        return tq.tq_gemm(x[last].contiguous(), *m.head)


def main():
    model = random_model()
    server = Server(model)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1024, (n,), generator=g).tolist() for n in (5, 40, 23, 70)]
    answers = [[] for _ in prompts]
    chunk = 32
    dev = model.embed.device
    settings = dict(temperature=torch.full((4,), 0.8, device=dev), top_k=torch.full((4,), 50, dtype=torch.int32, device=dev),
                    top_p=torch.full((4,), 0.95, device=dev))
    for step in range(12):
        feed = []
        for p, a in zip(prompts, answers):  # a chunk of the prompt, or the token sampled last
            feed.append([p.pop(0) for _ in range(min(chunk, len(p)))] if p else [a[-1]])
        logits = server.logits(feed)
        tokens, logprobs = tq.tq_sample(logits, torch.rand((4,), generator=g).to(dev), **settings)
        for b, t in enumerate(tokens.tolist()):
            if not prompts[b]:
                answers[b].append(t)
    for b, a in enumerate(answers):
        print(f"request {b}: {a}")
    print(f"log probabilities of the last step: {[round(x, 2) for x in logprobs.tolist()]}; "
          f"{int(server.head)} pages in use for {server.ctx.tolist()} tokens")
    assert all(math.isfinite(x) for x in logprobs.tolist())


if __name__ == "__main__":
    main()
