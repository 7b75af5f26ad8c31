"""A small decoder served with the library's calls alone for the heavy work: packed 4- and 5-bit
projections, page tables, KV append, paged attention and sampling, in the order a server makes
them. Random weights; norms, rotary positions and the embedding lookup are plain torch.

    python examples/serving_step.py [--experts 16]

serves four requests: their prompts in chunks (a step holds up to 64 tokens, what a projection
call takes), then decode steps in which every request draws its next token with its own settings.
With experts, the SwiGLU blocks are layers of experts with 8-bit weights, each token taking the best two.
All lengths, tables and settings stay on the GPU; only the tokens come back.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from weight_only_groupwise_gb300 import nq  # noqa: E402

STEP = 64            # tokens of a step


def packed(bits: int, K: int, N: int, g):
    """A random K x N weight of 4- or 5-bit codes, outputs of about unit variance for unit inputs."""
    word = lambda n: torch.randint(-2 ** 31, 2 ** 31, (N, n), device="cuda", generator=g).to(torch.int32)  # noqa: E731
    std = (2 ** (2 * bits) - 1) ** 0.5 / 12 ** 0.5
    s = torch.full((N, K // 64), K ** -0.5 / std, device="cuda", dtype=torch.float16)
    return nq.pack_q4(word(K // 8), s, K, N) if bits == 4 else nq.pack_q5(word(K // 8), word(K // 32), s, K, N)


def coded(E: int, N: int, K: int, g):
    """Random 8-bit weights of E experts with their block scales, outputs of about unit variance for unit inputs."""
    codes = (105 * torch.randn((E, N, K), device="cuda", generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, torch.full((E, -(-N // 128), -(-K // 128)), K ** -0.5 / 105, device="cuda")


class Decoder:
    """Layers of grouped-query attention (5-bit projections) and a SwiGLU block (4-bit), or `experts` of them
    (8-bit) of which each token takes `chosen`."""

    def __init__(self, layers=2, hidden=1024, heads=8, kv_heads=2, dim=128, inner=2816, vocab=32000, seed=0, experts=0, chosen=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.inner, self.hidden, self.vocab = heads, kv_heads, dim, inner, hidden, vocab
        self.experts, self.chosen = experts, chosen
        self.embed = torch.randn((vocab, hidden), device="cuda", generator=g).to(torch.bfloat16)
        self.layers = [{"q": packed(5, hidden, heads * dim, g), "k": packed(5, hidden, kv_heads * dim, g),
                        "v": packed(5, hidden, kv_heads * dim, g), "o": packed(5, heads * dim, hidden, g),
                        **self.block(g)} for _ in range(layers)]
        self.head = packed(4, hidden, vocab, g)

    def block(self, g):
        E, hidden, inner = self.experts, self.hidden, self.inner
        if E:
            return {"router": packed(5, hidden, E, g), "gate": coded(E, inner, hidden, g), "up": coded(E, inner, hidden, g),
                    "down": coded(E, hidden, inner, g)}
        return {"gate": packed(4, hidden, inner, g), "up": packed(4, hidden, inner, g), "down": packed(4, inner, hidden, g)}

    def feed(self, x, w):
        """x plus its SwiGLU block, or plus its experts'."""
        h = self.norm(x)
        if not self.experts:
            return x + nq.gemm_q4(nq.swiglu_q4(h, *w["gate"], *w["up"], self.inner), *w["down"], self.hidden)
        _, weights, offsets, rows, slots = nq.moe_route(nq.gemm_q5(h, *w["router"], self.experts), self.chosen)
        inner = nq.swiglu_fp8_experts(*nq.quant_fp8(h), *w["gate"], *w["up"], offsets, rows=rows, dtype=torch.float8_e4m3fn)
        return nq.moe_combine(nq.gemm_fp8_experts(*inner, *w["down"], offsets), slots, weights, base=x)

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def rotate(self, x, positions):
        half = self.dim // 2
        angle = positions.clamp(min=0)[:, None, None] * 10000.0 ** (-torch.arange(half, device="cuda") / half)
        a, b = x.float().split(half, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).to(torch.bfloat16)

    def __call__(self, tokens, step, table, caches):
        """Logits [tokens][vocab] of a step: flat tokens, what page_tables gave for them, the block
        table and each layer's paged caches."""
        q_start, kv_lens, positions, slots, _ = step
        x = self.embed[tokens]
        for w, (k_cache, v_cache) in zip(self.layers, caches):
            h = self.norm(x)
            width = self.kv_heads * self.dim
            q, k, v = nq.gemm_q5_grouped(h, [(*w["q"], self.heads * self.dim), (*w["k"], width), (*w["v"], width)])
            q = self.rotate(q.view(-1, self.heads, self.dim), positions)
            k = self.rotate(k.view(-1, self.kv_heads, self.dim), positions)
            nq.kv_append(k, v.view(-1, self.kv_heads, self.dim), slots, k_cache, v_cache)
            a = nq.attn_paged(q, k_cache, v_cache, table, q_start, kv_lens)
            x = x + nq.gemm_q5(a.view(-1, self.heads * self.dim), *w["o"], self.hidden)
            x = self.feed(x, w)
        return nq.gemm_q4(self.norm(x), *self.head, self.vocab)


class Server:
    """The requests of one batch over a paged pool: lengths, block table and free list on the GPU."""

    def __init__(self, model: Decoder, requests: int, blocks: int = 256, page: int = 64, most_blocks: int = 32):
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        self.model, self.page = model, page
        self.lens, self.table = i32(requests), i32(requests, most_blocks)
        self.free = torch.randperm(blocks, device="cuda").to(torch.int32)
        self.num_free, self.refused = i32(1) + blocks, i32(1)
        shape = (blocks, page, model.kv_heads, model.dim)
        self.caches = [[torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in model.layers]

    def step(self, tokens, new_lens):
        """Runs the flat new tokens (new_lens of each request) and returns their logits."""
        step = nq.page_tables(self.lens, new_lens, self.free, self.num_free, self.table, self.page, tokens.numel())
        q_start, kv_lens, positions, slots, counts = step
        logits = self.model(tokens, step, self.table, self.caches)
        # the lengths grow, the blocks taken leave the front of the free list
        self.lens = torch.where(kv_lens > 0, kv_lens, self.lens)
        self.free = self.free[(torch.arange(self.free.numel(), device="cuda") + counts[1]) % self.free.numel()]
        self.num_free -= counts[1]
        self.refused += counts[2]
        return logits, q_start

    def prompt(self, prompts, chunk: int):
        """Feeds the prompts, up to `chunk` tokens a request a step; the logits after each."""
        last = torch.empty((len(prompts), self.model.vocab), dtype=torch.bfloat16, device="cuda")
        for at in range(0, max(map(len, prompts)), chunk):
            parts = [p[at:at + chunk] for p in prompts]
            new = torch.tensor([len(p) for p in parts], dtype=torch.int32, device="cuda")
            logits, q_start = self.step(torch.cat(parts), new)
            ends = q_start[1:].long() - 1
            last = torch.where(new[:, None] > 0, logits[ends], last)
        return last

    def generate(self, logits, steps: int, generator, **settings):
        """Draws `steps` tokens for every request, each from the logits of the one before."""
        tokens, one = [], torch.ones_like(self.lens)
        for _ in range(steps):
            noise = torch.empty(logits.shape, device="cuda").exponential_(generator=generator)
            tokens.append(nq.sample(logits, noise, **settings))
            logits, _ = self.step(tokens[-1].long(), one)
        return torch.stack(tokens, 1)


def main(experts: int = 0):
    model = Decoder(experts=experts, inner=768 if experts else 2816)
    server = Server(model, 4)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (n,), device="cuda", generator=g) for n in (5, 70, 130, 33)]
    logits = server.prompt(prompts, STEP // len(prompts))
    f32 = lambda *v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    out = server.generate(logits, 16, g, temperature=f32(0.0, 0.7, 1.0, 1.0), top_p=f32(1.0, 0.9, 0.95, 1.0),
                          min_p=f32(0.0, 0.0, 0.0, 0.05),
                          top_k=torch.tensor([0, 50, 0, 200], dtype=torch.int32, device="cuda"))
    nq.device_error()
    assert int(server.refused) == 0, "the pool is full"
    for r, t in enumerate(out.tolist()):
        print(f"request {r}: prompt of {len(prompts[r])}, then {t}")
    print("blocks left:", int(server.num_free), "lengths:", server.lens.tolist())


if __name__ == "__main__":
    main(int(sys.argv[2]) if sys.argv[1:2] == ["--experts"] else 0)
