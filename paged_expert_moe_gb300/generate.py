"""Samples continuations of one prompt from a small random-weight decoder: the paged cache, the
attention over a shared prefix, the paged experts and the sampling as they run together.

The prompt goes through the model once. Its keys and values fill pages that every
continuation then reads as the shared prefix, followed by pages of its own:

    moe_kv_append          head norm, rotation, keys and values into the pages
    moe_prefix_attention   the prompt itself: row t sees t + 1 keys of one sequence;
                           continuations: the prompt's pages, then the row's own
    moe_router_gemm_topk   the router
    moe_paged_forward      the experts, copied in as they miss, plus the residual
    moe_sample_tokens      temperature, top-k, top-p, min-p and the draw

The projections between them are plain matrix products. The weights are random, so the text
means nothing; a user's model takes the place of `Decoder`'s tensors.

    python -m paged_expert_moe_gb300.generate --prompt 1000 --samples 8 --tokens 64
"""

import argparse
import time
from dataclasses import dataclass

import numpy as np
import torch
import torch.nn.functional as F

from . import _lib as pm


@dataclass(frozen=True)
class Shape:
    vocab: int = 32000
    layers: int = 4
    hidden: int = 1024
    q_heads: int = 16
    kv_heads: int = 2
    head_dim: int = 64
    experts: int = 32
    top_k: int = 4
    intermediate: int = 256
    slots: int = 32
    page: int = 64
    theta: float = 1e6
    eps: float = 1e-6


class Decoder:
    """Random weights of a `Shape`, its expert cache, and a cache of `pages` pages a layer."""

    def __init__(self, shape, pages, max_tokens, e4m3=False, seed=0):
        s = self.shape = shape
        self.max_tokens = max_tokens
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*size, scale):
            return (torch.randn(size, generator=g, device="cuda") * scale).to(torch.bfloat16)

        heads = s.q_heads + 2 * s.kv_heads
        self.embed = normal(s.vocab, s.hidden, scale=1.0)
        self.head = normal(s.vocab, s.hidden, scale=4 * s.hidden ** -0.5)
        self.qkv = [normal(heads * s.head_dim, s.hidden, scale=s.hidden ** -0.5) for _ in range(s.layers)]
        self.out = [normal(s.hidden, s.q_heads * s.head_dim, scale=(s.q_heads * s.head_dim) ** -0.5)
                    for _ in range(s.layers)]
        self.router = [normal(s.experts, s.hidden, scale=2 * s.hidden ** -0.5) for _ in range(s.layers)]
        self.norm = torch.ones(s.head_dim, device="cuda", dtype=torch.bfloat16)  # of q's and k's heads
        at = torch.arange(s.head_dim // 2, device="cuda", dtype=torch.float64)
        self.inv_freq = (s.theta ** (-2 * at / s.head_dim)).float()
        self.experts = pm.ExpertCache(s.experts, s.top_k, s.hidden, s.intermediate, s.slots, num_layers=s.layers,
                                      max_tokens=max_tokens)
        for layer in range(s.layers):
            for e in range(s.experts):
                w = normal(3 * s.intermediate * s.hidden, scale=s.hidden ** -0.5)  # gate, up, down
                self.experts.expert_cache_load_expert(layer, e, w.view(torch.uint8).cpu().numpy())
        size = (s.layers, pages, s.kv_heads, s.page, s.head_dim)
        self.k_cache, self.v_cache = (torch.zeros(size, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        self.scale = None
        if e4m3:
            self.k_cache, self.v_cache = self.k_cache.to(torch.float8_e4m3fn), self.v_cache.to(torch.float8_e4m3fn)
            # a head's values have a mean square of 1 after the norm: 448 / 16 leaves room for 16
            self.scale = torch.full((s.kv_heads,), 16 / 448, device="cuda")
        self.scratch = None
        self.routes = None  # a list, if the routing of every call is to be kept

    def close(self):
        self.experts.close()

    def reserve(self, rows, prefix_len, max_suffix):
        """Scratch for attention calls of up to these sizes, kept for all of them."""
        n = pm.moe_prefix_attention_scratch_bytes(self.k_cache[0], self.v_cache[0], rows, self.shape.q_heads, prefix_len,
                                                  max_suffix)
        if self.scratch is None or self.scratch.numel() < n:
            self.scratch = torch.empty(n, dtype=torch.uint8, device="cuda")

    def forward(self, tokens, positions, slots, prefix_pages, prefix_len, page_table, suffix_len, max_suffix, row_seq=None):
        """Hidden states (bf16 [T, hidden]) of T tokens, whose keys and values are appended."""
        s = self.shape
        x = self.embed[tokens]
        T = x.shape[0]
        for layer in range(s.layers):
            qkv = (F.rms_norm(x, (s.hidden,), eps=s.eps) @ self.qkv[layer].T).view(T, -1, s.head_dim)
            q, k, v = qkv.split([s.q_heads, s.kv_heads, s.kv_heads], dim=1)
            kc, vc = self.k_cache[layer], self.v_cache[layer]
            q = pm.moe_kv_append(kc, vc, q, k, v, positions, slots, self.inv_freq, q_norm=self.norm, k_norm=self.norm,
                                 eps=s.eps, k_scale=self.scale, v_scale=self.scale)
            o = pm.moe_prefix_attention(kc, vc, q, prefix_pages, prefix_len, page_table, suffix_len, max_suffix,
                                        row_seq=row_seq, k_scale=self.scale, v_scale=self.scale, scratch=self.scratch)
            x = x + o.view(T, -1) @ self.out[layer].T
            h = F.rms_norm(x, (s.hidden,), eps=s.eps)
            ids, w = pm.moe_router_gemm_topk(h, self.router[layer], s.top_k)
            x = self.experts.moe_paged_forward(layer, h, ids, w, residual=x)
            if self.routes is not None:
                self.routes.append((ids, w))
        return x

    def logits(self, x):
        return (F.rms_norm(x, (self.shape.hidden,), eps=self.shape.eps) @ self.head.T).float()


def pages_needed(shape, prompt, samples, tokens):
    """Pages of the prompt, and of each continuation."""
    return -(-prompt // shape.page), -(-tokens // shape.page)


def generate(model, prompt, samples, tokens, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0, seed=0, on_logits=None):
    """`samples` continuations of `tokens` tokens each of one prompt (int tensor [n] on the
    GPU): int32 [samples, tokens]. on_logits(logits) sees what each step draws from."""
    s, n = model.shape, prompt.numel()
    dev = prompt.device
    head, own = pages_needed(s, n, samples, tokens)
    assert model.k_cache.shape[1] >= head + samples * own and model.max_tokens >= max(n, samples)
    prefix_pages = torch.arange(head, device=dev, dtype=torch.int32)
    table = head + torch.arange(samples * own, device=dev, dtype=torch.int32).view(samples, own)
    model.reserve(n, 0, n)
    model.reserve(samples, n, tokens)

    # the prompt: one sequence, whose row t sees its first t + 1 keys
    at = torch.arange(n, device=dev, dtype=torch.int32)
    x = model.forward(prompt, at, at, prefix_pages, 0, prefix_pages.view(1, -1), at + 1, n, row_seq=torch.zeros_like(at))

    fill = lambda v, dt: torch.full((samples,), v, dtype=dt, device=dev)  # noqa: E731
    cut = dict(temperature=fill(temperature, torch.float32), top_k=fill(top_k, torch.int32),
               top_p=fill(top_p, torch.float32), min_p=fill(min_p, torch.float32))
    u = torch.rand((tokens, samples), generator=torch.Generator(device=dev).manual_seed(seed), device=dev)
    drawn = torch.empty((tokens, samples), dtype=torch.int32, device=dev)
    logits = model.logits(x[-1:]).repeat(samples, 1)
    for i in range(tokens):
        if on_logits is not None:
            on_logits(logits)
        pm.moe_sample_tokens(logits, u[i], ids_out=drawn[i], **cut)
        if i + 1 < tokens:
            slots = table[:, i // s.page] * s.page + i % s.page
            x = model.forward(drawn[i].long(), fill(n + i, torch.int32), slots, prefix_pages, n, table,
                              fill(i + 1, torch.int32), tokens)
            logits = model.logits(x)
    return drawn.T.contiguous()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--prompt", type=int, default=1000, help="tokens of the prompt")
    p.add_argument("--samples", type=int, default=8)
    p.add_argument("--tokens", type=int, default=64, help="tokens of a continuation")
    p.add_argument("--layers", type=int, default=Shape.layers)
    p.add_argument("--slots", type=int, default=Shape.slots, help="resident experts a layer, of %d" % Shape.experts)
    p.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    p.add_argument("--temperature", type=float, default=0.8)
    p.add_argument("--top-k", type=int, default=50)
    p.add_argument("--top-p", type=float, default=0.95)
    p.add_argument("--min-p", type=float, default=0.0)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    shape = Shape(layers=a.layers, slots=a.slots)
    head, own = pages_needed(shape, a.prompt, a.samples, a.tokens)
    model = Decoder(shape, head + a.samples * own, max(a.prompt, a.samples), e4m3=a.cache == "e4m3", seed=a.seed)
    prompt = torch.from_numpy(np.random.default_rng(a.seed).integers(0, shape.vocab, a.prompt)).cuda()
    for _ in range(2):  # the first run pages the experts in
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        ids = generate(model, prompt, a.samples, a.tokens, a.temperature, a.top_k, a.top_p, a.min_p, a.seed)
        torch.cuda.synchronize()
        t1 = time.perf_counter()
    for row in ids.tolist():
        print(" ".join(str(t) for t in row))
    print("%d continuations of %d tokens after a prompt of %d: %.1f ms, %.0f tokens/s" %
          (a.samples, a.tokens, a.prompt, 1e3 * (t1 - t0), a.samples * a.tokens / (t1 - t0)))
    model.close()


if __name__ == "__main__":
    main()
