"""Serves prompts of different lengths at once with a small random-weight decoder: every step is a
mixture of pieces of prompts and of single tokens, over pages that requests take and give back.

    moe_batch_tables       pages, slots, positions and row ranges of the step's tokens
    moe_kv_append          head norm, rotary positions, append to the pages
    moe_chunk_attention    each request's new tokens over its own pages; every other layer
                           with a sliding window and first keys that stay visible
    moe_router_select      experts by sigmoid scores, a balance bias and expert groups
    moe_paged_forward      the paged experts
    moe_adjust_logits      penalties for repeated tokens, biases, a grammar's mask
    moe_sample_tokens      the draw

The projections between them are plain matrix products. The weights are random, so the text
means nothing; a user's model takes the place of the tensors.

    python -m paged_expert_moe_gb300.serve --requests 12 --tokens 40
"""

import argparse
import time
from dataclasses import dataclass, field

import numpy as np
import torch
import torch.nn.functional as F

from . import _lib as pm
from .generate import Decoder, Shape


@dataclass(frozen=True)
class ServeShape(Shape):
    groups: int = 4          # of experts
    top_groups: int = 2
    route_scale: float = 2.5
    window: int = 256        # of every other layer
    sinks: int = 4


@dataclass
class Request:
    prompt: list
    tokens: int                     # how many to generate
    repetition: float = 1.0
    frequency: float = 0.0
    presence: float = 0.0
    biases: dict = field(default_factory=dict)   # token id: what is added to its logit
    allowed: list = None            # token ids that a grammar allows, or None
    output: list = field(default_factory=list)

    def done(self):
        return len(self.output) >= self.tokens


class Server:
    """`seats` requests at a time, steps of up to `rows` tokens, a cache of `pages` pages a layer."""

    def __init__(self, shape, seats, rows, pages, longest, max_biases=16, e4m3=False, seed=0):
        self.shape, self.seats, self.rows, self.pages, self.longest = shape, seats, rows, pages, longest
        self.model = Decoder(shape, pages, rows, e4m3=e4m3, seed=seed)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.balance = [torch.randn(shape.experts, generator=g, device="cuda") * 0.05 for _ in range(shape.layers)]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.zeros((seats, -(-longest // shape.page)), **i32)
        self.free = torch.arange(pages, **i32)
        self.free_count = torch.tensor([pages], **i32)
        self.lens = torch.zeros(seats, **i32)
        self.err = torch.zeros(1, **i32)
        self.history = torch.zeros((seats, longest), **i32)
        self.max_biases = max_biases
        n = pm.moe_chunk_attention_scratch_bytes(self.model.k_cache[0], self.model.v_cache[0], rows, shape.q_heads, seats)
        self.scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.generator = torch.Generator(device="cuda").manual_seed(seed + 2)
        self.seated, self.read = [None] * seats, [0] * seats  # requests, and how much of each is in the cache
        self.ended = []   # seats whose pages go back with the next step
        self.routes = None  # a list, if the routing of every call is to be kept

    def close(self):
        self.model.close()

    def hidden(self, tokens, t):
        """Hidden states of a step's tokens, whose keys and values are appended."""
        s, m = self.shape, self.model
        x = m.embed[tokens]
        T = x.shape[0]
        for layer in range(s.layers):
            qkv = (F.rms_norm(x, (s.hidden,), eps=s.eps) @ m.qkv[layer].T).view(T, -1, s.head_dim)
            q, k, v = qkv.split([s.q_heads, s.kv_heads, s.kv_heads], dim=1)
            kc, vc = m.k_cache[layer], m.v_cache[layer]
            q = pm.moe_kv_append(kc, vc, q, k, v, t.positions, t.slots, m.inv_freq, q_norm=m.norm, k_norm=m.norm, eps=s.eps,
                                 k_scale=m.scale, v_scale=m.scale, err_out=self.err)
            o = torch.zeros_like(q)  # (rows of no request stay as they are)
            pm.moe_chunk_attention(kc, vc, q, t.q_start, t.lens, self.table, window=s.window if layer % 2 else 0, sinks=s.sinks,
                                   k_scale=m.scale, v_scale=m.scale, out=o, scratch=self.scratch, err_out=self.err)
            x = x + o.view(T, -1) @ m.out[layer].T
            h = F.rms_norm(x, (s.hidden,), eps=s.eps)
            ids, w = pm.moe_router_select((h @ m.router[layer].T), s.top_k, scoring="sigmoid", bias=self.balance[layer],
                                          groups=s.groups, top_groups=s.top_groups, group_top=2, scale=s.route_scale)
            x = m.experts.moe_paged_forward(layer, h, ids, w, residual=x)
            if self.routes is not None:
                self.routes.append((ids, w))
        return x

    def check(self, r):
        """Refuses what would index beyond the model's tensors or the server's buffers."""
        def refuse(what):
            raise AssertionError(f"request: {what}")

        if not r.prompt or r.tokens < 1 or r.output:
            refuse("a prompt, at least one token to generate and no output so far are needed")
        if len(r.prompt) + r.tokens > self.longest:
            refuse(f"{len(r.prompt)} + {r.tokens} tokens, {self.longest} at most")
        if len(r.biases) > self.max_biases:
            refuse(f"{len(r.biases)} biases, {self.max_biases} at most")
        if r.allowed is not None and len(r.allowed) == 0:
            refuse("no token is allowed")
        for name, ids in (("prompt", r.prompt), ("biases", r.biases), ("allowed", () if r.allowed is None else r.allowed)):
            for v in ids:
                if not 0 <= v < self.shape.vocab:
                    refuse(f"{name}: token {v} of {self.shape.vocab}")

    def plan(self, waiting):
        """Seats requests, and gives each seat its tokens of this step: (seat, token ids)."""
        for seat in range(self.seats):
            if self.seated[seat] is None and seat not in self.ended and waiting:
                self.check(waiting[0])
                self.seated[seat], self.read[seat] = waiting.pop(0), 0
        room, work = self.rows, {}
        # generating requests first, one token each; then pieces of prompts
        for started in (True, False):
            for seat, r in enumerate(self.seated):
                if r is None or bool(r.output) != started or room == 0:
                    continue
                ids = r.output[-1:] if started else r.prompt[self.read[seat]:self.read[seat] + room]
                work[seat] = ids
                room -= len(ids)
        return work

    def step(self, waiting, temperature=1.0, top_k=50, top_p=0.95, on_logits=None):
        """One step; False when there is nothing left to do. on_logits(seats, logits, adjusted) sees what the step draws from."""
        s = self.shape
        work = self.plan(waiting)
        if not work and not self.ended:
            return False
        new = np.zeros(self.seats, np.int32)
        tokens = np.zeros(self.rows, np.int64)
        new[self.ended] = -1
        at = 0
        for seat in sorted(work):
            ids = work[seat]
            new[seat] = len(ids)
            tokens[at:at + len(ids)] = ids
            at += len(ids)
        self.ended = []
        t = pm.moe_batch_tables(self.table, self.free, self.free_count, self.lens, torch.from_numpy(new).cuda(), self.rows, s.page,
                                self.pages, lens_out=self.lens, free_count_out=self.free_count, err_out=self.err)
        x = self.hidden(torch.from_numpy(tokens).cuda(), t)

        # the requests whose prompt is through draw their next token
        draws = []
        for seat in sorted(work):
            self.read[seat] += len(work[seat])
            r = self.seated[seat]
            if r.output or self.read[seat] == len(r.prompt):
                draws.append(seat)
        if draws:
            seats = torch.tensor(draws, device="cuda")
            rows = t.q_start[1:][seats].long() - 1
            logits = F.rms_norm(x[rows], (s.hidden,), eps=s.eps) @ self.model.head.T
            adjusted = pm.moe_adjust_logits(logits, err_out=self.err, **self.settings(draws))
            if on_logits is not None:
                on_logits(draws, logits, adjusted)
            full = lambda v, dt: torch.full((len(draws),), v, dtype=dt, device="cuda")  # noqa: E731
            u = torch.rand(len(draws), generator=self.generator, device="cuda")
            ids = pm.moe_sample_tokens(adjusted, u, temperature=full(temperature, torch.float32), top_k=full(top_k, torch.int32),
                                       top_p=full(top_p, torch.float32)).tolist()
            for seat, token in zip(draws, ids):
                r = self.seated[seat]
                if token < 0:
                    raise RuntimeError(f"seat {seat}: no token's logit is above -inf")
                r.output.append(token)
                if r.done():
                    self.seated[seat] = None
                    self.ended.append(seat)
        if int(self.err):
            raise RuntimeError(f"device error bits {int(self.err)}")
        return True

    def settings(self, draws):
        """The penalties, biases and masks of the requests in seats `draws`, for moe_adjust_logits."""
        rs = [self.seated[seat] for seat in draws]
        up = lambda a, dt: torch.tensor(a, dtype=dt, device="cuda")  # noqa: E731
        said = [r.prompt + r.output for r in rs]
        history = np.zeros((len(rs), max(len(x) for x in said)), np.int32)
        for row, x in zip(history, said):
            row[:len(x)] = x
        out = dict(history=torch.from_numpy(history).cuda(), prompt_len=up([len(r.prompt) for r in rs], torch.int32),
                   history_len=up([len(x) for x in said], torch.int32),
                   repetition=up([r.repetition for r in rs], torch.float32), frequency=up([r.frequency for r in rs], torch.float32),
                   presence=up([r.presence for r in rs], torch.float32))
        if any(r.biases for r in rs):
            ids, values = np.full((len(rs), self.max_biases), -1, np.int32), np.zeros((len(rs), self.max_biases), np.float32)
            for i, r in enumerate(rs):
                ids[i, :len(r.biases)], values[i, :len(r.biases)] = list(r.biases), list(r.biases.values())
            out.update(bias_ids=torch.from_numpy(ids).cuda(), bias=torch.from_numpy(values).cuda())
        if any(r.allowed is not None for r in rs):
            bits = np.full((len(rs), -(-self.shape.vocab // 32)), 0xffffffff, np.uint32)
            for row, r in zip(bits, rs):
                if r.allowed is not None:
                    row[:] = 0
                    np.bitwise_or.at(row, np.array(r.allowed) // 32, np.uint32(1) << (np.array(r.allowed) % 32).astype(np.uint32))
            out["mask"] = torch.from_numpy(bits.view(np.int32)).cuda()
        return out

    def run(self, requests, **how):
        """Serves the requests; their outputs are filled in. Returns the number of steps."""
        for r in requests:
            self.check(r)
        waiting, steps = list(requests), 0
        while self.step(waiting, **how):
            steps += 1
        return steps


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--requests", type=int, default=12)
    p.add_argument("--seats", type=int, default=8, help="requests at a time")
    p.add_argument("--rows", type=int, default=256, help="tokens of a step, at most")
    p.add_argument("--prompt", type=int, default=600, help="tokens of the longest prompt")
    p.add_argument("--tokens", type=int, default=40, help="tokens to generate for each request")
    p.add_argument("--layers", type=int, default=ServeShape.layers)
    p.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    p.add_argument("--repetition", type=float, default=1.1)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    shape = ServeShape(layers=a.layers)
    longest = a.prompt + a.tokens
    server = Server(shape, a.seats, a.rows, a.seats * -(-longest // shape.page), longest, e4m3=a.cache == "e4m3", seed=a.seed)
    rng = np.random.default_rng(a.seed)
    for _ in range(2):  # the first run pages the experts in
        requests = [Request(rng.integers(0, shape.vocab, rng.integers(1, a.prompt + 1)).tolist(), a.tokens, repetition=a.repetition)
                    for _ in range(a.requests)]
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        steps = server.run(requests)
        torch.cuda.synchronize()
        t1 = time.perf_counter()
    for r in requests:
        print(" ".join(str(t) for t in r.output))
    n = sum(len(r.prompt) + len(r.output) for r in requests)
    print("%d requests, %d tokens in %d steps: %.1f ms, %.0f tokens/s" % (len(requests), n, steps, 1e3 * (t1 - t0), n / (t1 - t0)))
    server.close()


if __name__ == "__main__":
    main()
