"""The serving example against a plain model: batch tables, append, attention of new tokens, expert
selection, paged experts, logit adjustment and draws together, over requests of different lengths.

The plain model computes every request by itself, from its first token, in 64 bits, with the routing
of the run, so that a near tie of two experts does not count as an error. The run rounds some 9
activations a layer to bf16, each within 2^-9 of its value, and their errors add up like independent
ones; the experts' weights are multiplied by the routing scale: sqrt(9 * 2 + 4) * 2^-9 * 2.5 = 0.023 of the
logits' norm, 3 times of which is allowed. e4m3 keys and values are within 2^-4, on average 2^-5.8
of theirs; with two layers, keys and values, and the scale: sqrt(4) * 2^-5.8 * 2.5 = 0.09 more, again with 3
times allowed.
"""

import numpy as np
import pytest

from oracle import steps

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

SIZES = dict(vocab=500, layers=2, hidden=256, q_heads=8, kv_heads=2, head_dim=64, experts=8, top_k=2, intermediate=128,
             slots=6, page=16, groups=4, top_groups=2, window=40, sinks=3)


def f64(t):
    return t.detach().double().cpu()


def rms(x, eps):
    return x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()


def plain_logits(server, tokens, routes):
    """Logits of every position of one request; routes: per layer, (ids, w) of its tokens."""
    m, s, n = server.model, server.shape, len(tokens)
    x = f64(m.embed)[tokens]
    ang = torch.arange(n, dtype=torch.float64)[:, None, None] * f64(m.inv_freq)
    cos, sin = ang.cos(), ang.sin()

    def rotate(t):
        a, b = rms(t, s.eps).chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)

    for layer in range(s.layers):
        qkv = (rms(x, s.eps) @ f64(m.qkv[layer]).T).view(n, -1, s.head_dim)
        q, k, v = qkv.split([s.q_heads, s.kv_heads, s.kv_heads], dim=1)
        q, k = rotate(q), rotate(k)
        k, v = (t.repeat_interleave(s.q_heads // s.kv_heads, dim=1) for t in (k, v))
        att = torch.einsum("qhd,khd->hqk", q, k) * s.head_dim ** -0.5
        p, j = torch.arange(n)[:, None], torch.arange(n)[None]
        hidden = j > p
        if layer % 2:
            hidden |= (j <= p - s.window) & (j >= s.sinks)
        att = att.masked_fill(hidden, -torch.inf).softmax(-1)
        x = x + torch.einsum("hqk,khd->qhd", att, v).reshape(n, -1) @ f64(m.out[layer]).T
        h = rms(x, s.eps)
        ids, w = routes[layer]
        store = torch.from_numpy(m.experts.host_store(layer)[:, :m.experts.expert_bytes].copy())
        store = store.view(torch.bfloat16).double().view(s.experts, 3, -1)
        gate, up = (store[:, i].view(s.experts, s.intermediate, s.hidden) for i in (0, 1))
        down = store[:, 2].view(s.experts, s.hidden, s.intermediate)
        y = torch.zeros_like(x)
        for r in range(s.top_k):
            e = ids[:, r].long()
            g = torch.einsum("th,tih->ti", h, gate[e])
            act = g * torch.sigmoid(g) * torch.einsum("th,tih->ti", h, up[e])
            y += w[:, r:r + 1].double() * torch.einsum("ti,thi->th", act, down[e])
        x = x + y
    return rms(x, s.eps) @ f64(m.head).T


def requests(rng, n, vocab, longest, tokens):
    from paged_expert_moe_gb300.serve import Request
    out = []
    for i in range(n):
        prompt = rng.integers(0, vocab, rng.integers(1, longest)).tolist()
        r = Request(prompt, int(rng.integers(1, tokens + 1)), repetition=float(rng.uniform(1, 1.3)), frequency=0.2, presence=0.1)
        if i % 3 == 1:
            r.biases = {int(v): float(b) for v, b in zip(rng.integers(0, vocab, 5), rng.normal(0, 3, 5))}
        if i % 3 == 2:
            r.allowed = sorted({int(v) for v in rng.integers(0, vocab, 60)})
        out.append(r)
    return out


@pytest.mark.parametrize("e4m3,seats,rows,bound", [(False, 3, 24, 0.07), (False, 1, 7, 0.07), (True, 4, 50, 0.34)])
def test_logits_of_requests(e4m3, seats, rows, bound):
    from paged_expert_moe_gb300 import serve as ex
    shape = ex.ServeShape(**SIZES)
    rng = np.random.default_rng(seats)
    todo = requests(rng, 7, shape.vocab, 80, 12)
    server = ex.Server(shape, seats, rows, seats * 6 + 1, 92, e4m3=e4m3, seed=3)
    server.routes, seen, adjusted, spans = [], {id(r): [] for r in todo}, {id(r): [] for r in todo}, {id(r): [] for r in todo}
    waiting = list(todo)
    while True:
        before = list(server.seated)

        def look(draws, logits, changed):
            for i, seat in enumerate(draws):
                r = server.seated[seat]
                n = len(r.prompt) + len(r.output)
                seen[id(r)].append(f64(logits[i]))
                words = None if r.allowed is None else np.zeros((1, -(-shape.vocab // 32)), np.uint32)
                for v in r.allowed or []:
                    words[0, v // 32] |= np.uint32(1 << (v % 32))
                want, size = steps.adjust_logits(
                    logits[i:i + 1].float().cpu().numpy(), np.array([r.prompt + r.output]), [len(r.prompt)], [n],
                    [np.float32(r.repetition)], [np.float32(r.frequency)], [np.float32(r.presence)],
                    np.array([list(r.biases)], int) if r.biases else None,
                    np.array([list(r.biases.values())], np.float32) if r.biases else None,
                    None if words is None else words.view(np.int32))
                got = changed[i].double().cpu().numpy()
                assert np.array_equal(np.isneginf(got), np.isneginf(want[0]))
                fine = ~np.isneginf(got)
                assert np.all(np.abs(got - want[0])[fine] <= 4 * 2.0 ** -24 * size[0][fine])

        plan = server.plan(waiting)  # (seats what fits; the step finds the same)
        first = len(server.routes)
        at = 0
        for seat in sorted(plan):
            spans[id(server.seated[seat])].append((first, at, at + len(plan[seat])))
            at += len(plan[seat])
        del before
        if not server.step(waiting, on_logits=look):
            break
    for r in todo:
        assert r.done() and (r.allowed is None or set(r.output) <= set(r.allowed))
        row = torch.tensor(r.prompt + r.output[:-1])
        routes = []
        for layer in range(shape.layers):
            parts = [tuple(t[a:b].cpu() for t in server.routes[f + layer]) for f, a, b in spans[id(r)]]
            routes.append(tuple(torch.cat(t) for t in zip(*parts)))
        assert routes[0][0].shape[0] == len(row)
        want = plain_logits(server, row, routes)[len(r.prompt) - 1:]
        got = torch.stack(seen[id(r)])
        err = ((got - want).norm() / want.norm()).item()
        assert err <= bound, err
    # every page came back
    assert int(server.free_count) == server.pages and sorted(server.free[:server.pages].tolist()) == list(range(server.pages))
    server.close()


def test_greedy_requests_do_not_depend_on_their_neighbours():
    """The same requests through one seat and through many: the same tokens, but for near ties."""
    from paged_expert_moe_gb300 import serve as ex
    shape = ex.ServeShape(**SIZES)
    outs = []
    for seats, rows in ((1, 16), (5, 64)):
        server = ex.Server(shape, seats, rows, seats * 6, 92, seed=1)
        todo = requests(np.random.default_rng(5), 5, shape.vocab, 60, 8)
        server.run(todo, temperature=0.0)
        outs.append([r.output[0] for r in todo])
        assert all(r.done() for r in todo)
        server.close()
    assert sum(a == b for a, b in zip(*outs)) >= 4


def test_command_line(capsys):
    from paged_expert_moe_gb300 import serve as ex
    ex.main(["--requests", "3", "--seats", "2", "--rows", "32", "--prompt", "50", "--tokens", "4", "--layers", "2"])
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 4 and len(lines[0].split()) == 4 and "tokens/s" in lines[3]
