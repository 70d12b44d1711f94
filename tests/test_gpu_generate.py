"""The sampling example against a plain model: the prompt's cache, the shared prefix, the paged
experts and the draws together.

The plain model computes every continuation by itself, from its first token, in 64 bits, and
takes the routing of the run, so that a near tie of two experts does not count as an error.
The run rounds some 8 activations a layer to bf16, each within 2^-9 of its value, and their
errors add up like independent ones: sqrt(8 * 2 + 4) * 2^-9 = 0.009 of the logits' norm, 3 times
of which is allowed. e4m3 keys and values are within 2^-4, on average 2^-5.8 of theirs; with
two layers, keys and values: sqrt(4) * 2^-5.8 = 0.036 more, again with 3 times allowed.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

SIZES = dict(vocab=500, layers=2, hidden=256, q_heads=8, kv_heads=2, head_dim=64, experts=8, top_k=2, intermediate=128,
             slots=6, page=16)


def f64(t):
    return t.detach().double().cpu()


def rms(x, eps):
    return x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()


def plain_logits(model, tokens, routes):
    """Logits of every position of one sequence; routes: per layer, (ids, w) of its tokens."""
    s, n = model.shape, len(tokens)
    x = f64(model.embed)[tokens]
    ang = torch.arange(n, dtype=torch.float64)[:, None, None] * f64(model.inv_freq)
    cos, sin = ang.cos(), ang.sin()

    def rotate(t):
        a, b = rms(t, s.eps).chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)

    for layer in range(s.layers):
        qkv = (rms(x, s.eps) @ f64(model.qkv[layer]).T).view(n, -1, s.head_dim)
        q, k, v = qkv.split([s.q_heads, s.kv_heads, s.kv_heads], dim=1)
        q, k = rotate(q), rotate(k)
        k, v = (t.repeat_interleave(s.q_heads // s.kv_heads, dim=1) for t in (k, v))
        att = torch.einsum("qhd,khd->hqk", q, k) * s.head_dim ** -0.5
        att = att.masked_fill(torch.ones(n, n).triu(1).bool(), -torch.inf).softmax(-1)
        x = x + torch.einsum("hqk,khd->qhd", att, v).reshape(n, -1) @ f64(model.out[layer]).T
        h = rms(x, s.eps)
        ids, w = routes[layer]
        store = torch.from_numpy(model.experts.host_store(layer)[:, :model.experts.expert_bytes].copy())
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
    return rms(x, s.eps) @ f64(model.head).T


@pytest.mark.parametrize("e4m3,prompt_len,samples,tokens,bound", [(False, 37, 5, 20, 0.027), (False, 1, 1, 3, 0.027),
                                                                  (False, 64, 3, 2, 0.027), (True, 50, 4, 17, 0.135)])
def test_logits_of_continuations(e4m3, prompt_len, samples, tokens, bound):
    from paged_expert_moe_gb300 import generate as ex
    shape = ex.Shape(**SIZES)
    head, own = ex.pages_needed(shape, prompt_len, samples, tokens)
    model = ex.Decoder(shape, head + samples * own, max(prompt_len, samples), e4m3=e4m3, seed=3)
    prompt = torch.from_numpy(np.random.default_rng(4).integers(0, shape.vocab, prompt_len)).cuda()
    model.routes, seen = [], []
    ids = ex.generate(model, prompt, samples, tokens, temperature=1.0, seed=5, on_logits=lambda x: seen.append(f64(x)))
    assert ids.shape == (samples, tokens) and int(ids.min()) >= 0 and int(ids.max()) < shape.vocab
    routes = [(i.cpu(), w.cpu()) for i, w in model.routes]
    for b in range(samples):
        row = torch.cat([prompt.cpu(), ids[b, :-1].long().cpu()])
        own_routes = []
        for layer in range(shape.layers):
            steps = [routes[layer]] + [(i[b:b + 1], w[b:b + 1]) for i, w in routes[shape.layers + layer::shape.layers]]
            own_routes.append(tuple(torch.cat(t) for t in zip(*steps)))
        want = plain_logits(model, row, own_routes)[prompt_len - 1:]
        got = torch.stack([x[b] for x in seen])
        err = ((got - want).norm() / want.norm()).item()
        assert err <= bound, (b, err)
    model.close()


def test_same_seed_same_tokens_and_greedy():
    from paged_expert_moe_gb300 import generate as ex
    shape = ex.Shape(**SIZES)
    model = ex.Decoder(shape, 3 + 4 * 2, 40, seed=1)
    prompt = torch.arange(40, device="cuda")
    a = ex.generate(model, prompt, 4, 20, seed=7)
    assert torch.equal(a, ex.generate(model, prompt, 4, 20, seed=7))
    assert len({tuple(r) for r in a.tolist()}) > 1
    seen = []
    b = ex.generate(model, prompt, 4, 20, temperature=0.0, on_logits=lambda x: seen.append(x.argmax(-1)))
    assert torch.equal(b, torch.stack(seen, dim=1).int())
    assert all(r == b[0].tolist() for r in b.tolist())
    model.close()


def test_command_line(capsys):
    from paged_expert_moe_gb300 import generate as ex
    ex.main(["--prompt", "20", "--samples", "2", "--tokens", "5", "--layers", "1", "--slots", "8"])
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 3 and len(lines[0].split()) == 5 and "tokens/s" in lines[2]
