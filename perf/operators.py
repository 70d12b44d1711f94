"""The attention and sampling operators around the paged-expert layer, as measurable cases.

A serving step needs three things next to the MoE layer: the token's keys and values have
to reach the paged cache (``moe_kv_append``: head norm, rotation, append), its queries have
to attend to the cache (``moe_prefix_attention``: one prefix that the whole batch shares,
then each sequence's own pages), and the logits have to become a token
(``moe_sample_tokens``). Each case below is one call of one of them.

``run`` computes a case either through the package (``own``) or in its plain form, in
elementary torch operations in 32 bits; ``exact`` gives the same outputs from the
definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # One token of one request: what a step costs when nothing but latency counts.
        dict(name="append_1", op="append", T=1, Hq=32, Hkv=4, D=128, page=16, kv="bf16", rot=128, axes=1,
             interleaved=False, norm=True, skip=0.0, max_pos=40000),
        # A decode batch into an 8-bit cache.
        dict(name="append_256_e4m3", op="append", T=256, Hq=32, Hkv=4, D=128, page=64, kv="e4m3", rot=128, axes=1,
             interleaved=False, norm=True, skip=0.0, max_pos=130000),
        # Image tokens: time, height and width positions, interleaved pairs, a head that is
        # rotated in part, heads of 64 without grouping, padding tokens that are not appended.
        dict(name="append_4099_image", op="append", T=4099, Hq=16, Hkv=16, D=64, page=32, kv="bf16", rot=48, axes=3,
             interleaved=True, norm=False, skip=0.03, max_pos=2000),
        # A prompt chunk.
        dict(name="append_8192", op="append", T=8192, Hq=32, Hkv=4, D=128, page=16, kv="bf16", rot=128, axes=1,
             interleaved=False, norm=True, skip=0.0, max_pos=9000),
        # Few requests on a short system prompt: latency.
        dict(name="attend_4_short", op="attend", T=4, Hq=32, Hkv=4, D=128, page=16, kv="bf16", prefix=500, suffix=64,
             lse=False),
        # Two requests on a long document: the cache read has to be split over its length.
        dict(name="attend_2_long", op="attend", T=2, Hq=32, Hkv=4, D=128, page=16, kv="bf16", prefix=100003,
             suffix=256, lse=False),
        # An ordinary batch on one prompt of 8k tokens.
        dict(name="attend_64_8k", op="attend", T=64, Hq=32, Hkv=4, D=128, page=16, kv="bf16", prefix=8192, suffix=512,
             lse=True),
        # An 8-bit cache, five query heads to a key head, heads of 64, nothing a round number.
        dict(name="attend_47_e4m3", op="attend", T=47, Hq=40, Hkv=8, D=64, page=32, kv="e4m3", prefix=12345,
             suffix=777, lse=True),
        # A large batch on a long prompt: the prefix part is bound by the tensor cores.
        dict(name="attend_256_32k", op="attend", T=256, Hq=32, Hkv=4, D=128, page=64, kv="bf16", prefix=32768,
             suffix=1024, lse=False),
        # One row of logits: latency.
        dict(name="sample_1", op="sample", T=1, V=32000, dtype="f32"),
        # A decode batch, logits as the projection leaves them in bf16.
        dict(name="sample_64_bf16", op="sample", T=64, V=131072, dtype="bf16"),
        # A large batch, rows of odd length.
        dict(name="sample_256", op="sample", T=256, V=160001, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "sample"])
    if op == "sample":
        return dict(op="sample", T=_log_int(rng, 1, 256), V=_log_int(rng, 1000, 160001), dtype=rng.choice(["f32", "bf16"]))
    heads = rng.choice([(32, 4), (32, 8), (16, 16), (40, 8), (28, 4), (12, 2), (16, 1), (6, 3)])
    c = dict(op=op, Hq=heads[0], Hkv=heads[1], D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             kv=rng.choice(["bf16", "e4m3"]))
    if op == "append":
        axes = rng.choice([1, 1, 3])
        rot = c["D"] if rng.random() < 0.6 else rng.choice([16, 32, 48])
        c.update(T=_log_int(rng, 1, 8192), rot=rot, axes=axes, interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
                 skip=rng.choice([0.0, 0.0, 0.05]), max_pos=_log_int(rng, 100, 130000))
        return c
    while True:
        c.update(T=_log_int(rng, 1, 256), prefix=_log_int(rng, 16, 100000), suffix=_log_int(rng, 1, 1024),
                 lse=rng.random() < 0.5)
        if c["T"] * c["Hq"] * (c["prefix"] + c["suffix"]) <= 256 * 32 * 32768:
            return c


def _suffix_mean(c):
    return (1 + c["suffix"]) / 2


def work(case):
    c = case
    if c["op"] == "sample":
        n = c["T"] * c["V"]
        # one pass over the logits; a difference, a product, an exponential and a sum each
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + c["T"] * 28, "flops": 4 * n}
    eb = 2 if c["kv"] == "bf16" else 1
    if c["op"] == "append":
        T, D = c["T"], c["D"]
        read = T * (c["Hq"] + 2 * c["Hkv"]) * D * 2 + T * 4 * (c["axes"] + 1)
        write = T * c["Hq"] * D * 2 + int(T * (1 - c["skip"])) * 2 * c["Hkv"] * D * eb
        return {"bytes": read + write, "flops": T * (c["Hq"] + c["Hkv"]) * (3 * c["rot"] + (4 * D if c["norm"] else 0))}
    keys = c["prefix"] + c["T"] * _suffix_mean(c)
    return {"bytes": keys * c["Hkv"] * c["D"] * 2 * eb + 2 * c["T"] * c["Hq"] * c["D"] * 2,
            "flops": 4 * c["T"] * c["Hq"] * c["D"] * (c["prefix"] + _suffix_mean(c))}


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _cache(g, pages, c):
    shape = (pages, c["Hkv"], c["page"], c["D"])
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if c["kv"] == "bf16":
        return k, v, None, None
    # codes that use the format's range; the scales take them back to the values' size
    ks = torch.rand(c["Hkv"], generator=g, device=DEV) * 0.02 + 0.01
    vs = torch.rand(c["Hkv"], generator=g, device=DEV) * 0.02 + 0.01
    return (k * 64).to(torch.float8_e4m3fn), (v * 64).to(torch.float8_e4m3fn), ks, vs


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "sample":
        T, V = c["T"], c["V"]
        # a broad bulk and a few likely tokens, as a language model's head gives them
        x = torch.randn((T, V), generator=g, device=DEV) * 2.5
        hot = torch.randint(0, V, (T, 40), generator=g, device=DEV)
        x.scatter_add_(1, hot, torch.rand((T, 40), generator=g, device=DEV) * 12)
        pick = torch.randint(0, 4, (4, T), generator=g, device=DEV)
        of = lambda i, values, dt: torch.tensor(values, dtype=dt, device=DEV)[pick[i]].contiguous()  # noqa: E731
        return dict(c=c, logits=x.to(torch.bfloat16) if c["dtype"] == "bf16" else x,
                    u=torch.rand(T, generator=g, device=DEV),
                    temperature=of(0, [0.0, 0.6, 0.8, 1.0], torch.float32), top_k=of(1, [0, 20, 50, 1000], torch.int32),
                    top_p=of(2, [1.0, 0.95, 0.9, 0.8], torch.float32), min_p=of(3, [0.0, 0.0, 0.02, 0.1], torch.float32),
                    ids=torch.empty(T, dtype=torch.int32, device=DEV), logprob=torch.empty(T, device=DEV))
    T, Hq, Hkv, D, page = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    if c["op"] == "append":
        pages = -(-(T + T // 4) // page) + 1
        kc, vc, ks, vs = _cache(g, pages, c)
        # the projection's output, from which q, k and v are views
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV, dtype=torch.bfloat16) * 1.5
        q, k, v = (t.view(T, -1, D) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].to(torch.int32)
        if c["skip"]:
            slots[torch.rand(T, generator=g, device=DEV) < c["skip"]] = -1
        pairs = c["rot"] // 2
        at = torch.arange(pairs, device=DEV)
        norm = (lambda: (torch.rand(D, generator=g, device=DEV) + 0.5).to(torch.bfloat16)) if c["norm"] else (lambda: None)
        return dict(c=c, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, q=q, k=k, v=v, slots=slots,
                    positions=torch.randint(0, c["max_pos"], (c["axes"], T), generator=g, device=DEV, dtype=torch.int32),
                    pair_axis=(at * c["axes"] // pairs).to(torch.int32) if c["axes"] > 1 else None,
                    inv_freq=torch.pow(torch.tensor(1e6, dtype=torch.float64, device=DEV), -at.double() / pairs).float(),
                    q_norm=norm(), k_norm=norm(), q_out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV))
    per = -(-c["suffix"] // page)
    n_prefix = -(-c["prefix"] // page)
    pages = n_prefix + T * per + 3
    kc, vc, ks, vs = _cache(g, pages, c)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    lens = torch.randint(1, c["suffix"] + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
    return dict(c=c, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                q=torch.randn((T, Hq, D), generator=g, device=DEV, dtype=torch.bfloat16) * 2,
                prefix_pages=order[:n_prefix].contiguous(),
                page_table=order[n_prefix:n_prefix + T * per].reshape(T, per).contiguous(), suffix_len=lens,
                out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV),
                lse=torch.empty((T, Hq), device=DEV) if c["lse"] else None)


# ---------------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if own:
        import paged_expert_moe_gb300 as pm
        if op == "append":
            pm.moe_kv_append(s["k_cache"], s["v_cache"], s["q"], s["k"], s["v"], s["positions"], s["slots"],
                             s["inv_freq"], pair_axis=s["pair_axis"], interleaved=c["interleaved"], q_norm=s["q_norm"],
                             k_norm=s["k_norm"], eps=1e-6, k_scale=s["k_scale"], v_scale=s["v_scale"],
                             q_out=s["q_out"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if op == "attend":
            pm.moe_prefix_attention(s["k_cache"], s["v_cache"], s["q"], s["prefix_pages"], c["prefix"],
                                    s["page_table"], s["suffix_len"], c["suffix"], k_scale=s["k_scale"],
                                    v_scale=s["v_scale"], out=s["out"], lse_out=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        pm.moe_sample_tokens(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                             min_p=s["min_p"], ids_out=s["ids"], logprob_out=s["logprob"])
        return {"ids": s["ids"], "logprob": s["logprob"]}
    return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[op](s, c)


def _plain_turn(x, w, cos, sin, interleaved, rot):
    """Head norm (w given) and rotation of x [T, heads, D], in 32 bits."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_store(cache, rows, keep, slots, scale):
    if scale is not None:
        rows = (rows / scale[:, None]).clamp(-448, 448)
    rows = rows.to(cache.dtype)
    page = cache.shape[2]
    at = slots[keep].long()
    bits = torch.uint8 if cache.dtype == torch.float8_e4m3fn else torch.int16
    cache.view(bits)[at // page, :, at % page] = rows.view(bits)[keep]


def _plain_append(s, c):
    axis = s["pair_axis"].long() if s["pair_axis"] is not None else torch.zeros(c["rot"] // 2, dtype=torch.long, device=DEV)
    angle = s["positions"].float()[axis].T * s["inv_freq"]
    cos, sin = angle.cos(), angle.sin()
    q = _plain_turn(s["q"], s["q_norm"], cos, sin, c["interleaved"], c["rot"])
    k = _plain_turn(s["k"], s["k_norm"], cos, sin, c["interleaved"], c["rot"])
    s["q_out"].copy_(q)
    keep = s["slots"] >= 0
    _plain_store(s["k_cache"], k, keep, s["slots"], s["k_scale"])
    _plain_store(s["v_cache"], s["v"].float(), keep, s["slots"], s["v_scale"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_rows(cache, pages, scale):
    """The rows of `pages` [..., n] as [..., Hkv, n * page, D] in 32 bits."""
    x = cache.view(torch.uint8 if scale is not None else torch.int16)[pages.long()].view(cache.dtype).float()
    if scale is not None:
        x = x * scale[:, None, None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _plain_attend(s, c):
    T, Hq, Hkv, D, L = c["T"], c["Hq"], c["Hkv"], c["D"], c["prefix"]
    G = Hq // Hkv
    q = s["q"].float().view(T, Hkv, G, D) * D ** -0.5
    kp = _plain_rows(s["k_cache"], s["prefix_pages"], s["k_scale"])[:, :L]
    vp = _plain_rows(s["v_cache"], s["prefix_pages"], s["v_scale"])[:, :L]
    ks = _plain_rows(s["k_cache"], s["page_table"], s["k_scale"])
    vs = _plain_rows(s["v_cache"], s["page_table"], s["v_scale"])
    seen = torch.arange(ks.shape[2], device=DEV) < s["suffix_len"][:, None]
    a = torch.matmul(q.permute(1, 0, 2, 3).reshape(Hkv, T * G, D), kp.transpose(1, 2))
    a = a.view(Hkv, T, G, L).transpose(0, 1)
    b = torch.matmul(q, ks.transpose(2, 3)).masked_fill(~seen[:, None, None], -math.inf)
    m = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
    a, b = torch.exp(a - m), torch.exp(b - m)
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    o = torch.matmul(a.transpose(0, 1).reshape(Hkv, T * G, L), vp).view(Hkv, T, G, D).transpose(0, 1)
    o = o + torch.matmul(b, torch.where(seen[:, None, :, None], vs, 0.0))
    lse = (m + total.log()).reshape(T, Hq) if c["lse"] else None
    return {"out": (o / total).reshape(T, Hq, D).to(torch.bfloat16), "lse": lse}


# A row's tokens weigh w = exp((logit - largest) / temperature) in 32 bits, held as whole
# multiples of 2^-31; all sums and shares of sums are whole numbers, so that no order of
# summation changes a draw. The shares are in steps of 2^-24.
def _share(total, part):
    """floor(total * part), part = n * 2^-24, without leaving 63 bits."""
    n = (part.double() * 2 ** 24).long()
    return (total >> 24) * n + (((total & (2 ** 24 - 1)) * n) >> 24)


def _plain_sample(s, c):
    V = c["V"]
    x = s["logits"].float()
    greedy = s["temperature"] <= 0
    order = torch.sort(x, dim=1, descending=True, stable=True)
    z = (order.values - order.values[:, :1]) * (1 / torch.where(greedy, 1.0, s["temperature"]))[:, None]
    w = torch.exp(z)
    n = (w * 2.0 ** 31).long()
    rank = torch.arange(V, device=DEV)
    k = torch.where((s["top_k"] <= 0) | (s["top_k"] > V), V, s["top_k"])
    k = torch.where(greedy, 1, k)
    n = torch.where(rank < k[:, None], n, 0)
    upto = n.cumsum(1)
    total = upto[:, -1]
    least = torch.where(s["top_p"] >= 1, total, _share(total, s["top_p"]))
    kept = (upto - n < least[:, None]) | (rank == 0)
    n = torch.where(kept & (w >= s["min_p"][:, None]) & (n > 0), n, 0)
    by_id = torch.zeros_like(n).scatter_(1, order.indices, n)
    upto = by_id.cumsum(1)
    total = upto[:, -1]
    ids = (upto <= _share(total, s["u"])[:, None]).sum(1)
    p = by_id.gather(1, ids[:, None])[:, 0]
    return {"ids": ids.to(torch.int32), "logprob": torch.log(p.float() / total.float())}


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s, case)


def _exact_append(s, c):
    pairs = c["rot"] // 2
    first = [2 * i if c["interleaved"] else i for i in range(pairs)]
    second = [2 * i + 1 if c["interleaved"] else i + pairs for i in range(pairs)]
    axis = [int(a) for a in s["pair_axis"]] if s["pair_axis"] is not None else [0] * pairs
    angle = torch.stack([s["positions"][axis[i]].double() * float(s["inv_freq"][i]) for i in range(pairs)], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
        y = torch.complex(x[..., first], x[..., second]) * turn
        x = x.clone()
        x[..., first], x[..., second] = y.real, y.imag
        return x

    q, k, v = turned(s["q"], s["q_norm"]), turned(s["k"], s["k_norm"]), s["v"].double()
    caches = []
    for cache, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], v, s["v_scale"])):
        flat = cache.double().transpose(1, 2).reshape(-1, c["Hkv"], c["D"]).clone()
        if scale is not None:
            x = (x / scale.double()[:, None]).clamp(-448, 448)
        there = s["slots"] >= 0
        flat[s["slots"][there].long()] = x[there]
        caches.append(flat.view(-1, c["page"], c["Hkv"], c["D"]).transpose(1, 2).contiguous())
    return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attend(s, c):
    T, G, L, page = c["T"], c["Hq"] // c["Hkv"], c["prefix"], c["page"]
    if 4 * T * c["Hq"] * c["D"] * (L + c["suffix"]) > 4e11:
        return None
    out = torch.zeros((T, c["Hq"], c["D"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((T, c["Hq"]), dtype=torch.float64, device=DEV)
    lens = s["suffix_len"].tolist()
    wide = torch.uint8 if c["kv"] == "e4m3" else torch.int16

    def rows(cache, scale, pages, n, h):
        x = cache.view(wide)[pages.long(), h].view(cache.dtype).double().reshape(-1, c["D"])[:n]
        return x if scale is None else x * scale[h].double()

    for h in range(c["Hkv"]):
        kp, vp = (rows(x, y, s["prefix_pages"], L, h) for x, y in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
        for t in range(T):
            mine = s["page_table"][t, :-(-lens[t] // page)]
            kk = torch.cat([kp, rows(s["k_cache"], s["k_scale"], mine, lens[t], h)])
            vv = torch.cat([vp, rows(s["v_cache"], s["v_scale"], mine, lens[t], h)])
            a = s["q"][t, h * G:(h + 1) * G].double() @ kk.T / math.sqrt(c["D"])
            lse[t, h * G:(h + 1) * G] = torch.logsumexp(a, -1)
            out[t, h * G:(h + 1) * G] = torch.softmax(a, -1) @ vv
    return {"out": out, "lse": lse if c["lse"] else None}


def _exact_sample(s, c):
    # row by row in 64 bits; the ids are whole numbers and are left to the plain form
    got = torch.zeros(c["T"], dtype=torch.float64, device=DEV)
    one = {k: s[k].tolist() for k in ("u", "temperature", "top_k", "top_p", "min_p")}
    for t in range(c["T"]):
        x = s["logits"][t].double()
        if one["temperature"][t] <= 0:
            continue
        w = torch.exp((x - x.max()) / one["temperature"][t])
        order = torch.argsort(x, descending=True, stable=True)
        if one["top_k"][t] > 0:
            order = order[:one["top_k"][t]]
        n = torch.floor(w[order] * 2 ** 31)
        if one["top_p"][t] < 1:
            order = order[:int((torch.cumsum(n, 0) < one["top_p"][t] * n.sum()).sum()) + 1]
        order = order[w[order] >= one["min_p"][t]].sort().values
        n = torch.floor(w[order] * 2 ** 31)
        n = n[n > 0]
        i = min(int((torch.cumsum(n, 0) <= one["u"][t] * n.sum()).sum()), len(n) - 1)
        got[t] = torch.log(n[i] / n.sum())
    return {"ids": None, "logprob": got}
