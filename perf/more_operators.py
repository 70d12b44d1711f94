"""The operators of a step over requests of different lengths, as measurable cases.

A server's step mixes requests that generate one token each with pieces of prompts. Around
the paged experts it needs the requests' pages, slots and positions (``moe_batch_tables``),
attention of each request's new tokens over its own pages (``moe_chunk_attention``, with a
sliding window and first tokens that stay visible where the model has them), the choice of
the experts by scores with a balance bias and expert groups (``moe_router_select``), and,
before the draw, the penalties, biases and grammar masks of each request
(``moe_adjust_logits``). Each case below is one call of one of them.

``run`` computes a case either through the package (``own``) or in its plain form, in
elementary torch operations; ``exact`` gives the computed numbers from the definitions in
64 bits.
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # A decode batch: one token a request, some requests resting, some that ended.
        dict(name="tables_256", op="tables", R=256, T=256, chunk=1, page=16, cached=4000, rest=0.05, done=0.05, pad=0),
        # A thousand requests, a tenth of them with prompts to read, in a batch padded to a fixed size.
        dict(name="tables_1000", op="tables", R=1000, T=32768, chunk=500, page=64, cached=20000, rest=0.02, done=0.03,
             pad=777),
        # Four single tokens on short contexts: latency.
        dict(name="attend_decode_4", op="attend", decode=4, chunks=0, chunk=1, ctx=2000, full=False, Hq=32, Hkv=4, D=128,
             page=16, kv="bf16", window=0, sinks=0, lse=False),
        # A large decode batch of a model with a window and sinks: bound by reading the cache.
        dict(name="attend_decode_256_window", op="attend", decode=256, chunks=0, chunk=1, ctx=20000, full=False, Hq=32,
             Hkv=4, D=128, page=64, kv="bf16", window=4096, sinks=4, lse=False),
        # Decoding requests and pieces of three prompts in one step; an 8-bit cache, five query heads
        # to a key head, heads of 64, nothing a round number.
        dict(name="attend_mixed_e4m3", op="attend", decode=61, chunks=3, chunk=1500, ctx=9000, full=False, Hq=40, Hkv=8,
             D=64, page=32, kv="e4m3", window=2500, sinks=7, lse=True),
        # A whole prompt of 8k tokens.
        dict(name="attend_prompt_8192", op="attend", decode=0, chunks=1, chunk=8192, ctx=0, full=True, Hq=32, Hkv=4, D=128,
             page=16, kv="bf16", window=0, sinks=0, lse=False),
        # A piece of 4,096 tokens of a long document.
        dict(name="attend_chunk_60k", op="attend", decode=0, chunks=1, chunk=4096, ctx=60001, full=True, Hq=32, Hkv=4,
             D=128, page=64, kv="bf16", window=0, sinks=0, lse=False),
        # A few tokens: latency.
        dict(name="route_4", op="route", T=4, E=256, k=8, scoring="sigmoid", bias=True, groups=8, top_groups=4, group_top=2,
             renorm=True, dtype="f32"),
        # A prompt's tokens.
        dict(name="route_16384", op="route", T=16384, E=256, k=8, scoring="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, renorm=True, dtype="f32"),
        # One row with a grammar: latency.
        dict(name="adjust_1", op="adjust", T=1, V=32000, dtype="bf16", history=1000, biases=0, mask=True),
        # A batch with biases, logits as the projection leaves them in bf16.
        dict(name="adjust_64_bf16", op="adjust", T=64, V=131072, dtype="bf16", history=4000, biases=100, mask=True),
        # A large batch, rows of odd length, no grammar.
        dict(name="adjust_256", op="adjust", T=256, V=160001, dtype="f32", history=2000, biases=30, mask=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "attend", "attend", "route", "adjust"])
    if op == "tables":
        R = _log_int(rng, 1, 1000)
        chunk = _log_int(rng, 1, 500)
        return dict(op=op, R=R, T=min(32768, max(R, R * chunk // rng.choice([1, 2, 8]))), chunk=chunk,
                    page=rng.choice([16, 32, 64, 128, 256]), cached=_log_int(rng, 20, 20000), rest=rng.choice([0.0, 0.1]),
                    done=rng.choice([0.0, 0.05]), pad=rng.choice([0, 0, 13, 300]))
    if op == "route":
        E, groups = rng.choice([(256, 8), (160, 8), (128, 1), (64, 1), (384, 1), (60, 4), (512, 16), (128, 4)])
        top_groups = 1 if groups == 1 else rng.choice([groups // 2, max(1, groups // 4)])
        k = min(rng.choice([1, 4, 6, 8, 10]), E // groups * top_groups)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k, scoring=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.6, groups=groups, top_groups=top_groups, group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.7, dtype=rng.choice(["f32", "bf16"]))
    if op == "adjust":
        return dict(op=op, T=_log_int(rng, 1, 256), V=_log_int(rng, 1000, 160001), dtype=rng.choice(["f32", "bf16"]),
                    history=_log_int(rng, 1, 4000), biases=rng.choice([0, 5, 100, 300]), mask=rng.random() < 0.5)
    heads = rng.choice([(32, 4), (32, 8), (16, 16), (40, 8), (28, 4), (12, 2), (16, 1), (6, 3)])
    c = dict(op=op, Hq=heads[0], Hkv=heads[1], D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]),
             kv=rng.choice(["bf16", "e4m3"]), full=False, lse=rng.random() < 0.5)
    while True:
        c.update(decode=rng.choice([0, _log_int(rng, 1, 256)]), chunks=rng.choice([0, 1, _log_int(rng, 1, 8)]),
                 chunk=_log_int(rng, 2, 8192), ctx=_log_int(rng, 1, 60001))
        c.update(rng.choice([dict(window=0, sinks=0), dict(window=_log_int(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 100]))]))
        w = work(c) if c["decode"] + c["chunks"] else None
        keys = (c["decode"] + c["chunks"]) * c["ctx"] + c["chunks"] * c["chunk"]
        if w and w["flops"] <= 4.2e12 and keys * c["Hkv"] * c["D"] <= 1.4e9:
            return c


def _mean_keys(c, cached, n):
    """(keys read, keys seen summed over the rows) of a request with n new tokens after `cached`."""
    if not c["window"]:
        return cached + n, n * cached + n * (n + 1) / 2
    full = c["window"] + c["sinks"]
    rise = max(0, min(n, full - cached))  # rows that see everything
    return min(cached + n, full + n - 1), rise * cached + rise * (rise + 1) / 2 + (n - rise) * full


def work(case):
    c = case
    if c["op"] == "tables":
        # lengths in and out, new pages, and five numbers a token
        tokens = c["T"] - c["pad"]
        return {"bytes": 4 * (5 * c["R"] + 5 * c["T"] + 2 * tokens / c["page"]), "flops": 10 * c["R"] + 5 * c["T"]}
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + c["T"] * c["k"] * 8 + c["E"] * 4,
                "flops": n * (6 + c["k"])}
    if c["op"] == "adjust":
        n = c["T"] * c["V"]
        return {"bytes": n * (4 + (4 if c["dtype"] == "f32" else 2) + (0.125 if c["mask"] else 0)) +
                c["T"] * (4 * c["history"] + 8 * c["biases"]), "flops": 2 * n}
    read = seen = rows = 0.0
    steps = 1 if c["full"] else 8  # lengths are uniform below their bounds
    for i in range(steps):
        cached = c["ctx"] if c["full"] else int(c["ctx"] * (i + 0.5) / steps)
        for count, n in ((c["decode"], 1), (c["chunks"], c["chunk"] if c["full"] else (1 + c["chunk"]) / 2)):
            a, b = _mean_keys(c, cached, n)
            read, seen, rows = read + count * a / steps, seen + count * b / steps, rows + count * n / steps
    eb = 2 if c["kv"] == "bf16" else 1
    return {"bytes": read * c["Hkv"] * c["D"] * 2 * eb + rows * c["Hq"] * c["D"] * 4,
            "flops": 4 * seen * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _up(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    return {"tables": _make_tables, "attend": _make_attend, "route": _make_route, "adjust": _make_adjust}[case["op"]](
        case, _gen(seed), torch.Generator().manual_seed(seed))


def _make_tables(c, g, h):
    R, page = c["R"], c["page"]
    u = torch.rand(R, generator=h)
    new = torch.ones(R, dtype=torch.int64)
    long = torch.rand(R, generator=h) < 0.1
    if c["chunk"] > 1:
        new[long] = torch.randint(1, c["chunk"] + 1, (int(long.sum()),), generator=h)
    new[u < c["rest"]] = 0
    new[(u >= c["rest"]) & (u < c["rest"] + c["done"])] = -1
    room = c["T"] - c["pad"]
    total = new.clamp(min=0).cumsum(0)
    new[(total > room) & (new > 0)] = 0  # what the step has no room for waits
    if c["chunk"] > 1 and int(total[-1]) < room:
        new[0] = max(int(new[0]), 0) + room - int(total[-1])  # one prompt fills the batch
    cached = torch.randint(0, c["cached"] + 1, (R,), generator=h)
    have = (cached + page - 1) // page
    most = -(-c["cached"] // page)  # pages of a request so far
    width = most + -(-c["T"] // page) + 1
    pages = R * (most + 1) + -(-c["T"] // page) + 50
    order = torch.randperm(pages, generator=h).to(torch.int32)
    used = int(have.sum())
    table = torch.full((R, width), -1, dtype=torch.int32)
    table[torch.arange(width) < have[:, None]] = order[:used]
    free = torch.full((pages,), -1, dtype=torch.int32)
    free[:pages - used] = order[used:]
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(c=c, pages=pages, table=table.to(DEV), free=free.to(DEV), free_count=_up([pages - used]),
                lens=cached.to(torch.int32).to(DEV), new_len=new.to(torch.int32).to(DEV), lens_out=i32(R),
                free_count_out=i32(1), q_start=i32(R + 1), positions=i32(c["T"]), slots=i32(c["T"]), row_seq=i32(c["T"]),
                row_len=i32(c["T"]))


def _pieces(c, h):
    """The lengths of the prompts' pieces: any, with a sum that is the case's."""
    n = c["chunks"]
    if n == 0:
        return []
    rows = max(n, n * (c["chunk"] + 1) // 2)
    cuts = sorted((torch.randperm(rows - 1, generator=h)[:n - 1] + 1).tolist())
    return [b - a for a, b in zip([0] + cuts, cuts + [rows])]


def _make_attend(c, g, h):
    R, page, Hkv, D = c["decode"] + c["chunks"], c["page"], c["Hkv"], c["D"]
    if c["full"]:
        cached, new = [c["ctx"]] * R, [1] * c["decode"] + [c["chunk"]] * c["chunks"]
    else:
        cached = torch.randint(0, c["ctx"] + 1, (R,), generator=h).tolist()
        new = [1] * c["decode"] + _pieces(c, h)
    lens = [a + b for a, b in zip(cached, new)]
    width = -(-max(lens) // page)
    have = torch.tensor([-(-n // page) for n in lens])
    pages = int(have.sum()) + 3
    table = torch.zeros((R, width), dtype=torch.int32)
    table[torch.arange(width) < have[:, None]] = torch.randperm(pages, generator=h)[:pages - 3].to(torch.int32)
    shape = (pages, Hkv, page, D)
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    ks = vs = None
    if c["kv"] == "e4m3":
        # codes that use the format's range; the scales take them back to the values' size
        ks = torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.01
        vs = torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.01
        k, v = (k * 64).to(torch.float8_e4m3fn), (v * 64).to(torch.float8_e4m3fn)
    T = sum(new)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return dict(c=c, new=new, lens=lens, start=start, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, page_table=table.to(DEV),
                q_start=_up(start), kv_len=_up(lens), seen=_up(lens),
                q=torch.randn((T, c["Hq"], D), generator=g, device=DEV, dtype=torch.bfloat16) * 2,
                out=torch.empty((T, c["Hq"], D), dtype=torch.bfloat16, device=DEV),
                lse_out=torch.empty((T, c["Hq"]), device=DEV) if c["lse"] else None)


def _make_route(c, g, h):
    T, E, k = c["T"], c["E"], c["k"]
    x = torch.randn((T, E), generator=g, device=DEV) * 1.5 + torch.randn(E, generator=g, device=DEV) * 0.5
    bias = torch.randn(E, generator=g, device=DEV) * (0.1 if c["scoring"] == "sigmoid" else 0.01) if c["bias"] else None
    return dict(c=c, logits=x.to(torch.bfloat16) if c["dtype"] == "bf16" else x, bias=bias,
                ids=torch.empty((T, k), dtype=torch.int32, device=DEV), w=torch.empty((T, k), device=DEV))


def _make_adjust(c, g, h):
    T, V, H, B = c["T"], c["V"], c["history"], c["biases"]
    x = torch.randn((T, V), generator=g, device=DEV) * 3
    total = torch.randint(max(1, H // 2), H + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
    prompt = (total * torch.rand(T, generator=g, device=DEV)).to(torch.int32)
    # text repeats its frequent tokens
    history = (torch.rand((T, H), generator=g, device=DEV) ** 3 * V).to(torch.int32).clamp(max=V - 1)
    of = lambda lo, hi: torch.rand(T, generator=g, device=DEV) * (hi - lo) + lo  # noqa: E731
    ids = bias = None
    if B:
        ids = (torch.arange(B, device=DEV) * (V // B) + torch.randint(0, V // B, (T, B), generator=g, device=DEV)).to(torch.int32)
        ids[torch.rand((T, B), generator=g, device=DEV) < 0.3] = -1
        bias = torch.randn((T, B), generator=g, device=DEV) * 5
    mask = None
    if c["mask"]:
        # a grammar that allows some tokens of a few regions; every other row has none
        words = -(-V // 32)
        bits = torch.randint(-2 ** 31, 2 ** 31, (T, words), generator=g, device=DEV, dtype=torch.int64)
        bits = bits & torch.randint(-2 ** 31, 2 ** 31, (T, words), generator=g, device=DEV, dtype=torch.int64)
        bits = torch.where(torch.rand((T, words), generator=g, device=DEV) < 0.2, bits, 0)
        bits[1::2] = -1
        mask = bits.to(torch.int32)
    return dict(c=c, logits=x.to(torch.bfloat16) if c["dtype"] == "bf16" else x, history=history, prompt_len=prompt,
                history_len=total, repetition=of(1.0, 1.3), frequency=of(0.0, 0.5), presence=of(-0.2, 0.6), bias_ids=ids,
                bias=bias, mask=mask, out=torch.empty((T, V), device=DEV))


# ---------------------------------------------------------------------------- one pass

TABLE_OUT = ("lens_out", "free_count_out", "q_start", "positions", "slots", "row_seq", "row_len")


def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if not own:
        return {"tables": _plain_tables, "attend": _plain_attend, "route": _plain_route, "adjust": _plain_adjust}[op](s, c)
    import paged_expert_moe_gb300 as pm
    if op == "tables":
        pm.moe_batch_tables(s["table"], s["free"], s["free_count"], s["lens"], s["new_len"], c["T"], c["page"], s["pages"],
                            **{n: s[n] for n in TABLE_OUT})
        return {"table": s["table"], "free": s["free"], **{n: s[n] for n in TABLE_OUT}}
    if op == "attend":
        pm.moe_chunk_attention(s["k_cache"], s["v_cache"], s["q"], s["q_start"], s["kv_len"], s["page_table"],
                               window=c["window"], sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                               out=s["out"], lse_out=s["lse_out"])
        return {"out": s["out"], "lse": s["lse_out"]}
    if op == "route":
        pm.moe_router_select(s["logits"], c["k"], scoring=c["scoring"], bias=s["bias"], groups=c["groups"],
                             top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"], scale=2.5,
                             ids_out=s["ids"], w_out=s["w"])
        return {"ids": s["ids"], "w": s["w"]}
    pm.moe_adjust_logits(s["logits"], history=s["history"], prompt_len=s["prompt_len"], history_len=s["history_len"],
                         repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                         bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"], out=s["out"])
    return {"out": s["out"]}


def _plain_tables(s, c):
    """Whole numbers throughout. A request that ended gives its pages back first; the others'
    new pages come off the top of the free pages, in order; a request whose pages or rows do
    not all fit gets none."""
    R, T, page = c["R"], c["T"], c["page"]
    table, width = s["table"], s["table"].shape[1]
    new, lens = s["new_len"].long(), s["lens"].long()
    done = new < 0
    n = new.clamp(min=0)
    have = (lens + page - 1) // page
    at = torch.arange(width, device=DEV)
    back = torch.where(done, have, 0)
    upto = back.cumsum(0)
    count = s["free_count"].long()
    free = torch.cat([s["free"], s["free"][:1]])  # one place more, for what goes nowhere
    to = torch.where(at < back[:, None], count + (upto - back)[:, None] + at, s["free"].shape[0])
    free[to.flatten()] = table.flatten()
    s["free"].copy_(free[:-1])
    count = count + upto[-1]
    end = n.cumsum(0)
    fits = (lens + n <= width * page) & (end <= T)
    need = torch.where(fits, (lens + n + page - 1) // page - have, 0)
    upto = need.cumsum(0)
    fits &= (need == 0) | (upto <= count)
    need = torch.where(fits, need, 0)
    first = upto - need
    fresh = (at >= have[:, None]) & (at < (have + need)[:, None])
    top = (count - 1 - first[:, None] - (at - have[:, None])).clamp(min=0)
    table.copy_(torch.where(fresh, s["free"][top], table))
    s["free_count_out"].copy_(count - torch.where(fits, upto, 0).amax())
    s["lens_out"].copy_(torch.where(done, 0, torch.where(fits, lens + n, lens)))
    s["q_start"][0] = 0
    s["q_start"][1:] = end.clamp(max=T)
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(end, t, right=True)
    live = seq < R
    seq = seq.clamp(max=R - 1)
    pos = lens[seq] + t - (end - n)[seq]
    stored = live & fits[seq]
    slot = table[seq, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    s["positions"].copy_(torch.where(live, pos, 0))
    s["slots"].copy_(torch.where(stored, slot, -1))
    s["row_seq"].copy_(torch.where(live, seq, -1))
    s["row_len"].copy_(torch.where(stored, pos + 1, 0))
    return {"table": table, "free": s["free"], **{k: s[k] for k in TABLE_OUT}}


def _plain_rows(cache, pages, scale):
    """The rows of `pages` [..., n] as [..., Hkv, n * page, D] in 32 bits."""
    x = cache.view(torch.uint8 if scale is not None else torch.int16)[pages.long()].view(cache.dtype).float()
    if scale is not None:
        x = x * scale[:, None, None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _plain_softmax(a, visible, v):
    """softmax over the visible keys, times v; and the log of the sum."""
    a = a.masked_fill(~visible, -math.inf)
    m = a.amax(-1, keepdim=True)
    a = torch.exp(a - m)
    total = a.sum(-1, keepdim=True)
    return torch.matmul(a, v) / total, (m + total.log())[..., 0]


def _plain_attend(s, c):
    Hq, Hkv, D, page, W, S = c["Hq"], c["Hkv"], c["D"], c["page"], c["window"], c["sinks"]
    G = Hq // Hkv
    q = s["q"].float().view(-1, Hkv, G, D) * D ** -0.5
    start, lens = s["start"], s["lens"]
    out, lse = s["out"].view(-1, Hkv, G, D), None if s["lse_out"] is None else s["lse_out"].view(-1, Hkv, G)
    # single tokens together, as many as 4 GB hold: the pages that some of them see, key by key
    most = max([n for n in lens[:c["decode"]]], default=0)
    head = -(-S // page) if W else 0
    if W and most > W + (head + 1) * page:
        per, picked = head + W // page + 2, True
    else:
        per, picked = -(-most // page), False
    rows = max(1, int(4e9 / max(1, per * page * Hkv * D * 8)))
    at = torch.arange(per * page, device=DEV)
    for r in range(0, c["decode"], rows):
        e = min(c["decode"], r + rows)
        n = s["seen"][r:e].long()[:, None]
        which = torch.arange(per, device=DEV).expand(e - r, per)
        if picked:  # the first pages, and those that the window reaches
            low = ((n - W).clamp(min=0) // page).clamp(min=head)
            which = torch.where(which < head, which, low + which - head)
        key = which.repeat_interleave(page, 1) * page + at % page
        visible = key < n
        if W:
            visible &= (key >= n - W) | (key < S)
        which = which.clamp(max=s["page_table"].shape[1] - 1)
        pages = s["page_table"][r:e].gather(1, which)
        k, v = (_plain_rows(x, pages, y) for x, y in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
        a = torch.matmul(q[r:e], k.transpose(2, 3))
        o, total = _plain_softmax(a, visible[:, None, None], v)
        out[r:e] = o.to(torch.bfloat16)
        if lse is not None:
            lse[r:e] = total
    # the others one by one, some rows of one key head at a time
    for r in range(c["decode"], len(lens)):
        n, L = s["new"][r], lens[r]
        pages = s["page_table"][r, :-(-L // page)]
        k, v = (_plain_rows(x, pages, y)[:, :L] for x, y in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
        step = max(1, int(1e9 / (G * L)))
        key = torch.arange(L, device=DEV)
        for i in range(0, n, step):
            e = min(n, i + step)
            pos = L - n + torch.arange(i, e, device=DEV)[:, None]
            lo, hi = (max(0, L - n + i + 1 - W) if W else 0), L - n + e
            keep = torch.cat([key[:min(S, lo)], key[lo:hi]])
            visible = keep <= pos
            if W:
                visible &= (keep > pos - W) | (keep < S)
            visible = visible[:, None].expand(-1, G, -1).flatten(0, 1)
            t = start[r] + i
            for h in range(Hkv):
                qq = q[t:t + e - i, h].flatten(0, 1)
                kk, vv = k[h, lo:hi], v[h, lo:hi]
                if min(S, lo):
                    kk, vv = torch.cat([k[h, :min(S, lo)], kk]), torch.cat([v[h, :min(S, lo)], vv])
                o, total = _plain_softmax(qq @ kk.T, visible, vv)
                out[t:t + e - i, h] = o.view(-1, G, D).to(torch.bfloat16)
                if lse is not None:
                    lse[t:t + e - i, h] = total.view(-1, G)
    return {"out": s["out"], "lse": s["lse_out"]}


def _plain_route(s, c):
    # scores in 64 bits: two experts' order must not hang on a rounding
    x = s["logits"].double()
    T, E, k, g = c["T"], c["E"], c["k"], c["groups"]
    if c["scoring"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    choice = score + s["bias"].double() if s["bias"] is not None else score
    if g > 1:
        rank = torch.sort(choice.view(T, g, E // g), dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        best = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros((T, g), dtype=torch.bool, device=DEV).scatter_(1, best, True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // g, 1), -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": (w * 2.5).float()}


def _plain_adjust(s, c):
    V, H = c["V"], c["history"]
    x = s["logits"].float()
    at = torch.arange(H, device=DEV)
    said = at < s["history_len"][:, None]
    made = said & (at >= s["prompt_len"][:, None])
    ids = s["history"].long()
    any_ = torch.zeros_like(x, dtype=torch.int32).scatter_add_(1, ids, said.to(torch.int32))
    count = torch.zeros_like(x, dtype=torch.int32).scatter_add_(1, ids, made.to(torch.int32))
    r = s["repetition"][:, None]
    x = torch.where(any_ > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias_ids"] is not None:
        there = s["bias_ids"] >= 0
        x.scatter_add_(1, s["bias_ids"].long().clamp(min=0), torch.where(there, s["bias"], 0.0))
    if s["mask"] is not None:
        token = torch.arange(V, device=DEV)
        allowed = (s["mask"][:, token // 32] >> (token % 32).to(torch.int32)) & 1
        x = x.masked_fill(allowed == 0, -math.inf)
    s["out"].copy_(x)
    return {"out": s["out"]}


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"attend": _exact_attend, "route": _exact_route, "adjust": _exact_adjust}[case["op"]](s, case)


def _exact_attend(s, c):
    if work(c)["flops"] > 5e12:
        return None
    G, page = c["Hq"] // c["Hkv"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    wide = torch.uint8 if c["kv"] == "e4m3" else torch.int16
    for r, (n, L) in enumerate(zip(s["new"], s["lens"])):
        mine = s["page_table"][r, :(L + page - 1) // page].long()
        p = torch.arange(L - n, L, device=DEV).view(-1, 1)
        j = torch.arange(L, device=DEV).view(1, -1)
        hidden = j > p
        if c["window"]:
            hidden = hidden | ((p - j >= c["window"]) & (j >= c["sinks"]))
        for h in range(c["Hq"]):
            kv = []
            for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
                x = cache.view(wide)[mine, h // G].view(cache.dtype).double().reshape(-1, c["D"])[:L]
                kv.append(x if scale is None else x * scale[h // G].double())
            for i in range(0, n, 512):
                rows = slice(s["start"][r] + i, s["start"][r] + min(n, i + 512))
                a = s["q"][rows, h].double() @ kv[0].T / math.sqrt(c["D"])
                a[hidden[i:i + 512]] = -math.inf
                lse[rows, h] = torch.logsumexp(a, -1)
                out[rows, h] = torch.softmax(a, -1) @ kv[1]
    return {"out": out, "lse": lse if c["lse"] else None}


def _exact_route(s, c):
    # the weights of each token's experts, found group by group; the ids are whole numbers
    x = s["logits"].double().cpu()
    score = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, 1)
    choice = score + (s["bias"].double().cpu() if s["bias"] is not None else 0)
    size = c["E"] // c["groups"]
    kept = choice.clone()
    if c["groups"] > 1:
        parts = choice.split(size, dim=1)
        value = torch.stack([p.topk(min(c["group_top"], size), dim=1).values.sum(1) for p in parts], 1)
        floor = value.topk(c["top_groups"], dim=1).values[:, -1:]
        kept[(value < floor).repeat_interleave(size, dim=1)] = -math.inf
    ids = kept.topk(c["k"], dim=1).indices
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        w /= w.sum(1, keepdim=True)
    return {"ids": None, "w": (2.5 * w).to(DEV)}


def _exact_adjust(s, c):
    got = s["logits"].double()
    of = {n: s[n].tolist() for n in ("prompt_len", "history_len", "repetition", "frequency", "presence")}
    for t in range(c["T"]):
        mine = s["history"][t, :of["history_len"][t]].long()
        seen = torch.unique(mine)
        x = got[t, seen]
        got[t, seen] = torch.where(x > 0, x / of["repetition"][t], x * of["repetition"][t])
        made, times = torch.unique(mine[of["prompt_len"][t]:], return_counts=True)
        got[t, made] -= of["frequency"][t] * times + of["presence"][t]
        if s["bias_ids"] is not None:
            ids = s["bias_ids"][t].long()
            got[t, ids[ids >= 0]] += s["bias"][t][ids >= 0].double()
        if s["mask"] is not None:
            bits = (s["mask"][t].view(-1, 1) >> torch.arange(32, device=DEV)) & 1
            got[t, bits.flatten()[:c["V"]] == 0] = -math.inf
    return {"out": got}
