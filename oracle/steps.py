"""A step over requests of different lengths in float64 and whole numbers: the plain definitions.

batch_tables goes request by request and page by page; chunk_attention row by row of a request;
router_select and adjust_logits token by token.
"""

import numpy as np


def batch_tables(page_table, free_pages, free_count, lens, new_len, T, page_size, num_pages):
    """(page_table, free_pages, free_count, lens, q_start, positions, slots, row_seq, row_len,
    denied) after the step, the inputs left as they are."""
    table, free = np.array(page_table), list(free_pages[:free_count])
    R, width = table.shape
    pages = lambda n: -(-int(n) // page_size)  # noqa: E731
    for r in range(R):
        if new_len[r] == -1:
            free += [int(p) for p in table[r, :pages(lens[r])]]
    stack = np.array(free_pages)
    stack[:len(free)] = free
    out_lens, start, rows, denied, wanted, top = [], [0], [], [], 0, len(free)
    for r in range(R):
        n, old = max(int(new_len[r]), 0), int(lens[r])
        end = start[-1] + n
        need = pages(old + n) - pages(old)
        fits = end <= T and old + n <= width * page_size
        if fits:
            wanted += need  # of all requests up to this one, whether they get theirs or not
            fits = need == 0 or wanted <= len(free)
        if fits:
            for i in range(need):
                top -= 1
                table[r, pages(old) + i] = free[top]
        denied.append(n > 0 and not fits)
        for i in range(n):
            p = old + i
            page = int(table[r, p // page_size]) if fits else -1
            ok = fits and 0 <= page < num_pages
            rows.append((p, page * page_size + p % page_size if ok else -1, r, p + 1 if fits else 0))
        out_lens.append(0 if new_len[r] == -1 else old + n if fits else old)
        start.append(end)
    rows = (rows + [(0, -1, -1, 0)] * T)[:T]
    cols = np.array(rows, np.int32).reshape(T, 4).T
    return (table, stack, top, np.array(out_lens, np.int32), np.minimum(start, T).astype(np.int32), cols[0], cols[1], cols[2],
            cols[3], np.array(denied, bool))


def chunk_attention(k_cache, v_cache, q, q_start, kv_len, page_table, scale, window=0, sinks=0):
    """out [T, q_heads, D], lse [T, q_heads], per output element the sum of weight * |v|, and the
    number of visible keys of each row (-1: a row of no request). Caches are float64 arrays [pages,
    kv_heads, page_size, D]."""
    T, hq, D = q.shape
    hk, page = k_cache.shape[1], k_cache.shape[2]
    out, lse, mag = np.zeros((T, hq, D)), np.full((T, hq), -np.inf), np.zeros((T, hq, D))
    count = np.full(T, -1)
    for r in range(len(kv_len)):
        t0, t1, L = int(q_start[r]), int(q_start[r + 1]), int(kv_len[r])
        if t1 <= t0:
            continue
        n = t1 - t0
        pos = L - n + np.arange(n)
        at = np.array([page_table[r][j // page] for j in range(L)], int), np.arange(L) % page
        j = np.arange(L)
        seen = j[None] <= pos[:, None]
        if window:
            seen &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
        count[t0:t1] = seen.sum(1)
        if L == 0:
            continue
        some = seen.any(0)  # what no row sees may be anything
        for h in range(hq):
            k, v = k_cache[at[0], h // (hq // hk), at[1]], v_cache[at[0], h // (hq // hk), at[1]]
            k, v = np.where(some[:, None], k, 0), np.where(some[:, None], v, 0)
            s = np.where(seen, scale * (q[t0:t1, h] @ k.T), -np.inf)
            m = s.max(1, keepdims=True)
            w = np.exp(s - np.where(np.isinf(m), 0, m))
            total = w.sum(1, keepdims=True)
            safe = np.where(total > 0, total, 1)
            out[t0:t1, h] = w @ v / safe
            mag[t0:t1, h] = w @ np.abs(v) / safe
            with np.errstate(divide="ignore"):
                lse[t0:t1, h] = (m + np.log(total))[:, 0]
    return out, lse, mag, count


def router_select(logits, top_k, scoring, bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    """(ids, weights, margin) of every token: margin is the least difference of two values whose order
    decides something."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    T, E = x.shape
    ids, w, margin = np.zeros((T, top_k), np.int32), np.zeros((T, top_k)), np.full(T, np.inf)
    for t in range(T):
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1 / (1 + np.exp(-x[t]))
        else:
            m = x[t].max()
            with np.errstate(invalid="ignore"):
                e = np.where(x[t] == m, 1.0, np.exp(x[t] - m))
            s = e / e.sum()
        c = s if bias is None else s + np.where(np.isnan(bias), -np.inf, np.asarray(bias, np.float64))
        order = x[t] if bias is None else c  # the score rises with the logit
        alive = list(range(E))
        if groups > 1 and top_groups < groups:
            size = E // groups
            best = order if bias is None and min(group_top, size) == 1 else c  # (a sum needs the scores)
            value = [sum(sorted(best[g * size:(g + 1) * size], reverse=True)[:group_top]) for g in range(groups)]
            rank = sorted(range(groups), key=lambda g: (-value[g], g))
            margin[t] = min(margin[t], value[rank[top_groups - 1]] - value[rank[top_groups]])
            alive = [e for e in alive if e // size in rank[:top_groups]]
        rank = sorted(alive, key=lambda e: (-order[e], e))
        with np.errstate(invalid="ignore"):
            gaps = [order[a] - order[b] for a, b in zip(rank[:top_k], rank[1:top_k + 1])]
        margin[t] = min([margin[t]] + gaps)
        ids[t] = rank[:top_k]
        got = s[ids[t]]
        w[t] = scale * (got / got.sum() if renormalize and got.sum() > 0 else got)
    return ids, w, margin


def adjust_logits(logits, history=None, prompt_len=None, history_len=None, repetition=None, frequency=None, presence=None,
                  bias_ids=None, bias=None, mask=None):
    """float64 [T, V], and the sum of the magnitudes that each value went through."""
    x = np.array(logits, np.float64)
    T, V = x.shape
    size = np.abs(x)
    for t in range(T):
        if history is not None:
            n = min(max(int(history_len[t]), 0), history.shape[1])
            p = 0 if prompt_len is None else min(max(int(prompt_len[t]), 0), n)
            ids = [int(v) for v in history[t][:n]]
            r = 1.0 if repetition is None else float(repetition[t])
            for v in {v for v in ids if 0 <= v < V}:
                x[t, v] = x[t, v] / r if x[t, v] > 0 else x[t, v] * r
                size[t, v] += abs(x[t, v])
                times = ids[p:].count(v)
                if times:
                    f = 0.0 if frequency is None else float(frequency[t])
                    y = 0.0 if presence is None else float(presence[t])
                    x[t, v] -= f * times + y
                    size[t, v] += abs(f * times) + abs(y)
        if bias_ids is not None:
            for v, b in {int(i): float(b) for i, b in zip(bias_ids[t], bias[t]) if 0 <= i < V}.items():
                x[t, v] += b
                size[t, v] += abs(b)
        if mask is not None:
            words = np.asarray(mask[t]).view(np.uint32)
            v = np.arange(V)
            x[t, (words[v // 32] >> (v % 32).astype(np.uint32) & 1) == 0] = -np.inf
    return x, size
