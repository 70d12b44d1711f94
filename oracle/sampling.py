"""The draw of a token in float64: weights as whole multiples of 2^-31 of the largest."""

import numpy as np


def _share(total, part):
    return total * int(np.float32(part) * 2.0 ** 24) >> 24


def sample_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """x [V] float64 -> (id, log probability, margin): margin is the least distance, relative
    to the sum it is compared in, by which a rounding of the weights could change the draw."""
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max()
    if m == -np.inf:
        return -1, -np.inf, np.inf
    if not temperature > 0:
        return int(np.argmax(x)), 0.0, np.inf
    with np.errstate(invalid="ignore"):
        w = np.where(x == m, 1.0, np.exp((x - m) / temperature))
    n = [int(v) for v in np.floor(w * 2.0 ** 31)]
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    if 0 < top_k < len(x):
        order = order[:top_k]
    margin = np.inf
    if top_p < 1:
        total = sum(n[i] for i in order)
        least = max(1, _share(total, max(top_p, 0.0)))
        run, kept = 0, []
        for i in order:
            if run >= least:
                break
            kept.append(i)
            run += n[i]
            margin = min(margin, abs(run - least) / total)
        order = kept
    if min_p > 0:
        min_p = min(min_p, 1.0)
        margin = min([margin] + [abs(w[i] - min_p) / min_p for i in order if w[i] != 1.0])
        order = [i for i in order if w[i] >= min_p]
    order = sorted(i for i in order if n[i] > 0)
    S = sum(n[i] for i in order)
    target = _share(S, u)
    run = 0
    for i in order:
        margin = min(margin, abs(run - target) / S if run else np.inf)
        run += n[i]
        if run > target:
            return i, float(np.log(n[i] / S)), min(margin, (run - target) / S)
    raise AssertionError("no token reached the target")
