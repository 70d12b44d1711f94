"""moe_sample_tokens against the float64 oracle where no list of candidates decides a row: more
than 1,200 tokens kept by top-k, or lists that overflow, with and without the other cuts.

The kernel's weight of a token is exp2 of y = (x - m) * r, r = log2(e) / temperature, all fp32: y
is off by the roundings of x - m, of log2(e), of r and of the product, 4 x 2^-24 of itself, which
for weights that count (|y| <= 31) is 31 x 2^-22 and changes the weight by ln 2 x 31 x 2^-22 <
2^-17.5 of it; exp2 adds 2^-22. So weights, and sums of weights, are within 2^-17 of float64's, and
the rounding down to whole units of 2^-31 of the largest weight adds at most one unit a token, V
2^-31 of a sum (which has the largest in it). Rows in which a sum or weight comes nearer than that
to what it is compared with are left out, and have to be few.
"""

import numpy as np
import pytest

from oracle import sampling as osamp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def threshold_bin(x, k):
    """Logits in the sixteenth, by distance from the row's largest, that holds the k-th."""
    d = np.floor((x.max() - x) * 16)
    return int((d == np.sort(d)[k - 1]).sum())


FEW, MANY = [(12, 6000, False, 1.0), (8, 32000, True, 2.0)], [(8, 50001, False, 0.06), (6, 131072, True, 0.05), (5, 50000, False, 0.0)]


# (over rows as flat as MANY's no cut by top-p alone is farther from a token than near)
@pytest.mark.parametrize("T,V,bf16,spread,cut", [(*c, cut) for c in FEW + MANY for cut in ("k", "kp", "km", "kpm")] +
                         [(*c, cut) for c in FEW for cut in ("p", "pm")])
def test_draws_over_many_tokens(pm, T, V, bf16, spread, cut):
    rng = np.random.default_rng(V + len(cut))
    x = torch.from_numpy((rng.standard_normal((T, V)) * spread).astype(np.float32)).cuda()
    x = x.to(torch.bfloat16) if bf16 else x
    xs = x.float().cpu().numpy().astype(np.float64)
    near = 2.0 ** -17 + V * 2.0 ** -31
    temperature = rng.uniform(0.7, 1.4, T).astype(np.float32)
    top_k = rng.integers(1201, 5000, T).astype(np.int32) if "k" in cut else np.zeros(T, np.int32)
    top_p = rng.uniform(0.3, 0.97, T).astype(np.float32) if "p" in cut else np.ones(T, np.float32)
    min_p = rng.uniform(0.001, 0.3, T).astype(np.float32) if "m" in cut else np.zeros(T, np.float32)
    if "k" in cut:  # the bin of the threshold fits one CTA's list in the first two, not in the others
        assert (threshold_bin(xs[0], int(top_k[0])) > 2048) == (spread < 1)
    u = (rng.integers(0, 1 << 24, T) / 2.0 ** 24).astype(np.float32)
    lp = torch.empty(T, device="cuda")
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    ids = pm.moe_sample_tokens(x, up(u), up(temperature), up(top_k), up(top_p), up(min_p), logprob_out=lp).tolist()
    sure = 0
    for t in range(T):
        want, wlp, margin = osamp.sample_row(xs[t], u[t], float(temperature[t]), int(top_k[t]), float(top_p[t]), float(min_p[t]))
        if margin > near:
            sure += 1
            assert ids[t] == want, (t, ids[t], want, margin)
            assert abs(float(lp[t]) - wlp) <= 2 * near + 2.0 ** -22 * abs(wlp) + 2.0 ** -22
    assert sure >= T // 4, sure
