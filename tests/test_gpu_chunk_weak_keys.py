"""moe_chunk_attention with an e4m3 cache and keys whose weights are far below the strongest one's.

All keys but one are alike and their value is 1, the strong one's is 0, so that an output is the weak
keys' share w n / (1 + w n), w = 2^-below. Weights are rounded to fp16 as multiples of at least 2^-7 of the
strongest's: by 2^-11 of themselves, or where they lie below fp16's normal numbers by 2^-25 of 2^7,
2^-32 of the strongest's, each. The rest (scores that are exact but for 2^-23 of the softmax scale, exp2 2^-21,
fp32 sums of n terms 2 n 2^-24) as in test_gpu_chunk_attention.py: a share is within
(2^-11 + 2^-18 + 2 n 2^-24) of itself + n 2^-32 before it is rounded to bf16.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def to_bf16(x):
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
    return np.rint(x / 2.0 ** (e - 7)) * 2.0 ** (e - 7)


def shares(pm, D, keys, new, requests, at, below, window=0, sinks=0):
    """Outputs and log-sum-exps of `requests` requests on the same pages; key `at` is the strong one."""
    page = 64
    pages = -(-keys // page)
    k = torch.zeros((pages, 1, page, D), device="cuda")
    v = torch.ones((pages, 1, page, D), device="cuda")
    k[at // page, 0, at % page] = 1
    v[at // page, 0, at % page] = 0
    one = torch.ones(1, device="cuda")
    ints = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    T = requests * new
    lse = torch.empty((T, 1), device="cuda")
    out = pm.moe_chunk_attention(
        k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), torch.ones((T, 1, D), dtype=torch.bfloat16, device="cuda"),
        ints(np.arange(requests + 1) * new), ints([keys] * requests), ints(np.tile(np.arange(pages), (requests, 1))), window, sinks,
        scale=below * np.log(2) / D, k_scale=one, v_scale=one, lse_out=lse)
    return out.double().cpu().numpy()[:, 0], lse.double().cpu().numpy()[:, 0]


# requests of one token that a CTA takes whole, tokens of a piece, and one that all CTAs share
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("requests,new,keys", [(304, 1, 100001), (2, 300, 100001), (1, 1, 100001), (40, 1, 1000)])
@pytest.mark.parametrize("below", [20.0, 24.6, 25.5, 29.0])
def test_weak_keys_behind_a_strong_one(pm, D, requests, new, keys, below):
    for at in (0, keys - new - 70):
        out, lse = shares(pm, D, keys, new, requests, at, below)
        n = (keys - new + np.tile(np.arange(new), requests)).astype(np.float64)  # weak keys that a row sees
        weak = n * 2.0 ** -below
        share = weak / (1 + weak)
        tol = (2.0 ** -11 + 2.0 ** -18 + 2 * n * 2.0 ** -24) * share + n * 2.0 ** -32
        assert np.all(to_bf16(share - tol)[:, None] <= out) and np.all(out <= to_bf16(share + tol)[:, None])
        want = below * np.log(2) + np.log1p(weak)
        assert np.all(np.abs(lse - want) <= 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -21 * want)


def test_weak_keys_beside_a_sink(pm):
    """The strong key stays visible beside a window."""
    for below in (24.6, 25.5):
        out, _ = shares(pm, 64, 60001, 1, 304, 0, below, window=50000, sinks=1)
        weak = 50000 * 2.0 ** -below
        share = weak / (1 + weak)
        tol = (2.0 ** -11 + 2.0 ** -18 + 1e5 * 2.0 ** -24) * share + 50000 * 2.0 ** -32
        assert np.all(to_bf16(share - tol) <= out) and np.all(out <= to_bf16(share + tol))


@pytest.mark.parametrize("D", [64, 128])
def test_a_maximum_that_grows_by_less_than_it_moves_for(pm, D):
    """Scores that rise by up to 2^8 in weight without a new base: the largest weights fp16 has to hold."""
    keys, page = 4000, 64
    pages = -(-keys // page)
    k = torch.zeros((pages, 1, page, D), device="cuda")
    for i in range(pages):  # steps of a quarter to a page, over tiles of 128 keys
        k[i] = min(i // 2 * 0.25, 14.0)
    k = k.to(torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(D)
    v = (torch.randn((pages, 1, page, D), generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    one = torch.ones(1, device="cuda")
    ints = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.ones((3, 1, D), dtype=torch.bfloat16, device="cuda")
    scale = 7.9 * np.log(2) / D
    out = pm.moe_chunk_attention(k, v, q, ints([0, 3]), ints([keys]), ints(np.arange(pages)[None]), scale=scale, k_scale=one, v_scale=one)
    s = k.double().cpu().reshape(-1, D).numpy().sum(1) * np.float32(scale)
    vv = v.double().cpu().reshape(-1, D).numpy()
    for t in range(3):
        n = keys - 2 + t
        w = np.exp(s[:n] - s[:n].max())
        want, mag = (w @ vv[:n]) / w.sum(), (w @ np.abs(vv[:n])) / w.sum()
        ds = (D + 8) * 2.0 ** -24 * np.abs(s[:n]).max()
        tol = (2.0 ** -11 + 2 * ds + 2.0 ** -20 + 2 * n * 2.0 ** -24) * mag + n * 2.0 ** -32 * 448
        got = out[t, 0].double().cpu().numpy()
        assert np.all(to_bf16(want - tol) <= got) and np.all(got <= to_bf16(want + tol))
