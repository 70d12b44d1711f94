"""moe_sample_tokens against the float64 oracle.

The kernel's weights are fp32 exponentials (argument and result within 2^-22 of a weight
for the arguments here, |z| < 32: 32 2^-24 + 2 ulp), so a draw can differ from the float64
one only where a sum lies within 2^-18 of what it is compared with (relative): those rows
are left out, and have to be few. Rows of equal logits have exact weights and are compared
everywhere. A log probability is off by at most twice the weights' error and 2^-22.
"""

import numpy as np
import pytest

from oracle import sampling as osamp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -18


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def dev(a, dtype=None):
    return None if a is None else torch.as_tensor(np.asarray(a), dtype=dtype).cuda()


def draw(pm, x, u, temperature=None, top_k=None, top_p=None, min_p=None, **more):
    T = x.shape[0]
    lp = torch.empty(T, device="cuda")
    ids = pm.moe_sample_tokens(x, dev(u, torch.float32), dev(temperature, torch.float32), dev(top_k, torch.int32),
                               dev(top_p, torch.float32), dev(min_p, torch.float32), logprob_out=lp, **more)
    return ids.cpu().numpy(), lp.cpu().numpy()


def check(x, ids, lp, u, temperature=None, top_k=None, top_p=None, min_p=None):
    xs = x.float().cpu().numpy().astype(np.float64)
    sure = 0
    for t in range(len(ids)):
        one = [d if a is None else a[t] for a, d in ((temperature, 1.0), (top_k, 0), (top_p, 1.0), (min_p, 0.0))]
        one = [float(np.float32(v)) if i != 1 else int(v) for i, v in enumerate(one)]
        want, wlp, margin = osamp.sample_row(xs[t], u[t], *one)
        if margin > NEAR:
            sure += 1
            assert ids[t] == want, (t, ids[t], want, one, margin)
            assert lp[t] == wlp or abs(lp[t] - wlp) <= 2 * NEAR
    return sure / len(ids)


@pytest.mark.parametrize("T,V,bf16", [(1, 1, False), (3, 2, True), (16, 33, False), (9, 1000, True), (8, 2049, False),
                                      (6, 4097, True), (5, 32000, False), (4, 50001, False), (3, 131072, True),
                                      (2, 262144, False), (2, 262143, True)])
@pytest.mark.parametrize("cut", ["none", "k", "p", "m", "kpm"])
def test_draws_match_oracle(pm, T, V, bf16, cut):
    rng = np.random.default_rng(V * 10 + T)
    x = torch.from_numpy(rng.standard_normal((T, V)).astype(np.float32) * 3).cuda()
    x = x.to(torch.bfloat16) if bf16 else x
    u = rng.random(T).astype(np.float32) * np.float32(0.999)
    args = dict(temperature=rng.uniform(0.6, 1.5, T))
    if "k" in cut:
        args["top_k"] = rng.integers(1, max(2, min(V, 300)), T)
    if "p" in cut:
        args["top_p"] = rng.uniform(0.3, 0.99, T)
    if "m" in cut:
        args["min_p"] = rng.uniform(0.001, 0.2, T)
    ids, lp = draw(pm, x, u, **args)
    sure = check(x, ids, lp, u, **args)
    assert T < 3 or sure >= 0.6


def test_many_rows_of_mixed_settings(pm):
    rng = np.random.default_rng(1)
    T, V = 300, 700
    x = torch.from_numpy(rng.standard_normal((T, V)).astype(np.float32) * 4).cuda()
    u = rng.random(T).astype(np.float32)
    args = dict(temperature=rng.choice([0.0, -1.0, 0.5, 1.0, 2.0], T), top_k=rng.choice([-5, 0, 1, 2, 40, 699, 700, 5000], T),
                top_p=rng.choice([-1.0, 0.0, 0.5, 0.9, 1.0, 2.0], T), min_p=rng.choice([-1.0, 0.0, 0.05, 1.0, 3.0], T))
    ids, lp = draw(pm, x, u, **args)
    assert check(x, ids, lp, u, **args) > 0.95


@pytest.mark.parametrize("V", [7, 5000, 20011])
def test_equal_logits_are_exact(pm, V):
    """All weights are 2^31: ties are cut in id order and the draw is floor(u k)."""
    T = 64
    rng = np.random.default_rng(V)
    x = torch.full((T, V), -3.25, device="cuda")
    u = (rng.integers(0, 1 << 24, T) / 2.0 ** 24).astype(np.float32)
    u[:2] = [0.0, 1 - 2.0 ** -24]
    k = rng.integers(1, V + 1, T)
    ids, lp = draw(pm, x, u, top_k=k)
    S = [int(n) << 31 for n in k]
    want = [((s * int(v * 2.0 ** 24)) >> 24) >> 31 for s, v in zip(S, u.astype(np.float64))]
    assert ids.tolist() == want
    p = (rng.integers(1, 1 << 24, T) / 2.0 ** 24).astype(np.float32)
    ids, lp = draw(pm, x, u, top_p=p)
    kept = [max(1, -(-(((V << 31) * int(v * 2.0 ** 24)) >> 24) // (1 << 31))) for v in p.astype(np.float64)]
    want = [((n << 31) * int(v * 2.0 ** 24) >> 24) >> 31 for n, v in zip(kept, u.astype(np.float64))]
    assert ids.tolist() == want
    assert np.allclose(lp, -np.log(kept), atol=2.0 ** -18)


def test_two_values_with_ties_at_the_threshold(pm):
    """Half the row at 0, half at -1: the cut falls inside the lower ties, in id order."""
    V, T = 9000, 32
    rng = np.random.default_rng(3)
    high = rng.permutation(V)[:V // 2]
    row = np.full(V, -1.0, np.float32)
    row[high] = 0
    x = torch.from_numpy(np.tile(row, (T, 1))).cuda()
    u = rng.random(T).astype(np.float32)
    k = rng.integers(1, V, T)
    ids, lp = draw(pm, x, u, top_k=k)
    assert check(x, ids, lp, u, top_k=k) > 0.9
    p = rng.uniform(0.1, 0.999, T)
    ids, lp = draw(pm, x, u, top_p=p)
    assert check(x, ids, lp, u, top_p=p) > 0.9


def test_infinities_nan_and_empty_rows(pm):
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[-inf, -inf, -inf, -inf], [nan, nan, nan, nan], [nan, -inf, 1.0, nan], [-inf, inf, 0.0, inf],
                      [-3.4028235e38] * 3 + [-inf], [3.4028235e38, -3.4028235e38, 0.0, nan], [-0.0, 0.0, -1.0, -inf]],
                     device="cuda")
    T = x.shape[0]
    for u in (0.0, 0.5, 0.99):
        for top_k, top_p in ((0, 1.0), (2, 1.0), (0, 0.5), (3, 0.9)):
            ids, lp = draw(pm, x, [u] * T, top_k=[top_k] * T, top_p=[top_p] * T)
            assert ids[0] == ids[1] == -1 and np.isneginf(lp[0]) and np.isneginf(lp[1])
            assert ids[2] == 2 and lp[2] == 0
            assert ids[3] in (1, 3) and ids[4] in (0, 1, 2) and ids[5] == 0 and ids[6] in (0, 1, 2)
            if top_k == 0 and top_p == 1.0:
                assert ids[3] == (1 if u < 0.5 else 3) and ids[4] == int(u * 3)
                assert abs(lp[3] + np.log(2)) < 1e-6
    ids, lp = draw(pm, x, [0.3] * T, temperature=[0.0] * T)
    assert ids.tolist() == [-1, -1, 2, 1, 0, 0, 0] and lp[2] == 0


def test_strided_rows_streams_and_graphs(pm):
    rng = np.random.default_rng(4)
    for dtype in (torch.float32, torch.bfloat16):
        wide = torch.from_numpy(rng.standard_normal((6, 30013)).astype(np.float32) * 3).cuda().to(dtype)
        for off in (0, 1, 3):  # rows that start anywhere in a 16-byte vector
            x = wide[:, off:off + 30001]
            u = rng.random(6).astype(np.float32)
            ids, lp = draw(pm, x, u, top_p=[0.9] * 6)
            assert check(x, ids, lp, u, top_p=[0.9] * 6) > 0.5
            ud, pd = dev(u, torch.float32), dev([0.9] * 6, torch.float32)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            other = pm.moe_sample_tokens(x, ud, top_p=pd, stream=s)
            s.synchronize()
            assert ids.tolist() == other.tolist()
    out = torch.empty(6, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pm.moe_sample_tokens(x, ud, ids_out=out)
    g.replay()
    assert out.tolist() == pm.moe_sample_tokens(x, ud).tolist()


def test_sampling_refusals(pm):
    u = torch.zeros(2, device="cuda")
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_sample_tokens(torch.zeros((2, 262145), device="cuda"), u)
    assert e.value.status == pm.PMOE_EINVAL
    assert pm.moe_sample_tokens(torch.zeros((0, 8), device="cuda"), u[:0]).numel() == 0


@pytest.mark.parametrize("T,V,bf16", [(640, 40000, True), (400, 17001, False), (320, 39999, False), (64, 131072, True)])
def test_rows_do_not_depend_on_the_batch(pm, T, V, bf16):
    """How many CTAs take a row depends on the rows and their length; what is drawn does not."""
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, V)).astype(np.float32) * 2.5).cuda()
    x = x.to(torch.bfloat16) if bf16 else x
    u = torch.from_numpy(rng.random(T).astype(np.float32)).cuda()
    dev = lambda v, dt: torch.from_numpy(np.asarray(v).astype(dt)).cuda()  # noqa: E731
    args = dict(temperature=dev(rng.choice([0.0, 0.6, 1.0], T), np.float32), top_k=dev(rng.choice([0, 20, 1000, 2000], T), np.int32),
                top_p=dev(rng.choice([1.0, 0.95, 0.8], T), np.float32), min_p=dev(rng.choice([0.0, 0.0, 0.05], T), np.float32))
    lp = torch.empty(T, device="cuda")
    ids = pm.moe_sample_tokens(x, u, logprob_out=lp, **args)
    for i in range(0, T, 8):
        few = torch.empty(8, device="cuda")
        got = pm.moe_sample_tokens(x[i:i + 8], u[i:i + 8], logprob_out=few, **{k: v[i:i + 8] for k, v in args.items()})
        assert torch.equal(got, ids[i:i + 8]) and torch.equal(few, lp[i:i + 8])
