"""moe_chunk_attention against the float64 oracle: pieces, single tokens, windows, stale cache.

Tolerance, from what the kernels round. A score is an fp32 sum of D products (exact in
fp32 with bf16 and e4m3 operands; q goes to fp16 with an e4m3 cache, exact but 2^-25 of its
row's largest): off by ds <= (D + 8) 2^-24 scale sum |q k|. A weight is off by ds and 2^-21
(exp2, rescaling) and is rounded to 16 bits: by up to r = 2^-8 of itself in bf16, 2^-11 in
fp16 (and 2^-25 of the largest weight below the normals). Sums of n terms add n 2^-24. So
before its rounding to bf16, which is monotonic, an output is within
tol = (r + 2 ds + 2^-20 + 2 n 2^-24) sum w |v| + n 2^-25 max |v| (e4m3)
of float64's, and |lse - ref| <= ds + 2^-20 + n 2^-24 + 2^-22 |ref|.
"""

import numpy as np
import pytest

from oracle import steps

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def make(seed, news, lens, Hq, Hkv, D, page, e4m3, window=0, sinks=0, qscale=2.0, page_gap=0, q_gap=0, pad=0, first=0):
    """Requests with news[r] new tokens, lens[r] keys in all; `first` rows before, `pad` behind them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    R = len(news)
    width = max(1, -(-max(list(lens) + [1]) // page))
    have = [-(-n // page) for n in lens]
    pages = sum(have) + 2
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((R, width), -7, np.int32)  # no entry beyond a request's pages is read
    at = 0
    for r in range(R):
        table[r, :have[r]] = order[at:at + have[r]]
        at += have[r]
    caches = []
    for _ in range(2):
        x = torch.randn((pages, Hkv * page * D + page_gap), generator=g, device="cuda")
        x = (x * 64).to(torch.float8_e4m3fn) if e4m3 else x.to(torch.bfloat16)
        caches.append(x[:, :Hkv * page * D].unflatten(1, (Hkv, page, D)))
    scales = [torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2)] if e4m3 else [None, None]
    start = first + np.concatenate([[0], np.cumsum(news)])
    T = int(start[-1]) + pad
    q = (torch.randn((T, Hq * D + q_gap), generator=g, device="cuda") * qscale).to(torch.bfloat16)
    q = q[:, :Hq * D].unflatten(1, (Hq, D))
    return dict(k=caches[0], v=caches[1], ks=scales[0], vs=scales[1], q=q, start=start.astype(np.int32),
                lens=np.asarray(lens, np.int32), table=table, window=window, sinks=sinks)


def bits(x):
    return x.view(torch.uint8 if x.dtype == torch.float8_e4m3fn else torch.int16)


def nan_code(x):
    return 0x7f if x.dtype == torch.float8_e4m3fn else 0x7fc0


def poison_unseen(c):
    """NaN into every cache row that no query row of any request sees."""
    page = c["k"].shape[2]
    seen = torch.zeros((c["k"].shape[0], page), dtype=torch.bool)
    for r, L in enumerate(c["lens"]):
        n = int(c["start"][r + 1] - c["start"][r])
        low = max(0, L - n - c["window"] + 1) if c["window"] else 0
        for j in range(L if n else 0):
            if j >= low or j < c["sinks"]:
                seen[c["table"][r][j // page], j % page] = True
    for x in (c["k"], c["v"]):
        bits(x)[(~seen).cuda()[:, None, :].expand(x.shape[:3])] = nan_code(x)


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(pm, c, **more):
    out = torch.full(c["q"].shape, 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["q"].shape[:2], 77.0, device="cuda")
    pm.moe_chunk_attention(c["k"], c["v"], c["q"], up(c["start"]), up(c["lens"]), up(c["table"]), window=c["window"],
                           sinks=c["sinks"], k_scale=c["ks"], v_scale=c["vs"], out=out, lse_out=lse, **more)
    return out, lse


def to_bf16(x):
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
    return np.rint(x / 2.0 ** (e - 7)) * 2.0 ** (e - 7)


def f64(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def check(c, out, lse, scale=None, rows=None):
    D = c["q"].shape[2]
    k, v, q = f64(c["k"]), f64(c["v"]), f64(c["q"])
    if c["ks"] is not None:
        k, v = k * f64(c["ks"])[:, None, None], v * f64(c["vs"])[:, None, None]
    scale = D ** -0.5 if scale is None else scale
    ref, rlse, mag, count = steps.chunk_attention(k, v, q, c["start"], c["lens"], c["table"], scale, c["window"], c["sinks"])
    kmax, vmax = np.nan_to_num(np.abs(k)).max(), np.nan_to_num(np.abs(v)).max()
    ds = (D + 8) * 2.0 ** -24 * abs(scale) * np.abs(q).sum(-1) * kmax
    n = np.maximum(count, 0)[:, None] * np.ones(q.shape[:2])
    r = 2.0 ** -8 if c["ks"] is None else 2.0 ** -11
    tol = (r + 2 * ds + 2.0 ** -20 + 2 * n * 2.0 ** -24)[..., None] * mag
    if c["ks"] is not None:
        tol += n[..., None] * 2.0 ** -25 * vmax
    got, glse = f64(out), f64(lse)
    sel = np.ones(len(q), bool) if rows is None else np.isin(np.arange(len(q)), rows)
    none = count < 0
    assert np.all(got[none] == 77) and np.all(glse[none] == 77)
    sel &= ~none
    assert np.all(to_bf16(ref - tol)[sel] <= got[sel]) and np.all(got[sel] <= to_bf16(ref + tol)[sel])
    empty = np.isinf(rlse)
    assert np.array_equal(np.isneginf(glse)[sel], empty[sel])
    fine = ~empty & sel[:, None]
    ltol = ds + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(fine, rlse, 0))
    assert np.all(np.abs(glse[fine] - rlse[fine]) <= ltol[fine])
    assert np.all(got[empty & sel[:, None]] == 0)


SIZES = [
    # new tokens, keys, Hq, Hkv, D, page, e4m3, window, sinks
    ([1], [1], 1, 1, 64, 16, False, 0, 0),
    ([1], [1], 1, 1, 128, 16, True, 0, 0),
    ([1, 1, 1], [5, 128, 129], 8, 2, 128, 16, False, 0, 0),
    ([1, 1, 1], [700, 17, 1300], 32, 4, 128, 32, True, 0, 0),
    ([7], [7], 8, 1, 64, 32, False, 0, 0),
    ([130], [130], 8, 2, 128, 16, False, 0, 0),
    ([33, 1, 64], [500, 900, 64], 16, 2, 64, 64, True, 0, 0),
    ([65, 0, 1], [65, 40, 700], 8, 8, 128, 128, False, 0, 0),
    ([300], [1000], 4, 4, 64, 256, False, 0, 0),
    ([257, 3, 1, 1], [1200, 260, 77, 1], 12, 2, 128, 16, False, 0, 0),
    ([100, 50], [400, 300], 28, 4, 64, 16, True, 0, 0),
    ([40], [2000], 64, 1, 128, 64, False, 0, 0),
    ([30], [200], 60, 1, 64, 16, True, 0, 0),
    ([600], [600], 5, 1, 128, 128, True, 0, 0),
    ([500], [1500], 7, 7, 64, 16, False, 0, 0),
    # windows and sinks
    ([1, 1, 1, 1], [1, 50, 200, 1500], 8, 1, 128, 16, False, 100, 4),
    ([1, 1], [3000, 260], 16, 2, 64, 64, True, 128, 1),
    ([200, 1], [900, 900], 8, 2, 128, 32, False, 64, 0),
    ([300, 5, 1], [1100, 1000, 300], 8, 2, 128, 16, False, 333, 130),
    ([300, 5, 1], [1100, 1000, 300], 8, 2, 64, 16, True, 333, 130),
    ([150], [800], 32, 4, 128, 16, False, 1, 0),
    ([150], [800], 16, 4, 64, 16, False, 1, 1),
    ([400], [400], 6, 3, 128, 256, True, 17, 300),
    ([260], [700], 2, 1, 64, 128, False, 600, 20),
    ([90], [2000], 16, 1, 128, 64, False, 129, 257),
    ([1], [1200], 16, 16, 128, 16, False, 5000, 3),
]


@pytest.mark.parametrize("news,lens,Hq,Hkv,D,page,e4m3,window,sinks", SIZES)
def test_attention_matches_oracle(pm, news, lens, Hq, Hkv, D, page, e4m3, window, sinks):
    c = make(sum(lens) + D + window, news, lens, Hq, Hkv, D, page, e4m3, window, sinks)
    poison_unseen(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(pm, c, err_out=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(c, out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("news,lens", [([1, 1], [900, 1200]), ([100, 1, 300], [800, 300, 300])])
def test_peaked_and_shifted_scores(pm, e4m3, news, lens):
    """Large scores of either sign: the running maximum moves far between tiles."""
    c = make(77, news, lens, 16, 2, 128, 16, e4m3, qscale=30.0)
    out, lse = run(pm, c)
    check(c, out, lse)
    out, lse = run(pm, c, scale=-0.05)
    check(c, out, lse, scale=-0.05)
    out, lse = run(pm, c, scale=0.0)
    check(c, out, lse, scale=0.0)


def test_many_requests_and_padded_layouts(pm):
    rng = np.random.default_rng(3)
    news = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 9, 40], 300)]
    lens = [n + int(x) for n, x in zip(news, rng.integers(0, 200, 300))]
    for window, sinks in ((0, 0), (50, 3)):
        c = make(5, news, lens, 8, 2, 64, 16, False, window, sinks, page_gap=128, q_gap=24, pad=9, first=4)
        poison_unseen(c)
        out, lse = run(pm, c)
        check(c, out, lse)


def test_more_requests_than_a_block_plans_at_once(pm):
    rng = np.random.default_rng(4)
    news = [int(x) for x in rng.choice([0, 1, 1, 2], 2300)]
    lens = [n + int(x) for n, x in zip(news, rng.integers(0, 20, 2300))]
    c = make(6, news, lens, 2, 1, 64, 16, False)
    out, lse = run(pm, c)
    check(c, out, lse)


def at_rows(c, rows):
    """The given rows as requests of one token each."""
    r = np.searchsorted(c["start"], rows, side="right") - 1
    lens = c["lens"][r] - (c["start"][r + 1] - 1 - np.asarray(rows))
    return {**c, "q": c["q"][up(np.asarray(rows))], "start": np.arange(len(rows) + 1, dtype=np.int32),
            "lens": lens.astype(np.int32), "table": c["table"][r]}


def test_more_row_tiles_than_a_block_plans_at_once(pm):
    for window in (0, 300):
        c = make(7, [4500, 1, 4], [4500, 300, 4], 64, 1, 64, 64, False, window=window, sinks=2)
        out, lse = run(pm, c)
        rows = list(range(0, 4500, 150)) + [4499, 4500, 4501, 4504]
        check(at_rows(c, rows), out[rows], lse[rows])


def test_rows_before_the_first_key(pm):
    """More new tokens than keys: the first ones see nothing."""
    for e4m3 in (False, True):
        c = make(8, [1, 70, 300, 5], [0, 40, 20, 5], 8, 2, 128, 16, e4m3)
        poison_unseen(c)
        out, lse = run(pm, c)
        check(c, out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_a_value_reaches_the_rows_that_see_it_alone(pm, e4m3, D):
    """NaN and infinities among the values of a piece's own tokens, at a window's lower edge, and in another
    request."""
    kinds = [float("nan")] if e4m3 else [float("nan"), float("inf")]
    for bad in kinds:
        for window, sinks in ((0, 0), (90, 5)):
            c = make(9, [200, 1, 3], [500, 300, 10], 8, 2, D, 16, e4m3, window, sinks)
            poisons = [(0, 350, 1), (0, 480, 0), (0, 3, 1), (0, 280, 0)]
            page = 16
            for r, j, h in poisons:
                at = (int(c["table"][r][j // page]), h, j % page, 5 + j % 50)
                if e4m3:
                    bits(c["v"])[at] = 0x7f
                else:
                    c["v"][at] = bad
            out, lse = run(pm, c)
            clean = {**c, "v": c["v"].clone()}
            for r, j, h in poisons:
                bits(clean["v"])[int(c["table"][r][j // page]), h, j % page, 5 + j % 50] = 0
            got, hit = f64(out), np.zeros(out.shape, bool)
            for t in range(200):
                p = 300 + t
                for r, j, h in poisons:
                    if j <= p and (not window or j > p - window or j < sinks):
                        hit[t, h * 4:(h + 1) * 4, 5 + j % 50] = True
            assert not np.isfinite(got[hit]).any()
            if not e4m3 and np.isinf(bad):
                assert np.all(got[hit] == np.inf)
            want, _ = run(pm, clean)
            assert np.array_equal(got[~hit], f64(want)[~hit])
            check(clean, want, lse)


@pytest.mark.parametrize("news,lens", [([1, 1, 1], [300, 40, 100]), ([100, 1, 90], [300, 40, 100])])
def test_bad_pages_lengths_and_starts_are_reported(pm, news, lens):
    c = make(10, news, lens, 8, 1, 64, 16, False)
    good = {k: (x.copy() if isinstance(x, np.ndarray) else x) for k, x in c.items()}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    others = list(range(c["start"][1], c["start"][3]))
    for bad in (c["k"].shape[0], -1):
        c["table"][0][3] = bad
        err.zero_()
        out, lse = run(pm, c, err_out=err)
        assert int(err) == 64
        check(good, out, lse, rows=others)
    c = {k: (x.copy() if isinstance(x, np.ndarray) else x) for k, x in good.items()}
    c["lens"][0] = c["table"].shape[1] * 16 + 1
    err.zero_()
    out, lse = run(pm, c, err_out=err)
    assert int(err) & 128
    check(good, out, lse, rows=others)
    c["lens"][0] = -5
    err.zero_()
    out, lse = run(pm, c, err_out=err)
    assert int(err) == 128
    check(good, out, lse, rows=others)
    assert bool((out[:c["start"][1]] == 0).all())
    c = {k: (x.copy() if isinstance(x, np.ndarray) else x) for k, x in good.items()}
    c["start"][1] = 1 << 29  # beyond T: the first request has too many rows, the second none
    err.zero_()
    run(pm, c, err_out=err)
    assert int(err) & 128
    c["start"] = np.array([0, c["q"].shape[0], 0, c["q"].shape[0]], np.int32)  # goes back
    err.zero_()
    run(pm, c, err_out=err)
    assert int(err) & 128


@pytest.mark.parametrize("news,lens", [([1] * 40, [700] * 40), ([500, 1], [3000, 900])])
def test_same_bits_twice_on_another_stream_and_in_a_graph(pm, news, lens):
    c = make(11, news, lens, 16, 2, 128, 16, False, window=600, sinks=4)
    out, lse = run(pm, c)
    again, _ = run(pm, c)
    assert torch.equal(out, again)
    args = (c["k"], c["v"], c["q"], up(c["start"]), up(c["lens"]), up(c["table"]), 600, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = pm.moe_chunk_attention(*args, stream=s)
    s.synchronize()
    assert torch.equal(out, other)
    size = pm.moe_chunk_attention_scratch_bytes(c["k"], c["v"], c["q"].shape[0], 16, len(news))
    scratch = torch.empty(size, dtype=torch.uint8, device="cuda")
    held = torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pm.moe_chunk_attention(*args, out=held, scratch=scratch)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, held)
    # other lengths in the same tensors
    args[4].sub_(60)
    c["lens"] = c["lens"] - 60
    g.replay()
    want, lse = run(pm, c)
    assert torch.equal(held, want)
    check(c, want, lse)


@pytest.mark.parametrize("news", [[1, 1], [150, 3]])
def test_offsets_past_32_bits(pm, news):
    """Pages beyond 2^32 elements into the cache."""
    page, D, Hkv = 256, 128, 8
    pages = 2 ** 32 // (page * D * Hkv) + 3
    c = make(12, news, [200, 256], 32, 8, 128, 256, True)
    k = torch.zeros((pages, Hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    table = c["table"].copy()
    for i in range(2):
        p = int(c["table"][i][0])
        bits(k)[pages - 1 - i], bits(v)[pages - 1 - i] = bits(c["k"])[p], bits(c["v"])[p]
        table[i][0] = pages - 1 - i
    out, lse = run(pm, {**c, "k": k, "v": v, "table": table})
    check(c, out, lse)


def test_one_call_equals_calls_of_its_requests(pm):
    """The same requests in one call and one by one: another cut into runs, the same values to rounding."""
    c = make(13, [1, 80, 1, 400], [900, 800, 33, 1400], 16, 4, 64, 32, False, 300, 2)
    out, lse = run(pm, c)
    for r in range(4):
        t0, t1 = int(c["start"][r]), int(c["start"][r + 1])
        one = {**c, "q": c["q"][t0:t1], "start": np.array([0, t1 - t0], np.int32), "lens": c["lens"][r:r + 1],
               "table": c["table"][r:r + 1]}
        got, glse = run(pm, one)
        check(one, got, glse)
        check(one, out[t0:t1], lse[t0:t1])


def test_refusals(pm):
    c = make(14, [4, 2], [40, 20], 8, 2, 64, 16, False)
    args = (c["k"], c["v"], c["q"], up(c["start"]), up(c["lens"]), up(c["table"]))
    for more in (dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
                 dict(scratch=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(pm.PmoeError) as e:
            pm.moe_chunk_attention(*args, **more)
        assert e.value.status == pm.PMOE_EINVAL
    with pytest.raises(pm.PmoeError) as e:  # 130 query heads to a kv head
        pm.moe_chunk_attention(c["k"], c["v"], torch.zeros((4, 260, 64), dtype=torch.bfloat16, device="cuda"), *args[3:])
    assert e.value.status == pm.PMOE_EUNSUPPORTED
    with pytest.raises(AssertionError, match="q_start"):
        pm.moe_chunk_attention(*args[:3], args[3][:2], *args[4:])
    with pytest.raises(AssertionError, match="kv_len"):
        pm.moe_chunk_attention(*args[:4], args[4].long(), args[5])
    out = pm.moe_chunk_attention(c["k"], c["v"], c["q"][:0], *args[3:])
    assert out.shape == (0, 8, 64)
