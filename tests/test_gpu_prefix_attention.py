"""moe_prefix_attention against the float64 oracle: sizes, layouts, empty rows, stale cache.

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

from oracle import attention as oatt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def make(seed, T, Hq, Hkv, D, page, e4m3, prefix, suffix, lens=None, seqs=None, qscale=2.0, page_gap=0, q_gap=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    n_prefix, per = -(-prefix // page), -(-suffix // page)
    S = T if seqs is None else seqs
    pages = n_prefix + S * per + 2
    order = rng.permutation(pages).astype(np.int32)
    caches = []
    for _ in range(2):
        x = torch.randn((pages, Hkv * page * D + page_gap), generator=g, device="cuda")
        x = (x * 64).to(torch.float8_e4m3fn) if e4m3 else x.to(torch.bfloat16)
        caches.append(x[:, :Hkv * page * D].unflatten(1, (Hkv, page, D)))
    scales = [torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2)] if e4m3 else [None, None]
    q = (torch.randn((T, Hq * D + q_gap), generator=g, device="cuda") * qscale).to(torch.bfloat16)
    q = q[:, :Hq * D].unflatten(1, (Hq, D))
    if lens is None:
        lens = rng.integers(0, suffix + 1, T) if suffix else np.zeros(T)
    return dict(k=caches[0], v=caches[1], ks=scales[0], vs=scales[1], q=q, prefix=prefix, suffix=suffix,
                pp=order[:n_prefix], pt=order[n_prefix:n_prefix + S * per].reshape(S, per),
                lens=np.asarray(lens, np.int32), row_seq=None if seqs is None else rng.integers(0, seqs, T).astype(np.int32))


def poison_unseen(c):
    """NaN into every cache row that no query row sees."""
    page = c["k"].shape[2]
    seen = torch.zeros((c["k"].shape[0], page), dtype=torch.bool)
    for j in range(c["prefix"]):
        seen[c["pp"][j // page], j % page] = True
    for t, n in enumerate(c["lens"]):
        row = c["pt"][t if c["row_seq"] is None else c["row_seq"][t]]
        for j in range(n):
            seen[row[j // page], j % page] = True
    for x in (c["k"], c["v"]):
        bits = x.view(torch.uint8 if x.dtype == torch.float8_e4m3fn else torch.int16)
        bits[(~seen).cuda()[:, None, :].expand(x.shape[:3])] = 0x7f if x.dtype == torch.float8_e4m3fn else 0x7fc0


def run(pm, c, **more):
    up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    out = pm.moe_prefix_attention(c["k"], c["v"], c["q"], up(c["pp"]), c["prefix"], up(c["pt"]), up(c["lens"]), c["suffix"],
                                  row_seq=up(c["row_seq"]), k_scale=c["ks"], v_scale=c["vs"], lse_out=lse, **more)
    return out, lse


def to_bf16(x):
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
    return np.rint(x / 2.0 ** (e - 7)) * 2.0 ** (e - 7)


def check(c, out, lse, scale=None, rows=None):
    D = c["q"].shape[2]
    f64 = lambda x: x.detach().float().cpu().numpy().astype(np.float64)  # noqa: E731
    k, v, q = f64(c["k"]), f64(c["v"]), f64(c["q"])
    if c["ks"] is not None:
        k, v = k * f64(c["ks"])[:, None, None], v * f64(c["vs"])[:, None, None]
    scale = D ** -0.5 if scale is None else scale
    ref, rlse, mag = oatt.prefix_attention(k, v, q, c["pp"], c["prefix"], c["pt"], c["lens"], scale, c["row_seq"])
    kmax = np.nan_to_num(np.abs(k)).max()
    vmax = np.nan_to_num(np.abs(v)).max()
    ds = (D + 8) * 2.0 ** -24 * abs(scale) * np.abs(q).sum(-1) * kmax
    n = (c["prefix"] + c["lens"])[:, None] * np.ones(q.shape[:2])
    r = 2.0 ** -8 if c["ks"] is None else 2.0 ** -11
    tol = (r + 2 * ds + 2.0 ** -20 + 2 * n * 2.0 ** -24)[..., None] * mag
    if c["ks"] is not None:
        tol += n[..., None] * 2.0 ** -25 * vmax
    got, glse = f64(out), f64(lse)
    sel = slice(None) if rows is None else rows
    assert np.all(to_bf16(ref - tol)[sel] <= got[sel]) and np.all(got[sel] <= to_bf16(ref + tol)[sel])
    empty = np.isinf(rlse)
    assert np.array_equal(np.isneginf(glse)[sel], empty[sel])
    fine = ~empty
    if rows is not None:
        keep = np.zeros_like(fine)
        keep[rows] = True
        fine &= keep
    ltol = ds + 2.0 ** -20 + n * 2.0 ** -24
    assert np.all(np.abs(glse[fine] - rlse[fine]) <= (ltol[fine] + 2.0 ** -22 * np.abs(rlse[fine])))
    assert np.all(got[empty] == 0)


SIZES = [
    # T, Hq, Hkv, D, page, e4m3, prefix, suffix
    (1, 1, 1, 64, 16, False, 1, 0),
    (1, 1, 1, 128, 16, True, 0, 1),
    (1, 32, 4, 128, 16, False, 17, 5),
    (3, 8, 8, 64, 32, False, 63, 65),
    (4, 32, 4, 128, 16, False, 500, 64),
    (5, 16, 1, 128, 64, True, 129, 200),
    (7, 40, 8, 64, 32, True, 1001, 77),
    (2, 48, 2, 64, 16, False, 300, 130),
    (2, 64, 1, 128, 128, True, 260, 33),
    (2, 60, 1, 64, 16, True, 100, 33),
    (17, 12, 2, 128, 256, False, 700, 300),
    (33, 16, 2, 64, 16, True, 257, 20),
    (47, 40, 8, 64, 32, True, 345, 77),
    (40, 8, 1, 128, 64, False, 1000, 64),
    (130, 8, 1, 128, 16, False, 3000, 5),
    (70, 8, 2, 128, 16, True, 640, 16),
    (64, 16, 1, 64, 128, False, 999, 0),
    (131, 4, 2, 128, 32, False, 385, 40),
    (9, 32, 4, 128, 16, False, 0, 50),
    (130, 7, 7, 64, 16, False, 130, 3),
    # enough rows and keys for the tensor-core kernel
    (300, 16, 2, 128, 16, False, 1000, 20),
    (300, 16, 2, 64, 32, True, 1100, 20),
    (257, 8, 1, 128, 64, True, 900, 0),
    (520, 4, 2, 64, 128, False, 900, 33),
    (1100, 2, 1, 128, 256, False, 641, 17),
    (290, 10, 1, 128, 16, True, 1281, 9),
    # rows beyond one block of the stream kernel
    (2050, 1, 1, 64, 16, False, 5, 3),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,page,e4m3,prefix,suffix", SIZES)
def test_attention_matches_oracle(pm, T, Hq, Hkv, D, page, e4m3, prefix, suffix):
    c = make(T * 7 + prefix + D, T, Hq, Hkv, D, page, e4m3, prefix, suffix)
    if suffix:
        c["lens"][0] = 0
        c["lens"][-1] = suffix
    poison_unseen(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(pm, c, err_out=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(c, out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hq", [(2, 8), (40, 16), (300, 16)])
def test_peaked_and_shifted_scores(pm, e4m3, T, Hq):
    """Large scores of either sign: the running maximum moves far between tiles."""
    c = make(77, T, Hq, 2, 128, 16, e4m3, 900, 200, qscale=30.0)
    out, lse = run(pm, c)
    check(c, out, lse)
    out, lse = run(pm, c, scale=-0.05)
    check(c, out, lse, scale=-0.05)


@pytest.mark.parametrize("T,prefix", [(12, 100), (400, 1300)])
def test_rows_share_sequences_and_padded_layouts(pm, T, prefix):
    c = make(5, T, 8, 2, 64, 16, False, prefix, 90, seqs=3, page_gap=128, q_gap=24)
    out, lse = run(pm, c)
    check(c, out, lse)


def test_no_visible_key(pm):
    c = make(6, 5, 8, 2, 128, 16, False, 0, 40, lens=[0, 40, 0, 1, 0])
    poison_unseen(c)
    out, lse = run(pm, c)
    check(c, out, lse)
    c = make(6, 5, 8, 2, 128, 16, False, 0, 0)
    out, lse = run(pm, c)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_a_row_is_not_touched_by_other_rows_values(pm):
    """NaN and infinities in one sequence's own pages reach that sequence alone."""
    for value in (float("nan"), float("inf")):
        c = make(7, 6, 16, 2, 64, 16, False, 200, 64, lens=[64, 30, 64, 5, 0, 64])
        page = int(c["pt"][2][1])
        c["v"][page, :, 3] = value
        out, lse = run(pm, c)
        check({**c, "v": torch.nan_to_num(c["v"], nan=0.0, posinf=0.0)}, out, lse, rows=[0, 1, 3, 4, 5])
        assert not bool(torch.isfinite(out[2]).any())


@pytest.mark.parametrize("T", [2, 40])
def test_bad_pages_lengths_and_rows_are_reported(pm, T):
    c = make(8, T, 8, 1, 64, 16, False, 300, 64)
    c["lens"][:] = 64
    good = {k: (x.copy() if isinstance(x, np.ndarray) else x) for k, x in c.items()}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c["pt"][1][2] = c["k"].shape[0]
    out, lse = run(pm, c, err_out=err)
    assert int(err) == 64
    check(good, out, lse, rows=[i for i in range(T) if i != 1])
    c["pt"][1][2] = -1
    c["lens"][0] = 65
    out, lse = run(pm, c, err_out=err)
    assert int(err) == 64 | 128
    check(good, out, lse, rows=[i for i in range(T) if i != 1])
    c = {k: (x.copy() if isinstance(x, np.ndarray) else x) for k, x in good.items()}
    c["pp"][7] = -3
    err.zero_()
    run(pm, c, err_out=err)
    assert int(err) == 64
    c = {**good, "row_seq": np.arange(T, dtype=np.int32)}
    c["row_seq"][1] = T
    err.zero_()
    out, lse = run(pm, c, err_out=err)
    assert int(err) == 64
    check(good, out, lse, rows=[i for i in range(T) if i != 1])


@pytest.mark.parametrize("prefix", [300, 8000])
def test_same_bits_twice_on_another_stream_and_in_a_graph(pm, prefix):
    c = make(9, 40, 16, 2, 128, 16, False, prefix, 100)
    out, lse = run(pm, c)
    again, _ = run(pm, c)
    assert torch.equal(out, again)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    args = (c["k"], c["v"], c["q"], up(c["pp"]), c["prefix"], up(c["pt"]), up(c["lens"]), c["suffix"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = pm.moe_prefix_attention(*args, stream=s)
    s.synchronize()
    assert torch.equal(out, other)
    scratch = torch.empty(pm.moe_prefix_attention_scratch_bytes(c["k"], c["v"], 40, 16, prefix, 100), dtype=torch.uint8,
                          device="cuda")
    held = torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pm.moe_prefix_attention(*args, out=held, scratch=scratch)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, held)


@pytest.mark.parametrize("T", [40, 160])
def test_offsets_past_32_bits(pm, T):
    """Pages beyond 2^32 elements into the cache, in the prefix and the suffix."""
    page, D, Hkv = 256, 128, 8
    pages = 2 ** 32 // (page * D * Hkv) + 3
    c = make(10, T, 32, 8, 128, 256, True, 256, 256, lens=[200] * T, seqs=2)
    k = torch.zeros((pages, Hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    far = {}
    for i, p in enumerate([int(c["pp"][0]), int(c["pt"][0][0]), int(c["pt"][1][0])]):
        far[p] = pages - 1 - i
        k[far[p]], v[far[p]] = c["k"][p], c["v"][p]
    big = {**c, "k": k, "v": v, "pp": np.array([far[int(c["pp"][0])]], np.int32),
           "pt": np.array([[far[int(x[0])]] for x in c["pt"]], np.int32)}
    out, lse = run(pm, big)
    check(c, out, lse)


def test_a_bad_prefix_page_is_reported_by_the_tensor_core_kernel(pm):
    for e4m3 in (False, True):
        c = make(12, 300, 16, 2, 128, 16, e4m3, 1000, 20)
        c["pp"][7] = c["k"].shape[0]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        run(pm, c, err_out=err)
        assert int(err) == 64


def test_attention_refusals(pm):
    c = make(11, 4, 8, 2, 64, 16, False, 40, 20)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    args = (c["k"], c["v"], c["q"], up(c["pp"]), 40, up(c["pt"]), up(c["lens"]))
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_prefix_attention(*args, 64)  # the table has two pages a row
    assert e.value.status == pm.PMOE_EINVAL
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_prefix_attention(*args, 20, scratch=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pm.PMOE_EINVAL
    with pytest.raises(pm.PmoeError) as e:  # 130 query heads to a kv head
        pm.moe_prefix_attention(c["k"], c["v"], torch.zeros((4, 260, 64), dtype=torch.bfloat16, device="cuda"), *args[3:], 20)
    assert e.value.status == pm.PMOE_EUNSUPPORTED
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_prefix_attention(*args, 20, scale=float("nan"))
    assert e.value.status == pm.PMOE_EINVAL
    out = pm.moe_prefix_attention(c["k"], c["v"], c["q"][:0], args[3], 40, args[5], args[6][:0], 20)
    assert out.shape == (0, 8, 64)


@pytest.mark.parametrize("T,Hq,Hkv,D,page,e4m3,prefix,suffix", [
    # one CTA an item; clusters of 2, 4 and 8, with less than a tile a warp and with several
    (3, 32, 4, 128, 16, False, 0, 33), (20, 12, 4, 64, 32, True, 60, 60), (14, 8, 4, 128, 16, True, 500, 40),
    (8, 40, 4, 64, 64, False, 1500, 70), (5, 64, 2, 128, 128, False, 700, 300), (1, 8, 1, 128, 16, False, 6000, 100),
    (2, 16, 2, 64, 32, True, 3000, 200), (1, 48, 1, 128, 256, True, 250, 1)])
def test_short_calls_without_parts(pm, T, Hq, Hkv, D, page, e4m3, prefix, suffix):
    c = make(T + prefix, T, Hq, Hkv, D, page, e4m3, prefix, suffix)
    c["lens"][0] = 0
    c["lens"][-1] = suffix
    poison_unseen(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(pm, c, err_out=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(c, out, lse)
