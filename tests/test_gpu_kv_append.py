"""moe_kv_append against the float64 oracle: norms, rotations, layouts, skipped tokens.

Tolerance: an output is one rounding (to bf16 or e4m3, to nearest even) of an fp32 value
that is off by at most eps = 2^-20 of |a| + |b| of its pair: the norm's sum, square root and
products 2^-21, sine and cosine 2^-22 each, three roundings 2^-24 each, the angle's corrected
rounding (third order) below 2^-26 for positions up to 2^17. Rounding is monotonic, so the
output has to lie between the roundings of the float64 value - eps and + eps.
"""

import numpy as np
import pytest

from oracle import attention as oatt
from workloads import generators as gen
from tests import _harness as hz

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def bf16(rng, *shape, scale=1.0):
    bits = gen.bf16_bits(rng.standard_normal(shape) * scale)
    return hz.to_device_bf16(bits), gen.bf16_bits_to_float(bits).astype(np.float64)


def case(rng, T, Hq, Hkv, D, page, e4m3, rot, axes, interleaved, norm, max_pos=1 << 17, gap=0, page_gap=0):
    pages = -(-T // page) + 2
    width = (Hq + 2 * Hkv) * D + gap
    qkv, x = bf16(rng, T, width, scale=1.5)
    cut = [0, Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D]
    dev = [qkv[:, a:b].unflatten(1, (-1, D)) for a, b in zip(cut, cut[1:])]
    ref = [x[:, a:b].reshape(T, -1, D) for a, b in zip(cut, cut[1:])]
    raw = torch.randint(0, 100, (pages, Hkv * page * D + page_gap), device="cuda", dtype=torch.uint8)
    caches = []
    for _ in range(2):
        c = (raw.to(torch.float8_e4m3fn) if e4m3 else raw.to(torch.bfloat16)).clone()
        caches.append(c[:, :Hkv * page * D].unflatten(1, (Hkv, page, D)))
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    pos = rng.integers(0, max_pos, (axes, T)).astype(np.int32)
    pair_axis = rng.integers(0, axes, rot // 2).astype(np.int32) if axes > 1 else None
    freq = (10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
    scales = [(rng.random(Hkv) * 0.02 + 0.01).astype(np.float32) for _ in range(2)] if e4m3 else [None, None]
    norms = [gen.bf16_bits(rng.random(D) + 0.5) for _ in range(2)] if norm else None
    return dict(dev=dev, ref=ref, caches=caches, slots=slots, pos=pos, pair_axis=pair_axis, freq=freq, scales=scales,
                norms=norms, interleaved=interleaved)


def run(pm, c, **more):
    up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    n = [None, None] if c["norms"] is None else [hz.to_device_bf16(b) for b in c["norms"]]
    return pm.moe_kv_append(*c["caches"], *c["dev"], up(c["pos"]), up(c["slots"]), up(c["freq"]) if len(c["freq"]) else None,
                            pair_axis=up(c["pair_axis"]), interleaved=c["interleaved"], q_norm=n[0], k_norm=n[1],
                            k_scale=up(c["scales"][0]), v_scale=up(c["scales"][1]), **more)


def rounded(x, dtype):
    """float64 -> the nearest bf16 or e4m3 value, ties to even, saturating at 448 for e4m3."""
    bits, least = (8, -126) if dtype == torch.bfloat16 else (4, -6)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 1e-300))), least)
    y = np.rint(x / 2.0 ** (e - bits + 1)) * 2.0 ** (e - bits + 1)
    return y if dtype == torch.bfloat16 else np.clip(y, -448, 448)


def check(c, q_out, before):
    norms = [None, None] if c["norms"] is None else [gen.bf16_bits_to_float(b) for b in c["norms"]]
    turn = lambda x, w: oatt.turn_heads(x, c["pos"], c["freq"], c["pair_axis"], c["interleaved"], w)  # noqa: E731
    q, k, v = turn(c["ref"][0], norms[0]), turn(c["ref"][1], norms[1]), c["ref"][2]

    def eps(x):  # 2^-20 of |a| + |b|: at most twice the head's largest element
        return 2.0 ** -20 * 2 * np.abs(x).max(axis=-1, keepdims=True) + 0 * x

    got = hz.bf16_to_f64(q_out)
    assert np.all(rounded(q - 2 * eps(q), torch.bfloat16) <= got)
    assert np.all(got <= rounded(q + 2 * eps(q), torch.bfloat16))
    for cache, old, rows, scale in zip(c["caches"], before, (k, v), c["scales"]):
        new = cache.float().cpu().numpy().astype(np.float64)
        e = 2 * eps(rows)
        if scale is not None:
            s = scale.astype(np.float64)[:, None]
            rows, e = rows / s, e / s
        for sign in (1, -1):
            want = old.copy()
            oatt.append(want, rounded(rows + sign * e, cache.dtype), c["slots"])
            assert np.all(sign * want >= sign * new)


@pytest.mark.parametrize("T,Hq,Hkv,D,page,e4m3,rot,axes,inter,norm,gap", [
    (1, 32, 4, 128, 16, False, 128, 1, False, True, 0),
    (1, 1, 1, 64, 16, True, 64, 1, True, False, 0),
    (5, 6, 3, 64, 32, False, 32, 1, False, True, 8),
    (33, 8, 8, 128, 64, True, 128, 3, True, True, 0),
    (67, 40, 8, 64, 128, True, 48, 3, False, False, 16),
    (19, 16, 1, 128, 256, False, 16, 2, True, False, 0),
    (7, 3, 1, 128, 16, False, 0, 1, False, True, 0),
    (2049, 4, 2, 64, 16, False, 64, 1, False, True, 0),
    (3, 71, 1, 64, 16, False, 64, 1, False, True, 0),
])
def test_append_matches_oracle(pm, T, Hq, Hkv, D, page, e4m3, rot, axes, inter, norm, gap):
    rng = np.random.default_rng(T * 31 + D + rot)
    c = case(rng, T, Hq, Hkv, D, page, e4m3, rot, axes, inter, norm, gap=gap)
    c["slots"][rng.random(T) < 0.2] = -1
    before = [x.float().cpu().numpy().astype(np.float64) for x in c["caches"]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = run(pm, c, err_out=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(c, q_out, before)


def test_append_with_padded_pages_leaves_the_padding(pm):
    rng = np.random.default_rng(5)
    c = case(rng, 21, 4, 2, 64, 16, False, 64, 1, False, False, page_gap=64)
    whole = [x._base for x in c["caches"]]
    pad = [w[:, -64:].clone() for w in whole]
    before = [x.float().cpu().numpy().astype(np.float64) for x in c["caches"]]
    q_out = run(pm, c)
    check(c, q_out, before)
    assert all(torch.equal(w[:, -64:], p) for w, p in zip(whole, pad))


def test_bad_slots_and_axes_are_skipped_and_reported(pm):
    rng = np.random.default_rng(6)
    c = case(rng, 8, 4, 2, 64, 16, False, 32, 2, False, False)
    rows = c["caches"][0].shape[0] * 16
    c["slots"][[1, 4, 6]] = [rows, -2, 2 ** 31 - 1]
    before = [x.float().cpu().numpy().astype(np.float64) for x in c["caches"]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = run(pm, c, err_out=err)
    assert int(err) == 4
    check(c, q_out, before)
    c["pair_axis"][3] = 2
    run(pm, c, err_out=err)
    assert int(err) == 4 | 32
    c["pair_axis"][3] = 0  # what a bad axis counts as
    check(c, run(pm, c), before)


def test_offsets_past_32_bits(pm):
    """A cache of more than 2^32 elements: the last page's rows land where they should."""
    page, D, Hkv = 256, 128, 8
    pages = 2 ** 32 // (page * D * Hkv) + 2
    k = torch.empty((pages, Hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.empty_like(k)
    one = torch.ones(Hkv, device="cuda")
    slots = torch.tensor([pages * page - 1, (pages - 2) * page], dtype=torch.int32, device="cuda")
    x = torch.randint(-8, 9, (2, 3 * Hkv, D), device="cuda").to(torch.bfloat16)
    pm.moe_kv_append(k, v, x[:, :Hkv], x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:], None, slots, None, k_scale=one, v_scale=one)
    for t, (p, r) in enumerate(((pages - 1, page - 1), (pages - 2, 0))):
        assert torch.equal(k[p, :, r].float(), x[t, Hkv:2 * Hkv].float())
        assert torch.equal(v[p, :, r].float(), x[t, 2 * Hkv:].float())


def test_append_saturates_and_keeps_nan(pm):
    x = torch.zeros((1, 3, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 2, :4] = torch.tensor([1e30, -1e30, float("nan"), float("inf")])
    k = torch.zeros((1, 1, 16, 64), dtype=torch.float8_e4m3fn, device="cuda")
    v, one = torch.zeros_like(k), torch.ones(1, device="cuda")
    pm.moe_kv_append(k, v, x[:, :1], x[:, 1:2], x[:, 2:], None, torch.zeros(1, dtype=torch.int32, device="cuda"), None,
                     k_scale=one, v_scale=one)
    got = v[0, 0, 0, :4].float().cpu()
    assert got[0] == 448 and got[1] == -448 and torch.isnan(got[2]) and got[3] == 448


def test_append_on_another_stream_and_in_a_graph(pm):
    rng = np.random.default_rng(8)
    c = case(rng, 9, 8, 2, 128, 32, False, 128, 1, False, True)
    before = [x.float().cpu().numpy().astype(np.float64) for x in c["caches"]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q_out = run(pm, c, stream=s)
    s.synchronize()
    check(c, q_out, before)
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    args = (up(c["pos"]), up(c["slots"]), up(c["freq"]))
    out = torch.empty_like(q_out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pm.moe_kv_append(*c["caches"], *c["dev"], *args, q_out=out)
    g.replay()
    torch.cuda.synchronize()
    c["norms"] = None
    check(c, out, before)


def test_append_refusals(pm):
    rng = np.random.default_rng(9)
    c = case(rng, 4, 4, 2, 64, 16, False, 64, 1, False, False)
    with pytest.raises(pm.PmoeError) as e:  # an odd number of pairs per 16-byte vector
        pm.moe_kv_append(*c["caches"], *c["dev"], torch.zeros((1, 4), dtype=torch.int32, device="cuda"),
                         torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(5, device="cuda"))
    assert e.value.status == pm.PMOE_EINVAL
    small = [torch.zeros((2, 2, 8, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_kv_append(*small, *c["dev"], None, torch.zeros(4, dtype=torch.int32, device="cuda"), None)
    assert e.value.status == pm.PMOE_EUNSUPPORTED
    none = [x[:0] for x in c["dev"]]
    out = pm.moe_kv_append(*c["caches"], *none, None, torch.zeros(0, dtype=torch.int32, device="cuda"), None)
    assert out.shape == (0, 4, 64)
