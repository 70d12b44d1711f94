"""moe_router_select against the float64 oracle.

The ids are those of float64 wherever two values that had to be told apart differ by more than
2^-48 (float64's own rounding of a score and a sum); rows below that are left out and are few. A
weight is a score (the exponential within 2^-21, a sum of up to 32 terms a lane and 5 exchanges
with 2^-24 each, a division) over a sum of up to 32 of them, times the scale: within 2^-17 of it.
"""

import numpy as np
import pytest

from oracle import router, steps

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


def check(pm, x, top_k, scoring, bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0, few=0.0, **more):
    ids, w = pm.moe_router_select(x, top_k, scoring=scoring, bias=bias, groups=groups, top_groups=top_groups,
                                  group_top=group_top, renormalize=renormalize, scale=scale, **more)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32 and ids.shape == w.shape == (x.shape[0], top_k)
    want, ww, margin = steps.router_select(x.float().cpu().numpy(), top_k, scoring, None if bias is None else bias.cpu().numpy(),
                                           groups, top_groups, group_top, renormalize, float(np.float32(scale)))
    sure = (margin > 2.0 ** -48) | (margin == 0)  # equal values: the lower id
    assert np.mean(~sure) <= few
    assert np.array_equal(ids.cpu().numpy()[sure], want[sure])
    assert np.all(np.abs(w.cpu().numpy().astype(np.float64) - ww)[sure] <= 2.0 ** -17 * np.abs(ww)[sure] + 1e-37)
    return ids, w


@pytest.mark.parametrize("T,E,k,groups,top_groups", [
    (1, 1, 1, 1, 1), (3, 8, 2, 1, 1), (5, 33, 5, 1, 1), (9, 60, 4, 4, 2), (17, 64, 8, 8, 3), (40, 128, 8, 1, 1),
    (33, 160, 6, 8, 3), (70, 256, 8, 8, 4), (8, 256, 32, 32, 4), (20, 384, 8, 1, 1), (6, 512, 10, 16, 2), (4, 1024, 32, 32, 1),
    (11, 96, 3, 3, 1), (5, 32, 32, 32, 32), (7, 30, 4, 30, 5)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased,group_top,bf16", [(True, 2, False), (False, 2, True), (True, 1, True), (False, 1, False)])
def test_selection_matches_oracle(pm, T, E, k, groups, top_groups, scoring, biased, group_top, bf16):
    rng = np.random.default_rng(T * 1000 + E)
    x = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32)).cuda()
    x = x.to(torch.bfloat16) if bf16 else x
    bias = torch.from_numpy((rng.standard_normal(E) * (0.1 if scoring == "sigmoid" else 0.02)).astype(np.float32)).cuda()
    check(pm, x, k, scoring, bias if biased else None, groups, top_groups, group_top, renormalize=T % 2 == 0, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_near_ties_are_decided_as_in_64_bits(pm, scoring):
    """Biases that cancel the scores' differences but for some 2^-26: fp32 cannot tell their order."""
    rng = np.random.default_rng(5)
    T, E = 64, 64
    x = (rng.standard_normal((1, E)) * 2).astype(np.float32)
    s = 1 / (1 + np.exp(-x.astype(np.float64))) if scoring == "sigmoid" else np.exp(x.astype(np.float64)) / np.exp(x.astype(np.float64)).sum()
    bias = (0.75 - s[0]).astype(np.float32)  # c = 0.75 within a rounding of the bias
    xs = torch.from_numpy(np.repeat(x, T, 0)).cuda()
    ids, _ = check(pm, xs, 8, scoring, torch.from_numpy(bias).cuda())
    assert bool((ids == ids[0]).all())
    check(pm, xs, 6, scoring, torch.from_numpy(bias).cuda(), groups=8, top_groups=2, group_top=2)


def test_equal_values_go_to_the_lower_id_and_group(pm):
    x = torch.zeros((3, 64), device="cuda")
    for scoring in ("softmax", "sigmoid"):
        ids, w = check(pm, x, 8, scoring)
        assert ids[0].tolist() == list(range(8))
        ids, _ = check(pm, x, 4, scoring, torch.zeros(64, device="cuda"), 8, 2, 2)
        assert ids[0].tolist() == [0, 1, 2, 3]
    x = -torch.zeros((1, 8), device="cuda")
    x[0, 3] = 0.0
    assert check(pm, x, 2, "softmax")[0].tolist() == [[0, 1]]


def test_infinite_and_nan_logits_and_biases(pm):
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[1.0, nan, 3.0, -inf, 2.0, 0.0, -1.0, 0.5], [-inf] * 8, [nan] * 8, [inf, 1.0, inf, 0.0, 2.0, 3.0, 4.0, 5.0],
                      [1.0, 2.0, -inf, -inf, -inf, -inf, -inf, -inf]], device="cuda")
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            check(pm, x, 3, scoring, renormalize=renormalize)
    bias = torch.tensor([0.0, 1.0, nan, 0.0, -inf, inf, 0.25, 0.0], device="cuda")
    for scoring in ("softmax", "sigmoid"):
        ids, w = pm.moe_router_select(x, 3, scoring=scoring, bias=bias)
        assert bool((ids[:, 0] == 5).all()) and not bool(((ids == 2) | (ids == 4)).any())
    x = torch.tensor([[100.0, -100.0, 90.0, -90.0, 80.0, -80.0, 0.0, 1e30]], device="cuda")
    check(pm, x, 8, "sigmoid")


def test_without_bias_or_groups_it_is_the_plain_router(pm):
    x = torch.randn((100, 128), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    ids, w = check(pm, x, 8, "softmax")
    want, ww = router.router_topk(x.cpu().numpy(), 8)
    assert np.array_equal(ids.cpu().numpy(), want) and np.abs(w.cpu().numpy() - ww).max() <= 2.0 ** -17
    plain_ids, plain_w = pm.moe_router_topk(x, 8)
    assert torch.equal(ids, plain_ids) and float((w - plain_w).abs().max()) <= 2.0 ** -17


def test_strided_rows_streams_and_graphs(pm):
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn((50, 301), generator=g, device="cuda")
    bias = torch.randn(256, generator=g, device="cuda") * 0.1
    x = wide[:, 17:273]
    how = dict(scoring="sigmoid", bias=bias, groups=8, top_groups=4, group_top=2, scale=2.5)
    ids, w = pm.moe_router_select(x, 8, **how)
    want, ww = pm.moe_router_select(x.contiguous(), 8, **how)
    assert torch.equal(ids, want) and torch.equal(w, ww)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids, w = pm.moe_router_select(x, 8, stream=s, **how)
    s.synchronize()
    assert torch.equal(ids, want) and torch.equal(w, ww)
    ids.zero_(), w.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pm.moe_router_select(x, 8, ids_out=ids, w_out=w, **how)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, want) and torch.equal(w, ww)
    empty, _ = pm.moe_router_select(x[:0], 8, **how)
    assert empty.shape == (0, 8)


def test_refusals(pm):
    x = torch.zeros((2, 64), device="cuda")
    for change in (dict(top_k=0), dict(top_k=33), dict(groups=5), dict(groups=64), dict(groups=8, top_groups=9),
                   dict(groups=8, top_groups=1, top_k=9), dict(group_top=3), dict(scale=float("inf")), dict(top_groups=0)):
        with pytest.raises(pm.PmoeError) as e:
            pm.moe_router_select(x, **{"top_k": 4, **change})
        assert e.value.status == pm.PMOE_EINVAL
    for change, name in ((dict(bias=x[0, :63]), "bias"), (dict(bias=x[0].double()), "bias"), (dict(scoring="relu"), "scoring"),
                         (dict(logits=x.t()), "logits"), (dict(logits=x.half()), "logits"), (dict(w_out=x), "w_out")):
        with pytest.raises(AssertionError, match=name):
            pm.moe_router_select(**{"logits": x, "top_k": 4, **change})
