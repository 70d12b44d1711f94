"""moe_router_select where fp32 has the order of two values wrong by more than their difference.

float64 computes each c = score + bias within 2^-53 of c and a few 2^-53 of the score: with biases of up
to 1,000 within 2^-43, a sum of two within 2^-41. All differences that decide something here are above
2^-38 (2^-48 with biases of up to 1: asserted), so that the ids have to be the oracle's.
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


def same_ids(pm, x, top_k, scoring, bias, least, **how):
    """least: what every margin has to be above, or the case says nothing."""
    x, bias = np.asarray(x, np.float32), np.asarray(bias, np.float32)
    want, _, margin = steps.router_select(x, top_k, scoring, bias, **how)
    assert margin.min() > least
    ids, _ = pm.moe_router_select(torch.from_numpy(x).cuda(), top_k, scoring=scoring, bias=torch.from_numpy(bias).cuda(), **how)
    assert np.array_equal(ids.cpu().numpy(), want)


def test_a_group_whose_two_best_cancel(pm):
    """fp32 has 1.000061 and 1 for the groups' sums, which are 1.000032 and 1.000044."""
    s = np.array([[3.2e-5, 0, 2.9e-5, 1.5e-5]])
    same_ids(pm, 4 * s, 1, "sigmoid", [1000, -1000, 1000, -1000], 1e-6, groups=2, top_groups=1, group_top=2)


@pytest.mark.parametrize("scoring,spread", [("sigmoid", 2e-4), ("softmax", 2e-2)])
@pytest.mark.parametrize("E,groups,top_groups", [(16, 4, 1), (64, 8, 3), (256, 8, 4), (160, 8, 2), (60, 4, 2), (1024, 32, 5)])
def test_groups_of_large_biases_of_both_signs(pm, scoring, spread, E, groups, top_groups):
    """Two experts of each group have biases B and -B, the others less: a group's sum is that of two
    scores, and fp32 has lost up to 2^-15 of each on the way."""
    rng = np.random.default_rng(E + groups)
    size = E // groups
    bias = np.full((groups, size), -3000.0)
    for g in range(groups):
        a, b = rng.permutation(size)[:2]
        bias[g, a] = 2.0 ** rng.uniform(4, 9.95)
        bias[g, b] = -np.float32(bias[g, a])
    x = rng.standard_normal((200, E)) * spread
    same_ids(pm, x, 2 * top_groups, scoring, bias.ravel(), 2.0 ** -38, groups=groups, top_groups=top_groups, group_top=2)


@pytest.mark.parametrize("E", [64, 256, 60])
def test_groups_of_the_lowest_and_infinite_biases(pm, E):
    """Experts that a bias of the type's lowest value or -inf takes out, with groups of nothing else."""
    rng = np.random.default_rng(E)
    lowest = float(np.finfo(np.float32).min)
    x = rng.standard_normal((50, E)) * 2
    for out in (lowest, -1e30, -np.inf):
        bias = rng.standard_normal(E) * 0.1
        bias.reshape(4, -1)[1] = out      # a group of none
        bias.reshape(4, -1)[2, 1:] = out  # of one
        bias[rng.integers(0, E // 4, 5)] = out
        x32, b32 = x.astype(np.float32), bias.astype(np.float32)
        for scoring in ("sigmoid", "softmax"):
            want, _, margin = steps.router_select(x32, 6, scoring, b32, 4, 2, 2)
            sure = margin > 2.0 ** -48
            assert sure.mean() > 0.9
            ids, _ = pm.moe_router_select(torch.from_numpy(x32).cuda(), 6, scoring=scoring, bias=torch.from_numpy(b32).cuda(),
                                          groups=4, top_groups=2, group_top=2)
            assert np.array_equal(ids.cpu().numpy()[sure], want[sure])


@pytest.mark.parametrize("top_k", [1, 3, 8])
@pytest.mark.parametrize("E,at", [(512, 256), (512, 0), (1024, 512), (1024, 992), (256, 128), (1000, 640)])
def test_an_expert_of_a_large_score_and_a_negative_bias(pm, E, at, top_k):
    """Softmax rows with nearly all of the sum at one expert, whose own c is off by more in fp32 than the c of
    the experts of small scores around it: it is told apart from each of them, not from its neighbours alone."""
    low = np.float32(-11.2463)  # its exponential is 109.5 times 2^-23: added to 1, each one is off by half of that
    x = np.full((3, E), low)
    x[:, at] = 0
    e = np.exp(x[0].astype(np.float64))
    score = e / e.sum()
    first, second = (2, 1) if at == 0 else (1, E - 1)
    for gap in (3e-7, 5e-7, 7e-7, 1e-6, 2e-6):
        for ahead in (2e-7, 5e-7, 8e-7, -2e-7, -5e-7, -8e-7):
            bias = np.full(E, -1.0)
            others = [i for i in range(3, 200) if i not in (at, first, second)][:top_k - 1]
            bias[others] = np.linspace(1, 0.5, len(others))
            bias[first] = 0.01
            bias[second] = 0.01 - gap
            bias[at] = np.float32(0.01) + score[first] + ahead - score[at]
            same_ids(pm, x, top_k, "softmax", bias, 2.0 ** -48)


@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_of_one_expert_whose_scores_are_equal_in_64_bits(pm, group_top):
    """Without a bias the logits decide, also where a group's value is a single score: 1 for 45 as for 50."""
    x = torch.tensor([[0.0, 45.0, 50.0, 48.0, -3.0, 60.0, 47.0, 44.0]], device="cuda")
    ids, _ = pm.moe_router_select(x, 2, scoring="sigmoid", groups=8, top_groups=3, group_top=group_top)
    assert ids.tolist() == [[5, 2]]
    assert steps.router_select(x.cpu().numpy(), 2, "sigmoid", None, 8, 3, group_top)[0].tolist() == [[5, 2]]
