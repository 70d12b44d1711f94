"""How exact moe_router_select's weights are where scores are small.

With u = 2^-24: an exponential is within 4 u (two units in the last place), a score of a sigmoid adds
1 u for the sum and 4 u for the quotient, each at most of itself: 9 u, with the scale 10 u. Softmax: the
difference of logits is taken without an error, so an exponential over the row's sum. That sum's terms are
off by 4 u and by 2.23 u of their exponents' arguments, whose mean is at most log(1024) = 7, and 10 u of adding:
30 u with the quotient, 36 u with the exponential and the product, 37 u with the scale. Renormalised: two of these
(the row's sum drops out of softmax: 6 u each), 5 u of adding, 4 u of the quotient and 1 u of the scale: 28 u and 22 u.
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


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E,k,low", [(64, 8, -30), (256, 8, -60), (256, 32, -66), (1024, 10, -80), (33, 33 - 1, -50)])
def test_weights_of_low_logits(pm, scoring, renormalize, E, k, low):
    """All logits low (of softmax: all but one, which the bias takes out)."""
    rng = np.random.default_rng(E + k)
    x = (rng.uniform(low - 6, low + 6, (100, E))).astype(np.float32)
    bias = np.zeros(E, np.float32)
    if scoring == "softmax":
        x[:, 3] = 5.0
        bias[3] = -np.inf
        if k == E - 1:
            bias[:] = np.arange(E) % 2
            bias[3] = -np.inf
    else:
        bias[::5] = 0.5
    want, ww, _ = steps.router_select(x, k, scoring, bias, renormalize=renormalize, scale=2.5)
    ids, w = pm.moe_router_select(torch.from_numpy(x).cuda(), k, scoring=scoring, bias=torch.from_numpy(bias).cuda(),
                                  renormalize=renormalize, scale=2.5)
    same = (ids.cpu().numpy() == want).all(1)  # (scores of 2^-90 beside a bias of 0.5 are equal in 64 bits)
    s = 1 / (1 + np.exp(-x.astype(np.float64)))
    if scoring == "softmax":
        e = np.exp(x.astype(np.float64) - x.max(1, keepdims=True))
        s = e / e.sum(1, keepdims=True)
    got = np.take_along_axis(s, ids.cpu().numpy().astype(np.int64), 1)
    if renormalize:
        got = got / got.sum(1, keepdims=True)
    u = {("sigmoid", False): 10, ("sigmoid", True): 28, ("softmax", False): 37, ("softmax", True): 22}[scoring, renormalize]
    assert np.all(np.abs(w.double().cpu().numpy() - 2.5 * got) <= u * 2.0 ** -24 * 2.5 * got + 2.0 ** -125)
    assert same.any() or scoring == "sigmoid"
