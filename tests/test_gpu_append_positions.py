"""moe_kv_append at positions an int32 can hold, not only those a float can.

Tolerance: as in test_gpu_kv_append an output is one rounding of an fp32 value that is off by at
most 2^-20 of |a| + |b| of its pair, and by the error of the angle: the position goes into two
floats and the product into two, whose low part, at most |angle| 2^-23, is rounded twice: 2^-46
|angle|. The float64 product position * inv_freq is off by 2^-53 |angle| itself.
"""

import numpy as np
import pytest

from oracle import attention as oatt
from tests import _harness as hz
from tests.test_gpu_kv_append import case, rounded, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


@pytest.mark.parametrize("D,rot,interleaved,axes", [(128, 128, False, 1), (64, 32, True, 1), (64, 64, False, 3)])
def test_rotation_at_large_positions(pm, D, rot, interleaved, axes):
    special = np.array([2 ** 17 + 1, 2 ** 20 + 7, -2 ** 20 - 7, 2 ** 22 - 1, 5000011, 2 ** 24 - 1, 2 ** 24 + 1, 2 ** 24 + 3,
                        -2 ** 24 - 1, 2 ** 27 + 13, 10 ** 9 + 7, 2 ** 30 + 1, 2 ** 31 - 1, 2 ** 31 - 65, -2 ** 31,
                        -2 ** 31 + 1], np.int64).astype(np.int32)
    rng = np.random.default_rng(D + rot)
    c = case(rng, len(special), 4, 2, D, 16, False, rot, axes, interleaved, False)
    c["pos"] = np.stack([np.roll(special, i) for i in range(axes)])
    c["freq"] = (1.0 / (1.0 + 0.37 * np.arange(rot // 2))).astype(np.float32)
    got = hz.bf16_to_f64(run(pm, c))
    want = oatt.turn_heads(c["ref"][0], c["pos"], c["freq"], c["pair_axis"], c["interleaved"])
    angle = np.abs(c["pos"].astype(np.float64)).max(axis=0)[:, None, None]
    eps = (2.0 ** -20 + (2.0 ** -46 + 2.0 ** -53) * angle) * 2 * np.abs(want).max(axis=-1, keepdims=True) * 2
    assert np.all(rounded(want - eps, torch.bfloat16) <= got) and np.all(got <= rounded(want + eps, torch.bfloat16))
