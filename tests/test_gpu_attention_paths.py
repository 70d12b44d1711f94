"""moe_prefix_attention against the float64 oracle on the paths that the sizes of
test_gpu_prefix_attention, with the tolerances derived there, do not reach: groups of several
16-row items in parts, joins of many parts, row blocks behind the tensor-core kernel, bounds of
the own keys far above the lengths, launches that do not overlap. test_attention_plan holds the
sizes, and that they reach these paths.
"""

import os
import subprocess
import sys

import numpy as np
import pytest

from tests.test_attention_plan import ALL_PATHS
from tests.test_gpu_prefix_attention import check, make, poison_unseen, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


@pytest.mark.parametrize("T,Hq,Hkv,D,page,e4m3,prefix,suffix", ALL_PATHS)
def test_paths_match_oracle(pm, T, Hq, Hkv, D, page, e4m3, prefix, suffix):
    c = make(T * 3 + prefix + D, T, Hq, Hkv, D, page, e4m3, prefix, suffix)
    if suffix:
        c["lens"][0] = 0
        c["lens"][-1] = suffix
    poison_unseen(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(pm, c, err_out=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(c, out, lse)


@pytest.mark.parametrize("T,Hq,Hkv,D,page,e4m3,prefix,suffix", [
    (300, 16, 2, 128, 16, False, 1000, 20), (40, 16, 2, 128, 16, False, 385, 200), (4, 16, 2, 64, 16, True, 0, 64),
    (2, 8, 1, 64, 32, False, 100, 20), (70, 4, 4, 64, 16, True, 3000, 90)])
@pytest.mark.parametrize("bound", [500, 20000, 100000])
def test_loose_bounds_of_the_own_keys(pm, T, Hq, Hkv, D, page, e4m3, prefix, suffix, bound):
    """max_suffix above every length: the table's entries beyond the lengths are never used."""
    c = make(T + prefix, T, Hq, Hkv, D, page, e4m3, prefix, suffix)
    c["lens"][0] = 0
    poison_unseen(c)
    wide = np.full((T, -(-bound // page)), -1, np.int32)
    wide[:, :c["pt"].shape[1]] = c["pt"]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(pm, {**c, "pt": wide, "suffix": bound}, err_out=err)
    assert int(err) == 0
    check(c, out, lse)


def test_without_overlapping_launches():
    """PMOE_NO_PDL=1: every kernel waits for the one before it to end."""
    names = ["tests/test_gpu_kv_append.py::test_append_matches_oracle", "tests/test_gpu_sample.py::test_draws_match_oracle",
             "tests/test_gpu_prefix_attention.py::test_attention_matches_oracle", "tests/test_gpu_generate.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", *names], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), env={**os.environ, "PMOE_NO_PDL": "1"})
    assert r.returncode == 0, r.stdout[-3000:]
