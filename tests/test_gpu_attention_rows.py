"""moe_prefix_attention with a table row or a prefix page out of range: its keys count as zeros, on
every path, and no other sequence's pages are read in their place."""

import numpy as np
import pytest

from tests.test_gpu_prefix_attention import check, make, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_expert_moe_gb300 as pm
    pm.load()
    return pm


PATHS = [(3, 16, 2, 64, 16, True, 100, 33), (2, 16, 2, 128, 32, False, 1500, 40), (40, 16, 2, 128, 16, False, 385, 200),
         (300, 16, 2, 128, 16, True, 1000, 20), (300, 16, 2, 64, 64, False, 1100, 70)]


def zeroed_page(c):
    """A page that nothing refers to, filled with zeros."""
    used = set(c["pp"].tolist()) | set(c["pt"].ravel().tolist())
    spare = next(p for p in range(c["k"].shape[0]) if p not in used)
    for x in (c["k"], c["v"]):
        x[spare] = torch.zeros((), dtype=x.dtype, device="cuda")
    return spare


@pytest.mark.parametrize("T,Hq,Hkv,D,page,e4m3,prefix,suffix", PATHS + [(2, 8, 1, 64, 16, False, 0, 40)])
@pytest.mark.parametrize("bad", ["beyond", -1, -2 ** 31, 2 ** 31 - 1])
def test_keys_of_a_bad_table_row_are_zeros(pm, T, Hq, Hkv, D, page, e4m3, prefix, suffix, bad):
    c = make(T + prefix, T, Hq, Hkv, D, page, e4m3, prefix, suffix, lens=[suffix] * T)
    spare = zeroed_page(c)
    c["row_seq"] = np.arange(T, dtype=np.int32)
    want = {**c, "pt": c["pt"].copy(), "row_seq": c["row_seq"].copy()}
    want["pt"][1] = spare
    c["row_seq"][1] = T if bad == "beyond" else bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(pm, c, err_out=err)
    assert int(err) == 64
    check(want, out, lse)


@pytest.mark.parametrize("T,Hq,Hkv,D,page,e4m3,prefix,suffix", PATHS)
@pytest.mark.parametrize("bad", ["beyond", -1])
def test_keys_of_a_bad_prefix_page_are_zeros(pm, T, Hq, Hkv, D, page, e4m3, prefix, suffix, bad):
    c = make(T + prefix, T, Hq, Hkv, D, page, e4m3, prefix, suffix)
    want = {**c, "pp": c["pp"].copy()}
    want["pp"][[1, -1]] = zeroed_page(c)
    c["pp"][[1, -1]] = c["k"].shape[0] if bad == "beyond" else bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(pm, c, err_out=err)
    assert int(err) == 64
    check(want, out, lse)
