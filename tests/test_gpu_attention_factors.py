"""moe_prefix_attention where the factor of the scores is zero, negative or vanishes: e4m3 scales
of any sign, a softmax scale of zero, queries so small that the factor leaves fp32's range. The
answer is the formula's on every path, with prefixes that end inside a tile. Tolerances: those of
test_gpu_prefix_attention, whose score error is proportional to the factor.
"""

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


# a CTA an item; a cluster an item; parts of the stream kernel; the tensor-core kernel
PATHS = [(3, 16, 2, 64, 100, 33), (2, 16, 2, 128, 1500, 40), (40, 16, 2, 128, 385, 200), (300, 16, 2, 128, 1000, 20),
         (300, 16, 2, 64, 1100, 0)]


@pytest.mark.parametrize("T,Hq,Hkv,D,prefix,suffix", PATHS)
@pytest.mark.parametrize("k_scale", [(0.0, 0.013), (0.013, -0.02), (-0.011, 0.0), (-0.0, -3.0)])
def test_key_scales_of_any_sign(pm, T, Hq, Hkv, D, prefix, suffix, k_scale):
    c = make(T + prefix, T, Hq, Hkv, D, 16, True, prefix, suffix)
    c["ks"] = torch.tensor(k_scale, device="cuda")
    out, lse = run(pm, c)
    check(c, out, lse)
    out, lse = run(pm, c, scale=-0.07)
    check(c, out, lse, scale=-0.07)


@pytest.mark.parametrize("T,Hq,Hkv,D,prefix,suffix", PATHS)
@pytest.mark.parametrize("v_scale", [(0.0, 0.013), (0.013, -0.02)])
def test_value_scales_of_any_sign(pm, T, Hq, Hkv, D, prefix, suffix, v_scale):
    c = make(T + prefix, T, Hq, Hkv, D, 16, True, prefix, suffix)
    c["vs"] = torch.tensor(v_scale, device="cuda")
    out, lse = run(pm, c)
    check(c, out, lse)


@pytest.mark.parametrize("T,Hq,Hkv,D,prefix,suffix", PATHS)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("qscale", [2.0, 1e-30, 1e33])
def test_a_softmax_scale_of_zero_weighs_all_keys_alike(pm, T, Hq, Hkv, D, prefix, suffix, e4m3, qscale):
    c = make(T + prefix, T, Hq, Hkv, D, 16, e4m3, prefix, suffix, qscale=qscale)
    for scale in (0.0, -0.0):
        out, lse = run(pm, c, scale=scale)
        check(c, out, lse, scale=scale)


@pytest.mark.parametrize("T,Hq,Hkv,D,prefix,suffix", PATHS)
def test_scores_below_the_range_of_fp32(pm, T, Hq, Hkv, D, prefix, suffix):
    c = make(T + prefix, T, Hq, Hkv, D, 16, True, prefix, suffix, qscale=1e-36)
    c["ks"] = torch.tensor([1e-12, -1e-15], device="cuda")
    out, lse = run(pm, c)
    check(c, out, lse)
