"""moe_prefix_attention's plan, which is made on the host and needs no GPU."""

import ctypes

import numpy as np
import pytest


class Plan(ctypes.Structure):
    _fields_ = [("scratch_bytes", ctypes.c_uint64), ("scratch_bound", ctypes.c_uint64)] + \
        [(n, ctypes.c_int32) for n in ("cluster", "tc_ctas", "prefix_parts", "suffix_parts", "join_warps")]


def plan(T, Hq, Hkv, D, page, e4m3, prefix, suffix, sms=152):
    import paged_expert_moe_gb300 as pm
    lib = pm.load()
    d = pm._lib.pmoe_kv_desc(0x10000, 0x20000, Hkv * page * D, 0x30000, 0x40000, 4, page, Hkv, D, int(e4m3))
    p = Plan()
    assert lib.pmoe_attention_plan(ctypes.byref(d), T, Hq, prefix, suffix, sms, ctypes.byref(p)) == 0
    return p


def test_fewer_rows_may_need_more_scratch():
    """Why the size of a call is no bound for smaller ones."""
    need = {T: plan(T, 32, 4, 128, 16, False, 100003, 256).scratch_bytes for T in (2, 8)}
    assert need[2] > need[8]


@pytest.mark.parametrize("sms", [152, 132, 16])
def test_the_bound_holds_for_every_smaller_call(sms):
    rng = np.random.default_rng(sms)
    log = lambda hi: int(2 ** rng.uniform(0, np.log2(hi + 1)))  # noqa: E731
    for _ in range(3000):
        Hkv = int(rng.choice([1, 2, 3, 4, 8, 16]))
        Hq = Hkv * int(rng.choice([1, 2, 4, 5, 7, 8, 12, 16, 17, 33, 48, 64]))
        D, e4m3 = int(rng.choice([64, 128])), bool(rng.integers(2))
        T, prefix, suffix = log(5000), log(200000) - 1, log(40000) - 1
        most = plan(T, Hq, Hkv, D, 16, e4m3, prefix, suffix, sms).scratch_bound
        for _ in range(6):
            t, p, s = log(T), int(rng.integers(prefix + 1)), int(rng.integers(suffix + 1))
            small = plan(t, Hq, Hkv, D, 16, e4m3, p, s, sms)
            assert small.scratch_bytes <= small.scratch_bound <= most, (Hq, Hkv, D, T, prefix, suffix, t, p, s)


def test_every_batch_below_a_size_fits_its_bound():
    for prefix, suffix, Hq, Hkv, D in ((1000, 64, 32, 4, 128), (8192, 512, 32, 4, 128), (100003, 256, 32, 4, 128),
                                       (0, 4096, 16, 1, 64), (30000, 0, 8, 8, 64), (5000, 5000, 48, 1, 128)):
        most = plan(512, Hq, Hkv, D, 16, False, prefix, suffix).scratch_bound
        assert all(plan(T, Hq, Hkv, D, 16, False, prefix, suffix).scratch_bytes <= most for T in range(1, 513))


# T, Hq, Hkv, D, page, e4m3, prefix, suffix of test_gpu_attention_paths, by what they have to reach
LARGE_GROUPS = [(3, 64, 2, 128, 128, False, 900, 5000), (70, 60, 1, 64, 16, True, 100, 300), (60, 40, 1, 128, 16, True, 300, 600)]
MANY_PARTS = [(1, 16, 4, 128, 16, False, 30001, 100), (2, 32, 4, 64, 32, True, 30000, 256), (1, 1, 1, 64, 16, False, 0, 60000),
              (2, 5, 1, 128, 64, False, 0, 33333), (3, 4, 4, 64, 16, True, 0, 9000)]
TWO_ROUNDS = [(1, 8, 1, 64, 16, False, 100000, 40), (2, 8, 1, 128, 16, True, 40000, 0)]
TC_MANY_PARTS = [(16, 16, 1, 128, 16, False, 20000, 30), (32, 8, 1, 64, 64, True, 20011, 0), (16, 16, 1, 64, 32, True, 12000, 300)]
TC_LARGE_GROUP = [(5, 64, 1, 128, 16, False, 20000, 64)]
TC_ROW_BLOCKS = [(2100, 2, 1, 64, 16, False, 700, 5), (2050, 4, 2, 128, 32, True, 600, 20), (4100, 1, 1, 64, 16, False, 2000, 3)]
ALL_PATHS = LARGE_GROUPS + MANY_PARTS + TWO_ROUNDS + TC_MANY_PARTS + TC_LARGE_GROUP + TC_ROW_BLOCKS


def parts(p):
    return p.prefix_parts + p.suffix_parts


def test_the_sizes_reach_their_paths():
    for c in LARGE_GROUPS:  # several 16-row items of a token and kv head, in parts of the stream kernel
        p = plan(*c)
        assert p.cluster == 0 and p.tc_ctas == 0 and c[1] // c[2] > 16 and p.suffix_parts > 1 and p.prefix_parts > 1
    for c in MANY_PARTS + TWO_ROUNDS:
        p = plan(*c)
        assert p.cluster == 0 and p.tc_ctas == 0 and parts(p) > 64 and p.join_warps == 16
    for c in TWO_ROUNDS:  # a lane of the join looks at more than one part
        assert parts(plan(*c)) > 32 * 16
    for c in TC_MANY_PARTS:
        p = plan(*c)
        assert p.tc_ctas > 0 and parts(p) > 64 and p.join_warps == 16
    for c in TC_LARGE_GROUP:
        assert plan(*c).tc_ctas > 0 and c[1] // c[2] > 16
    for c in TC_ROW_BLOCKS:  # more rows than one launch of the stream kernel takes
        assert plan(*c).tc_ctas > 0 and c[0] > 2048 and c[7] > 0
