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
