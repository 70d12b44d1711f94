"""The cut of moe_chunk_attention's work into runs, compiled for the host: whole numbers against Python's."""

import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_expert_moe_gb300", "csrc")
SOURCE = """
#include "runs.h"
extern "C" long long start(long long units, int ctas, int c) { return pmoe::chunk::run_start(units, ctas, c); }
extern "C" int owner(long long units, int ctas, long long u) { return pmoe::chunk::cta_of(units, ctas, u); }
"""


@pytest.fixture(scope="module")
def runs(tmp_path_factory):
    d = tmp_path_factory.mktemp("runs")
    (d / "runs.cpp").write_text(SOURCE)
    out = str(d / "runs.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "runs.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.start.argtypes, lib.start.restype = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int], ctypes.c_longlong
    lib.owner.argtypes, lib.owner.restype = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong], ctypes.c_int
    return lib


# 2^33 units are 2^20 single tokens on 2^20 keys each, 2^39 are the most that the call's limits allow
@pytest.mark.parametrize("units", [1, 7, 152, 153, 1000, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 5, 3 * 2 ** 32 - 1, 2 ** 33, 2 ** 39])
@pytest.mark.parametrize("ctas", [1, 3, 152])
def test_runs_and_their_owners(runs, units, ctas):
    ctas = min(ctas, units)
    rng = random.Random(units)
    for c in range(ctas + 1):
        assert runs.start(units, ctas, c) == units * c // ctas
    at = {0, 1, 2, units - 1, units // 2} | {units * c // ctas + d for c in range(ctas) for d in (-1, 0, 1)}
    at |= {rng.randrange(units) for _ in range(200)} | {rng.randrange(min(units, 1 << 26)) for _ in range(200)}
    for u in at:
        if 0 <= u < units:
            c = ((u + 1) * ctas - 1) // units
            assert runs.owner(units, ctas, u) == c
            assert units * c // ctas <= u < units * (c + 1) // ctas
