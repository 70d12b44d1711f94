"""moe_adjust_logits against the float64 oracle.

A value goes through at most four fp32 operations, each off by 2^-24 of its result, whose
magnitude the oracle's running sum bounds: 4 x 2^-24 of that; a bf16 output rounds once more, to
within half a step, 2^-8 of it at most.
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


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make(seed, T, V, H=0, B=0, mask=None, bf16=False, scale=3.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((T, V)) * scale).astype(np.float32)).cuda()
    a = {}
    if H:
        a["history"] = (rng.random((T, H)) ** 2 * V).astype(np.int32)
        a["history_len"] = rng.integers(0, H + 1, T).astype(np.int32)
        a["history_len"][0] = H
        a["prompt_len"] = (rng.random(T) * a["history_len"]).astype(np.int32)
        a["repetition"] = rng.uniform(0.8, 1.4, T).astype(np.float32)
        a["frequency"] = rng.uniform(-0.3, 0.6, T).astype(np.float32)
        a["presence"] = rng.uniform(-0.3, 0.6, T).astype(np.float32)
    if B:
        a["bias_ids"] = rng.integers(-1, V, (T, B)).astype(np.int32)
        a["bias"] = (rng.standard_normal((T, B)) * 4).astype(np.float32)
    if mask is not None:
        words = -(-V // 32)
        m = rng.integers(0, 2 ** 32, (T, words), dtype=np.uint32)
        if mask == "sparse":
            m[rng.random((T, words)) < 0.9] = 0
        if mask == "none":
            m[:] = 0
        if mask == "all":
            m[:] = 0xffffffff
        a["mask"] = m.view(np.int32)
    return x.to(torch.bfloat16) if bf16 else x, a


def check(x, a, out, untouched_equal=True):
    want, size = steps.adjust_logits(x.float().cpu().numpy(), **a)
    got = out.float().cpu().numpy().astype(np.float64)
    off = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), off)
    tol = 4 * 2.0 ** -24 * size
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(np.where(off, 0, want))
    assert np.all(np.abs(got - want)[~off] <= tol[~off])


@pytest.mark.parametrize("T,V", [(1, 1), (2, 31), (3, 33), (5, 1000), (4, 8191), (3, 8193), (2, 32000), (7, 50001), (2, 131072),
                                 (1, 262144), (200, 1024)])
@pytest.mark.parametrize("H,B,mask", [(50, 0, None), (0, 7, None), (0, 0, "sparse"), (300, 20, "half"), (1, 1, "none"), (0, 0, None),
                                      (9, 0, "all")])
@pytest.mark.parametrize("bf16,out_bf16", [(False, False), (True, False), (True, True), (False, True)])
def test_adjusted_logits_match_oracle(pm, T, V, H, B, mask, bf16, out_bf16):
    if bf16 != out_bf16 and (T, V) not in ((3, 33), (7, 50001), (2, 131072)):
        pytest.skip("mixed types at some sizes")
    x, a = make(T * V + H, T, V, H, B, mask, bf16)
    out = torch.full((T, V), 5.0, dtype=torch.bfloat16 if out_bf16 else torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = x.clone()
    pm.moe_adjust_logits(x, out=out, err_out=err, **{k: dev(v) for k, v in a.items()})
    assert int(err) == 0 and torch.equal(x, before)
    check(x, a, out)
    if bf16 == out_bf16:  # in place: the same bits
        pm.moe_adjust_logits(x, out=x, **{k: dev(v) for k, v in a.items()})
        assert torch.equal(x, out)


def test_one_token_over_and_over(pm):
    """Counts far beyond one, in prompt and output, in every position of the history."""
    T, V, H = 3, 700, 5000
    x, a = make(1, T, V, H)
    a["history"][:] = 123
    a["history_len"][:] = [H, H, 1]
    a["prompt_len"][:] = [0, H, 1]
    out = pm.moe_adjust_logits(x, **{k: dev(v) for k, v in a.items()})
    check(x, a, out)
    assert out.dtype == torch.float32


def test_each_setting_alone(pm):
    x, full = make(2, 4, 999, 80, 6, "half")
    for drop in (["repetition"], ["frequency"], ["presence"], ["prompt_len"], ["repetition", "frequency", "presence"], ["mask"],
                 ["bias", "bias_ids"], ["history", "history_len", "prompt_len"]):
        a = {k: v for k, v in full.items() if k not in drop}
        out = pm.moe_adjust_logits(x, **{k: dev(v) for k, v in a.items()})
        check(x, a, out)


def test_infinities_pass_through(pm):
    x, a = make(3, 2, 100, 30, 0, "half")
    x[:, ::7] = float("-inf")
    x[:, 3] = float("inf")
    out = pm.moe_adjust_logits(x, **{k: dev(v) for k, v in a.items()}).cpu().numpy()
    want, _ = steps.adjust_logits(x.cpu().numpy(), **a)
    for f in (np.isneginf, np.isposinf, np.isnan):
        assert np.array_equal(f(out), f(want))
    x, a = make(4, 2, 100, 30)
    x[:, 50] = float("nan")
    out = pm.moe_adjust_logits(x, **{k: dev(v) for k, v in a.items()})
    assert bool(torch.isnan(out[:, 50]).all()) and int(torch.isnan(out).sum()) == 2


def test_the_last_bias_of_a_token_counts(pm):
    x, _ = make(5, 2, 50)
    a = dict(bias_ids=np.array([[4, 9, 4, -1, 9, 4], [49, -1, -1, 0, 0, -1]], np.int32),
             bias=np.arange(12, dtype=np.float32).reshape(2, 6) + 1)
    out = pm.moe_adjust_logits(x, **{k: dev(v) for k, v in a.items()})
    check(x, a, out)


@pytest.mark.parametrize("shift,out_shift", [(0, 0), (1, 1), (3, 3), (1, 2), (0, 3)])
@pytest.mark.parametrize("bf16", [False, True])
def test_strides_and_alignment(pm, shift, out_shift, bf16):
    T, V = 5, 9001
    x, a = make(6 + shift, T, V, 60, 3, "half", bf16)
    wide = torch.zeros((T, V + 11), dtype=x.dtype, device="cuda")
    view = wide[:, shift:shift + V]
    view.copy_(x)
    hist = np.full((T, 77), -1, np.int32)
    hist[:, :60] = a["history"]
    mask = np.zeros((T, -(-V // 32) + 3), np.int32)
    mask[:, :a["mask"].shape[1]] = a["mask"]
    room = torch.full((T, V + 9), 3.0, device="cuda")
    args = {k: dev(v) for k, v in a.items()}
    args.update(history=dev(hist)[:, :60], mask=dev(mask))
    pm.moe_adjust_logits(view, out=room[:, out_shift:out_shift + V], **args)
    check(x, a, room[:, out_shift:out_shift + V])
    assert bool((room[:, :out_shift] == 3).all()) and bool((room[:, out_shift + V:] == 3).all())


def test_ids_and_lengths_out_of_range_are_reported(pm):
    x, a = make(7, 4, 500, 40, 5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for name, value, bit in (("history", 500, 512), ("history", -1, 512), ("history", 1 << 30, 512), ("bias_ids", 500, 512),
                             ("bias_ids", -2, 512), ("history_len", 41, 128), ("history_len", -1, 128), ("prompt_len", 41, 128),
                             ("prompt_len", -7, 128)):
        b = {k: v.copy() for k, v in a.items()}
        b["history_len"][:] = 40
        b[name][1, ...] = value
        err.zero_()
        out = pm.moe_adjust_logits(x, err_out=err, **{k: dev(v) for k, v in b.items()})
        assert int(err) == bit, name
        check(x, b, out)


def test_streams_and_graphs(pm):
    x, a = make(8, 6, 20000, 100, 9, "sparse", True)
    args = {k: dev(v) for k, v in a.items()}
    want = pm.moe_adjust_logits(x, **args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pm.moe_adjust_logits(x, stream=s, **args)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pm.moe_adjust_logits(x, out=out, **args)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert pm.moe_adjust_logits(x[:0], **{k: v[:0] for k, v in args.items()}).shape == (0, 20000)


def test_refusals(pm):
    x, a = make(9, 2, 100, 10, 3, "half")
    args = {k: dev(v) for k, v in a.items()}
    for change, name in ((dict(mask=args["mask"][:, :3]), "mask"), (dict(bias=None), "bias"), (dict(history_len=None), "history_len"),
                         (dict(history=args["history"][:1]), "history"), (dict(repetition=args["repetition"].double()), "repetition"),
                         (dict(out=torch.empty((2, 99), device="cuda")), "out"), (dict(logits=x.t()), "logits")):
        with pytest.raises(AssertionError, match=name):
            pm.moe_adjust_logits(**{"logits": x, **args, **change})
    big = torch.zeros((1, 262145), device="cuda")
    with pytest.raises(pm.PmoeError) as e:
        pm.moe_adjust_logits(big)
    assert e.value.status == pm.PMOE_EINVAL
