"""Pins of the attention and sampling oracles, each independent of their own formulas."""

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import sampling as osamp

torch = pytest.importorskip("torch")


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 2, 8))
    pos, freq = rng.integers(0, 50, (1, 4)), np.array([1.0, 0.3, 0.1], np.float32)
    for inter in (False, True):
        y = oatt.turn_heads(x, pos, freq, interleaved=inter)
        a, b = (np.s_[..., 0:6:2], np.s_[..., 1:6:2]) if inter else (np.s_[..., 0:3], np.s_[..., 3:6])
        want = (x[a] + 1j * x[b]) * np.exp(1j * pos[0][:, None, None] * freq.astype(np.float64))
        assert np.allclose(y[a], want.real) and np.allclose(y[b], want.imag) and np.array_equal(y[..., 6:], x[..., 6:])


def test_rotation_axes_and_norm():
    x = np.ones((1, 1, 4))
    y = oatt.turn_heads(x, [[0], [np.pi / 2]], [1.0, 1.0], pair_axis=[0, 1])
    assert np.allclose(y[0, 0], [1, -1, 1, 1])  # pair 0 does not turn, pair 1 turns by a right angle
    y = oatt.turn_heads(3 * x, [[0]], [], norm=np.array([1.0, 2.0, 3.0, 4.0]), eps=0.0)
    assert np.allclose(y[0, 0], [1, 2, 3, 4])
    z = torch.nn.functional.rms_norm(torch.arange(1.0, 5.0).double(), (4,), eps=1e-6).numpy()
    assert np.allclose(oatt.turn_heads(np.arange(1.0, 5.0)[None, None], [[0]], [], norm=np.ones(4))[0, 0], z)


def test_append_places_rows():
    cache = np.zeros((3, 2, 4, 1))
    oatt.append(cache, np.arange(6.0).reshape(3, 2, 1) + 1, [9, -1, 0])
    assert cache[2, :, 1, 0].tolist() == [1, 2] and cache[0, :, 0, 0].tolist() == [5, 6] and cache.sum() == 14


def test_attention_is_the_library_attention_of_the_gathered_rows():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 5, 2, 4, 8))
    q = rng.standard_normal((2, 6, 8))
    out, lse, mag = oatt.prefix_attention(k, v, q, [3, 1], 6, [[0, 4], [2, 0]], [0, 7], 0.5)
    flat = lambda x, pages, n: x[pages].transpose(1, 0, 2, 3).reshape(2, -1, 8)[:, :n]  # noqa: E731
    for t, (pages, n) in enumerate((([0, 4], 0), ([2, 0], 7))):
        kk, vv = (np.concatenate([flat(x, [3, 1], 6), flat(x, pages, n)], 1).repeat(3, 0) for x in (k, v))
        a, b, c = (torch.from_numpy(x)[None] for x in (q[t][:, None], kk, vv))
        ref = torch.nn.functional.scaled_dot_product_attention(a, b, c, scale=0.5)[0, :, 0].numpy()
        assert np.allclose(out[t], ref)
        assert np.allclose(lse[t], torch.logsumexp(0.5 * torch.from_numpy(np.einsum("hd,hnd->hn", q[t], kk)), -1))
    assert np.all(mag >= np.abs(out))
    out, lse, _ = oatt.prefix_attention(k, v, q, [], 0, [[0], [1]], [0, 1], 0.5)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(out[1], v[1, :, 0].repeat(3, 0))


def test_sampling_frequencies_follow_the_cut_softmax():
    x = np.log(np.array([0.4, 0.1, 0.3, 0.2]))
    n = 4000
    grid = (np.arange(n) + 0.5) / n
    for args, want in ((dict(), [0.4, 0.1, 0.3, 0.2]), (dict(top_k=2), [4 / 7, 0, 3 / 7, 0]),
                       (dict(top_p=0.71), [4 / 9, 0, 3 / 9, 2 / 9]), (dict(min_p=0.3), [4 / 9, 0, 3 / 9, 2 / 9]),
                       (dict(temperature=0.5), [16 / 30, 1 / 30, 9 / 30, 4 / 30]), (dict(temperature=0.0), [1, 0, 0, 0])):
        ids = [osamp.sample_row(x, u, **args)[0] for u in grid]
        assert np.allclose(np.bincount(ids, minlength=4) / n, want, atol=2 / n), args
        assert ids == sorted(ids)  # ascending ids with ascending u


def test_sampling_ties_and_empty_rows():
    assert osamp.sample_row(np.zeros(5), 0.99, top_k=2)[0] == 1
    assert osamp.sample_row(np.full(3, -np.inf), 0.5)[0] == -1
    assert osamp.sample_row(np.array([np.nan, 2.0, 2.0]), 0.5, temperature=0)[0] == 1
    assert osamp.sample_row(np.array([0.0, np.inf, np.inf]), 0.6)[:2] == (2, pytest.approx(-np.log(2)))
