"""The oracle of a step over unequal requests: pins worked out by hand."""

import numpy as np

from oracle import attention, steps


def test_tables_by_hand():
    table = np.array([[4, 9, -1], [7, -1, -1], [2, 3, -1]])
    got = steps.batch_tables(table, np.array([5, 6, 8, 0, 0, 0]), 3, [17, 16, 20], [1, 2, -1], 5, 16, 10)
    assert got[0].tolist() == [[4, 9, -1], [7, 3, -1], [2, 3, -1]]  # page 3, given back last, goes out first
    assert got[1].tolist() == [5, 6, 8, 2, 3, 0] and got[2] == 4
    assert got[3].tolist() == [18, 18, 0] and got[4].tolist() == [0, 1, 3, 3]
    assert got[5].tolist() == [17, 16, 17, 0, 0]
    assert got[6].tolist() == [9 * 16 + 1, 3 * 16, 3 * 16 + 1, -1, -1]
    assert got[7].tolist() == [0, 1, 1, -1, -1] and got[8].tolist() == [18, 17, 18, 0, 0]
    got = steps.batch_tables(table, np.array([5]), 1, [16, 16, 20], [1, 1, 1], 9, 16, 10)
    assert got[9].tolist() == [False, True, False] and got[3].tolist() == [17, 16, 21]


def test_chunk_attention_of_single_tokens_is_the_paged_attention():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 5, 2, 16, 8))
    q = rng.standard_normal((2, 4, 8))
    table = np.array([[3, 1], [4, 0]])
    a = steps.chunk_attention(k, v, q, [0, 1, 2], [20, 7], table, 0.4)
    b = attention.prefix_attention(k, v, q, [], 0, table, [20, 7], 0.4)
    for x, y in zip(a[:3], b):
        assert np.allclose(x, y, rtol=1e-13, atol=1e-13)
    assert a[3].tolist() == [20, 7]


def test_chunk_attention_limits():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 2, 1, 16, 4))
    q = rng.standard_normal((9, 1, 4))
    out, lse, _, count = steps.chunk_attention(k, v, q, [1, 7], [4], np.array([[1, 0]]), 1.0, 2, 1)
    assert count.tolist() == [-1, 0, 0, 1, 2, 3, 3, -1, -1]  # positions -2 .. 3, a window of 2 and one sink
    assert np.allclose(out[3, 0], v[1, 0, 0]) and np.all(out[1:3] == 0) and np.all(np.isneginf(lse[:3]))
    s = np.array([q[6, 0] @ k[1, 0, j] for j in (0, 2, 3)])
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[6, 0], w @ v[1, 0, [0, 2, 3]])


def test_selection_by_hand():
    x = np.log(np.array([[1.0, 3.0, 2.0, 2.0, 9.0, 1.0, 1.0, 1.0]]))  # softmax: twentieths
    ids, w, _ = steps.router_select(x, 2, "softmax", groups=4, top_groups=2, group_top=2, renormalize=False)
    assert ids.tolist() == [[4, 1]] or ids.tolist() == [[4, 2]]
    ids, w, _ = steps.router_select(x, 2, "softmax", groups=4, top_groups=1, group_top=2, renormalize=False, scale=2.0)
    assert ids.tolist() == [[4, 5]] and np.allclose(w, [[0.9, 0.1]])
    bias = np.array([0.0, 0, 0.9, 0, 0, 0, 0, 0])
    ids, w, _ = steps.router_select(x, 2, "softmax", bias)
    assert ids.tolist() == [[2, 4]] and np.allclose(w, [[2 / 11, 9 / 11]])  # the bias is not in the weights
    ids, w, _ = steps.router_select(np.zeros((1, 8)), 2, "sigmoid", groups=4, top_groups=1, group_top=1, renormalize=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 0.5)


def test_adjusting_by_hand():
    x, _ = steps.adjust_logits(np.array([[2.0, -2.0, 1.0, 4.0, 5.0]]), np.array([[0, 1, 2, 2, 99]]), [2], [4], [2.0], [0.5], [0.25],
                               np.array([[4, -1, 4]]), np.array([[7.0, 1.0, -1.0]]), np.array([[0b10111]], np.int32))
    assert x.tolist() == [[1.0, -4.0, 0.5 - 1.0 - 0.25, -np.inf, 4.0]]
