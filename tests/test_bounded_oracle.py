"""Pins of the definitions of a bounded cache's operators (oracle/decode.py): closed forms and brute force."""
import itertools

import numpy as np

from oracle import decode as D


def test_axes_that_agree_are_plain_positions():
    rng = np.random.default_rng(0)
    q, k, v = (rng.normal(size=(5, h, 8)) for h in (4, 2, 2))
    pages = rng.normal(size=(3, 2, 4, 8)), rng.normal(size=(3, 2, 4, 8))
    table = rng.normal(size=(9, 6))
    at, slots = rng.integers(0, 9, 5), np.array([0, 3, -1, 11, 7])
    a = D.append(q, k, v, at, slots, table, 6, True, None, None, 0.0, *pages)
    b = D.append_axes(q, k, v, np.stack([at] * 3, 1), [0, 1, 2], slots, table, 6, True, None, None, 0.0, *pages)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_a_pair_turns_by_its_own_axis():
    """Two pairs on two axes: a quarter turn for one, none for the other."""
    table = np.array([[1, 1, 0, 0], [0, 0, 1, 1]], float)         # position 1 turns by 90 degrees
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    q, _, _ = D.append_axes(x, x, x, [[1, 0]], [0, 1], [-1], table, 4, False, None, None, 0.0, np.zeros((1, 1, 1, 4)), np.zeros((1, 1, 1, 4)))
    assert np.allclose(q[0, 0], [-3, 2, 1, 4])                     # (1, 3) -> (-3, 1); (2, 4) stays


def attention_case(n, length, n_q=4, n_kv=2, d=6, page=4, masks=None, decay=0.5):
    rng = np.random.default_rng(n + length)
    pages = -(-length // page)
    k = rng.normal(size=(pages + 1, n_kv, page, d))
    table = rng.permutation(pages + 1)[None, :pages]
    q, w = rng.normal(size=(n, n_q, d)), rng.random((pages + 1, n_kv, page))
    new, gain, _ = D.attention_weights(q, k, [0, n], [length], table, masks, 0.7, w, decay)
    at = [(table[0][c // page], c % page) for c in range(length)]
    return q, k, w, new, gain, at, table


def test_weights_of_a_softmax_sum_to_its_rows():
    _, _, w, new, gain, at, _ = attention_case(3, 17)
    for h in range(2):
        assert np.isclose(sum(gain[p, h, o] for p, o in at), 3 * 2)        # rows: three tokens of two heads
        for c, (p, o) in enumerate(at):
            assert np.isclose(new[p, h, o], gain[p, h, o] + (0.5 * w[p, h, o] if c < 14 else 0.0))
    seen = {(p, o) for p, o in at}
    for p, o in itertools.product(range(w.shape[0]), range(4)):
        if (p, o) not in seen:
            assert np.array_equal(new[p, :, o], w[p, :, o])


def test_weights_are_the_probabilities_of_the_attention():
    """With values that are one-hot, the attention's output is the weights."""
    q, k, w, new, gain, at, table = attention_case(2, 6, decay=0.0)
    v = np.zeros((*k.shape[:3], 6))
    for c, (p, o) in enumerate(at):
        v[p, :, o, c] = 1
    out, _, _ = D.tree_attention(q, k, v, [0, 2], [6], table, None, 0.7)
    for h in range(2):
        assert np.allclose(out[:, 2 * h: 2 * h + 2].sum((0, 1)), [new[p, h, o] for p, o in at])


def test_rows_that_see_nothing_add_nothing():
    _, _, w, new, gain, at, _ = attention_case(3, 3, masks=[np.zeros((3, 3), bool)])
    assert not gain.any() and all((new[p, :, o] == 0).all() for p, o in at)


def test_evicted_tokens_have_the_lowest_scores():
    rng = np.random.default_rng(4)
    for trial in range(40):
        length, page = int(rng.integers(2, 20)), 4
        keep = int(rng.integers(0, length))
        first, recent = int(rng.integers(0, 4)), int(rng.integers(0, 4))
        pages = -(-length // page)
        scores = rng.integers(0, 4, (pages, 1, page)).astype(float)
        table = rng.permutation(pages)[None]
        ids = np.arange(pages * page, dtype=float).reshape(pages, 1, page)
        (moved,), kept, lens = D.evict([ids], scores, [length], table, [keep], first, recent)
        f = [scores[table[0][c // page], 0, c % page] for c in range(length)]
        last = min(recent, keep)
        begin = min(first, keep - last)
        must = set(range(begin)) | set(range(length - last, length))
        got = kept[0][0]
        assert lens[0] == keep and must <= set(got.tolist()) and list(got) == sorted(got)
        rest, gone = [c for c in got if c not in must], [c for c in range(length) if c not in got]
        assert all((f[a], -a) > (f[b], -b) for a in rest for b in gone)
        for j, c in enumerate(got):
            assert moved[table[0][j // page], 0, j % page] == ids[table[0][c // page], 0, c % page]


def test_order_of_odd_scores():
    scores = np.array([[[np.nan, -np.inf, -0.0, 0.0, np.inf, np.nan, 1.0, -1.0]]])
    for keep, chosen in ((1, [4]), (2, [4, 6]), (3, [2, 4, 6]), (4, [2, 3, 4, 6]), (5, [2, 3, 4, 6, 7]), (6, [1, 2, 3, 4, 6, 7]),
                         (7, [0, 1, 2, 3, 4, 6, 7])):
        _, kept, _ = D.evict([scores], scores, [8], np.array([[0]]), [keep], 0, 0)
        assert kept[0][0].tolist() == chosen


def test_requests_within_their_budget_stay():
    planes, kept, lens = D.evict([np.arange(8.0).reshape(1, 1, 8)], np.ones((1, 1, 8)), [8, 5], np.array([[0], [0]]), [-1, 5], 1, 1)
    assert kept == [None, None] and lens.tolist() == [8, 5] and np.array_equal(planes[0].ravel(), np.arange(8))
