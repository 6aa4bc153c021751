"""Pins of the step oracle: worked cases and invariants (CPU only)."""
import numpy as np

from oracle import step_oracle as so


def test_plan_by_hand():
    # pages of 4: sequence 0 grows 3 -> 6 (one page), 1 drops 9 -> 4 (two pages back), 2 stays, 3 grows 0 -> 1
    table = np.array([[5, -1, -1], [2, 7, 1], [9, -1, -1], [-1, -1, -1]])
    free = np.array([0, 3, -9, -9, -9, -9, -9, -9, -9, -9])
    r = so.plan([3, -5, 0, 1], [3, 9, 2, 0], table, free, 2, 6, 4, 10, 12)
    # given back: 7, 1 on top of 0, 3; taken: 1 by sequence 0, 7 by sequence 3
    assert r["free"][:4].tolist() == [0, 3, 7, 1] and r["n_free"] == 2
    assert r["table"].tolist() == [[5, 1, -1], [2, 7, 1], [9, -1, -1], [7, -1, -1]]
    assert r["q_start"].tolist() == [0, 3, 3, 3, 4] and r["kv_len"].tolist() == [6, 4, 2, 1]
    assert r["positions"].tolist() == [3, 4, 5, 0, 0, 0] and r["slots"].tolist() == [23, 4, 5, 28, -1, -1]
    assert not r["bad"]


def test_plan_leaves_out_from_the_first_that_finds_too_little():
    table, free = np.full((4, 3), -1), np.array([4, 5, 6, 0, 0, 0, 0])
    for T, n_free in ((8, 7), (20, 2)):  # rows, or pages, run out at the second
        r = so.plan([4, 8, 1, -1], [0, 0, 0, 2], np.array([[-1] * 3] * 3 + [[1, -1, -1]]), free, n_free, T, 4, 7, 12)
        assert r["q_start"].tolist() == [0, 4, 4, 4, 4] and r["kv_len"].tolist() == [4, 0, 0, 1] and r["bad"]
    r = so.plan([1, 1], [0, 13], table[:2], free, 3, 4, 4, 7, 12)  # one beyond its bound hinders nobody
    assert r["q_start"].tolist() == [0, 1, 1] and r["kv_len"].tolist() == [1, 13] and r["bad"]


def test_pages_are_never_lost():
    rng = np.random.default_rng(3)
    page, n_pages, B, width = 16, 60, 12, 5
    table, lens, free, n_free = np.full((B, width), -1), np.zeros(B, int), rng.permutation(n_pages), n_pages
    for _ in range(200):
        new = rng.integers(-30, 30, B)
        new = np.where(lens + new < 0, -lens, np.where(lens + new > page * width, 0, new))
        r = so.plan(new.tolist(), lens.tolist(), table, free, n_free, 400, page, n_pages, page * width)
        table, lens, free, n_free = r["table"], r["kv_len"], r["free"], r["n_free"]
        held = [table[b, i] for b in range(B) for i in range(-(-lens[b] // page))]
        assert sorted(held + free[:n_free].tolist()) == list(range(n_pages))


def test_head_norm_by_hand():
    y = so.head_norm([[3.0, 4.0, 0.0, 0.0]], [1.0, 2.0, 1.0, 1.0], 0.0)
    assert np.allclose(y, [[3 / 2.5, 8 / 2.5, 0, 0]], rtol=1e-15)
    assert np.allclose(so.head_norm([[0.0, 0.0]], [1, 1], 1e-6), 0) and np.allclose(so.head_norm([[1e-3] * 2], [1, 1], 1e-6), 2 ** -0.5)


def test_window_by_hand():
    s = so.window_sees(3, 8, 2, 1).astype(int).tolist()
    assert s == [[1, 0, 0, 0, 1, 1, 0, 0], [1, 0, 0, 0, 0, 1, 1, 0], [1, 0, 0, 0, 0, 0, 1, 1]]
    assert so.window_sees(4, 2, 1, 0).astype(int).tolist() == [[0, 0], [0, 0], [1, 0], [0, 1]]


def test_attention_of_what_a_row_sees():
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(4, 2, 8)), rng.normal(size=(9, 1, 8)), rng.normal(size=(9, 1, 8))
    from oracle import attn_oracle as ao
    for o, r in zip(so.attend(q, k, v, 0.3, 2, so.window_sees(4, 9, 9, 0)), ao.attend(q, k, v, 0.3, 2)):
        assert np.allclose(o, r, atol=1e-14)
    one = so.attend(q, k, v, 0.3, 2, so.window_sees(4, 9, 1, 0))[0]
    assert np.allclose(one, np.repeat(v[5:, :1], 2, 1))
    keep = [0, 1, 6, 7, 8]
    last = so.attend(q, k, v, 0.3, 2, so.window_sees(4, 9, 3, 2))[0][3]
    assert np.allclose(last, so.attend(q[3:], k[keep], v[keep], 0.3, 2, np.ones((1, 5), bool))[0][0])
