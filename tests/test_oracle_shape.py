"""Pins of the oracle's logit shaping and token state."""

import numpy as np

from oracle import shape as OS


def _state(g, V):
    counts = g.integers(0, 4, V) * (g.random(V) < 0.3)
    seen = (counts > 0) | (g.random(V) < 0.2)
    return seen, counts


def test_neutral_values_change_nothing():
    g = np.random.default_rng(1)
    V = 96
    row = g.normal(0, 3, V)
    row[3], row[4] = -np.inf, np.nan
    seen, counts = _state(g, V)
    out, mag = OS.shape_row(row, [1, 2], seen, counts, bias=[(5, 0.0)], allowed=np.ones(V, bool))
    assert np.array_equal(out, row, equal_nan=True)
    assert mag[[3, 4]].sum() == 0


def test_formula_by_hand():
    row = np.array([2.0, -2.0, 0.0, 1.0, 5.0, 1.5, np.nan, 7.0])
    seen = np.array([1, 1, 1, 0, 0, 0, 0, 0], bool)
    counts = np.array([3, 0, 1, 9, 0, 0, 0, 0])   # token 3 has no bit: its count is no count
    allowed = np.array([1, 1, 1, 1, 1, 1, 0, 0], bool)
    out, _ = OS.shape_row(row, [4, 4, 9, -1], seen, counts, 2.0, 0.5, 0.25, [(5, 1.0), (5, -3.0), (99, 1.0)],
                          allowed)
    assert np.array_equal(out, [2 / 2 - 1.5 - 0.25, -4.0, 0 - 0.5 - 0.25, 1.0, 5 / 2 - 1.0 - 0.25, -1.5, -np.inf,
                                -np.inf])


def test_drafted_tokens_equal_state_tokens():
    g = np.random.default_rng(2)
    V = 64
    row = g.normal(0, 3, V)
    seen, counts = _state(g, V)
    written = [3, 3, 17, 60]
    s2, c2 = seen.copy(), counts * seen
    OS.enter_tokens(s2, c2, written)
    a, _ = OS.shape_row(row, written, seen, counts, 1.3, 0.4, 0.2)
    b, _ = OS.shape_row(row, [], s2, c2, 1.3, 0.4, 0.2)
    assert np.array_equal(a, b)


def test_lists_in_pieces_and_prompts():
    g = np.random.default_rng(3)
    V = 40
    toks = g.integers(-2, V + 2, 50)
    a = np.zeros(V, bool), np.zeros(V, int)
    b = np.ones(V, bool), np.full(V, 7)
    OS.enter_tokens(*a, toks, prompt_len=20)
    OS.enter_tokens(*b, toks[:30], prompt_len=20, reset=True)
    OS.enter_tokens(*b, toks[30:])
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    ok = toks[(toks >= 0) & (toks < V)]
    assert np.array_equal(np.nonzero(a[0])[0], np.unique(ok))
    tail = toks[20:]
    assert np.array_equal(a[1], np.bincount(tail[(tail >= 0) & (tail < V)], minlength=V))


def test_bits_roundtrip():
    g = np.random.default_rng(4)
    for V in (8, 31, 32, 40, 96, 104):
        rows = g.random((3, V)) < 0.4
        assert np.array_equal(OS.unpack_bits(OS.pack_bits(rows), V), rows)
        assert OS.pack_bits(rows, 9).shape == (3, 9)
    assert OS.pack_bits(np.arange(64)[None, :] == 31)[0, 0] == np.int32(-2**31)
