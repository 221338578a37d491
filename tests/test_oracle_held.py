"""Pin of the oracle: a request that a call of the step refused keeps what it
had, whatever verification accepted of its rows."""

import numpy as np
import pytest

from oracle import slots as OS


@pytest.mark.parametrize("bits,held", [(0, False), (1, False), (8, False), (16, False), (64, False), (1 | 8 | 64, False),
                                       (2, True), (4, True), (32, True), (32 | 64, True), (127, True)])
def test_a_refused_request_is_held(bits, held):
    bs, q = 4, 5
    table = np.array([[0, 1, 2], [3, 4, -1]], np.int32)
    free = np.array([9, 8, -1, -1, -1, -1, -1, -1, -1, -1], np.int32)
    seq, ell, tokens = np.array([6, 3]), np.array([4, 2]), np.arange(10).reshape(2, 5) + 100
    status = np.array([bits, 0], np.int32)
    got = OS.commit(seq, ell, np.array([3, 2]), table, free, 2, bs, q, tokens, np.array([50, 51], np.int32), status)
    assert got["n_new"].tolist() == [0 if held else 4, 3]
    assert got["seq_len"].tolist() == [6 if held else 10, 6]
    assert got["x0"].tolist() == [50 if held else 103, 107]
    # 11 positions were reserved in 3 blocks: a held request keeps 2 of them
    assert got["free_count"][0] == (3 if held else 2) and free[2] == (2 if held else -1)
    assert status.tolist() == [bits, 0]
