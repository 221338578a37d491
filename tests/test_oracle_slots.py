"""Pins of the oracle's slot bookkeeping: a long random run in which the pool
stays a partition and every slot is the one a dictionary remembers."""

import numpy as np
import pytest

from oracle import slots as OS


@pytest.mark.parametrize("seed", range(4))
def test_pool_stays_a_partition(seed):
    g = np.random.default_rng(seed)
    R, bs, mb, q = 6, int(g.integers(1, 9)), 7, 5
    pool = R * mb - 10   # tight: some requests go short
    table = np.full((R, mb), -1, np.int32)
    free = g.permutation(pool).astype(np.int32)
    F = pool
    seq = np.zeros(R, np.int64)
    held = {r: [] for r in range(R)}
    where = {}
    for step in range(200):
        ell = g.integers(-1, q, R).astype(np.int32)
        padded = bool(step % 2)
        rows = R * q if padded else int(g.integers(1, R * q + 1))
        o = OS.reserve(seq, ell, table, free, F, bs, q, rows, padded)
        F = int(o["free_count"][0])
        n = o["ell"] + 1
        assert np.array_equal(np.diff(o["cu_rows"]), n) and o["batch"][0] == n.sum()
        assert (n <= np.maximum(np.minimum(ell, q - 1) + 1, 0)).all()
        for r in range(R):
            b = OS.blocks_of(int(seq[r] + n[r]), bs)
            assert list(table[r, :len(held[r])]) == held[r]
            held[r] = list(table[r, :b])
        for e in range(rows):
            r = o["row_req"][e]
            if r < 0:
                assert o["row_pos"][e] == o["row_slot"][e] == -1
                continue
            where[(int(r), int(o["row_pos"][e]))] = int(o["row_slot"][e])
            assert o["row_slot"][e] // bs == held[r][o["row_pos"][e] // bs]
        used = sum(held.values(), []) + list(free[:F])
        assert sorted(used) == list(range(pool))
        if not padded and rows == R * q:
            short = o["status"] & OS.NO_SLOT != 0
            assert not short.any() or F == 0 or (seq + ell + 1 > bs * mb).any()
        release = g.random(R) < 0.1
        acc = g.integers(0, q, R)
        status = np.where(g.random(R) < 0.1, 2, 0).astype(np.int32)
        c = OS.commit(seq, o["ell"], acc, table, free, F, bs, q, status=status, release=release)
        F = int(c["free_count"][0])
        seq = c["seq_len"]
        for r in range(R):
            held[r] = held[r][:OS.blocks_of(int(seq[r]), bs)]
            for p in range(int(seq[r])):
                assert where[(r, p)] == held[r][p // bs] * bs + p % bs
        used = sum(held.values(), []) + list(free[:F])
        assert sorted(used) == list(range(pool))
