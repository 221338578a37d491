"""sd_slot_reserve and sd_slot_commit against the oracle, bit for bit."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from oracle import slots as OS
from tests.parity_util import to_np

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _t(a, dt=torch.int32):
    return None if a is None else torch.as_tensor(np.ascontiguousarray(a), dtype=dt).to(DEV)


def _pool(g, R, mb, held, spare):
    """A table, the free list and its count for `held` blocks per request."""
    pool = int(held.sum()) + spare
    perm = g.permutation(pool).astype(np.int32)
    table = np.full((R, mb), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :held[r]] = perm[at:at + held[r]]
        at += held[r]
    free = np.full(pool, -5, np.int32)
    free[:spare] = perm[at:]
    return table, free, spare


def _reserve(seq, ell, table, free, F, bs, q, rows, padded, x0=None, tokens=None, alias=False):
    ts, te, tt, tf, tF = _t(seq, torch.int64), _t(ell), _t(table), _t(free), _t([F])
    out = dict(row_req=torch.full((rows,), 9, dtype=torch.int32, device=DEV))
    if alias:
        out.update(ell=te, free_count=tF)
    got = sdv.sd_slot_reserve(ts, te, tt, tf, tF, bs, q, padded=padded, x0=_t(x0), tokens=_t(tokens), out=out)
    torch.cuda.synchronize()
    want_table = table.copy()
    want = OS.reserve(seq, ell, want_table, free, F, bs, q, rows, padded, x0, tokens)
    for k, v in want.items():
        if k == "row_token" and x0 is None and tokens is None:
            assert got[k] is None
            continue
        assert np.array_equal(to_np(got[k]), v), (k, to_np(got[k])[:20], v[:20])
    assert np.array_equal(to_np(tt), want_table)
    assert np.array_equal(to_np(ts), seq) and np.array_equal(to_np(tf), free)
    return want, want_table


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("R,q,bs,mb", [(1, 1, 1, 1), (1, 9, 16, 8), (4, 5, 16, 32), (64, 9, 24, 40), (300, 6, 16, 20),
                                       (513, 17, 64, 33), (1024, 2, 8, 12), (1025, 3, 16, 9), (5000, 5, 7, 11),
                                       (3, 3000, 16, 400), (4, 70000, 32, 3000)])
def test_reserve(R, q, bs, mb, padded):
    g = np.random.default_rng(R + q)
    cap = bs * mb
    for spare_share in (1.0, 0.6, 0.0):
        seq = g.integers(0, cap + 1, R)
        seq[g.random(R) < 0.1] = 0
        ell = g.integers(-1, q + 2, R)
        held = -(-seq // bs)
        need = int((-(-np.minimum(seq + np.clip(ell, -1, q - 1) + 1, cap) // bs) - held).sum())
        table, free, F = _pool(g, R, mb, held, int(spare_share * need))
        rows = R * q if padded else max(1, int(g.integers(R * q // 3, R * q + 9)))
        x0, tokens = g.integers(0, 1 << 20, R), g.integers(0, 1 << 20, (R, q))
        _reserve(seq, ell, table, free, F, bs, q, rows, padded, x0, tokens, alias=spare_share == 0.6)
    _reserve(seq, ell, table, free, F, bs, q, rows, padded, None, tokens)
    _reserve(seq, ell, table, free, F, bs, q, rows, padded)


def test_reserve_extremes():
    """Bad lengths, counts and block ids, extreme ell, rows behind the batch."""
    g = np.random.default_rng(3)
    bs, mb, q = 8, 4, 6
    seq = np.array([-1, 33, 32, 31, 0, 5, 1 << 40, -(1 << 40), 9, 17])
    ell = np.array([2, 2, 2, 2, -(1 << 31), (1 << 31) - 1, 1, 1, 3, 0])
    held = np.where((seq >= 0) & (seq <= 32), -(-seq // bs), 0)
    table, free, F = _pool(g, 10, mb, held, 12)
    want, _ = _reserve(seq, ell, table, free, F, bs, q, 80, False)
    assert want["status"].tolist()[:3] == [32, 32, 64]
    table[8, 1] = 10 ** 6       # the block that holds position 9
    table[9, 2] = -4
    want, _ = _reserve(seq, ell, table, free, F, bs, q, 80, True)
    assert want["status"].tolist()[8:] == [32, 32]
    free[F - 1] = 10 ** 8
    _reserve(seq, ell, table, free, F, bs, q, 80, False)
    for f in (-3, len(free) + 100):     # a count outside the list is clamped
        _reserve(seq, ell, table, free, f, bs, q, 80, False)


def _commit(seq, ell, acc, table, free, F, bs, q, tokens=None, x0=None, status=None, release=None, keep=None,
            alias=False):
    ts, tx, tf, tF, tst = _t(seq, torch.int64), _t(x0), _t(free), _t([F]), _t(status)
    out = dict(seq_len=ts, free_count=tF) if alias else None
    if alias and tokens is not None:
        out["x0"] = tx
    tt = _t(table)
    got = sdv.sd_slot_commit(ts, _t(ell), _t(acc), tt, tf, tF, bs, q_max=q, out_tokens=_t(tokens), x0=tx,
                             status=tst, release=_t(release), keep=_t(keep), out=out)
    torch.cuda.synchronize()
    wf, wst = free.copy(), None if status is None else status.copy()
    want = OS.commit(seq, ell, acc, table, wf, F, bs, q, tokens, x0 if tokens is not None else None, wst, release,
                     keep)
    for k, v in want.items():
        if v is None:
            assert got[k] is None
        else:
            assert np.array_equal(to_np(got[k]), v), (k, to_np(got[k])[:20], v[:20])
    assert np.array_equal(to_np(tf), wf)
    assert np.array_equal(to_np(tt), table)
    if status is not None:
        assert np.array_equal(to_np(tst), wst)
    return want


@pytest.mark.parametrize("R,q,bs,mb", [(1, 1, 1, 1), (1, 9, 16, 8), (4, 5, 16, 32), (64, 9, 24, 40), (300, 6, 16, 20),
                                       (513, 17, 64, 33), (1024, 2, 8, 12), (1025, 3, 16, 9), (5000, 5, 7, 11),
                                       (3, 3000, 16, 2100)])
def test_commit(R, q, bs, mb):
    g = np.random.default_rng(R + q)
    cap = bs * mb
    for k in range(3):
        ell = np.minimum(g.integers(-1, q, R), cap - 1)
        seq = (g.random(R) * (cap - ell)).astype(np.int64)
        table, free, F = _pool(g, R, mb, -(-(seq + ell + 1) // bs), 7)
        acc = g.integers(0, q, R)
        tokens, x0 = g.integers(0, 1 << 20, (R, q)), g.integers(0, 1 << 20, R)
        status = np.where(g.random(R) < 0.2, g.integers(0, 32, R), 0).astype(np.int32)
        release, keep = (g.random(R) < 0.3).astype(int), g.integers(-1, 4, R)
        _commit(seq, ell, acc, table, free, F, bs, q, tokens, x0, status, release if k else None,
                keep if k == 2 else None, alias=k == 1)
    _commit(seq, ell, acc, table, free, F, bs, q)


def test_commit_extremes():
    """Lengths and ell out of range leave the request as it is; blocks past
    the pool's size are dropped."""
    g = np.random.default_rng(5)
    bs, mb, q = 8, 4, 6
    seq = np.array([-1, 33, 30, 8, 8, 8, 0])
    ell = np.array([2, 2, 2, 6, -(1 << 31), 5, 3])
    table, free, F = _pool(g, 7, mb, np.array([0, 0, 0, 0, 1, 2, 1]), 3)
    status = np.zeros(7, np.int32)
    acc = np.array([1, 1, 1, 1, 1, -5, 99])
    want = _commit(seq, ell, acc, table, free, F, bs, q, status=status, release=np.ones(7, int))
    assert want["n_new"].tolist() == [0, 0, 0, 0, 0, 1, 4]
    want = _commit(seq, ell, acc, table, free, len(free) - 1, bs, q, status=status, release=np.ones(7, int))
    assert want["free_count"][0] == len(free)
    for f in (-3, len(free) + 100):
        _commit(seq, ell, acc, table, free, f, bs, q, status=status)


def test_slots_past_32_bits():
    """Block ids times the block size past 2^32."""
    bs, pool = 256, 1 << 25
    free = np.full(pool, -1, np.int32)
    free[:6] = pool - 1 - np.arange(6)
    table = np.full((2, 4), pool - 9, np.int32)
    seq, ell = np.array([5, 300]), np.array([600, 3])
    want, _ = _reserve(seq, ell, table, free, 6, bs, 700, 700, False)
    assert want["row_slot"].max() > 1 << 32 and (want["status"] == 0).all()


@pytest.mark.parametrize("rows", [0, 1, 700])
def test_a_step_without_requests(rows):
    i = lambda *k: torch.full(k, 9, dtype=torch.int32, device=DEV)  # noqa: E731
    seq = torch.zeros(0, dtype=torch.int64, device=DEV)
    for F, n in ((5, 5), (12, 8), (-2, 0)):
        for padded in (False, True):
            o = sdv.sd_slot_reserve(seq, i(0), i(0, 4), i(8), i(1) * 0 + F, 16, 3, max_rows=rows, padded=padded)
            assert int(o["batch"]) == 0 and int(o["free_count"]) == n and o["cu_rows"].tolist() == [0]
            assert all((o[k] == -1).all() and o[k].numel() == rows for k in ("row_req", "row_pos", "row_slot"))
        c = i(1) * 0 + F
        sdv.sd_slot_reserve(seq, i(0), i(0, 4), i(8), c, 16, 3, max_rows=rows, out=dict(free_count=c))
        assert int(c) == n
        assert int(sdv.sd_slot_commit(seq, i(0), i(0), i(0, 4), i(8), i(1) * 0 + F, 16, q_max=3)["free_count"]) == n


def test_a_step_is_repeated_with_the_old_count():
    g = np.random.default_rng(6)
    seq, ell = np.array([3, 9, 0]), np.array([4, 4, 4])
    table, free, F = _pool(g, 3, 8, -(-seq // 4), 10)
    a, ta = _reserve(seq, ell, table, free, F, 4, 5, 15, False)
    b, tb = _reserve(seq, ell, ta, free, F, 4, 5, 15, False)
    assert np.array_equal(ta, tb)
    for k in a:
        assert np.array_equal(a[k], b[k])


def test_refusals_of_the_binding():
    i = lambda *k: torch.zeros(k, dtype=torch.int32, device=DEV)  # noqa: E731
    seq = torch.zeros(2, dtype=torch.int64, device=DEV)
    ok = dict(seq_len=seq, ell=i(2), block_table=i(2, 4), free_list=i(8), free_count=i(1), block_size=16, q_max=3)
    sdv.sd_slot_reserve(*ok.values())
    for k, v in dict(ell=i(3), block_table=i(3, 4), free_count=i(2), free_list=i(8).float(), seq_len=i(2)).items():
        with pytest.raises((ValueError, TypeError)):
            sdv.sd_slot_reserve(**dict(ok, **{k: v}))
    with pytest.raises(ValueError, match="contiguous"):
        sdv.sd_slot_reserve(**dict(ok, block_table=i(4, 2).t()))
    with pytest.raises(ValueError, match="live on"):
        sdv.sd_slot_reserve(**dict(ok, ell=torch.zeros(2, dtype=torch.int32)))
    with pytest.raises(sdv.SdvError):
        sdv.sd_slot_reserve(**ok, max_rows=5, padded=True)
    with pytest.raises(ValueError):
        sdv.sd_slot_commit(seq, i(2), i(2), i(2, 4), i(8), i(1), 16)
    with pytest.raises(ValueError):
        sdv.sd_slot_commit(seq, i(2), i(2), i(2, 4), i(8), i(1), 16, out_tokens=i(3, 3), x0=i(2))
    x = torch.zeros((4, 64), device=DEV)
    with pytest.raises(ValueError, match="shape|elements"):
        sdv.sd_logit_shape(x, i(2), i(3), 64, gamma_max=1)
    with pytest.raises(ValueError, match="go together"):
        sdv.sd_logit_shape(x, i(2), i(2), 64, gamma_max=1, mask=i(2, 2))
    with pytest.raises(TypeError):
        sdv.sd_logit_shape(x.half(), i(2), i(2), 64, gamma_max=1)
    with pytest.raises(ValueError, match="shape|elements"):
        sdv.sd_logit_shape(x, i(2), i(2), 64, gamma_max=1, out=dict(logits=x[:2]))
    with pytest.raises(ValueError, match="start needs"):
        sdv.sd_token_counts(i(4), i(2, 2), None, 64, start=seq)
