"""A request that one call of a step refused (SD_ST_BAD_INPUT of the slots or
of the shaping) is held back by the commit: nothing of its step is kept."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from oracle import slots as OS
from tests.parity_util import to_np
from tests.test_gpu_slots import _commit, _pool
from tests.test_gpu_step import BS, DEV, G, MB, Q, R, V, Loop

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,q,bs,mb", [(1, 4, 8, 6), (4, 5, 16, 32), (5, 3, 4, 9), (64, 9, 24, 40), (300, 6, 16, 20),
                                       (1024, 2, 8, 12), (1100, 3, 16, 9)])
def test_every_status(n, q, bs, mb):
    g = np.random.default_rng(n)
    for k in range(3):
        ell = g.integers(-1, q, n)
        seq = (g.random(n) * (bs * mb - ell)).astype(np.int64)
        table, free, F = _pool(g, n, mb, -(-(seq + ell + 1) // bs), 7)
        status = np.where(g.random(n) < 0.6, g.integers(0, 128, n), 0).astype(np.int32)
        status[0] = [32, 96, 33][k]
        want = _commit(seq, ell, g.integers(0, q, n), table, free, F, bs, q, g.integers(0, 1 << 20, (n, q)),
                       g.integers(0, 1 << 20, n), status, (g.random(n) < 0.2).astype(int) if k else None,
                       alias=k == 1)
        assert want["n_new"][0] == 0


@pytest.mark.parametrize("n", [4, 300, 1024, 1100])
def test_more_blocks_than_the_pool_holds(n):
    """The bit that this adds to a status does not hold anything back."""
    g = np.random.default_rng(n)
    bs, mb, q = 4, 9, 8
    for room in (0, 3, n // 2, n):
        ell = g.integers(-1, q, n)
        seq = (g.random(n) * (bs * mb - ell)).astype(np.int64)
        table, free, _ = _pool(g, n, mb, -(-(seq + ell + 1) // bs), 7)
        status = np.where(g.random(n) < 0.2, g.integers(0, 128, n), 0).astype(np.int32)
        _commit(seq, ell, g.integers(0, 2, n), table, free, max(len(free) - room, 0), bs, q,
                g.integers(0, 99, (n, q)), g.integers(0, 99, n), status, (g.random(n) < 0.1).astype(int))


def test_commit_of_the_largest_ell():
    """ell + 1 is formed of an ell in range only."""
    top = (1 << 31) - 1
    g = np.random.default_rng(2)
    seq, ell = np.array([3, 3, 8, 0]), np.array([top, 2, top, top])
    table, free, F = _pool(g, 4, 4, np.array([1, 2, 2, 0]), 3)
    for alias in (False, True):
        want = _commit(seq, ell, np.array([1, 1, top, 0]), table, free, F, 4, 5, status=np.zeros(4, np.int32), alias=alias)
        assert want["n_new"].tolist() == [0, 2, 0, 0]


def _step(L):
    """Loop.step with the statuses of all its calls handed on."""
    s = sdv.sd_slot_reserve(L.seq, L.ell, L.table, L.free, L.F, BS, Q, x0=L.x0, tokens=L.drafts)
    rows = torch.index_select(L.model, 0, s["row_token"].clamp(0, V - 1))   # the target's pass
    z = sdv.sd_logit_shape(rows, s["row0"], s["ell"], V, draft_tokens=L.drafts, repetition=L.rep, frequency=L.freq,
                           presence=L.pres, seen=L.seen, counts=L.counts, mask=L.mask_w, mask_row0=L.m0,
                           out=dict(logits=rows))
    v = sdv.sd_verify(rows, s["row0"], L.drf, L.drf_row0, L.drafts, s["ell"], V, 1.0, 77, pos0=L.seq)
    status = s["status"] | z["status"] | v["status"]
    c = sdv.sd_slot_commit(L.seq, s["ell"], v["n_acc"], L.table, L.free, s["free_count"], BS, out_tokens=v["tokens"],
                           x0=L.x0, status=status, release=L.release)
    sdv.sd_token_counts(v["tokens"], L.seen, L.counts, V, length=c["n_new"])
    torch.cuda.synchronize()
    return s, z, v, c, status


def test_loop_holds_refused_requests():
    L = Loop(4)
    L.ell = torch.full((R,), G, dtype=torch.int32, device=DEV)
    L.rep[1] = float("nan")                          # refused by the shaping
    L.m0[4] = L.mask_w.shape[0] - 1                  # its grammar has rows missing
    pool = int(L.F[0])
    blocks = -(-Q // BS)
    good = L.free.clone()
    L.free[pool - 1 - 2 * blocks] = 10 ** 6          # request 2 gets a block that is not there
    L.drafts[3, 0] = V + 5                           # a bad token holds nothing back
    held = [1, 2, 4]
    before = {k: getattr(L, k).clone() for k in ("seq", "x0", "seen", "counts")}
    s, z, v, c, status = _step(L)
    assert (to_np(s["status"])[[2]] == sdv.SD_ST_BAD_INPUT).all() and (to_np(z["status"])[[1, 4]] & 32 == 32).all()
    assert to_np(z["status"])[3] & sdv.SD_ST_BAD_TOKEN
    n_new = to_np(c["n_new"])
    free = [r for r in range(R) if r not in held]
    assert (n_new[held] == 0).all() and (n_new[free] == to_np(v["n_acc"])[free] + 1).all()
    assert torch.equal(c["seq_len"][held], before["seq"][held]) and torch.equal(c["x0"][held], before["x0"][held])
    assert torch.equal(L.seen[held], before["seen"][held]) and torch.equal(L.counts[held], before["counts"][held])
    assert (to_np(L.counts.sum(1))[free] == n_new[free]).all()
    # their blocks are free again
    back = pool - len(free) * blocks
    assert int(c["free_count"]) >= back
    # put right, the step goes through
    L.seq, L.x0, L.F = c["seq_len"], c["x0"], c["free_count"]
    L.free.copy_(torch.where(L.free == 10 ** 6, good[pool - 1 - 2 * blocks], L.free))
    L.rep[1] = 1.5
    L.m0[4] = 4 * Q
    s, z, v, c, status = _step(L)
    assert (c["n_new"] == v["n_acc"] + 1).all() and ((s["status"] | z["status"]) & 32 == 0).all()


def test_overlapping_outputs_are_refused():
    """Refused on the host, whatever the kernel chosen; the in-place forms that
    the interface names are not."""
    i = lambda *k: torch.zeros(k, dtype=torch.int32, device=DEV)  # noqa: E731
    n, q = 9, 3
    seq, acc, tok, x0, table, free, F = torch.zeros(n, dtype=torch.int64, device=DEV), i(n), i(n, q), i(n), i(n, 4), \
        i(40), i(1)
    for out in (dict(n_new=acc), dict(x0=acc), dict(n_new=x0, x0=x0), dict(free_count=free[:1])):
        with pytest.raises(sdv.SdvError):
            sdv.sd_slot_commit(seq, i(n) - 1, acc, table, free, F, 16, out_tokens=tok, x0=x0, out=out)
    sdv.sd_slot_commit(seq, i(n) - 1, acc, table, free, F, 16, out_tokens=tok, x0=x0,
                       out=dict(seq_len=seq, x0=x0, free_count=F))
    ell = i(n) - 1
    for out in (dict(ctx_len=ell), dict(status=ell), dict(batch=F), dict(row0=x0), dict(row_token=tok.view(-1))):
        with pytest.raises(sdv.SdvError):
            sdv.sd_slot_reserve(seq, ell, table, free, F, 16, q, x0=x0, tokens=tok, out=out)
    sdv.sd_slot_reserve(seq, ell, table, free, F, 16, q, x0=x0, tokens=tok, out=dict(ell=ell, free_count=F))
    cu = i(n + 1) + 9
    got = sdv.sd_slot_reserve(seq, i(n), i(n, 4), torch.arange(40, dtype=torch.int32, device=DEV), i(1) + 40, 16, q,
                              out=dict(cu_rows=cu, batch=cu[n:]))
    assert cu.tolist() == list(range(n + 1)) and got["batch"].tolist() == [n]
    x = torch.zeros((2 * n, 64), device=DEV)
    row0, none = i(n), i(n) - 1
    with pytest.raises(sdv.SdvError):
        sdv.sd_logit_shape(x[:n], row0, none, 64, gamma_max=0, out=dict(logits=x[1:n + 1]))
    with pytest.raises(sdv.SdvError):
        sdv.sd_logit_shape(x, row0, none, 64, gamma_max=0, out=dict(status=none))
    sdv.sd_logit_shape(x[:n], row0, none, 64, gamma_max=0, out=dict(logits=x[n:]))
    with pytest.raises(sdv.SdvError):
        sdv.sd_token_counts(tok, i(n, 2), i(n, 64), 64, length=acc, out=dict(status=acc))
