"""Paged caches with contents and their fp64 values, and bounds for attention."""

import numpy as np
import torch

from oracle import heads as OH

DEV = "cuda"
U = 2.0 ** -24


def np64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def random_cache(g, kind, blocks, n_kv, bs, D, loud=1.0):
    """A cache full of values (also where no token will be), and [blocks][n_kv][bs][D] fp64 of both sides."""
    if kind == "bf16":
        cache = tuple((loud * torch.randn((blocks, n_kv, bs, D), generator=g)).to(torch.bfloat16) for _ in range(2))
        return tuple(t.to(DEV) for t in cache), [np64(t) for t in cache]
    codes = [torch.randint(0, 256, (blocks, n_kv, bs, D // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
    scale = [torch.randint(124, 129, (blocks, n_kv, bs, D // 32), generator=g, dtype=torch.uint8) for _ in range(2)]
    return tuple(t.to(DEV) for t in codes + scale), [OH.values(c.numpy(), s.numpy()) for c, s in zip(codes, scale)]


def random_batch(g, R, q_max, lo, hi, bs, spare=2, empty=True):
    """Rows and contexts of R requests: n, ctx, row0 (packed, with a gap), the table and its blocks' number."""
    n = torch.randint(1, q_max + 1, (R,), generator=g)
    n[0] = q_max
    if empty and R > 2:
        n[2] = 0
    ctx = torch.randint(lo, hi + 1, (R,), generator=g)
    ctx[0], ctx[-1] = hi, lo
    ctx = torch.maximum(ctx, n)
    row0 = torch.cumsum(n, 0) - n + 1
    held = (ctx + bs - 1) // bs
    mb = int(held.max()) + 1
    perm = torch.randperm(int(held.sum()) + spare, generator=g).to(torch.int32)
    table = torch.full((R, mb), -7, dtype=torch.int32)
    at = 0
    for r in range(R):
        table[r, :held[r]] = perm[at:at + int(held[r])]
        at += int(held[r])
    return n, ctx, row0, table, len(perm)


def tokens_of(side, table, r, T, bs):
    """[T][n_kv][D] of request r."""
    b = table[r, :-(-T // bs)].numpy() if isinstance(table, torch.Tensor) else table[r, :-(-T // bs)]
    x = side[b]                                   # [blocks][n_kv][bs][D]
    return x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])[:T]


def visible(n, T, causal, window):
    pos = T - n + np.arange(n)[:, None]
    t = np.arange(T)[None]
    see = t <= pos if causal else np.ones((n, T), bool)
    return see & (t > pos - window) if window else see


def check(got, got_lse, q, k, v, see, scale, tag=()):
    """One request's rows against fp64.  Bounds: D products summed in fp32
    leave a score within (D + 8) u of the sum of their sizes, its exponent is
    rounded once more, and weight and normaliser both carry that; a weight is
    rounded to bf16 (2^-8), sums over T tokens lose at most u for each, the
    result is rounded once (2^-8)."""
    want, lse, size = OH.attend(q, k, v, see, scale)
    n, n_q, D = q.shape
    T, G = k.shape[0], n_q // k.shape[1]
    big = np.zeros((n, n_q))
    for h in range(n_q):
        a = np.abs(q[:, h]) @ np.abs(np.where(np.isfinite(k[:, h // G]), k[:, h // G], 0.0)).T * scale
        big[:, h] = np.where(see, a, 0.0).max(-1, initial=0.0)
    e = 2 * (D + 24) * U * big + (T + 64) * U
    tol = 2.0 ** -8 * np.abs(want) + size * (2.0 ** -8 + 2 * e[..., None]) * (1 + 2.0 ** -7) + 1e-30
    ok = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), ok), (tag, np.argwhere(np.isfinite(got) != ok)[:5])
    bad = ok & (np.abs(np.where(ok, got, 0.0) - np.where(ok, want, 0.0)) > np.where(ok, tol, 0.0))
    assert not bad.any(), (tag, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])
    if got_lse is not None:
        fine = np.isfinite(lse)
        assert np.array_equal(np.isneginf(got_lse), np.isneginf(lse)), tag
        off = np.abs(np.where(fine, got_lse - np.where(fine, lse, 0), 0))
        assert (off <= np.where(fine, e + 8 * U * np.abs(np.where(fine, lse, 0)), 0) + 8 * U).all(), (tag, off.max())
