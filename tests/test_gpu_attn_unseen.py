"""sd_cache_attn over a cache in 4 bits whose scales reach past the largest
value: with byte 253 the levels 4 and 6 are infinite, with 254 those from 2 on,
with 255 all are NaN.  Where a row does not see them they do not touch it; where
it does, the infinite ones are infinite and the others what they stand for."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from oracle import heads as OH
from tests.attn_util import DEV, check, gen, np64, random_batch, random_cache, tokens_of, visible

pytestmark = pytest.mark.gpu

BS = 16
# D, query heads, key heads, rows: the forms for a few queries with 1 to 4 times 16 of them, and the others
FORMS = [(64, 4, 1, 1), (64, 4, 1, 7), (64, 8, 2, 10), (64, 4, 1, 14), (64, 8, 1, 12), (128, 4, 2, 1), (128, 4, 1, 7),
         (128, 8, 2, 10), (128, 4, 1, 30), (256, 2, 2, 1), (256, 4, 1, 4), (256, 4, 1, 9), (96, 4, 2, 3), (192, 4, 2, 9)]


def _reads(codes, scale):
    """What the codes are read as: bf16, infinite from 2^128 on."""
    x = OH.values(codes, scale)
    return np.where(np.abs(x) >= 2.0 ** 128, np.copysign(np.inf, x), x)


def _setup(D, n_q, n_kv, q_max, lo, hi, spoil):
    """spoil(request, its rows, its tokens): token -> (scale byte, codes or None) of values and keys."""
    g = gen(D + n_q + q_max)
    n, ctx, row0, table, blocks = random_batch(g, 4, q_max, lo, hi, BS, empty=False)
    cache, _ = random_cache(g, "fp4", blocks, n_kv, BS, D)
    host = [t.cpu() for t in cache]
    for b in range(4):
        for side, pos, byte, codes in spoil(b, int(n[b]), int(ctx[b])):
            block, off = int(table[b, pos // BS]), pos % BS
            host[2 + side][block, :, off, :] = byte
            if codes is not None:
                host[side][block, :, off, :] = codes
    cache = tuple(t.to(DEV) for t in host)
    sides = [_reads(host[i].numpy(), host[2 + i].numpy()) for i in range(2)]
    q = torch.randn((int(n.sum()) + 3, n_q, D), generator=g).to(torch.bfloat16).to(DEV)
    return n, ctx, row0, table, cache, sides, q


def _run(n, ctx, row0, table, cache, q, q_max, **mask):
    i32 = lambda t: t.to(torch.int32).to(DEV)  # noqa: E731
    plan = sdv.sd_attn_plan(i32(row0), i32(n - 1), i32(ctx), q_max, q.shape[1], cache, **mask)
    r = sdv.sd_cache_attn(q, cache, table.to(DEV), plan, lse=True)
    assert not r["status"].any()
    return np64(r["out"]), np64(r["lse"])


@pytest.mark.parametrize("D,n_q,n_kv,q_max", FORMS)
@pytest.mark.parametrize("byte", [253, 254, 255])
@pytest.mark.parametrize("window", [0, 40])
def test_unseen_scales(window, byte, D, n_q, n_kv, q_max):
    """Random codes under such scales behind the last token, in tokens that only
    the last row sees, and before every row's window, keys and values alike."""

    def spoil(b, n, T):
        for pos in range(T, -(-T // BS) * BS):
            yield 0, pos, byte, None
            yield 1, pos, byte, None
        if window:
            for pos in range(max(0, T - n - window - 20), T - n - window + 1):
                yield 0, pos, byte, None
                yield 1, pos, byte, None
        if b != 1 and n > 1:      # the last row's own values: 0, 6 and -6 alone
            yield 1, T - 1, byte, 0x7F if b == 0 else 0xF0

    n, ctx, row0, table, cache, sides, q = _setup(D, n_q, n_kv, q_max, q_max + 30, 300, spoil)
    out, lse = _run(n, ctx, row0, table, cache, q, q_max, window=window)
    for b in range(4):
        m, T, r0 = int(n[b]), int(ctx[b]), int(row0[b])
        k, v = (tokens_of(x, table, b, T, BS) for x in sides)
        see = visible(m, T, True, window)
        check(out[r0:r0 + m], lse[r0:r0 + m], np64(q)[r0:r0 + m], k, v, see, float(np.float32(D ** -0.5)), (b,))
        want = OH.attend(np64(q)[r0:r0 + m], k, v, see, float(np.float32(D ** -0.5)))[0]
        assert np.array_equal(np.isinf(want), np.isinf(out[r0:r0 + m]))
        assert (out[r0:r0 + m][np.isinf(want)] == want[np.isinf(want)]).all()


@pytest.mark.parametrize("D,n_q,n_kv,q_max", FORMS)
@pytest.mark.parametrize("byte", [252, 253, 254])
def test_seen_one_at_a_time(byte, D, n_q, n_kv, q_max):
    """Each row sees its own token alone: what comes out is its values, finite or not."""

    def spoil(b, n, T):
        for pos in range(max(0, T - n - 5), T):
            yield 1, pos, byte, None

    n, ctx, row0, table, cache, sides, q = _setup(D, n_q, n_kv, q_max, q_max + 5, 200, spoil)
    out, _ = _run(n, ctx, row0, table, cache, q, q_max, window=1)
    for b in range(4):
        m, T, r0 = int(n[b]), int(ctx[b]), int(row0[b])
        v = tokens_of(sides[1], table, b, T, BS)[T - m:]
        assert np.array_equal(out[r0:r0 + m], np.repeat(v, n_q // n_kv, 1))


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
@pytest.mark.parametrize("D,n_q,n_kv,q_max", FORMS)
def test_missing_blocks(kind, D, n_q, n_kv, q_max):
    """Blocks outside the pool while the pool's first block, nobody's, holds
    nothing finite; one request also sees an infinite value of its own."""
    g = gen(D + q_max + 1)
    n, ctx, row0, table, blocks = random_batch(g, 4, q_max, q_max + 120, 300, BS, empty=False)
    table = torch.where(table < 0, table, table + 1)
    cache, _ = random_cache(g, kind, blocks + 1, n_kv, BS, D)
    for side in range(2):
        if kind == "fp4":
            cache[2 + side][0] = torch.tensor([253, 254, 255, 253] * 4, dtype=torch.uint8, device=DEV)[None, :, None]
        else:
            cache[side][0] = float("inf") if side else float("nan")
    one = int(table[2, 1])
    if kind == "fp4":
        cache[1][one, :, 3], cache[3][one, :, 3] = 0x7F, 253
    else:
        cache[1][one, :, 3] = -float("inf")
    host = [t.cpu() for t in cache]
    sides = [_reads(host[i].numpy(), host[2 + i].numpy()) if kind == "fp4" else np64(host[i]) for i in range(2)]
    q = torch.randn((int(n.sum()) + 3, n_q, D), generator=g).to(torch.bfloat16).to(DEV)
    given = table.clone()
    given[0, 2], given[2, 4], given[3, 0] = -1, blocks + 1, 1 << 30
    i32 = lambda t: t.to(torch.int32).to(DEV)  # noqa: E731
    plan = sdv.sd_attn_plan(i32(row0), i32(n - 1), i32(ctx), q_max, n_q, cache)
    r = sdv.sd_cache_attn(q, cache, given.to(DEV), plan, lse=True)
    bad = sdv.SD_ST_BAD_INPUT
    assert r["status"].tolist() == [bad, 0, bad, bad]
    out, lse = np64(r["out"]), np64(r["lse"])
    for b, gone in enumerate((2, None, 4, 0)):
        m, T, r0 = int(n[b]), int(ctx[b]), int(row0[b])
        k, v = (tokens_of(x, table, b, T, BS) for x in sides)
        see = visible(m, T, True, 0)
        if gone is not None:
            see = see & (np.arange(T) // BS != gone)[None]
        check(out[r0:r0 + m], lse[r0:r0 + m], np64(q)[r0:r0 + m], k, v, see, float(np.float32(D ** -0.5)), (b,))
        assert np.isfinite(out[r0:r0 + m]).all() == (b != 2)
