"""sd_cache_attn with a sliding window whose blocks behind it have been given
back: what no row sees needs no block, what some row sees does."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from tests.attn_util import DEV, check, gen, np64, random_batch, random_cache, tokens_of, visible

pytestmark = pytest.mark.gpu

FORMS = [(64, 4, 1, 1), (64, 8, 1, 6), (64, 8, 2, 40), (128, 4, 2, 1), (128, 4, 1, 11), (128, 8, 1, 30), (256, 2, 2, 3),
         (256, 4, 1, 30), (96, 4, 2, 5), (192, 4, 1, 20)]


def _run(b, table, **mask):
    i32 = lambda t: t.to(torch.int32).to(DEV)  # noqa: E731
    plan = sdv.sd_attn_plan(i32(b["row0"]), i32(b["n"] - 1), i32(b["ctx"]), b["q_max"], b["q"].shape[1], b["cache"],
                            **mask)
    r = sdv.sd_cache_attn(b["q"], b["cache"], table.to(DEV), plan, lse=True)
    return np64(r["out"]), np64(r["lse"]), r["status"].tolist()


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
@pytest.mark.parametrize("bs", [16, 64, 5])
@pytest.mark.parametrize("D,n_q,n_kv,q_max", FORMS)
def test_blocks_behind_the_window(kind, bs, D, n_q, n_kv, q_max):
    g = gen(D + bs + q_max)
    R = 6
    n, ctx, row0, table, blocks = random_batch(g, R, q_max, q_max + 150, 700, bs, empty=False)
    cache, sides = random_cache(g, kind, blocks, n_kv, bs, D)
    q = torch.randn((int(n.sum()) + 3, n_q, D), generator=g).to(torch.bfloat16).to(DEV)
    b = dict(n=n, ctx=ctx, row0=row0, cache=cache, q=q, q_max=q_max)
    for window in (1, 17, 64, 100):
        for causal in (True, False):
            first = ctx - n - window + 1                  # the first token that a row sees
            given = table.clone()
            for r in range(R):
                given[r, :max(int(first[r]), 0) // bs] = (-1, 1 << 30)[r % 2]
            assert (given[:, :int(ctx.max()) // bs] != table[:, :int(ctx.max()) // bs]).any()
            out, lse, status = _run(b, given, window=window, causal=causal)
            assert status == [0] * R, (window, causal)
            for r in range(R):
                m, T, r0 = int(n[r]), int(ctx[r]), int(row0[r])
                k, v = (tokens_of(x, table, r, T, bs) for x in sides)
                check(out[r0:r0 + m], lse[r0:r0 + m], np64(q)[r0:r0 + m], k, v, visible(m, T, causal, window),
                      float(np.float32(D ** -0.5)), (r, window, causal))
            # the block of the first token that a row sees: its request is told, the others are not
            at = [int(first[r]) // bs for r in range(R)]
            for r in (0, 3):
                given[r, at[r]] = -1
            out, lse, status = _run(b, given, window=window, causal=causal)
            assert status == [sdv.SD_ST_BAD_INPUT if r in (0, 3) else 0 for r in range(R)], (window, causal)
            for r in (0, 2, 3):
                m, T, r0 = int(n[r]), int(ctx[r]), int(row0[r])
                k, v = (tokens_of(x, table, r, T, bs) for x in sides)
                see = visible(m, T, causal, window)
                if r != 2:
                    see = see & (np.arange(T) // bs != at[r])[None]
                check(out[r0:r0 + m], lse[r0:r0 + m], np64(q)[r0:r0 + m], k, v, see, float(np.float32(D ** -0.5)),
                      (r, window, causal))
