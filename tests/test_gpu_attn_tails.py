"""sd_cache_attn where a context ends inside a block, inside a unit of tokens and
inside the part of it that a wave loads: block sizes of whole such parts, and
contexts of each kind of rest, all requests live, the last block of the pool
full to its end."""

import pytest
import torch

import numpy as np

import draft_verification_amd as sdv
from tests.attn_util import DEV, check, gen, np64, random_cache, tokens_of, visible

pytestmark = pytest.mark.gpu

CTX = [416, 150, 1024, 33, 79, 80, 81, 159, 64, 63, 1, 768]
FORMS = [(64, 1, 1, 1), (64, 8, 1, 4), (64, 12, 2, 8), (64, 8, 2, 15), (64, 8, 1, 9), (64, 8, 1, 40), (128, 16, 2, 2),
         (128, 4, 1, 8), (128, 10, 2, 9), (128, 4, 1, 16), (128, 4, 1, 30), (256, 4, 2, 8), (256, 4, 1, 9),
         (256, 2, 1, 40), (96, 4, 4, 3), (96, 4, 1, 30), (192, 3, 1, 11), (192, 3, 1, 30)]


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
@pytest.mark.parametrize("bs", [16, 32, 64, 256])
@pytest.mark.parametrize("D,n_q,n_kv,q_max", FORMS)
def test_ends_of_contexts(kind, bs, D, n_q, n_kv, q_max):
    g = gen(17)
    R = len(CTX)
    ctx = torch.tensor(CTX)
    n = torch.minimum(torch.tensor([q_max if r % 3 == 0 else 1 + (5 * r) % q_max for r in range(R)]), ctx)
    row0 = torch.cumsum(n, 0) - n
    held = (ctx + bs - 1) // bs
    blocks = int(held.sum())
    perm = torch.randperm(blocks - 1, generator=g).to(torch.int32)
    # the pool's last block is the last of 1024 or of 768 tokens, which fill it
    table, at = torch.full((R, int(held.max())), -7, dtype=torch.int32), 0
    for r in range(R):
        table[r, :held[r]] = torch.cat([perm, torch.tensor([blocks - 1], dtype=torch.int32)])[at:at + int(held[r])]
        at += int(held[r])
    assert int(table[R - 1, int(held[R - 1]) - 1]) == blocks - 1 and CTX[-1] % bs == 0
    cache, sides = random_cache(g, kind, blocks, n_kv, bs, D)
    q = torch.randn((int(n.sum()), n_q, D), generator=g).to(torch.bfloat16).to(DEV)
    i32 = lambda t: t.to(torch.int32).to(DEV)  # noqa: E731
    plan = sdv.sd_attn_plan(i32(row0), i32(n - 1), i32(ctx), q_max, n_q, cache)
    r = sdv.sd_cache_attn(q, cache, table.to(DEV), plan, lse=True)
    out, lse, status = np64(r["out"]), np64(r["lse"]), r["status"].cpu()
    assert not status.any()
    for b in range(R):
        m, T, r0 = int(n[b]), int(ctx[b]), int(row0[b])
        k, v = (tokens_of(x, table, b, T, bs) for x in sides)
        check(out[r0:r0 + m], lse[r0:r0 + m], np64(q)[r0:r0 + m], k, v, visible(m, T, True, 0),
              float(np.float32(D ** -0.5)), (b, T))
