"""A plan is for one type of cache and one block size: others are refused."""

import pytest
import torch

import draft_verification_amd as sdv
from tests.attn_util import DEV, gen, random_cache

pytestmark = pytest.mark.gpu


def _plan(cache):
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return sdv.sd_attn_plan(i32(0, 2), i32(1, 1), i32(40, 64), 2, 4, cache)


def test_other_caches_are_refused():
    q = torch.randn((4, 4, 64), generator=gen(1)).to(torch.bfloat16).to(DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    caches = [random_cache(gen(2), kind, 8, 2, bs, 64)[0] for kind, bs in (("bf16", 16), ("fp4", 16), ("bf16", 32))]
    plans = [_plan(c) for c in caches]
    for i, cache in enumerate(caches):
        for k, plan in enumerate(plans):
            if i == k:
                assert sdv.sd_cache_attn(q, cache, table, plan)["out"].isfinite().all()
            else:
                with pytest.raises(ValueError, match="plan is for"):
                    sdv.sd_cache_attn(q, cache, table, plan)
    # one layer's plan serves another layer's cache of its kind
    other = random_cache(gen(3), "fp4", 9, 2, 16, 64)[0]
    assert sdv.sd_cache_attn(q, other, table, plans[1])["out"].isfinite().all()
