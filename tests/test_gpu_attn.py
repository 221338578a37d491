"""sd_attn_plan and sd_cache_attn against fp64, over a cache in bf16 and in 4 bits."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from tests.attn_util import DEV, check, gen, np64, random_batch, random_cache, tokens_of, visible

pytestmark = pytest.mark.gpu

BAD_INPUT = sdv.SD_ST_BAD_INPUT


def _i32(t):
    return torch.as_tensor(t).to(torch.int32).to(DEV)


def _setup(seed, kind, R, q_max, n_q, n_kv, D, bs, lo, hi, loud=1.0, empty=True):
    g = gen(seed)
    n, ctx, row0, table, blocks = random_batch(g, R, q_max, lo, hi, bs, empty=empty)
    cache, sides = random_cache(g, kind, blocks, n_kv, bs, D, loud)
    rows = int(n.sum()) + 3
    q = (1.5 * torch.randn((rows, n_q, D), generator=g)).to(torch.bfloat16).to(DEV)
    return dict(n=n, ctx=ctx, row0=row0, table=table, cache=cache, sides=sides, rows=rows, q=q, bs=bs, q_max=q_max,
                n_q=n_q, n_kv=n_kv, D=D, R=R)


def _run(s, causal=True, window=0, scale=None, plan=None, lse=True, q=None, out=None):
    if plan is None:
        plan = sdv.sd_attn_plan(_i32(s["row0"]), _i32(s["n"] - 1), _i32(s["ctx"]), s["q_max"], s["n_q"], s["cache"],
                                causal=causal, window=window)
    if out is None:
        out = dict(out=torch.full((s["rows"], s["n_q"], s["D"]), 77.0, dtype=torch.bfloat16, device=DEV))
        if lse:
            out["lse"] = torch.full((s["rows"], s["n_q"]), 77.0, device=DEV)
    r = sdv.sd_cache_attn(s["q"] if q is None else q, s["cache"], s["table"].to(DEV), plan, scale=scale, out=out)
    torch.cuda.synchronize()
    return r


def _compare(s, r, causal=True, window=0, scale=None, skip=(), see_of=None):
    out, q = np64(r["out"]), np64(s["q"])
    lse = None if r["lse"] is None else np64(r["lse"])
    scale = float(np.float32(s["D"] ** -0.5 if scale is None else scale))
    live = np.zeros(s["rows"], bool)
    for b in range(s["R"]):
        n, T, r0 = int(s["n"][b]), int(s["ctx"][b]), int(s["row0"][b])
        if n == 0 or b in skip:
            continue
        live[r0:r0 + n] = True
        k, v = (tokens_of(x, s["table"], b, T, s["bs"]) for x in s["sides"])
        see = visible(n, T, causal, window)
        if see_of is not None:
            see = see & see_of(b, T)[None]
        check(out[r0:r0 + n], None if lse is None else lse[r0:r0 + n], q[r0:r0 + n], k, v, see, scale, (b,))
    assert (out[~live] == 77.0).all()
    if lse is not None:
        assert (lse[~live] == 77.0).all()


SHAPES = [  # R, q_max, n_q, n_kv, D, bs, lo, hi
    (1, 1, 1, 1, 64, 1, 1, 1), (3, 1, 4, 2, 64, 16, 1, 70), (5, 1, 16, 2, 128, 16, 30, 400),
    (2, 1, 7, 1, 96, 5, 64, 129), (4, 3, 10, 2, 128, 33, 3, 200), (6, 5, 12, 3, 64, 64, 5, 640),
    (3, 9, 14, 2, 96, 48, 10, 300), (4, 12, 16, 4, 128, 64, 12, 500), (2, 17, 8, 1, 128, 17, 20, 260),
    (3, 4, 20, 4, 192, 16, 4, 300), (2, 1, 6, 6, 256, 100, 1, 500), (3, 13, 5, 1, 256, 256, 13, 300),
    (2, 40, 8, 2, 128, 16, 40, 333), (3, 150, 3, 1, 64, 32, 150, 400), (2, 70, 4, 2, 192, 128, 70, 200),
    (40, 2, 8, 4, 128, 16, 2, 90)]


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("R,q_max,n_q,n_kv,D,bs,lo,hi", SHAPES)
def test_attention(R, q_max, n_q, n_kv, D, bs, lo, hi, kind):
    s = _setup(R + D + bs, kind, R, q_max, n_q, n_kv, D, bs, lo, hi)
    r = _run(s)
    _compare(s, r)
    assert (r["status"] == 0).all()
    again = _run(s)          # the same bits, whatever the order of the workgroups
    assert torch.equal(again["out"], r["out"]) and torch.equal(again["lse"], r["lse"])


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 37), (True, 64), (False, 50), (True, 100000),
                                           (False, 1)])
def test_masks(causal, window, kind):
    for q_max, n_q, n_kv, D in ((6, 8, 2, 64), (40, 6, 1, 128), (1, 4, 4, 96)):
        s = _setup(window + q_max, kind, 5, q_max, n_q, n_kv, D, 16, q_max, 380)
        _compare(s, _run(s, causal, window, scale=0.21), causal, window, scale=0.21)


@pytest.mark.parametrize("kind,D,n_q,n_kv,q_max,T", [("bf16", 64, 2, 1, 1, 70001), ("fp4", 128, 4, 2, 2, 30011),
                                                    ("bf16", 128, 8, 1, 13, 20000), ("fp4", 256, 4, 1, 3, 9000)])
def test_long_context(kind, D, n_q, n_kv, q_max, T):
    """One request cut over many workgroups, and a short one beside it."""
    s = _setup(T, kind, 2, q_max, n_q, n_kv, D, 64, 20, T)
    _compare(s, _run(s))


def test_strides_and_no_lse():
    s = _setup(5, "bf16", 4, 5, 6, 2, 128, 16, 6, 200)
    wide = torch.randn((s["rows"], 10, 128), generator=gen(6)).to(torch.bfloat16).to(DEV)
    s["q"] = wide[:, 2:8]
    full = torch.full((s["rows"], 7, 128), 77.0, dtype=torch.bfloat16, device=DEV)
    r = _run(s, out=dict(out=full[:, :6]))
    assert r["lse"] is None and (full[:, 6] == 77.0).all()
    _compare(s, r)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("n_q,n_kv,q_max,D", [(8, 2, 1, 64), (4, 1, 5, 128), (16, 2, 5, 128), (16, 1, 8, 96),
                                              (8, 1, 9, 256)])
def test_what_is_masked_may_hold_anything(n_q, n_kv, q_max, D, kind):
    """NaN and infinities behind the last token, in drafts that earlier rows do
    not see, and before the window; rows that see them show it."""
    bs, window = 16, 40
    s = _setup(D + n_q, kind, 4, q_max, n_q, n_kv, D, bs, q_max + 30, 150, empty=False)
    k, v = s["cache"][:2] if kind == "bf16" else s["cache"][2:]
    odd = [float("nan"), float("inf"), -float("inf")]

    def spoil(t, b, pos, x):
        block, off = int(s["table"][b, pos // bs]), pos % bs
        if kind == "bf16":
            t[block, pos % n_kv, off, (7 * pos) % D] = x
        else:
            t[block, pos % n_kv, off, (7 * pos) % D // 32] = 255
    for b in range(4):
        T, n = int(s["ctx"][b]), int(s["n"][b])
        for pos in range(T, -(-T // bs) * bs):          # the page's stale end
            for t in (k, v):
                for x in odd:
                    spoil(t, b, pos, x)
        spoil(v, b, T - 1, odd[b % 3])                  # the last row's own value
        if b == 1 and n > 2:
            spoil(k, b, T - 2, odd[0])
        spoil(v, b, T - n - window, odd[(b + 1) % 3])   # before every row's window
        if n > 1:
            spoil(v, b, T - n - window + 1, odd[2])     # before every row's but the first's
    if kind == "bf16":
        s["sides"] = [np64(t) for t in s["cache"]]
    else:
        from oracle import heads as OH
        s["sides"] = [OH.values(s["cache"][i].cpu().numpy(), s["cache"][2 + i].cpu().numpy()) for i in range(2)]
    _compare(s, _run(s, True, window), True, window)
    _compare(s, _run(s, True, 0), True, 0)


def test_extreme_scores():
    """Scores of some thousand, a row whose scores are all -inf, and one of which is +inf."""
    s = _setup(9, "bf16", 3, 3, 4, 1, 64, 16, 20, 100, loud=40.0, empty=False)
    _compare(s, _run(s, scale=1.0), scale=1.0)
    k = s["cache"][0]
    T, n, r0 = int(s["ctx"][1]), int(s["n"][1]), int(s["row0"][1])
    for p in range(T):
        k[int(s["table"][1, p // 16]), 0, p % 16, 3] = -float("inf")
    s["q"][r0:r0 + n, :, 3] = 1.0
    T2, r2 = int(s["ctx"][2]), int(s["row0"][2])
    k[int(s["table"][2, 0]), 0, 1, 5] = float("inf")
    s["q"][r2:r2 + int(s["n"][2]), :, 5] = 2.0
    r = _run(s)
    assert (r["out"][r0:r0 + n] == 0).all() and (r["lse"][r0:r0 + n] == -float("inf")).all()
    assert T2 > 1 and r["out"][r2:r2 + int(s["n"][2])].isnan().all()
    s["sides"] = [np64(t) for t in s["cache"]]
    _compare(s, dict(out=r["out"].nan_to_num(77.0).where(r["out"].isnan() | (r["out"] != 0), 77.0), lse=None),
             skip=(1, 2))


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_blocks_outside_the_pool(kind):
    s = _setup(11, kind, 4, 6, 8, 2, 128, 16, 100, 300, empty=False)
    good = s["table"].clone()
    s["table"][1, 2], s["table"][1, 4] = -1, 1 << 30
    s["table"][3, 0] = s["cache"][0].shape[0]
    r = _run(s)
    assert r["status"].tolist() == [0, BAD_INPUT, 0, BAD_INPUT]
    pool, bad = s["cache"][0].shape[0], s["table"].numpy()
    s["table"] = good
    _compare(s, r, see_of=lambda b, T: ~np.isin(np.arange(T) // 16, np.flatnonzero((bad[b] < 0) | (bad[b] >= pool))))
    # none of a request's blocks in the pool: its rows see nothing
    s["table"] = good.clone()
    s["table"][2] = -1
    r = _run(s)
    r0, n = int(s["row0"][2]), int(s["n"][2])
    assert (r["out"][r0:r0 + n] == 0).all() and (r["lse"][r0:r0 + n] == -float("inf")).all()
    assert r["status"].tolist() == [0, 0, BAD_INPUT, 0]


def test_requests_out_of_range():
    s = _setup(12, "bf16", 6, 4, 4, 2, 64, 16, 30, 90, empty=False)
    s["ctx"][1] = int(s["n"][1]) - 1          # fewer tokens than rows
    s["row0"][2] = -1
    s["row0"][3] = s["rows"] - int(s["n"][3]) + 1      # past the row buffers
    ctx4, s["ctx"][4] = int(s["ctx"][4]), s["table"].shape[1] * 16 + 1     # past the table
    r = _run(s)
    assert r["status"].tolist() == [0, BAD_INPUT, BAD_INPUT, BAD_INPUT, BAD_INPUT, 0]
    s["ctx"][4] = ctx4
    _compare(s, r, skip=(1, 2, 3, 4))
    # ell past q_max - 1 counts as q_max - 1
    s = _setup(13, "bf16", 3, 4, 4, 2, 64, 16, 30, 90)
    plan = sdv.sd_attn_plan(_i32(s["row0"]), _i32(torch.where(s["n"] == 4, 1000, s["n"] - 1)), _i32(s["ctx"]), 4, 4,
                            s["cache"])
    _compare(s, _run(s, plan=plan))


def test_a_plan_for_other_sizes_writes_nothing():
    s = _setup(14, "bf16", 3, 4, 4, 2, 64, 16, 30, 90)
    plan = sdv.sd_attn_plan(_i32(s["row0"]), _i32(s["n"] - 1), _i32(s["ctx"]), 4, 4, s["cache"])
    r = _run(s, plan=dict(plan, q_max=3))
    assert (r["out"] == 77.0).all() and (r["lse"] == 77.0).all()
    with pytest.raises(ValueError, match="plan"):
        _run(s, plan=dict(plan, n_kv=4))
    _compare(s, _run(s, plan=plan))


def test_no_requests_and_no_rows():
    s = _setup(15, "bf16", 3, 4, 4, 2, 64, 16, 30, 90)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    plan = sdv.sd_attn_plan(e, e, e, 4, 4, s["cache"])
    r = sdv.sd_cache_attn(s["q"], s["cache"], torch.empty((0, 4), dtype=torch.int32, device=DEV), plan)
    assert r["out"].shape == s["q"].shape
    s["n"][:] = 0                               # a step in which every request sits out
    r = _run(s)
    assert (r["out"] == 77.0).all() and (r["status"] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_offsets_past_32_bits(kind):
    """Blocks behind 2^32 bytes of each side."""
    n_kv, bs, D = 2, 256, 128
    row = n_kv * bs * (D * 2 if kind == "bf16" else D // 2)
    blocks = (1 << 32) // row + 8
    s = _setup(16, kind, 2, 3, 4, n_kv, D, bs, 300, 1000)
    small = s["cache"]
    s["cache"] = tuple(torch.zeros((blocks,) + t.shape[1:], dtype=t.dtype, device=DEV) for t in small)
    for t, x in zip(s["cache"], small):
        t[-x.shape[0]:] = x
    table = s["table"]
    s["table"] = torch.where(table < 0, table, table + blocks - small[0].shape[0])
    r = _run(s)
    s["table"] = table
    _compare(s, r)
