"""sd_qk_rope, sd_cache_append and sd_cache_read against fp64.

Bounds, in units of u = 2^-24 (half a step of fp32): the sum of squares has up
to 13 roundings of positive terms (7 of a lane, one to start, 5 joins), half of
which pass through the root; the mean, eps, root, reciprocal and the two
products add 6; cosine and sine are within 2 steps of values up to 1 (4u) and
see an angle of up to pi half turns rounded once (1.6u); two products and their
sum add 3.  All of them stay below 24u of |a| + |b| of the pair.  Rounding to
bf16 adds 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from oracle import heads as OH

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy()


def _heads(g, n, h, D, dtype, pad=0, extra=0):
    """Rows of heads, cut from wider rows, and what lies around them."""
    full = torch.randn((n, extra + h * D + pad), generator=g) * 2
    full = full.to(TYPES[dtype]).to(DEV)
    return full[:, extra:extra + h * D].unflatten(1, (h, D)) if h else None


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _freq(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEV) if rot else None


def _near(got, want, size, dtype):
    tol = 24 * U * size + (2.0 ** -8 * np.abs(want) * (1 + 24 * U) if dtype == "bf16" else 0) + 1e-45
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,n_q,n_kv,D,rot,norm", [
    (1, 1, 1, 8, 8, "qk"), (3, 4, 1, 64, 64, "qk"), (17, 7, 1, 128, 64, ""), (5, 3, 3, 80, 24, "q"),
    (130, 5, 2, 96, 96, "k"), (33, 8, 8, 256, 128, "qk"), (2, 0, 3, 128, 128, "k"), (7, 3, 0, 192, 192, "q"),
    (64, 6, 2, 128, 0, "qk"), (4000, 9, 3, 64, 32, "qk"), (9, 70, 5, 40, 16, "")])
def test_rope(n, n_q, n_kv, D, rot, norm, interleaved, dtype):
    g = _gen(n + D + rot)
    if n_q == 0:      # the binding takes queries first: keys alone go there
        n_q, n_kv, norm = n_kv, 0, norm.replace("k", "q")
    q = _heads(g, n, n_q, D, dtype, 24, 16)
    k = _heads(g, n, n_kv, D, dtype, 8)
    pos = torch.randint(0, 1 << 20, (n,), generator=g).to(torch.int32)
    pos[0] = 0
    if n > 3:
        pos[1], pos[2] = -1, (1 << 31) - 1
    pos = pos.to(DEV)
    wq, wk = ((torch.randn(D, generator=g) + 1).to(DEV) if s in norm else None for s in "qk")
    out = dict(q=torch.full((n, n_q, D), 9.0, dtype=q.dtype, device=DEV))
    if n_kv:
        out["k"] = torch.full((n, n_kv, D), 9.0, dtype=q.dtype, device=DEV)
    f = _freq(rot)
    r = sdv.sd_qk_rope(q, k, pos, f, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved, out=out)
    torch.cuda.synchronize()
    live = (pos >= 0).cpu().numpy()
    for x, w, y in ((q, wq, r["q"]), (k, wk, r["k"])):
        if x is None:
            continue
        want, size = OH.turn(_np(x), None if w is None else _np(w), _np(pos), None if f is None else _np(f), 1e-5,
                             interleaved)
        _near(_np(y)[live], want[live], size[live], dtype)
        assert (_np(y)[~live] == 9.0).all()
    # in place: the same bits
    q2, k2 = q.clone(), None if k is None else k.clone()
    r2 = sdv.sd_qk_rope(q2, k2, pos, f, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved,
                        out=dict(q=q2, k=k2))
    torch.cuda.synchronize()
    for key in ("q", "k"):
        if r[key] is not None:
            assert torch.equal(r2[key][pos >= 0], r[key][pos >= 0])
    if n > 3:
        assert torch.equal(q2[1], q[1])


def test_zero_and_non_finite_heads():
    x = torch.randn((4, 3, 64), generator=_gen(1)).to(DEV)
    x[0, 0] = 0
    x[1, 1, 5] = float("inf")
    x[2, 2, 7] = float("nan")
    r = sdv.sd_qk_rope(x, None, torch.arange(4, dtype=torch.int32, device=DEV), _freq(64),
                       q_weight=torch.ones(64, device=DEV), eps=0.0)["q"]
    ok = torch.ones((4, 3), dtype=torch.bool)
    ok[0, 0] = ok[1, 1] = ok[2, 2] = False
    assert r.isfinite().all(-1).cpu().equal(ok)       # a head's fault stays in it
    r = sdv.sd_qk_rope(x, None, torch.arange(4, dtype=torch.int32, device=DEV), _freq(64),
                       q_weight=torch.ones(64, device=DEV), eps=1e-6)["q"]
    assert (r[0, 0] == 0).all()


def _cache(kind, blocks, n_kv, bs, D, fill=0x5A):
    if kind == "bf16":
        return tuple(torch.full((blocks, n_kv, bs, D), 0.125, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    return tuple(torch.full((blocks, n_kv, bs, c), fill, dtype=torch.uint8, device=DEV)
                 for c in (D // 2, D // 2, D // 32, D // 32))


def _at(cache, part, slots, bs):
    return cache[part][slots // bs, :, slots % bs].cpu().numpy() if cache[part].dtype == torch.uint8 else \
        _np(cache[part][slots // bs, :, slots % bs])


CASES = [(1, 0, 1, 32, 32, 1, 3), (5, 4, 2, 64, 64, 16, 2), (60, 8, 2, 128, 128, 16, 9), (33, 0, 3, 96, 32, 7, 11),
         (200, 16, 4, 192, 96, 64, 5), (17, 5, 5, 256, 256, 13, 4), (3000, 4, 1, 128, 64, 256, 14),
         (700, 3, 9, 64, 0, 100, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("n,n_q,n_kv,D,rot,bs,blocks", CASES)
def test_append_and_read(n, n_q, n_kv, D, rot, bs, blocks, kind, interleaved, dtype):
    g = _gen(n + D)
    q = _heads(g, n, n_q, D, dtype, 8)
    k, v = _heads(g, n, n_kv, D, dtype, 16, 8), _heads(g, n, n_kv, D, dtype)
    k[:, :, 3] *= 8
    slot = torch.randperm(blocks * bs, generator=g)[:n]
    assert len(slot) == min(n, blocks * bs)
    slot = torch.cat([slot, torch.full((n - len(slot),), -1)])
    pos = torch.randint(0, 100000, (n,), generator=g).to(torch.int32)
    if n > 4:
        slot[1], slot[2], pos[3] = -1, blocks * bs, -1      # no slot, past the cache, no request's
    slot, pos = slot.to(DEV), pos.to(DEV)
    wk = (torch.rand(D, generator=g) + 0.5).to(DEV)
    wq = (torch.rand(D, generator=g) + 0.5).to(DEV) if n_q else None
    cache = _cache(kind, blocks, n_kv, bs, D)
    before = [t.clone() for t in cache]
    f = _freq(rot)
    qo = torch.full((n, n_q, D), 9.0, dtype=k.dtype, device=DEV)
    r = sdv.sd_cache_append(k, v, cache, slot, row_pos=pos, inv_freq=f, q=q, q_weight=wq, k_weight=wk, eps=1e-6,
                            interleaved=interleaved, out=dict(q=qo))
    torch.cuda.synchronize()
    fn = None if f is None else _np(f)
    live = ((slot >= 0) & (slot < blocks * bs) & (pos >= 0)).cpu().numpy()
    if n_q:
        want, size = OH.turn(_np(q), _np(wq), _np(pos), fn, 1e-6, interleaved)
        on = (pos >= 0).cpu().numpy()
        _near(_np(r["q"])[on], want[on], size[on], dtype)
        assert (_np(r["q"])[~on] == 9.0).all()
    else:
        assert r["q"] is None
    want_k, size_k = OH.turn(_np(k), _np(wk), _np(pos), fn, 1e-6, interleaved)
    at = slot[torch.from_numpy(live).to(DEV)]
    if kind == "bf16":
        _near(_at(cache, 0, at, bs), want_k[live], size_k[live], "bf16")
        assert np.array_equal(_at(cache, 1, at, bs), _np(v.bfloat16())[live])
    else:
        for part, want, size in ((0, want_k[live], size_k[live]), (1, _np(v)[live], np.abs(_np(v))[live])):
            byte = _at(cache, 2 + part, at, bs)
            slack = 24 * U * size if part == 0 else 0 * size
            # the scale: the exact one's, or its neighbour's where the largest magnitude is that near to its border
            top = np.abs(want).reshape(want.shape[:2] + (-1, 32)).max(-1)
            room = slack.reshape(want.shape[:2] + (-1, 32)).max(-1)
            s = np.exp2(byte.astype(np.float64) - 127)
            assert (top - room <= 7 * s).all() and (top + room > 3.5 * s).all()
            got = OH.values(_at(cache, part, at, bs), byte)
            best = np.abs(OH.nearest(want, byte.astype(np.int64) - 127) - want)
            assert (np.abs(got - want) <= best + slack).all()
            exact = slack == 0
            assert np.array_equal(got[exact], OH.nearest(want, byte.astype(np.int64) - 127)[exact])
    # nothing else changed
    rest = torch.ones(blocks * bs, dtype=torch.bool, device=DEV)
    rest[at] = False
    rest = torch.nonzero(rest)[:, 0]
    for t, b in zip(cache, before):
        assert torch.equal(t[rest // bs, :, rest % bs], b[rest // bs, :, rest % bs])
    # and back, in both types, with a slot twice
    for dt in (torch.bfloat16, torch.float32):
        want = [OH.values(_at(cache, p, at, bs), _at(cache, 2 + p, at, bs)) if kind == "fp4" else _at(cache, p, at, bs)
                for p in range(2)]
        back = sdv.sd_cache_read(torch.cat([at, at]), cache, dtype=dt)
        for got, w in zip((back["k"], back["v"]), want):
            assert got.dtype == dt and np.array_equal(_np(got), np.concatenate([w, w]))
    o = dict(k=torch.full((n, n_kv, D), 3.0, device=DEV), v=torch.full((n, n_kv, D), 3.0, device=DEV))
    sdv.sd_cache_read(slot, cache, out=o)
    out = ((slot < 0) | (slot >= blocks * bs))
    assert (o["k"][out] == 3.0).all() and (o["v"][out] == 3.0).all()


def test_4bit_borders_and_faults():
    """Every border between levels, the scales' borders, zeros, tiny and huge
    values, and groups that are not finite."""
    v = torch.zeros((40, 1, 64), device=DEV)
    steps = [0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7]
    up = [float(np.nextafter(np.float32(s), np.float32(9))) for s in steps]
    v[0, 0, :16] = torch.tensor(steps)
    v[1, 0, :16] = -torch.tensor(steps)
    v[2, 0, :15], v[2, 0, 15] = torch.tensor(up[:15]), 7
    v[3, 0, 0] = up[15]                       # over 7: the next scale
    v[4, 0, 0] = 3.5
    v[5, 0, 0] = float(np.nextafter(np.float32(3.5), np.float32(9)))
    v[6, 0, 0], v[7, 0, 0] = 2.0 ** -126, 2.0 ** -149
    v[8, 0, 0], v[8, 0, 1] = 3.4e38, -1.7e38
    v[9, 0, 3], v[10, 0, 33], v[11, 0, 0] = float("nan"), float("inf"), -float("inf")
    v[12:] = torch.randn((28, 1, 64), generator=_gen(3)).to(DEV) * torch.exp2(torch.arange(-14., 14.))[:, None, None].to(DEV)
    slot = torch.arange(40, device=DEV)
    cache = _cache("fp4", 3, 1, 16, 64)
    sdv.sd_cache_append(v, v, cache, slot)
    x = _np(v)[:, 0]
    for part in range(2):
        byte = _at(cache, 2 + part, slot, 16)[:, 0]
        fine = np.isfinite(x).reshape(40, 2, 32).all(-1)
        assert (byte[~fine] == 255).all()
        e = OH.scale_exponent(np.where(np.isfinite(x), x, 0.0))
        assert np.array_equal(byte[fine].astype(int) - 127, e[fine])
        got = OH.values(_at(cache, part, slot, 16), _at(cache, 2 + part, slot, 16))[:, 0].reshape(40, 2, 32)
        assert np.isnan(got[~fine]).all()
        want = OH.nearest(np.where(np.isfinite(x), x, 0.0), e).reshape(40, 2, 32)
        assert np.array_equal(got[fine], want[fine])
        assert np.array_equal(np.signbit(got[fine]), np.signbit(want[fine]))
    back = sdv.sd_cache_read(slot, cache)["v"]
    assert back[9, 0, :32].isnan().all() and back[9, 0, 32:].isfinite().all()


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_offsets_past_32_bits(kind):
    """The last blocks of a cache of more than 2^32 bytes on each side."""
    n_kv, bs, D = 8, 256, 128
    blocks = (1 << 32) // (n_kv * bs * (D * 2 if kind == "bf16" else D // 2)) + 3
    shapes = [D] if kind == "bf16" else [D // 2, D // 32]
    dt = torch.bfloat16 if kind == "bf16" else torch.uint8
    cache = tuple(torch.zeros((blocks, n_kv, bs, c), dtype=dt, device=DEV) for c in shapes for _ in range(2))
    slot = torch.tensor([blocks * bs - 1, 0, (blocks - 2) * bs + 5], device=DEV)
    x = torch.randn((3, n_kv, D), generator=_gen(4)).to(torch.bfloat16).to(DEV)
    sdv.sd_cache_append(x, x, cache, slot)
    back = sdv.sd_cache_read(slot, cache)
    for t in (back["k"], back["v"]):
        if kind == "bf16":
            assert torch.equal(t, x)
        else:
            assert np.array_equal(_np(t), OH.nearest(_np(x), OH.scale_exponent(_np(x))))
    assert sum(int(t.count_nonzero(dim=(1, 2, 3)).count_nonzero()) for t in cache[:2]) == 6


def test_most_heads():
    """1024 heads of queries on one of keys, 256 channels each, two rows."""
    g = _gen(77)
    q, k = _heads(g, 2, 1024, 256, "bf16"), _heads(g, 2, 1, 256, "bf16")
    w, freq, pos = torch.ones(256, device=DEV), _freq(256), torch.tensor([5, 70000], dtype=torch.int32, device=DEV)
    r = sdv.sd_qk_rope(q, k, pos, freq, w, w)
    torch.cuda.synchronize()
    for x, y in ((q, r["q"]), (k, r["k"])):
        want, size = OH.turn(_np(x), _np(w), _np(pos), _np(freq), 1e-6, False)
        _near(_np(y), want, size, "bf16")


def test_no_rows():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    i = lambda dt=torch.int32: torch.empty(0, dtype=dt, device=DEV)  # noqa: E731
    cache = _cache("fp4", 2, 1, 16, 64)
    assert sdv.sd_qk_rope(e(0, 4, 64), e(0, 1, 64), i(), _freq(64))["q"].shape == (0, 4, 64)
    sdv.sd_cache_append(e(0, 1, 64), e(0, 1, 64), cache, i(torch.int64), row_pos=i(), inv_freq=_freq(64))
    assert sdv.sd_cache_read(i(torch.int64), cache)["k"].shape == (0, 1, 64)
