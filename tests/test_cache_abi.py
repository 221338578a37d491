"""Host checks of the paged cache's entry points: bad arguments, and written
arguments that overlap others, are refused before anything reaches the GPU, so
the addresses need not exist."""

import ctypes
import itertools

import pytest
import torch

import draft_verification_amd as sdv
from draft_verification_amd import _lib

OK, E, RANGE, U = _lib.SD_OK, _lib.SD_EINVAL, _lib.SD_ERANGE, _lib.SD_EUNSUPPORTED
BF, F32, C16, C4 = _lib.SD_DTYPE_BF16, _lib.SD_DTYPE_F32, _lib.SD_CACHE_BF16, _lib.SD_CACHE_FP4


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _far(names):
    """An address per argument, too far apart to meet."""
    return {n: (i + 1) << 44 for i, n in enumerate(names)}


ROPE = ("q", "k", "pos", "wq", "wk", "freq", "qo", "ko")


def _rope(n=6, D=64, dt=BF, n_q=4, ld_q=256, n_kv=2, ld_k=128, eps=1e-6, rot=64, inter=0, ld_qo=256, ld_ko=128, **at):
    a = {**_far(ROPE), **at}
    return sdv.lib().sd_qk_rope(None, n, D, dt, _p(a["q"]), n_q, ld_q, _p(a["k"]), n_kv, ld_k, _p(a["pos"]),
                                _p(a["wq"]), _p(a["wk"]), eps, _p(a["freq"]), rot, inter, _p(a["qo"]), ld_qo,
                                _p(a["ko"]), ld_ko)


def test_rope_host_validation():
    nan, inf = float("nan"), float("inf")
    for kw in (dict(n=-1), dict(D=0), dict(D=60), dict(dt=2), dict(n_q=-1), dict(n_kv=-1), dict(rot=-8),
               dict(rot=12), dict(rot=72), dict(inter=2), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
               dict(pos=None), dict(freq=None), dict(freq=264), dict(wq=264), dict(wk=264), dict(q=None), dict(k=None),
               dict(qo=None), dict(ko=None), dict(q=264), dict(k=264), dict(qo=264), dict(ko=264), dict(ld_q=248),
               dict(ld_q=260), dict(ld_k=120), dict(ld_qo=248), dict(ld_ko=132)):
        assert _rope(**kw) == E, kw
    assert _rope(D=264, ld_q=2048, ld_k=2048, ld_qo=2048, ld_ko=2048) == U
    assert _rope(n_q=1025, ld_q=1 << 17, ld_qo=1 << 17) == U
    assert _rope(n_kv=1025, ld_k=1 << 17, ld_ko=1 << 17) == U
    assert _rope(n=0, pos=None, q=None) == OK
    assert _rope(n_q=0, n_kv=0, q=None, k=None) == OK
    assert _rope(n=1 << 30, D=8, rot=8, n_q=1, n_kv=1, ld_q=8, ld_k=8, ld_qo=8, ld_ko=8) == U   # past one launch


APPEND = ("q", "k", "v", "pos", "slot", "wq", "wk", "freq", "qo", "kc", "vc", "ks", "vs")


def _append(n=6, D=64, dt=BF, n_q=4, ld_q=256, ld_k=128, ld_v=128, n_kv=2, eps=1e-6, rot=64, inter=0, ld_qo=256,
            ctype=C4, bs=16, blocks=8, **at):
    a = {**_far(APPEND), **at}
    return sdv.lib().sd_cache_append(None, n, D, dt, _p(a["q"]), n_q, ld_q, _p(a["k"]), ld_k, _p(a["v"]), ld_v, n_kv,
                                     _p(a["pos"]), _p(a["slot"]), _p(a["wq"]), _p(a["wk"]), eps, _p(a["freq"]), rot,
                                     inter, _p(a["qo"]), ld_qo, ctype, bs, blocks, _p(a["kc"]), _p(a["vc"]),
                                     _p(a["ks"]), _p(a["vs"]))


def test_append_host_validation():
    for kw in (dict(n=-1), dict(D=60), dict(D=40, rot=40), dict(dt=2), dict(n_q=-1), dict(n_kv=0), dict(rot=12),
               dict(inter=-1), dict(eps=-1.0), dict(pos=None), dict(slot=None), dict(freq=None), dict(ctype=2),
               dict(bs=0), dict(blocks=-1), dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(kc=None),
               dict(vc=None), dict(ks=None), dict(vs=None), dict(kc=264), dict(vc=264),
               dict(ks=260), dict(vs=264), dict(v=264), dict(ld_v=120),
               dict(ld_k=132), dict(ld_qo=120)):
        assert _append(**kw) == E, kw
    assert _append(D=288, ld_q=2048, ld_k=2048, ld_v=2048, ld_qo=2048) == U
    assert _append(bs=1 << 30, blocks=1 << 11) == U
    assert _append(n=0, slot=None, kc=None) == OK


READ = ("slot", "kc", "vc", "ks", "vs", "ko", "vo")


def _read(n=6, D=64, ctype=C4, n_kv=2, bs=16, blocks=8, dt=BF, ld_k=128, ld_v=128, **at):
    a = {**_far(READ), **at}
    return sdv.lib().sd_cache_read(None, n, D, _p(a["slot"]), ctype, n_kv, bs, blocks, _p(a["kc"]), _p(a["vc"]),
                                   _p(a["ks"]), _p(a["vs"]), dt, _p(a["ko"]), ld_k, _p(a["vo"]), ld_v)


def test_read_host_validation():
    for kw in (dict(n=-1), dict(D=60), dict(D=40), dict(dt=2), dict(n_kv=0), dict(ctype=2), dict(bs=0),
               dict(blocks=-1), dict(slot=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None),
               dict(ko=None), dict(vo=None), dict(kc=264), dict(ks=260), dict(vs=264), dict(ko=264), dict(ld_k=120), dict(ld_v=132)):
        assert _read(**kw) == E, kw
    assert _read(D=288, ld_k=2048, ld_v=2048) == U
    assert _read(n_kv=1025, ld_k=1 << 17, ld_v=1 << 17) == U
    assert _read(bs=1 << 30, blocks=1 << 11) == U
    assert _read(n=0, slot=None) == OK


def _size(R=6, q_max=5, n_q=8, n_kv=2, D=128):
    return sdv.sd_attn_workspace_size(R, q_max, n_q, n_kv, D)


PLAN = ("row0", "ell", "ctx", "status", "ws")


def _plan(R=6, q_max=5, n_q=8, n_kv=2, D=128, ctype=C16, bs=16, causal=1, window=0, size=None, **at):
    a = {**_far(PLAN), **at}
    return sdv.lib().sd_attn_plan(None, R, q_max, n_q, n_kv, D, ctype, bs, _p(a["row0"]), _p(a["ell"]), _p(a["ctx"]),
                                  causal, window, _p(a["status"]), _p(a["ws"]), _size() if size is None else size)


def test_plan_host_validation():
    for kw in (dict(R=-1), dict(q_max=0), dict(n_q=0), dict(n_kv=0), dict(n_q=7), dict(D=0), dict(ctype=2),
               dict(bs=0), dict(causal=2), dict(window=-1), dict(row0=None), dict(ell=None), dict(ctx=None),
               dict(status=None), dict(ws=None), dict(ws=128)):
        assert _plan(**kw) == E, kw
    for kw in (dict(D=80), dict(D=320), dict(n_q=2048), dict(R=1 << 15, q_max=1 << 14, n_q=64)):
        assert _plan(**kw) == U, kw
    assert _plan(size=128) == RANGE
    assert _plan(R=0, row0=None) == OK
    assert _size(D=80) == 0 and _size(R=-1) == 0 and _size(n_q=7) == 0
    # both types of cache, any block size, and smaller steps fit in what the size says
    assert _size(R=5) <= _size() and _size(q_max=4) <= _size()


ATTN = ("q", "kc", "vc", "ks", "vs", "table", "out", "lse", "status", "ws")


def _attn(R=6, q_max=5, n_q=8, n_kv=2, D=128, n=30, ld_q=1024, ctype=C4, bs=16, blocks=8, mb=4, scale=0.1, ld_out=1024,
          size=None, **at):
    a = {**_far(ATTN), **at}
    return sdv.lib().sd_cache_attn(None, R, q_max, n_q, n_kv, D, n, _p(a["q"]), ld_q, ctype, bs, blocks, _p(a["kc"]),
                                   _p(a["vc"]), _p(a["ks"]), _p(a["vs"]), _p(a["table"]), mb, scale, _p(a["out"]),
                                   ld_out, _p(a["lse"]), _p(a["status"]), _p(a["ws"]),
                                   _size() if size is None else size)


def test_attn_host_validation():
    for kw in (dict(R=-1), dict(q_max=0), dict(n_q=7), dict(ctype=2), dict(n=-1), dict(bs=0), dict(blocks=-1),
               dict(blocks=0), dict(mb=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(q=None), dict(out=None), dict(kc=None), dict(vc=None), dict(ks=None),
               dict(vs=None), dict(table=None), dict(status=None), dict(ws=None), dict(q=264), dict(out=264),
               dict(kc=264), dict(vc=264), dict(ks=260), dict(vs=264), dict(ws=128), dict(ld_q=1016), dict(ld_q=1028), dict(ld_out=1016),
               dict(ld_out=1028)):
        assert _attn(**kw) == E, kw
    for kw in (dict(D=80), dict(bs=1 << 20, mb=1 << 12), dict(bs=1 << 30, blocks=1 << 11, mb=1),
               dict(n_kv=8, bs=1 << 29, mb=1)):
        assert _attn(**kw) == U, kw
    assert _attn(size=128) == RANGE
    assert _attn(R=0, q=None) == OK and _attn(n=0, q=None) == OK


# (bytes, written) of what each call above is given
SIZES = {
    "rope": dict(q=(6 * 512, 0), k=(6 * 256, 0), pos=(24, 0), wq=(256, 0), wk=(256, 0), freq=(128, 0),
                 qo=(6 * 512, 1), ko=(6 * 256, 1)),
    "append": dict(q=(6 * 512, 0), k=(6 * 256, 0), v=(6 * 256, 0), pos=(24, 0), slot=(48, 0), wq=(256, 0),
                   wk=(256, 0), freq=(128, 0), qo=(6 * 512, 1), kc=(256 * 32, 1), vc=(256 * 32, 1), ks=(512, 1),
                   vs=(512, 1)),
    "read": dict(slot=(48, 0), kc=(256 * 32, 0), vc=(256 * 32, 0), ks=(512, 0), vs=(512, 0), ko=(6 * 256, 1),
                 vo=(6 * 256, 1)),
    "plan": dict(row0=(24, 0), ell=(24, 0), ctx=(24, 0), status=(24, 1), ws=(None, 1)),
    "attn": dict(q=(30 * 2048, 0), kc=(256 * 64, 0), vc=(256 * 64, 0), ks=(1024, 0), vs=(1024, 0), table=(96, 0),
                 out=(30 * 2048, 1), lse=(960, 1), status=(24, 1), ws=(None, 1)),
}
CALLS = dict(rope=_rope, append=_append, read=_read, plan=_plan, attn=_attn)
IN_PLACE = {("q", "qo"), ("k", "ko")}   # from the same start


@pytest.mark.parametrize("what", SIZES)
def test_overlaps_are_refused(what):
    sizes = {k: (_size() if n is None else n, w) for k, (n, w) in SIZES[what].items()}
    at = _far(sizes)
    for (x, (nx, wx)), (y, (ny, wy)) in itertools.combinations(sizes.items(), 2):
        if not (wx or wy):
            continue
        starts = [at[x] + (nx - 1) // 256 * 256]          # y begins in x's last bytes
        if (x, y) not in IN_PLACE or what == "append" and x == "k":
            starts.append(at[x])
        for s in starts:
            if s + ny > at[x] + (1 << 43) or s % 256:
                continue
            assert CALLS[what](**{x: at[x], y: s}) == E, (x, y, s - at[x])


def test_binding_refuses():
    z = lambda *k, t=torch.bfloat16: torch.zeros(k, dtype=t)  # noqa: E731
    i = lambda *k: z(*k, t=torch.int32)  # noqa: E731
    cache, slot = (z(4, 2, 16, 64), z(4, 2, 16, 64)), torch.zeros(6, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_qk_rope(z(6, 4, 64), z(6, 2, 64), i(6))
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_cache_append(z(6, 2, 64), z(6, 2, 64), cache, slot)
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_cache_read(slot, cache)
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_attn_plan(i(3), i(3), i(3), 5, 4, cache)
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_cache_attn(z(6, 4, 64), cache, i(3, 2), dict(n_q=4, n_kv=2, D=64, R=3, q_max=2))
    with pytest.raises(TypeError, match="tensor"):
        sdv.sd_qk_rope(None, None, None)
