"""Host checks of the entry points around a step (logit shaping, token counts,
cache slots): bad arguments are refused before anything reaches the GPU."""

import ctypes

import pytest
import torch

import draft_verification_amd as sdv
from draft_verification_amd import _lib

A = ctypes.c_void_p(256)


def _shape(R=2, g=2, V=64, ld=64, dt=1, n_rows=6, at=256, out=256, ld_seen=2, ld_counts=64, n_slots=2, n_bias=4,
           ld_mask=2, n_mask=4, counts=256, have=()):
    """have: which optional arguments are given."""
    P = lambda n: A if n in have else None  # noqa: E731
    v = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    req = [None if "no_" + n in have else A for n in ("row0", "ell", "status")]
    return sdv.lib().sd_logit_shape(
        None, R, g, V, ld, dt, v(at), v(out), n_rows, req[0], req[1], P("draft"), P("rep"), P("freq"), P("pres"),
        P("seen"), ld_seen, v(counts) if "counts" in have else None, ld_counts, n_slots, P("slot"), P("off"),
        P("tok"), P("val"), n_bias, P("mask"), ld_mask, n_mask, P("m0"), req[2])


def test_shape_host_validation():
    E, U = _lib.SD_EINVAL, _lib.SD_EUNSUPPORTED
    for kw in (dict(R=-1), dict(g=-1), dict(V=60), dict(V=0), dict(ld=56), dict(ld=68), dict(dt=2), dict(n_rows=-1),
               dict(at=None), dict(out=None), dict(at=264), dict(out=264), dict(have=("no_row0",)),
               dict(have=("no_ell",)), dict(have=("no_status",)),
               dict(have=("rep",)),                                   # penalties without seen
               dict(have=("freq", "seen")), dict(have=("pres", "seen")),   # ... without counts
               dict(have=("rep", "seen"), n_slots=0), dict(have=("rep", "seen"), ld_seen=1),
               dict(have=("freq", "seen", "counts"), ld_counts=60),
               dict(have=("freq", "seen", "counts"), ld_counts=66),
               dict(have=("freq", "seen", "counts"), counts=264),
               dict(have=("off",)), dict(have=("off", "tok")), dict(have=("off", "tok", "val"), n_bias=-1),
               dict(have=("mask",)), dict(have=("mask", "m0"), ld_mask=1), dict(have=("mask", "m0"), n_mask=-1)):
        assert _shape(**kw) == E, kw
    assert _shape(g=256) == U
    assert _shape(V=(1 << 24) + 8, ld=(1 << 24) + 8) == U
    assert _shape(have=("off", "tok", "val"), n_bias=(1 << 30) + 1) == U
    assert _shape(R=1 << 20, V=1 << 24, ld=1 << 24) == U          # more work-items than one launch holds
    assert _shape(R=0, at=None) == _lib.SD_OK                     # nothing to do


def _counts(R=2, V=64, tokens=256, n=8, width=4, start=None, length=None, seen=256, ld_seen=2, counts=256,
            ld_counts=64, n_slots=2, status=256):
    v = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return sdv.lib().sd_token_counts(None, R, V, v(tokens), n, width, v(start), v(length), None, None, None,
                                     v(seen), ld_seen, v(counts), ld_counts, n_slots, v(status))


def test_counts_host_validation():
    E = _lib.SD_EINVAL
    for kw in (dict(R=-1), dict(V=12), dict(n=-1), dict(width=-1), dict(tokens=None), dict(seen=None),
               dict(status=None), dict(n_slots=0), dict(ld_seen=1), dict(ld_counts=60), dict(ld_counts=66),
               dict(counts=260), dict(start=256)):
        assert _counts(**kw) == E, kw
    assert _counts(n=7) == _lib.SD_ERANGE                         # lists past the buffer
    assert _counts(V=(1 << 24) + 8, ld_counts=1 << 25) == _lib.SD_EUNSUPPORTED
    assert _counts(R=0, seen=None) == _lib.SD_OK


def _reserve(R=2, q=3, bs=16, mb=4, pool=8, rows=6, padded=0, ld=3, nulls=(), tokens=True, x0=True, ws=256,
             wsb=4096):
    P = lambda n: None if n in nulls else A  # noqa: E731
    return sdv.lib().sd_slot_reserve(
        None, R, q, bs, mb, pool, rows, padded, P("seq"), P("ell"), A if x0 else None, A if tokens else None, ld,
        P("table"), P("list"), P("count"), P("ell_out"), P("row0"), P("cu"), P("ctx"), P("batch"), P("left"),
        P("req"), P("pos"), P("slot"), P("token"), P("status"), ctypes.c_void_p(ws), wsb)


def test_reserve_host_validation():
    E, U = _lib.SD_EINVAL, _lib.SD_EUNSUPPORTED
    for kw in (dict(R=-1), dict(q=0), dict(bs=0), dict(mb=0), dict(pool=-1), dict(rows=-1), dict(padded=2),
               dict(tokens=False), dict(x0=False, tokens=False), dict(ws=260)):
        assert _reserve(**kw) == E, kw
    for n in ("seq", "ell", "table", "list", "count", "ell_out", "row0", "cu", "ctx", "batch", "left", "req", "pos",
              "slot", "status"):
        assert _reserve(nulls=(n,)) == E, n
    assert _reserve(rows=0) == _lib.SD_ERANGE
    assert _reserve(padded=1, rows=5) == _lib.SD_ERANGE           # reserved rows do not fit
    assert _reserve(ld=1) == _lib.SD_ERANGE                       # token rows too short
    assert _reserve(ld=2, x0=False) == _lib.SD_ERANGE
    assert _reserve(wsb=sdv.sd_slot_reserve_workspace_size(2) - 1) == _lib.SD_ERANGE
    assert _reserve(bs=1 << 16, mb=1 << 15) == U
    assert _reserve(R=1 << 16, q=1 << 15) == U
    assert _reserve(R=1 << 16, mb=1 << 15) == U
    assert _reserve(rows=(1 << 31) - 1) == U
    assert sdv.sd_slot_reserve_workspace_size(-1) == 0
    assert sdv.sd_slot_reserve_workspace_size(1) % 256 == 0


def _commit(R=2, q=3, bs=16, mb=4, pool=8, nulls=(), ws=256, wsb=4096):
    P = lambda n: None if n in nulls else A  # noqa: E731
    return sdv.lib().sd_slot_commit(
        None, R, q, bs, mb, pool, P("seq"), P("ell"), P("acc"), P("tokens"), P("x0"), None, None, P("table"),
        P("list"), P("count"), None, P("seq_out"), P("x0_out"), P("new"), P("count_out"), ctypes.c_void_p(ws), wsb)


def test_commit_host_validation():
    E, U = _lib.SD_EINVAL, _lib.SD_EUNSUPPORTED
    for kw in (dict(R=-1), dict(q=0), dict(bs=0), dict(mb=0), dict(pool=-1), dict(ws=260)):
        assert _commit(**kw) == E, kw
    for n in ("seq", "ell", "acc", "tokens", "x0", "table", "list", "count", "seq_out", "new", "count_out"):
        assert _commit(nulls=(n,)) == E, n
    assert _commit(wsb=sdv.sd_slot_commit_workspace_size(2) - 1) == _lib.SD_ERANGE
    assert _commit(bs=1 << 16, mb=1 << 15) == U
    assert _commit(R=1 << 16, q=1 << 15) == U
    assert _commit(R=1 << 16, mb=1 << 15) == U
    assert sdv.sd_slot_commit_workspace_size(-1) == 0


def test_binding_refuses_host_tensors():
    i = lambda *k: torch.zeros(k, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_logit_shape(torch.zeros(2, 64), i(2), i(2), 64, gamma_max=0)
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_token_counts(i(2, 3), i(2, 2), i(2, 64), 64)
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_slot_reserve(torch.zeros(2, dtype=torch.int64), i(2), i(2, 4), i(8), i(1), 16, 3)
    with pytest.raises(ValueError, match="GPU"):
        sdv.sd_slot_commit(torch.zeros(2, dtype=torch.int64), i(2), i(2), i(2, 4), i(8), i(1), 16, q_max=3)
    with pytest.raises(TypeError, match="tensor"):
        sdv.sd_logit_shape(None, i(2), i(2), 64, gamma_max=0)


def test_status_strings_of_the_new_bits():
    for bit in (sdv.SD_ST_BAD_INPUT, sdv.SD_ST_NO_SLOT):
        assert sdv.sd_status_string(bit) != "unknown status"
