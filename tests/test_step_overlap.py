"""Calls around a step whose written arguments overlap others are refused on the
host: nothing is launched, so the addresses need not exist."""

import ctypes
import itertools

import pytest
import torch

import draft_verification_amd as sdv
from draft_verification_amd import _lib

R, Q, BS, MB, POOL, ROWS, V, SLOTS = 6, 3, 16, 4, 40, 18, 64, 8

# (bytes, written) of every argument that is memory, in the order of the call
RESERVE = dict(seq=(8 * R, 0), ell=(4 * R, 0), x0=(4 * R, 0), tokens=(4 * R * Q, 0), table=(4 * R * MB, 1),
               free_list=(4 * POOL, 0), free_count=(4, 0), ell_out=(4 * R, 1), row0=(4 * R, 1), cu=(4 * R + 4, 1),
               ctx=(4 * R, 1), batch=(4, 1), left=(4, 1), row_req=(4 * ROWS, 1), row_pos=(4 * ROWS, 1),
               row_slot=(8 * ROWS, 1), row_token=(4 * ROWS, 1), status=(4 * R, 1), ws=(12 * R + 4, 1))
COMMIT = dict(seq=(8 * R, 0), ell=(4 * R, 0), n_acc=(4 * R, 0), tokens=(4 * R * Q, 0), x0=(4 * R, 0),
              release=(4 * R, 0), keep=(4 * R, 0), table=(4 * R * MB, 0), free_list=(4 * POOL, 1),
              free_count=(4, 0), status=(4 * R, 1), seq_out=(8 * R, 1), x0_out=(4 * R, 1), n_new=(4 * R, 1),
              left=(4, 1), ws=(12 * R, 1))
COUNTS = dict(tokens=(4 * 50, 0), start=(8 * R, 0), length=(4 * R, 0), prompt=(4 * R, 0), slot=(4 * R, 0),
              reset=(4 * R, 0), seen=(8 * SLOTS, 1), counts=(4 * SLOTS * V, 1), status=(4 * R, 1))
SHAPE = dict(logits=(4 * ROWS * V, 0), out=(4 * ROWS * V, 1), row0=(4 * R, 0), ell=(4 * R, 0), draft=(4 * R * 2, 0),
             rep=(4 * R, 0), freq=(4 * R, 0), pres=(4 * R, 0), seen=(8 * SLOTS, 0), counts=(4 * SLOTS * V, 0),
             slot=(4 * R, 0), off=(8 * R + 8, 0), tok=(4 * 30, 0), val=(4 * 30, 0), mask=(8 * ROWS, 0), m0=(4 * R, 0),
             status=(4 * R, 1))
# what a call may be given as input and output at once
SAME = {("ell", "ell_out"), ("free_count", "left"), ("seq", "seq_out"), ("x0", "x0_out"), ("logits", "out")}


def _call(what, at):
    a = {k: ctypes.c_void_p(v) for k, v in at.items()}
    L = sdv.lib()
    if what == "reserve":
        return L.sd_slot_reserve(None, R, Q, BS, MB, POOL, ROWS, 0, a["seq"], a["ell"], a["x0"], a["tokens"], Q,
                                 a["table"], a["free_list"], a["free_count"], a["ell_out"], a["row0"], a["cu"],
                                 a["ctx"], a["batch"], a["left"], a["row_req"], a["row_pos"], a["row_slot"],
                                 a["row_token"], a["status"], a["ws"], 1 << 12)
    if what == "commit":
        return L.sd_slot_commit(None, R, Q, BS, MB, POOL, a["seq"], a["ell"], a["n_acc"], a["tokens"], a["x0"],
                                a["release"], a["keep"], a["table"], a["free_list"], a["free_count"], a["status"],
                                a["seq_out"], a["x0_out"], a["n_new"], a["left"], a["ws"], 1 << 12)
    if what == "counts":
        return L.sd_token_counts(None, R, V, a["tokens"], 50, 0, a["start"], a["length"], a["prompt"], a["slot"],
                                 a["reset"], a["seen"], 2, a["counts"], V, SLOTS, a["status"])
    return L.sd_logit_shape(None, R, 2, V, V, 0, a["logits"], a["out"], ROWS, a["row0"], a["ell"], a["draft"],
                            a["rep"], a["freq"], a["pres"], a["seen"], 2, a["counts"], V, SLOTS, a["slot"], a["off"],
                            a["tok"], a["val"], 30, a["mask"], 2, ROWS, a["m0"], a["status"])


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that do not exist: only where nothing can be launched")
@pytest.mark.parametrize("what,args", [("reserve", RESERVE), ("commit", COMMIT), ("counts", COUNTS),
                                       ("shape", SHAPE)])
def test_overlaps_are_refused(what, args):
    apart = {k: (i + 1) << 20 for i, k in enumerate(args)}
    # what cannot be launched here is told from what is refused
    assert _call(what, apart) == _lib.SD_ELAUNCH
    for (a, (na, wa)), (b, (nb, wb)) in itertools.combinations(args.items(), 2):
        if not (wa or wb):      # inputs may share memory
            assert _call(what, dict(apart, **{b: apart[a]})) == _lib.SD_ELAUNCH, (a, b)
            continue
        same = _lib.SD_ELAUNCH if (a, b) in SAME else _lib.SD_EINVAL
        assert _call(what, dict(apart, **{b: apart[a]})) == same, (a, b)
        for off in {16 * ((na - 1) // 16), -16 * ((nb - 1) // 16)} - {0}:     # the last, the first bytes
            assert _call(what, dict(apart, **{b: apart[a] + off})) == _lib.SD_EINVAL, (a, b, off)
        for off in (16 * ((na + 15) // 16), -16 * ((nb + 15) // 16)):         # next to each other
            assert _call(what, dict(apart, **{b: apart[a] + off})) == _lib.SD_ELAUNCH, (a, b, off)


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that do not exist: only where nothing can be launched")
def test_rows_side_by_side_in_one_buffer():
    """Rows of one leading dimension interleave without meeting."""
    base, es, ld, rows = 1 << 20, 4, 160, 9

    def shape(shift, V=64, n=rows, dt=0):
        p = lambda x: ctypes.c_void_p(x)  # noqa: E731
        return sdv.lib().sd_logit_shape(None, 2, 2, V, ld, dt, p(base + (1 << 16)), p(base + (1 << 16) + shift), n,
                                        p(64), p(128), None, None, None, None, None, 0, None, 0, 0, None, None, None,
                                        None, 0, None, 0, 0, None, p(256))

    step = ld * es
    for k in range(-rows - 2, rows + 3):
        for off, free in ((0, False), (16, False), (240, False), (256, True), (320, True), (384, True), (400, False)):
            shift = k * step + off
            # row i of the one begins `off` behind row i + k of the other, and as far before row i + k + 1
            near = [k] * (off < 256) + [k + 1] * (off > step - 256)
            meets = any(abs(x) < rows for x in near) and not free
            want = _lib.SD_ELAUNCH if shift == 0 or not meets else _lib.SD_EINVAL
            assert shape(shift) == want, (k, off)
    state = lambda seen, ld_seen: sdv.lib().sd_token_counts(  # noqa: E731
        None, 2, 64, ctypes.c_void_p(64), 8, 4, None, None, None, None, None, ctypes.c_void_p(seen), ld_seen,
        ctypes.c_void_p(base), 72, 20, ctypes.c_void_p(256))
    # counts and bits of a slot in one row of 72 words
    assert state(base + 4 * 64, 72) == _lib.SD_ELAUNCH
    assert state(base + 4 * 63, 72) == _lib.SD_EINVAL
    assert state(base + 4 * 71, 72) == _lib.SD_EINVAL
    assert state(base + 4 * 64, 2) == _lib.SD_EINVAL
    assert state(base + 4 * 72 * 20, 2) == _lib.SD_ELAUNCH


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that do not exist: only where nothing can be launched")
def test_the_batch_may_end_the_prefix_sums():
    at = {k: (i + 1) << 20 for i, k in enumerate(RESERVE)}
    assert _call("reserve", dict(at, batch=at["cu"] + 4 * R)) == _lib.SD_ELAUNCH
    assert _call("reserve", dict(at, batch=at["cu"])) == _lib.SD_EINVAL
    assert _call("reserve", dict(at, batch=at["cu"] + 4 * R, row_pos=at["cu"])) == _lib.SD_EINVAL


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that do not exist: only where nothing can be launched")
def test_an_unbounded_list_length_meets_no_other_allocation_below():
    """n_tokens near 2^63 does not wrap round."""
    call = lambda seen: sdv.lib().sd_token_counts(  # noqa: E731
        None, 1, 64, ctypes.c_void_p(1 << 30), (1 << 63) - 1, 0, ctypes.c_void_p(64), ctypes.c_void_p(128), None, None,
        None, ctypes.c_void_p(seen), 2, None, 0, 1, ctypes.c_void_p(256))
    assert call((1 << 30) + 64) == _lib.SD_EINVAL
