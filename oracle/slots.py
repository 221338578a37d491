"""Rows and paged cache slots of a step (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

What it computes (LightSpec article, system section: token slots reserved for
the whole draft and cut after the fact; DSpark summary, "2.2": the verify
batch B = sum of 1 + l_r): one request after another takes its rows and
blocks, and after verification gives back what was not accepted.

Pins (tests/test_oracle_slots.py): the blocks of all requests and the free
list partition the pool after every step, and slots name what a dictionary
from (request, position) holds.
"""

import numpy as np

BAD_INPUT, NO_SLOT = 32, 64
HELD = 2 | 4 | BAD_INPUT   # a step of such a status is repeated


def blocks_of(n, block_size):
    return -(-n // block_size)


def reserve(seq_len, ell, table, free_list, free_count, block_size, q_max, max_rows, padded=False, x0=None,
            tokens=None):
    """Returns a dict like sd_slot_reserve's; `table` is updated in place."""
    R, max_blocks = table.shape
    pool = len(free_list)
    cap = block_size * max_blocks
    left = min(max(int(free_count), 0), pool)
    out = dict(ell=np.zeros(R, np.int32), row0=np.zeros(R, np.int32), cu_rows=np.zeros(R + 1, np.int32),
               ctx_len=np.zeros(R, np.int32), status=np.zeros(R, np.int32),
               row_req=np.full(max_rows, -1, np.int32), row_pos=np.full(max_rows, -1, np.int32),
               row_slot=np.full(max_rows, -1, np.int64), row_token=np.full(max_rows, -1, np.int32))
    row = 0           # rows of the requests before
    spoken_rows = 0   # rows the requests before wanted
    spoken = 0        # blocks the requests before needed
    for r in range(R):
        n0 = int(seq_len[r])
        asked = max(min(int(ell[r]), q_max - 1) + 1, 0)
        if n0 < 0 or n0 > cap:
            out["status"][r] |= BAD_INPUT
            n0 = asked = 0
        want = min(asked, cap - n0)
        wished = want
        if not padded:
            want = min(want, max(max_rows - spoken_rows, 0))
        spoken_rows += wished
        have = blocks_of(n0, block_size)
        need = blocks_of(n0 + want, block_size) - have
        got = min(need, max(min(max(int(free_count), 0), pool) - spoken, 0))
        n = min(want, (have + got) * block_size - n0)
        if n < asked:
            out["status"][r] |= NO_SLOT
        top = min(max(int(free_count), 0), pool) - 1 - spoken
        for k in range(got):
            table[r, have + k] = free_list[top - k]
        spoken += need
        left -= got
        first = r * q_max if padded else row
        out["row0"][r] = first if padded else min(first, max_rows - 1)
        out["cu_rows"][r] = row
        out["ell"][r] = n - 1
        out["ctx_len"][r] = 0 if out["status"][r] & BAD_INPUT else n0 + n
        for i in range(n):
            p = n0 + i
            block = int(table[r, p // block_size])
            good = 0 <= block < pool
            if not good:
                out["status"][r] |= BAD_INPUT
            out["row_req"][first + i] = r
            out["row_pos"][first + i] = p
            out["row_slot"][first + i] = block * block_size + p % block_size if good else -1
            if x0 is not None:
                out["row_token"][first + i] = x0[r] if i == 0 else tokens[r][i - 1]
            elif tokens is not None:
                out["row_token"][first + i] = tokens[r][i]
        row += n
    out["cu_rows"][R] = row
    out["batch"] = np.array([row], np.int32)
    out["free_count"] = np.array([left], np.int32)
    return out


def commit(seq_len, ell, n_acc, table, free_list, free_count, block_size, q_max, out_tokens=None, x0=None,
           status=None, release=None, keep=None):
    """Returns a dict like sd_slot_commit's; `free_list` and `status` are
    updated in place."""
    R, max_blocks = table.shape
    pool = len(free_list)
    cap = block_size * max_blocks
    at = min(max(int(free_count), 0), pool)
    out = dict(seq_len=np.array(seq_len, np.int64), n_new=np.zeros(R, np.int32),
               x0=None if x0 is None else np.array(x0, np.int32))
    for r in range(R):
        n0, L = int(seq_len[r]), int(ell[r])
        q = L + 1 if L >= 0 else 0
        st = 0 if status is None else int(status[r])
        if n0 < 0 or n0 > cap or L >= q_max or n0 + q > cap:
            if status is not None:
                status[r] |= BAD_INPUT
            continue
        acc = min(max(int(n_acc[r]), 0), max(L, 0))
        n_new = acc + 1 if q and not st & HELD else 0
        held = blocks_of(n0 + q, block_size)
        if release is not None and release[r]:
            new, kept = 0, min(max(0 if keep is None else int(keep[r]), 0), held)
        else:
            new = n0 + n_new
            kept = blocks_of(new, block_size)
        if held > kept and at + held - kept > pool and status is not None:
            status[r] |= BAD_INPUT
        for b in range(kept, held):
            if at < pool:
                free_list[at] = table[r, b]
            at += 1
        out["seq_len"][r] = new
        out["n_new"][r] = n_new
        if out["x0"] is not None and n_new:
            out["x0"][r] = out_tokens[r][acc]
    out["free_count"] = np.array([min(at, pool)], np.int32)
    return out
