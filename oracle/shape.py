"""Penalties, biases and grammar masks on target rows, and the token state
behind them (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

What it computes (speculative-decoding history page, "1.1 mechanism":
verification reproduces the distribution of the target rows it is given, so a
request's wishes are applied to those rows; the formulas are the usual ones of
sampling interfaces):

* row i of a request scores the token after its drafts x_1..x_i, which count
  as written there;
* a token seen in the prompt or written has its logit divided by the
  repetition penalty where positive, else multiplied by it; a token written n
  times loses frequency * n, and presence once;
* the request's bias is added (the last entry of a token counts), and a token
  that the row's grammar mask does not allow becomes -inf.

Pins (tests/test_oracle_shape.py): neutral values change nothing, drafting a
token equals having it in the state, a list entered in pieces equals the list
entered at once.
"""

import numpy as np


def pack_bits(rows, words=None):
    """[n][V] truth values -> [n][words] int32, token v in bit v % 32 of word v // 32."""
    rows = np.asarray(rows, bool)
    n, V = rows.shape
    words = (V + 31) // 32 if words is None else words
    out = np.zeros((n, words), np.uint32)
    for r, v in zip(*np.nonzero(rows)):
        out[r, v // 32] |= np.uint32(1) << np.uint32(v % 32)
    return out.view(np.int32)


def unpack_bits(words, V):
    w = np.asarray(words).view(np.uint32)
    v = np.arange(V)
    return ((w[:, v // 32] >> (v % 32).astype(np.uint32)) & 1).astype(bool)


def shape_row(row, written, seen, counts, repetition=1.0, frequency=0.0, presence=0.0, bias=(), allowed=None):
    """One row.  written: the drafts before it; seen, counts: the state row
    (truth values, numbers); bias: (token, value) pairs in list order; allowed:
    truth values or None.  Returns the shaped row and, per token, the sum of
    the magnitudes of the intermediate results (what fp32 rounds), 0 where no
    term touches the token."""
    row = np.array(row, np.float64)
    mag = np.zeros(row.shape[0])
    V = row.shape[0]
    more = {}
    for x in written:
        if 0 <= x < V:
            more[int(x)] = more.get(int(x), 0) + 1
    with np.errstate(invalid="ignore", over="ignore"):
        if repetition != 1.0 or frequency != 0.0 or presence != 0.0:
            for v in sorted(set(np.nonzero(seen)[0].tolist()) | set(more)):
                n = (int(counts[v]) if counts is not None and seen[v] else 0) + more.get(v, 0)
                x = row[v] / repetition if row[v] > 0 else row[v] * repetition
                y = x - frequency * n
                z = y - presence if n > 0 else y
                mag[v] += abs(x) + abs(frequency * n) + abs(y) + abs(z)
                row[v] = z
        last = {}
        for t, b in bias:
            if 0 <= t < V:
                last[int(t)] = float(b)
        for v, b in last.items():
            row[v] += b
            mag[v] += abs(row[v])
    if allowed is not None:
        row[~np.asarray(allowed, bool)] = -np.inf
        mag[~np.asarray(allowed, bool)] = 0.0
    return row, mag


def enter_tokens(seen, counts, tokens, prompt_len=0, reset=False):
    """Enter one list into a state row (seen truth values, counts or None), in
    place; tokens outside the vocabulary are skipped."""
    if reset:
        seen[:] = False
        if counts is not None:
            counts[:] = 0
    for i, t in enumerate(tokens):
        if 0 <= t < seen.shape[0]:
            seen[t] = True
            if counts is not None and i >= prompt_len:
                counts[t] += 1
