"""Heads between projection and attention, and the paged cache, in fp64: norm
and rotation of heads, the 4-bit format, attention over a list of tokens."""

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def turn(x, w, pos, inv_freq, eps, interleaved):
    """Heads x [rows][heads][D] normed (w [D] or None) and rotated: y, and the
    size of what each channel was summed from (for error bounds)."""
    x = np.asarray(x, np.float64).copy()
    if w is not None:
        x /= np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x *= np.asarray(w, np.float64)
    size = np.abs(x)
    r = 0 if inv_freq is None else 2 * len(inv_freq)
    if r:
        t = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        ia = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
        ib = ia + 1 if interleaved else ia + r // 2
        a, b = x[..., ia].copy(), x[..., ib].copy()
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return x, size


def scale_exponent(x):
    """The exponent of each group of 32 channels [..., D/32]: the smallest of
    at least -126 with max |x| <= 7 * 2^e."""
    top = np.abs(x.reshape(x.shape[:-1] + (-1, 32))).max(-1)
    m, e = np.frexp(np.where(top > 0, top, 2.0 ** -200))
    return np.maximum(np.where(m > 0.875, e - 2, e - 3), -126)


def nearest(x, e):
    """x [..., D] at the nearest levels of scales 2^e [..., D/32], ties to the
    even code, past the last level 6."""
    s = np.repeat(np.exp2(np.asarray(e, np.float64)), 32, -1)
    a = np.abs(x) / s
    d = np.abs(a[..., None] - LEVELS)
    best = d.min(-1, keepdims=True)
    even = np.arange(8) % 2 == 0
    code = np.argmin(np.where(d == best, np.where(even, 0, 1), 2), -1)
    return np.copysign(LEVELS[code], x) * s


def values(codes, scale):
    """fp64 values of codes [..., D/2] and scale bytes [..., D/32] (255: NaN)."""
    one = np.concatenate([LEVELS, -LEVELS])
    v = np.stack([one[codes & 15], one[codes >> 4]], -1).reshape(codes.shape[:-1] + (-1,))
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return v * np.repeat(s, 32, -1)


def attend(q, k, v, see, scale):
    """One request: q [n][n_q][D], k, v [T][n_kv][D], see [n][T].  Returns
    out [n][n_q][D], lse [n][n_q], and sum p |v| [n][n_q][D] (for error
    bounds); zeros and -inf where a row sees nothing."""
    n, n_q, D = q.shape
    G = n_q // k.shape[1]
    out, lse, size = np.zeros((n, n_q, D)), np.full((n, n_q), -np.inf), np.zeros((n, n_q, D))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for h in range(n_q):
            x = (q[:, h].astype(np.float64) @ k[:, h // G].T) * scale
            for i in range(n):
                at = np.flatnonzero(see[i])
                if not len(at):
                    continue
                m = x[i, at].max()
                if m == -np.inf:
                    continue
                p = np.exp(x[i, at] - m)
                z = p.sum()
                lse[i, h] = m + np.log(z)
                vv = v[at, h // G]
                out[i, h] = (p[:, None] * vv).sum(0) / z
                size[i, h] = (p[:, None] * np.abs(vv)).sum(0) / z
    return out, lse, size
