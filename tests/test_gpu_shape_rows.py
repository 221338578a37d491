"""Batches in which a wave of sd_logit_shape takes several rows of a request.

A batch is split over some 16384 waves: with R requests and c = ceil(V / 512)
pieces of a row a wave has about rows * R * c / 16384 rows of its request, one
in the small batches of the other tests.  Here it has from 3 rows to all of a
request's, in both dtypes, in place and not, streamed (a batch past the
last-level cache, by its size or by a large leading dimension) and not; the
lengths are ragged, so that groups of rows end anywhere.  Every batch has to
give the bits that its requests give a few at a time, one row per wave, and a
sample of the requests is compared with the oracle (tolerances as in
test_gpu_shape.py)."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from oracle import shape as OS
from tests.parity_util import to_np
from tests.test_gpu_shape import _compare, _expect

pytestmark = pytest.mark.gpu

DEV = "cuda"

# R, gmax, V, ld: rows per wave, and whether the batch is streamed
SIZES = [
    (300, 16, 4104, 4112),      # 3 rows; bf16 in place: not streamed
    (300, 16, 4104, 16000),     # 3 rows; streamed
    (17000, 6, 264, 264),       # 7 rows; bf16: not streamed
    (17000, 4, 64, 72),         # 5 rows of eight lanes; not streamed
    (1900, 16, 4104, 4104),     # 17 rows; streamed
    (600, 255, 24, 24),         # 10 of 256 rows, three lanes; not streamed
    (5600, 12, 1560, 1568),     # 13 rows; streamed
]


def _batch(R, gmax, V, ld, dtype, pen, bias, mask):
    g = torch.Generator(device=DEV).manual_seed(R + gmax + V)
    ints = lambda lo, hi, *k: torch.randint(lo, hi, k, generator=g, device=DEV, dtype=torch.int32)  # noqa: E731
    rand = lambda *k: torch.rand(k, generator=g, device=DEV)  # noqa: E731
    words = lambda *k: torch.randint(-(1 << 31), 1 << 31, k, generator=g, device=DEV).to(torch.int32)  # noqa: E731
    q, w, S = gmax + 1, (V + 31) // 32, R + 2
    b = dict(V=V, gmax=gmax, row0=torch.arange(R, device=DEV, dtype=torch.int32) * q, ell=ints(-1, q, R))
    b["ell"][:3] = torch.tensor([gmax, -1, 0])
    b["x"] = (4 * torch.randn((R * q + 1, ld), generator=g, device=DEV)).to(dtype)
    drafts = (V * rand(R, gmax) ** 2).to(torch.int32)
    for i in range(0, gmax - 2, 3):     # a token again, and its neighbour: the same lane's
        drafts[:, i + 1] = drafts[:, i]
        drafts[:, i + 2] = drafts[:, i] ^ 1
    if gmax > 4:
        drafts[::2, 4] = drafts[::2, 0]
    b["draft"], b["slot"] = drafts, torch.randperm(S, generator=g, device=DEV)[:R].to(torch.int32)
    b["seen"] = b["counts"] = b["rep"] = b["freq"] = b["pres"] = b["off"] = b["tok"] = b["val"] = None
    b["mask"] = b["m0"] = None
    if pen:
        b["seen"], b["counts"] = words(S, w) & words(S, w) & words(S, w), ints(0, 4, S, (V + 3) // 4 * 4)
        on = lambda: (rand(R) < 0.7).float()  # noqa: E731
        b["rep"], b["freq"], b["pres"] = 1 + on() * (rand(R) - 0.4), on() * (rand(R) - 0.3), on() * rand(R)
    if bias:
        n = ints(0, 7, R).long()
        b["off"] = torch.cat([n[:1] * 0, torch.cumsum(n, 0)])
        total = int(b["off"][-1])
        b["tok"], b["val"] = ints(0, V, total), torch.randn(total, generator=g, device=DEV)
    if mask:
        kind = ints(0, 4, R * q, 1)     # nothing allowed, everything, half, an eighth
        m = words(R * q, w)
        m = torch.where(kind == 3, m & words(R * q, w) & words(R * q, w), m)
        b["mask"] = torch.where(kind == 0, 0, torch.where(kind == 1, -1, m)).to(torch.int32)
        b["m0"] = torch.where(torch.arange(R, device=DEV) % 3 == 1, -1, b["row0"]).to(torch.int32)
    return b


def _call(b, src, dst, lo, hi):
    cut = lambda k, n=0: None if b[k] is None else b[k][lo:hi + n]  # noqa: E731
    got = sdv.sd_logit_shape(src, cut("row0"), cut("ell"), b["V"], draft_tokens=cut("draft"), repetition=cut("rep"),
                             frequency=cut("freq"), presence=cut("pres"), seen=b["seen"], counts=b["counts"],
                             slot=cut("slot"), bias=None if b["off"] is None else (cut("off", 1), b["tok"], b["val"]),
                             mask=b["mask"], mask_row0=cut("m0"), out=dict(logits=dst))
    return got["status"]


def _sample(b, requests, got, base):
    """Compare the rows of some requests with the oracle."""
    n = lambda t: None if t is None else to_np(t)  # noqa: E731
    V, q, i = b["V"], b["gmax"] + 1, torch.as_tensor(requests, device=DEV)
    rows = (i[:, None] * q + torch.arange(q, device=DEV)).flatten()
    k = len(requests)
    c = dict(R=k, gmax=b["gmax"], V=V, ell=n(b["ell"][i]), row0=np.arange(k) * q, x=b["x"][rows, :V].cpu(),
             slot=np.arange(k), draft=n(b["draft"][i]), rep=None, freq=None, pres=None, bias=None, allowed=None, m0=None,
             seen=np.zeros((k, V), bool), counts=np.zeros((k, V), int))
    if b["seen"] is not None:
        s = b["slot"][i].long()
        c["seen"], c["counts"] = OS.unpack_bits(n(b["seen"][s]), V), n(b["counts"][s])
        c.update({x: n(b[x][i]) for x in ("rep", "freq", "pres")})
    if b["off"] is not None:
        off, tok, val = n(b["off"]), n(b["tok"]), n(b["val"])
        c["bias"] = [list(zip(tok[off[r]:off[r + 1]], val[off[r]:off[r + 1]])) for r in requests]
    if b["m0"] is not None:
        c["m0"] = np.where(n(b["m0"][i]) < 0, -1, np.arange(k) * q)
        c["allowed"] = OS.unpack_bits(n(b["mask"][rows]), V)
    _compare(n(got[rows, :V]).astype(np.float64), *_expect(c, n(base[rows, :V]).astype(np.float64)))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("terms", ["all", "penalties", "mask", "bias"])
@pytest.mark.parametrize("R,gmax,V,ld", SIZES)
def test_rows_of_one_wave(R, gmax, V, ld, terms, dtype, in_place):
    b = _batch(R, gmax, V, ld, dtype, terms in ("all", "penalties"), terms in ("all", "bias"), terms in ("all", "mask"))
    dst = lambda: b["x"].clone() if in_place else torch.full_like(b["x"], 123.0)  # noqa: E731
    whole, parts = dst(), dst()
    base = whole.clone()
    status = _call(b, whole if in_place else b["x"], whole, 0, R)
    assert (status == 0).all()
    few = max(1, 16384 // (gmax + 1) // ((V + 511) // 512))
    for lo in range(0, R, few):
        _call(b, parts if in_place else b["x"], parts, lo, min(R, lo + few))
    torch.cuda.synchronize()
    word = torch.int16 if dtype is torch.bfloat16 else torch.int32
    assert torch.equal(whole.view(word), parts.view(word))
    assert torch.equal(whole[:, V:], base[:, V:])
    _sample(b, [0, 1, 2, R // 2, R - 1] if gmax > 100 else [0, 1, 2, 3, R // 3, R // 2, R - 2, R - 1], whole, base)
