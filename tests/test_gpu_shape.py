"""sd_logit_shape and sd_token_counts against the oracle in 64 bits.

Tolerance of a shaped logit: every fp32 operation rounds by at most half a
step, 2^-24 of its result, so the value before the last rounding is off by at
most 2^-24 times the sum of the magnitudes of the intermediate results (the
oracle gives that sum; second-order terms are below 1e-6 of it), and the
rounding to the rows' type adds half a step of that (bf16 2^-8, fp32 2^-24).
Below the normal range a half step is absolute: 2^-150 for each of at most six
fp32 results, 2^-134 for bf16.  Where no term touches a token the value is equal."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from oracle import shape as OS
from tests.parity_util import to_np

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 6 * 2.0 ** -150, torch.bfloat16: 2.0 ** -134 + 6 * 2.0 ** -150}


def _case(R, gmax, V, dtype=torch.bfloat16, pad=0, seed=0, packed=False, draft=True, rep=True, fp=True, bias=3,
          mask=True, slots=True, extra=0, ells=None, hist=20, wide=0):
    """Inputs as numpy on the host and as tensors on the GPU."""
    g = np.random.default_rng(seed)
    ell = g.integers(-1, gmax + 1, R) if ells is None else np.asarray(ells)
    n = np.maximum(ell + 1, 0)
    row0 = np.concatenate([[0], np.cumsum(n)[:-1]]) if packed else np.arange(R) * (gmax + 1)
    rows = max(1, int((row0 + n).max())) + 1
    x = torch.as_tensor(g.normal(0, 4, (rows, V + pad)), dtype=torch.float32).to(dtype)
    S = R + extra
    slot = g.permutation(S)[:R] if slots else np.arange(R)
    seen = np.zeros((S, V), bool)
    counts = np.zeros((S, V), np.int64)
    for s in range(S):
        OS.enter_tokens(seen[s], counts[s], (V * g.random(hist) ** 2).astype(int), prompt_len=hist // 2)
    c = dict(R=R, gmax=gmax, V=V, ell=ell, row0=row0, x=x, slot=slot, seen=seen, counts=counts, draft=None,
             rep=None, freq=None, pres=None, bias=None, allowed=None, m0=None)
    if draft:
        c["draft"] = (V * g.random((R, gmax)) ** 2).astype(int)
        if gmax > 1:
            c["draft"][:, 1] = c["draft"][:, 0]   # the same token twice
    if rep:
        c["rep"] = np.float32(np.where(g.random(R) < 0.3, 1.0, g.uniform(0.5, 2.0, R)))
    if fp:
        c["freq"] = np.float32(g.uniform(-0.5, 1.0, R) * (g.random(R) < 0.7))
        c["pres"] = np.float32(g.uniform(-0.5, 1.0, R) * (g.random(R) < 0.7))
    if bias:
        lists = [[(int(t), np.float32(b)) for t, b in zip(g.integers(0, V, k), g.normal(0, 3, k))]
                 for k in g.integers(0, bias + 1, R)]
        c["bias"] = lists
    if mask:
        masked = g.random(R) < 0.7
        c["m0"] = np.where(masked, np.arange(R) * (gmax + 1), -1)
        c["allowed"] = g.random((R * (gmax + 1), V)) < g.choice([0.0, 0.05, 0.5, 1.0], (R * (gmax + 1), 1))
    c["wide"] = wide
    return c


def _gpu(c, in_place=False, stream=None, out=None, raw=False, ld=None):
    i32 = lambda a: None if a is None else torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).to(DEV)  # noqa: E731
    f32 = lambda a: None if a is None else torch.as_tensor(a).to(DEV)  # noqa: E731
    V, w = c["V"], (c["V"] + 31) // 32 + c["wide"]
    x = c["x"].to(DEV)
    if ld is not None:   # the same rows further apart
        wide = torch.full((x.shape[0], ld), 7.0, dtype=x.dtype, device=DEV)
        wide[:, :V] = x[:, :V]
        x = wide
    cnt = np.full((c["counts"].shape[0], V + 4 * c["wide"]), 77)
    cnt[:, :V] = c["counts"]
    pen = c["rep"] is not None or c["freq"] is not None
    bias = None
    if c["bias"] is not None:
        flat = [e for b in c["bias"] for e in b]
        off = np.concatenate([[0], np.cumsum([len(b) for b in c["bias"]])])
        bias = (torch.as_tensor(off, dtype=torch.int64).to(DEV), i32([t for t, _ in flat]),
                torch.as_tensor([float(b) for _, b in flat], dtype=torch.float32).to(DEV))
    if out is None:
        dst = x if in_place else torch.full_like(x, 123.0)
        out = dict(logits=dst, status=torch.full((c["R"],), -9, dtype=torch.int32, device=DEV))
    got = sdv.sd_logit_shape(
        x, i32(c["row0"]), i32(c["ell"]), V, gamma_max=c["gmax"], draft_tokens=i32(c["draft"]),
        repetition=f32(c["rep"]), frequency=f32(c["freq"]), presence=f32(c["pres"]),
        seen=i32(OS.pack_bits(c["seen"], w)) if pen else None, counts=i32(cnt) if c["freq"] is not None else None,
        slot=i32(c["slot"]) if pen else None, bias=bias,
        mask=None if c["allowed"] is None else i32(OS.pack_bits(c["allowed"], w)), mask_row0=i32(c["m0"]),
        out=out, stream=stream)
    torch.cuda.synchronize()
    if raw:
        return got
    return to_np(got["logits"]).astype(np.float64), to_np(got["status"])


def _expect(c, base, skip=()):
    """(rows, tolerance) the call has to give on rows that were `base`."""
    ref, tol = base.copy(), np.zeros_like(base)
    x = to_np(c["x"]).astype(np.float64)
    V, half = c["V"], HALF[c["x"].dtype]
    one = lambda k, r, d: d if c[k] is None else float(c[k][r])  # noqa: E731
    for r in range(c["R"]):
        if r in skip:
            continue
        s = c["slot"][r]
        for i in range(min(c["ell"][r], c["gmax"]) + 1):
            row, mag = OS.shape_row(
                x[c["row0"][r] + i, :V], [] if c["draft"] is None else c["draft"][r][:i], c["seen"][s],
                c["counts"][s] if c["freq"] is not None else None, one("rep", r, 1.0), one("freq", r, 0.0),
                one("pres", r, 0.0), [] if c["bias"] is None else c["bias"][r],
                None if c["m0"] is None or c["m0"][r] < 0 else c["allowed"][c["m0"][r] + i])
            e = 2.0 ** -24 * mag * (1 + 1e-6)
            ref[c["row0"][r] + i, :V] = row
            with np.errstate(invalid="ignore"):
                t = np.where(mag > 0, e + half * (np.abs(row) + e) + TINY[c["x"].dtype], 0.0)
            tol[c["row0"][r] + i, :V] = np.where(np.isfinite(t), t, 0.0)
    return ref, tol


def _compare(got, ref, tol):
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        near = np.abs(got - ref) <= tol
    bad = np.argwhere(~(same | near))
    assert bad.size == 0, (len(bad), bad[:4], [(got[tuple(b)], ref[tuple(b)], tol[tuple(b)]) for b in bad[:4]])


def _check(c, in_place, status=0):
    got, st = _gpu(c, in_place)
    base = to_np(c["x"]).astype(np.float64) if in_place else np.full_like(got, 123.0)
    _compare(got, *_expect(c, base))
    assert (st == status).all(), st


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,gmax,V,pad", [(1, 0, 8, 0), (3, 2, 40, 8), (5, 4, 1000, 24), (4, 3, 2048, 0),
                                          (3, 5, 2056, 8), (2, 1, 16392, 0), (7, 16, 4104, 16), (2, 255, 64, 0),
                                          (40, 1, 96, 0)])
def test_sizes(R, gmax, V, pad, dtype, in_place):
    _check(_case(R, gmax, V, dtype, pad, seed=V + R, packed=bool(R % 2), extra=R % 3, wide=R % 2), in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kw", [dict(rep=False, fp=False, bias=0, mask=False), dict(rep=False), dict(fp=False),
                                dict(draft=False), dict(mask=False), dict(bias=0), dict(slots=False),
                                dict(rep=False, fp=False, mask=False), dict(rep=False, fp=False, bias=0),
                                dict(hist=4000), dict(bias=2500), dict(ells=[-1, -1, -1, -1])])
def test_terms(kw, in_place):
    _check(_case(4, 5, 5000, seed=len(str(kw)), **kw), in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", [dict(), dict(mask=False), dict(mask=False, bias=0), dict(mask=False, bias=900),
                                dict(mask=False, rep=False, fp=False), dict(mask=False, draft=False, hist=3000),
                                dict(mask=False, fp=False), dict(rep=False, fp=False)])
def test_batches_past_the_cache(kw, dtype, in_place):
    """Batches that do not fit the last-level cache take other kernels: with
    rows far apart they give the bits of the same rows packed (checked against
    the oracle), and leave the rest of the rows alone."""
    c = _case(9, 7, 17000, dtype, seed=21, packed=True, extra=1, wide=1, ells=[7, 7, 0, 3, -1, 7, 5, 6, 7], **kw)
    c["allowed"] = None if c["allowed"] is None else c["allowed"].copy()
    if c["allowed"] is not None:
        c["allowed"][:2] = True
        c["allowed"][8] = False
    _check(c, in_place)
    near = _gpu(c, in_place, raw=True)
    rows, esize = c["x"].shape[0], 2 if dtype is torch.bfloat16 else 4
    ld = (140 << 20) // (72 * esize * (1 if in_place else 2)) // 8 * 8
    far = _gpu(c, in_place, raw=True, ld=ld)
    assert torch.equal(near["status"], far["status"])
    V = c["V"]
    a, b = near["logits"][:, :V].contiguous(), far["logits"][:, :V].contiguous()
    word = torch.int16 if esize == 2 else torch.int32
    assert torch.equal(a.view(word), b.view(word))
    assert (far["logits"][:, V:] == (7.0 if in_place else 123.0)).all() and far["logits"].shape == (rows, ld)


@pytest.mark.parametrize("in_place", [False, True])
def test_full_vocabulary(in_place):
    _check(_case(3, 2, 151936, seed=5, hist=3000, bias=300, ells=[2, 0, 1]), in_place)


def test_ell_past_the_block_is_cut():
    c = _case(3, 2, 64, ells=[5, 2, 99], seed=8)
    c["x"] = torch.cat([c["x"]] * 2)
    _check(c, False)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_values(dtype, in_place):
    """NaN, infinities and the type's extremes, touched, untouched and masked;
    rows whose mask allows nothing; biases of -inf."""
    c = _case(4, 3, 512, dtype, seed=9, ells=[3, 3, 3, 3])
    odd = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max, torch.finfo(dtype).min,
                        torch.finfo(dtype).tiny, 0.0, -0.0])
    g = np.random.default_rng(1)
    at = torch.as_tensor(g.random(c["x"].shape) < 0.4)
    c["x"] = torch.where(at, odd[torch.as_tensor(g.integers(0, 8, c["x"].shape))].to(dtype), c["x"])
    c["allowed"][0:4] = False
    c["m0"] = np.array([0, 4, -1, 8])
    c["bias"] = [[(int(t), np.float32(-np.inf)) for t in g.integers(0, 512, 9)] for _ in range(4)]
    got, st = _gpu(c, in_place)
    ref, tol = _expect(c, to_np(c["x"]).astype(np.float64) if in_place else np.full_like(got, 123.0))
    # fp32 sums past the type's range round to infinity
    top = float(torch.finfo(dtype).max) * (1 + HALF[dtype])
    with np.errstate(invalid="ignore"):
        ref = np.where(np.abs(ref) >= top, np.copysign(np.inf, ref), ref)
    _compare(got, ref, tol)
    assert (st == 0).all()
    assert np.isneginf(got[c["row0"][0]][:512]).all()


def test_last_bias_entry_of_a_token_counts():
    c = _case(2, 1, 4096, seed=11, ells=[1, 0])
    g = np.random.default_rng(2)
    c["bias"] = [[(int(t), np.float32(b)) for t, b in zip(g.integers(0, 6, 700), g.normal(0, 3, 700))], []]
    _check(c, False)


def test_entries_outside_the_vocabulary_are_skipped_and_told():
    c = _case(3, 3, 256, seed=12, ells=[3, 3, 1])
    c["bias"] = [[(3, np.float32(1)), (256, np.float32(9)), (-1, np.float32(9))], [], []]
    c["draft"][1] = [5, -7, 1 << 20]
    c["draft"][2, 1:] = -1     # behind the request's drafts: not read
    got, st = _gpu(c)
    _compare(got, *_expect(c, np.full_like(got, 123.0)))
    assert st.tolist() == [sdv.SD_ST_BAD_TOKEN, sdv.SD_ST_BAD_TOKEN, 0]


@pytest.mark.parametrize("what", ["row", "row_end", "slot", "slot_end", "mask_end", "rep", "rep0", "rep_inf", "freq",
                                  "pres", "bias"])
def test_request_out_of_range_is_left_out(what):
    c = _case(3, 2, 300 // 4 * 8, seed=13, ells=[2, 2, 2], extra=1)
    if what == "row":
        c["row0"][1] = -1
    elif what == "row_end":
        c["row0"][1] = c["x"].shape[0] - 2
    elif what == "slot":
        c["slot"][1] = -1
    elif what == "slot_end":
        c["slot"][1] = 4
    elif what == "mask_end":
        c["m0"] = np.array([0, 7, -1])
    elif what == "rep":
        c["rep"][1] = np.nan
    elif what == "rep0":
        c["rep"][1] = 0.0
    elif what == "rep_inf":
        c["rep"][1] = np.inf
    elif what == "freq":
        c["freq"][1] = np.inf
    elif what == "pres":
        c["pres"][1] = np.nan
    else:
        c["bias"] = [[(1, np.float32(1.0))], [(2, np.float32(1.0))], [(3, np.float32(1.0))]]
    c["rep"][1] = 1.5 if what in ("slot", "slot_end") else c["rep"][1]
    if what == "bias":
        i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).to(DEV)  # noqa: E731
        x = c["x"].to(DEV)
        for off in ([0, 2, 1, 3], [0, 1, 4, 3], [-1, 1, 1, 1]):
            got = sdv.sd_logit_shape(x, i32(c["row0"]), i32(c["ell"]), c["V"], gamma_max=2,
                                     bias=(torch.tensor(off, device=DEV), i32([1, 2, 3]),
                                           torch.ones(3, device=DEV)), out=dict(logits=torch.full_like(x, 123.0)))
            st = to_np(got["status"])
            for r in range(3):
                bad = not 0 <= off[r] <= off[r + 1] <= 3
                assert (st[r] != 0) == bad
                rows = to_np(got["logits"])[c["row0"][r]:c["row0"][r] + 3, :c["V"]]
                assert (rows == 123.0).all() == bad
        return
    got, st = _gpu(c)
    _compare(got, *_expect(c, np.full_like(got, 123.0), skip=(1,)))
    assert st.tolist() == [0, sdv.SD_ST_BAD_INPUT, 0]


def test_rows_past_32_bit_offsets():
    """In place on rows more than 2^32 elements into the buffer."""
    V, n = 151936, 28400
    x = torch.empty((n, V), dtype=torch.bfloat16, device=DEV)
    assert (n - 4) * V > 1 << 32
    g = torch.Generator(device=DEV).manual_seed(3)
    x[n - 4:] = torch.randn((4, V), generator=g, device=DEV).to(torch.bfloat16)
    before = x[n - 4:].clone()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    mask = torch.zeros((2, V // 32), dtype=torch.int32, device=DEV)
    mask[:, 100] = 255
    off = torch.tensor([0, 1], device=DEV)
    got = sdv.sd_logit_shape(x, i32(n - 3), i32(1), V, gamma_max=1, bias=(off, i32(3201), torch.ones(1, device=DEV)),
                             mask=mask, mask_row0=i32(0), out=dict(logits=x))
    assert int(got["status"]) == 0
    after = x[n - 4:]
    assert torch.equal(after[0], before[0]) and torch.equal(after[3], before[3])
    keep = before[1:3, 3200:3208].float()
    keep[:, 1] += 1.0
    assert torch.equal(after[1:3, 3200:3208], keep.to(torch.bfloat16))
    assert int(torch.isneginf(after[1:3].float()).sum()) == 2 * (V - 8)


# ---------------------------------------------------------------------------
# token counts

def _counts_check(lists, V, prompt=None, slot=None, reset=None, fixed=None, extra=0, with_counts=True, seed=0,
                  wide=0):
    """lists entered in one call against the oracle, list by list."""
    g = np.random.default_rng(seed)
    R = len(lists)
    slot_ = np.arange(R) if slot is None else np.asarray(slot)
    S = max(R, int(slot_.max(initial=0)) + 1) + extra
    seen = g.random((S, V)) < 0.3
    counts = g.integers(0, 5, (S, V))
    i32 = lambda a: None if a is None else torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).to(DEV)  # noqa: E731
    w = (V + 31) // 32 + wide
    ts = i32(OS.pack_bits(seen, w))
    ts[:, (V + 31) // 32:] = 5
    tc = torch.full((S, V + 4 * wide), -3, dtype=torch.int32, device=DEV)
    tc[:, :V] = i32(counts)
    if fixed is not None:
        toks = np.full((R, fixed), -1)
        for r, x in enumerate(lists):
            toks[r, :len(x)] = x
        kw = dict(tokens=i32(toks))
    else:
        n = np.array([len(x) for x in lists])
        kw = dict(tokens=i32(np.concatenate([np.asarray(x, int) for x in lists] + [[1, 2]])),
                  start=torch.as_tensor(np.cumsum(n) - n, dtype=torch.int64).to(DEV), length=i32(n))
    got = sdv.sd_token_counts(seen=ts, counts=tc if with_counts else None, V=V, prompt_len=i32(prompt),
                              slot=i32(slot), reset=i32(reset), **kw)
    torch.cuda.synchronize()
    if reset is not None:
        for r in range(R):
            if reset[r]:
                OS.enter_tokens(seen[slot_[r]], counts[slot_[r]] if with_counts else None, [], reset=True)
    for r, x in enumerate(lists):
        OS.enter_tokens(seen[slot_[r]], counts[slot_[r]] if with_counts else None, x,
                        0 if prompt is None else prompt[r])
    want = OS.pack_bits(seen, w)
    want[:, (V + 31) // 32:] = 5
    assert np.array_equal(to_np(ts), want)
    assert np.array_equal(to_np(tc[:, :V]), counts)
    assert (to_np(tc[:, V:]) == -3).all()
    assert (to_np(got["status"]) == 0).all()


@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("V", [8, 40, 1000, 33000, 151936])
def test_counts_sizes(V, reset):
    g = np.random.default_rng(V)
    lists = [g.integers(0, V, k) for k in (0, 1, 3, 700, 64)] + [np.full(5000, V - 1), (V * g.random(9000) ** 3).astype(int)]
    _counts_check(lists, V, prompt=[0, 1, 2, 300, 64, 4000, 0], slot=[3, 7, 0, 1, 2, 5, 4],
                  reset=[1, 0, 1, 1, 0, 1, 1] if reset else None, extra=1, wide=1, seed=V)


def test_counts_of_verified_tokens():
    g = np.random.default_rng(4)
    lists = [g.integers(0, 96, k) for k in (1, 5, 0, 3)]
    _counts_check(lists, 96, fixed=6)
    _counts_check(lists, 96, fixed=6, with_counts=False, reset=[0, 1, 1, 0])


def test_counts_of_one_row_shared_by_requests():
    g = np.random.default_rng(5)
    _counts_check([g.integers(0, 64, 500) for _ in range(6)], 64, slot=[2, 2, 0, 2, 0, 2], reset=[1, 0, 0, 1, 0, 0])


def test_counts_of_long_lists_added():
    """Long lists without a reset, two of them into one state row."""
    g = np.random.default_rng(8)
    V = 40000
    lists = [(V * g.random(k) ** 2).astype(int) for k in (9000, 30000, 8193, 0, 4100)] + [np.full(20000, 32767)]
    lists[1][100:200] = [-1, V] * 50
    _counts_check(lists, V, prompt=[0, 20000, 8192, 0, 9000, 5], slot=[4, 1, 4, 2, 0, 3], extra=1)
    _counts_check(lists, V, slot=[4, 1, 4, 2, 0, 3], with_counts=False)


def test_counts_of_very_many_requests():
    g = np.random.default_rng(6)
    R = 4100
    _counts_check([g.integers(0, 40, k) for k in g.integers(0, 6, R)], 40, slot=g.permutation(R),
                  reset=(g.random(R) < 0.5).astype(int), prompt=g.integers(0, 4, R))


def test_counts_skip_tokens_outside_and_requests_out_of_range():
    V = 64
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32).to(DEV)  # noqa: E731
    _counts_check([[1, -1, 64, 2, 1 << 30, -(1 << 31)], [63, 0]], V)
    seen = torch.zeros((3, 2), dtype=torch.int32, device=DEV)
    counts = torch.zeros((3, V), dtype=torch.int32, device=DEV)
    toks = i32([1, 2, 3, 4])
    start = torch.tensor([0, -1, 3, 5, 0, 0, 4], device=DEV)
    got = sdv.sd_token_counts(toks, seen, counts, V, start=start, length=i32([2, 1, 2, 0, 1, -4, 0]),
                              slot=i32([0, 0, 0, 0, 3, 1, 2]), reset=i32([1] * 7))
    bad = sdv.SD_ST_BAD_INPUT
    assert to_np(got["status"]).tolist() == [0, bad, bad, bad, bad, 0, 0]
    assert int(counts.sum()) == 2 and int(counts[0, 1]) == 1 and int(counts[0, 2]) == 1
    assert int(seen[0, 0]) == 6 and int(seen.sum()) == 6


@pytest.mark.parametrize("reset", [False, True])
def test_counts_of_fixed_rows_with_lengths(reset):
    """A length past its row is refused; others end a row early."""
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32).to(DEV)  # noqa: E731
    toks = i32([[1, 2, 3], [4, 5, 6], [7, 8, 9], [10, 11, 12]])
    seen = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    counts = torch.full((4, 64), 2, dtype=torch.int32, device=DEV)
    got = sdv.sd_token_counts(toks, seen, counts, 64, length=i32([2, 4, 0, 3]),
                              reset=i32([1, 1, 1, 0]) if reset else None)
    assert to_np(got["status"]).tolist() == [0, sdv.SD_ST_BAD_INPUT, 0, 0]
    want = np.full((4, 64), 2)
    if reset:
        want[0] = want[2] = 0
    want[0, 1:3] += 1
    want[3, 10:13] += 1
    assert np.array_equal(to_np(counts), want)
    assert to_np(seen)[:, 0].tolist() == [6, 0, 0, 7 << 10]


def test_counts_of_short_lists_in_a_large_buffer():
    """start into a [R][n] buffer, lengths bounded or not: the same counts."""
    g = np.random.default_rng(12)
    R, n, V = 5, 20000, 3000
    toks = torch.as_tensor(g.integers(0, V, (R, n)), dtype=torch.int32).to(DEV)
    length = g.integers(0, 8, R)
    start = np.arange(R) * n + g.integers(0, n - 8, R)
    want = np.zeros((R, V), int)
    for r in range(R):
        np.add.at(want[r], to_np(toks).ravel()[start[r]:start[r] + length[r]], 1)
    for bound in (0, 7, 8):
        seen = torch.zeros((R, (V + 31) // 32), dtype=torch.int32, device=DEV)
        counts = torch.zeros((R, V), dtype=torch.int32, device=DEV)
        got = sdv.sd_token_counts(toks, seen, counts, V, start=torch.as_tensor(start).to(DEV),
                                  length=torch.as_tensor(length, dtype=torch.int32).to(DEV), max_length=bound)
        assert (got["status"] == 0).all()
        assert np.array_equal(to_np(counts), want) and np.array_equal(to_np(seen), OS.pack_bits(want > 0))
    got = sdv.sd_token_counts(toks, seen, counts, V, start=torch.as_tensor(start).to(DEV), max_length=3,
                              length=torch.as_tensor(length, dtype=torch.int32).to(DEV))
    assert np.array_equal(to_np(got["status"]) != 0, length > 3)
    with pytest.raises(ValueError, match="goes with start"):
        sdv.sd_token_counts(toks, seen, counts, V, max_length=4)


def test_state_and_lists_past_32_bit_offsets():
    """State rows past 2^32 elements and lists past 2^31 tokens."""
    V, S = 151936, 28400
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    seen = torch.empty((S, V // 32), dtype=torch.int32, device=DEV)
    counts = torch.empty((S, V), dtype=torch.int32, device=DEV)
    s = S - 2
    assert s * V > 1 << 32
    for t in (seen, counts):
        t[s - 1:] = 7
    at = (1 << 31) + 5
    toks = torch.empty(at + 20, dtype=torch.int32, device=DEV)
    toks[at:] = torch.arange(20, dtype=torch.int32, device=DEV) * 7000 + 11
    start = torch.tensor([at], device=DEV)
    for reset in (i32(1), None):     # through LDS, then through LDS and by atomics onto what is there
        sdv.sd_token_counts(toks, seen, counts, V, start=start, length=i32(20), slot=i32(s), reset=reset)
    sdv.sd_token_counts(toks[at:at + 20].view(1, 20), seen, counts, V, slot=i32(s))
    want = torch.zeros(V, dtype=torch.int32, device=DEV)
    want[toks[at:].long()] = 3
    assert torch.equal(counts[s], want)
    assert torch.equal(seen[s], torch.as_tensor(OS.pack_bits(to_np(want)[None] > 0)).to(DEV)[0])
    for t in (seen, counts):
        assert (t[s - 1] == 7).all() and (t[s + 1] == 7).all()
    x = torch.ones((1, V), device=DEV)
    f = lambda v: torch.full((1,), v, device=DEV)  # noqa: E731
    got = sdv.sd_logit_shape(x, i32(0), i32(0), V, gamma_max=0, repetition=f(2.0), frequency=f(0.25), seen=seen,
                             counts=counts, slot=i32(s))["logits"][0]
    assert torch.equal(got, torch.where(want > 0, 0.5 - 0.75, 1.0))


def test_nothing_to_do():
    i = lambda *k: torch.zeros(k, dtype=torch.int32, device=DEV)  # noqa: E731
    x = torch.ones((3, 64), device=DEV)
    assert sdv.sd_logit_shape(x, i(0), i(0), 64, gamma_max=2)["status"].numel() == 0
    got = sdv.sd_logit_shape(x, i(2), i(2), 64, gamma_max=0, mask=i(0, 2), mask_row0=i(2) - 1,
                             bias=(i(3).long(), i(0), torch.zeros(0, device=DEV)), out=dict(logits=x * 0))
    assert torch.equal(got["logits"][0], x[0]) and (got["status"] == 0).all()
    got = sdv.sd_logit_shape(x, i(1), i(1), 64, gamma_max=0, mask=i(0, 2), mask_row0=i(1))
    assert int(got["status"]) == sdv.SD_ST_BAD_INPUT      # a mask row that is not there
    assert sdv.sd_token_counts(i(0, 4), i(1, 2), None, 64)["status"].numel() == 0
    seen = i(2, 2) + 3
    for reset, want in ((None, 3), (i(2) + 1, 0)):
        assert (sdv.sd_token_counts(i(2, 0), seen, None, 64, reset=reset)["status"] == 0).all()
        assert (seen == want).all()


def test_counts_then_shape_equals_drafts_as_written():
    """Tokens entered into the state do to a row what the same tokens do as
    drafts before it."""
    R, V, g = 4, 2000, 6
    gen = torch.Generator(device=DEV).manual_seed(7)
    draft = torch.randint(0, V, (R, g), generator=gen, device=DEV, dtype=torch.int32)
    x = torch.randn((R * (g + 1), V), generator=gen, device=DEV)
    z = lambda *k: torch.zeros(k, dtype=torch.int32, device=DEV)  # noqa: E731
    seen, counts = z(R, 63), z(R, V)
    f = lambda v: torch.full((R,), v, device=DEV)  # noqa: E731
    kw = dict(repetition=f(1.3), frequency=f(0.4), presence=f(0.2), seen=seen, counts=counts)
    row0 = torch.arange(R, dtype=torch.int32, device=DEV) * (g + 1)
    a = sdv.sd_logit_shape(x, row0, z(R) + g, V, draft_tokens=draft, **kw)["logits"]
    sdv.sd_token_counts(draft, seen, counts, V)
    b = sdv.sd_logit_shape(x, row0 + g, z(R), V, gamma_max=0, **kw)["logits"]
    last = (row0 + g).long()
    assert torch.equal(a[last], b[last])
