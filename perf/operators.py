"""Cases of the operators around a verification step: shaping the target rows
(penalties, biases, grammar masks), the token counts behind the penalties, and
the paged cache's slots (reserved before the target's pass, committed after
verification).

``run`` computes each operator in its plain form (elementary torch operations)
or, where ``own`` is true, through the library's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
NO_SLOT = 64      # status bit: fewer rows than asked for


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one small fp32 batch with every term and a padded leading dimension: the latency of a call
        dict(name="shape_tiny_fp32", op="shape", R=4, gmax=4, V=1000, pad=24, dtype="fp32", hist=64, draft=True,
             penalties=True, bias=12, mask=True, packed=True, in_place=False, ragged=False),
        # one request decoding without drafts over a full vocabulary
        dict(name="shape_single_token", op="shape", R=1, gmax=0, V=151936, pad=0, dtype="bf16", hist=2000,
             draft=False, penalties=True, bias=40, mask=True, packed=False, in_place=False, ragged=False),
        # a middling packed verify batch, every term
        dict(name="shape_mid", op="shape", R=64, gmax=8, V=32000, pad=0, dtype="bf16", hist=1000, draft=True,
             penalties=True, bias=64, mask=True, packed=True, in_place=False, ragged=True),
        # the ragged asynchronous step's batch in reserved slots, every term
        dict(name="shape_ragged_large", op="shape", R=512, gmax=16, V=151936, pad=0, dtype="bf16", hist=1500,
             draft=True, penalties=True, bias=32, mask=True, packed=False, in_place=False, ragged=True),
        # constrained decoding without penalties: grammars and banned tokens, on the rows in place
        dict(name="shape_grammar_in_place", op="shape", R=128, gmax=16, V=129280, pad=0, dtype="bf16", hist=0,
             draft=True, penalties=False, bias=64, mask=True, packed=False, in_place=True, ragged=True),
        # a few short prompts admitted
        dict(name="counts_tiny", op="counts", R=4, V=1024, lo=1, hi=64, output=0.0, repeat=0.2),
        # long contexts resumed, with their own output and a stretch of one repeated token each
        dict(name="counts_long", op="counts", R=96, V=151936, lo=500, hi=131072, output=0.3, repeat=0.1),
        # a small verify batch's slots, in reserved rows
        dict(name="reserve_tiny", op="reserve", R=4, q_max=5, bs=16, max_blocks=32, padded=True, short=False),
        # the ragged step's slots, packed, the pool running out near the end
        dict(name="reserve_ragged", op="reserve", R=512, q_max=17, bs=64, max_blocks=512, padded=False, short=True),
        # prompts entering the cache in long pieces beside decoding requests
        dict(name="reserve_prefill", op="reserve", R=256, q_max=8192, bs=16, max_blocks=2048, padded=False,
             short=False),
        # one small batch's outcome
        dict(name="commit_tiny", op="commit", R=4, q_max=5, bs=16, max_blocks=32, release=0.0),
        # the ragged step's outcome, some requests finished and their blocks given back
        dict(name="commit_ragged", op="commit", R=512, q_max=17, bs=64, max_blocks=512, release=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shape", "shape", "shape", "counts", "reserve", "commit"])
    if op == "shape":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        gmax = rng.randint(0, 16)
        V = 8 * _log_int(rng, 32, 18992)
        in_place = rng.random() < 0.3
        # at most the large listed batch's bytes, masks and counts included
        most = int(2.4e9 / ((gmax + 1) * V * (4 if dtype == "fp32" else 2)))
        R = _log_int(rng, 1, max(1, min(512, most)))
        return dict(op=op, R=R, gmax=gmax, V=V, pad=8 * rng.randint(0, 3), dtype=dtype, hist=_log_int(rng, 8, 4096),
                    draft=rng.random() < 0.8, penalties=not in_place and rng.random() < 0.8,
                    bias=rng.choice([0, _log_int(rng, 1, 300)]), mask=in_place or rng.random() < 0.6,
                    packed=rng.random() < 0.5, in_place=in_place, ragged=rng.random() < 0.7)
    if op == "counts":
        hi = _log_int(rng, 4, 131072)
        R = _log_int(rng, 1, max(1, min(96, 6000000 // hi)))
        return dict(op=op, R=R, V=8 * _log_int(rng, 16, 18992), lo=rng.randint(0, 3) * hi // 8, hi=hi,
                    output=rng.choice([0.0, 0.3, 1.0]), repeat=rng.choice([0.0, 0.1, 0.5]))
    bs = rng.choice([8, 16, 32, 64, 128, 24])
    max_blocks = _log_int(rng, 4, 2048)
    q_max = min(_log_int(rng, 1, 4096), max(1, max_blocks * bs // 2))
    R = _log_int(rng, 1, max(1, min(1024, 500000 // q_max, 600000 // max_blocks)))
    if op == "reserve":
        return dict(op=op, R=R, q_max=q_max, bs=bs, max_blocks=max_blocks, padded=rng.random() < 0.4,
                    short=rng.random() < 0.3)
    return dict(op=op, R=R, q_max=q_max, bs=bs, max_blocks=max_blocks, release=rng.choice([0.0, 0.1, 0.5]))


# ---------------------------------------------------------------------------
# Inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _randint(g, lo, hi, *shape, dtype=torch.int32):
    """Integers lo..hi, both included."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=dtype)


def _pack_bits(b):
    """[n][V] truth values -> [n][ceil(V / 32)] int32 words, token v in bit v % 32 of word v // 32."""
    n, V = b.shape
    W = (V + 31) // 32
    x = torch.zeros((n, W * 32), dtype=torch.int64, device=b.device)
    x[:, :V] = b
    w = (x.view(n, W, 32) << torch.arange(32, device=b.device)).sum(2)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _unpack_bits(w, V):
    """The inverse: [n][W] int32 -> [n][V] truth values."""
    b = (w[:, :, None] >> torch.arange(32, device=w.device, dtype=torch.int32)) & 1
    return b.view(w.shape[0], -1)[:, :V] != 0


def _lengths(g, R, lo, hi):
    """Log-uniform whole lengths in lo..hi."""
    lo_, hi_ = math.log(lo + 1), math.log(hi + 1)
    return (torch.exp(lo_ + (hi_ - lo_) * _rand(g, R)) - 1).round().long().clamp(lo, hi)


def _prepare_shape(c, seed):
    g = _gen(seed)
    R, gmax, V = c["R"], c["gmax"], c["V"]
    ld, dt = V + c["pad"], torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    ell = _randint(g, 0, gmax, R) if c["ragged"] else torch.full((R,), gmax, dtype=torch.int32, device=DEV)
    if c["packed"]:
        row0 = (torch.cumsum(ell + 1, 0) - (ell + 1)).to(torch.int32)
    else:
        row0 = torch.arange(R, dtype=torch.int32, device=DEV) * (gmax + 1)
    n = R * (gmax + 1)
    rows = torch.empty((n + 1, ld), dtype=dt, device=DEV)   # one spare row behind the batch's
    for i in range(0, n + 1, 1024):
        x = torch.randn((min(1024, n + 1 - i), ld), generator=g, device=DEV)
        rows[i:i + 1024] = x * 2.0 + 0.15 * x * x * x   # heavy tails
    dst = rows if c["in_place"] else torch.zeros_like(rows)
    logits = rows[:n]
    # what the requests have seen: frequent tokens come first in a vocabulary
    S = R + 3
    slot = torch.randperm(S, generator=g, device=DEV)[:R].to(torch.int32)
    hist = max(1, c["hist"])
    toks = (V * _rand(g, R, hist) ** 3).long().clamp(max=V - 1)
    used = torch.arange(hist, device=DEV)[None, :] < _lengths(g, R, min(hist, max(1, hist // 8)), hist)[:, None]
    written = used & (torch.arange(hist, device=DEV)[None, :] >= int(0.6 * hist))
    at = slot.long()[:, None] * V + toks
    seen = torch.zeros(S * V, dtype=torch.int32, device=DEV).index_add_(0, at.view(-1), used.view(-1).to(torch.int32))
    counts = torch.zeros(S * V, dtype=torch.int32, device=DEV).index_add_(0, at.view(-1),
                                                                         written.view(-1).to(torch.int32))
    draft = None
    if c["draft"]:
        fresh = (V * _rand(g, R, gmax) ** 3).to(torch.int32).clamp(max=V - 1)
        again = torch.gather(toks, 1, _randint(g, 0, hist - 1, R, gmax, dtype=torch.int64)).to(torch.int32)
        draft = torch.where(_rand(g, R, gmax) < 0.5, again, fresh).contiguous()
    s = dict(c=c, logits=logits, row0=row0, ell=ell, draft=draft, slot=slot, seen=_pack_bits(seen.view(S, V) > 0),
             counts=counts.view(S, V), rep=None, freq=None, pres=None, bias=None, mask=None, mask_row0=None)
    if c["penalties"]:
        on = lambda p: (_rand(g, R) < p).float()  # noqa: E731
        s["rep"] = 1.0 + on(0.67) * 0.5 * _rand(g, R)
        s["freq"] = on(0.6) * (1.2 * _rand(g, R) - 0.2)
        s["pres"] = on(0.6) * (1.2 * _rand(g, R) - 0.2)
    if c["bias"]:
        k = min(c["bias"], V)
        nb = (_rand(g, R) < 0.5) * _randint(g, 1, k, R)
        off = torch.zeros(R + 1, dtype=torch.int64, device=DEV)
        off[1:] = torch.cumsum(nb, 0)
        total = max(1, int(off[-1]))
        e = torch.arange(total, device=DEV)
        r = (torch.searchsorted(off, e, right=True) - 1).clamp(0, R - 1)
        step = 1 + (_rand(g, R) * (V // k - 1)).long()
        tok = ((_rand(g, R) * V).long()[r] + (e - off[r]) * step[r]) % V
        val = 2.0 * torch.randn(total, generator=g, device=DEV)
        ban = float("-inf") if c["in_place"] else -100.0   # in place: what a second pass leaves as it is
        val = torch.where(_rand(g, total) < (2.0 if c["in_place"] else 0.3), torch.full_like(val, ban), val)
        s["bias"] = (off, tok.to(torch.int32), val)
    if c["mask"]:
        masked = _rand(g, R) < 0.6
        masked[0] = True
        m0 = torch.where(masked, (torch.cumsum(masked, 0) - 1) * (gmax + 1), -1).to(torch.int32)
        mask = torch.empty((int(masked.sum()) * (gmax + 1), (V + 31) // 32), dtype=torch.int32, device=DEV)
        for i in range(0, mask.shape[0], 256):
            k = min(256, mask.shape[0] - i)
            kind = _rand(g, k, 1)   # a few tokens allowed, most allowed, now and then none
            p = torch.where(kind < 0.05, 0.0, torch.where(kind < 0.6, 20.0 / V, 0.8))
            mask[i:i + k] = _pack_bits(_rand(g, k, V) < p)
        s["mask"], s["mask_row0"] = mask, m0
    s["dst"] = dst
    s["out"] = dict(logits=dst[:n], status=torch.empty(R, dtype=torch.int32, device=DEV))
    return s


def _prepare_counts(c, seed):
    g = _gen(seed)
    R, V = c["R"], c["V"]
    n = _lengths(g, R, c["lo"], c["hi"])
    off = torch.cumsum(n, 0) - n
    total = max(1, int(n.sum()))
    tokens = (V * _rand(g, total) ** 3).to(torch.int32).clamp(max=V - 1)
    e = torch.arange(total, device=DEV)
    r = (torch.searchsorted(off, e, right=True) - 1).clamp(0, R - 1)
    tokens = torch.where(e - off[r] < c["repeat"] * n[r], (r % V).to(torch.int32), tokens)
    S = R + 2
    out = dict(seen=torch.full((S, (V + 31) // 32), 5, dtype=torch.int32, device=DEV),
               counts=torch.full((S, V), 3, dtype=torch.int32, device=DEV),
               status=torch.empty(R, dtype=torch.int32, device=DEV))
    return dict(c=c, tokens=tokens, start=off, length=n.to(torch.int32),
                prompt=(n * (1.0 - c["output"])).to(torch.int32),
                slot=torch.randperm(S, generator=g, device=DEV)[:R].to(torch.int32),
                reset=torch.ones(R, dtype=torch.int32, device=DEV), **out)


def _held(n, bs):
    return torch.div(n + bs - 1, bs, rounding_mode="floor")


def _prepare_blocks(c, g, held, P):
    """A table of `held` blocks per request and the free list of the rest."""
    R, mb = c["R"], c["max_blocks"]
    perm = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    i = torch.arange(mb, device=DEV)
    take = (first[:, None] + i[None, :]).clamp(max=P - 1)
    table = torch.where(i[None, :] < held[:, None], perm[take], torch.full((), -1, dtype=torch.int32, device=DEV))
    return table.contiguous(), perm, int(held.sum())


def _packed_rows(c):
    """The rows a packed batch has room for."""
    return min(c["R"] * c["q_max"], int((0.6 if c["q_max"] <= 64 else 0.3) * c["R"] * c["q_max"]) + 2 * c["R"] + 8)


def _prepare_reserve(c, seed):
    g = _gen(seed)
    R, q, bs, mb = c["R"], c["q_max"], c["bs"], c["max_blocks"]
    cap = bs * mb
    seq = (_rand(g, R) * (cap - min(q, cap) + 1)).long()
    seq[_rand(g, R) < 0.1] = 0
    # a verify block each; with long pieces half of the requests decode a token or two
    ell = _randint(g, 0, q - 1, R)
    if q > 64:
        ell = torch.where(_rand(g, R) < 0.5, _randint(g, 0, 1, R), ell)
    ell = torch.where(_rand(g, R) < 0.05, torch.full_like(ell, -1), ell)   # requests that sit this step out
    held = _held(seq, bs)
    need = int((_held(seq + ell + 1, bs) - held).sum())
    free = max(1, int(0.9 * need)) if c["short"] else need + 16
    P = R * mb + 16
    table, perm, used = _prepare_blocks(c, g, held, P)
    free_list = torch.zeros(P, dtype=torch.int32, device=DEV)
    free_list[:free] = perm[used:used + free]
    rows = R * q if c["padded"] else _packed_rows(c)
    i32 = lambda *k: torch.empty(k, dtype=torch.int32, device=DEV)  # noqa: E731
    out = dict(ell=i32(R), row0=i32(R), cu_rows=i32(R + 1), ctx_len=i32(R), batch=i32(1), free_count=i32(1),
               row_req=i32(rows), row_pos=i32(rows), row_slot=torch.empty(rows, dtype=torch.int64, device=DEV),
               row_token=i32(rows), status=i32(R))
    s = dict(c=c, seq=seq, ell=ell, table=table, free_list=free_list, rows=rows,
             free_count=torch.tensor([free], dtype=torch.int32, device=DEV),
             x0=_randint(g, 0, 50000, R), tokens=_randint(g, 0, 50000, R, q), out=out)
    if own:
        import draft_verification_amd as sdv
        s["ws"] = torch.empty(sdv.sd_slot_reserve_workspace_size(R), dtype=torch.uint8, device=DEV)
    return s


def _prepare_commit(c, seed):
    g = _gen(seed)
    R, q, bs, mb = c["R"], c["q_max"], c["bs"], c["max_blocks"]
    cap = bs * mb
    seq = (_rand(g, R) * (cap - min(q, cap) + 1)).long()
    ell = _randint(g, 0, min(q, cap) - 1, R)
    ell = torch.where(_rand(g, R) < 0.05, torch.full_like(ell, -1), ell)
    held = _held(seq + ell + 1, bs)
    free = R
    P = R * mb + free
    table, perm, used = _prepare_blocks(c, g, held, P)
    free_list = torch.zeros(P, dtype=torch.int32, device=DEV)
    free_list[:free] = perm[used:used + free]
    n_acc = (_rand(g, R) * (ell + 1).clamp(min=1)).to(torch.int32)
    status = torch.where(_rand(g, R) < 0.02, 2, 0).to(torch.int32)   # a non-finite row now and then
    s = dict(c=c, seq=seq, ell=ell, n_acc=n_acc, status=status, table=table, free_list=free_list,
             free_count=torch.tensor([free], dtype=torch.int32, device=DEV),
             tokens=_randint(g, 0, 50000, R, q), x0=_randint(g, 0, 50000, R),
             release=(_rand(g, R) < c["release"]).to(torch.int32),
             keep=_randint(g, 0, 2, R),
             out=dict(seq_len=torch.empty(R, dtype=torch.int64, device=DEV),
                      x0=torch.empty(R, dtype=torch.int32, device=DEV),
                      n_new=torch.empty(R, dtype=torch.int32, device=DEV),
                      free_count=torch.empty(1, dtype=torch.int32, device=DEV)))
    if own:
        import draft_verification_amd as sdv
        s["ws"] = torch.empty(sdv.sd_slot_commit_workspace_size(R), dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    return {"shape": _prepare_shape, "counts": _prepare_counts, "reserve": _prepare_reserve,
            "commit": _prepare_commit}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# One pass

def _shape_own(s):
    import draft_verification_amd as sdv
    c = s["c"]
    pen = c["penalties"]
    sdv.sd_logit_shape(s["logits"], s["row0"], s["ell"], c["V"], gamma_max=c["gmax"], draft_tokens=s["draft"],
                       repetition=s["rep"], frequency=s["freq"], presence=s["pres"],
                       seen=s["seen"] if pen else None, counts=s["counts"] if pen else None, slot=s["slot"],
                       bias=s["bias"], mask=s["mask"], mask_row0=s["mask_row0"], out=s["out"])
    return s["out"]


def _shape_plain(s):
    """Position by position over all requests at once."""
    c, out = s["c"], s["out"]
    R, gmax, V = c["R"], c["gmax"], c["V"]
    src, dst = s["logits"], s["dst"]
    pen = c["penalties"]
    if pen:
        slot = s["slot"].long()
        seen, cnt = _unpack_bits(s["seen"][slot], V), s["counts"][slot].float()
        rep, freq, pres = (s[k][:, None] for k in ("rep", "freq", "pres"))
    if s["bias"] is not None:
        off, tok, val = s["bias"]
        e = torch.arange(tok.numel(), device=DEV)
        r = (torch.searchsorted(off, e, right=True) - 1).clamp(0, R - 1)
        bias = torch.zeros((R + 1, V), device=DEV)   # the last row takes a list's unused end
        bias.view(-1)[torch.where(e < off[R], r, R) * V + tok] = val
        bias = bias[:R]
    req = torch.arange(R, device=DEV)
    for i in range(gmax + 1):
        act = s["ell"] >= i   # the others take their first row and write to the spare one
        x = src[s["row0"].long() + torch.where(act, i, 0), :V].float()
        if pen:
            if i > 0 and s["draft"] is not None:   # the drafts before this position count as written
                x1 = s["draft"][:, i - 1].long()
                seen[req, x1] = True
                cnt[req, x1] += 1.0
            x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
            x = x - freq * cnt - pres * (cnt > 0)
        if s["bias"] is not None:
            x = x + bias
        if s["mask"] is not None:
            m0 = s["mask_row0"].long()
            allowed = _unpack_bits(s["mask"][m0.clamp(min=0) + i], V)
            x = torch.where(allowed | (m0 < 0)[:, None], x, float("-inf"))
        dst[torch.where(act, s["row0"].long() + i, dst.shape[0] - 1), :V] = x.to(dst.dtype)
    out["status"].zero_()
    return out


def _counts_own(s):
    import draft_verification_amd as sdv
    sdv.sd_token_counts(s["tokens"], s["seen"], s["counts"], s["c"]["V"], start=s["start"], length=s["length"],
                        prompt_len=s["prompt"], slot=s["slot"], reset=s["reset"], out=dict(status=s["status"]))
    return s["seen"], s["counts"], s["status"]


def _counts_plain(s):
    c = s["c"]
    R, V = c["R"], c["V"]
    slot = s["slot"].long()
    tok = s["tokens"].long()
    e = torch.arange(tok.numel(), device=DEV)
    r = (torch.searchsorted(s["start"], e, right=True) - 1).clamp(0, R - 1)
    i = e - s["start"][r]
    inside = i < s["length"][r]
    n = torch.zeros(R * V, dtype=torch.int32, device=DEV)
    n.index_add_(0, r * V + tok, (inside & (i >= s["prompt"][r])).to(torch.int32))
    b = torch.zeros(R * V, dtype=torch.int32, device=DEV)
    b.index_add_(0, r * V + tok, inside.to(torch.int32))
    s["counts"][slot] = n.view(R, V)
    s["seen"][slot] = _pack_bits(b.view(R, V) > 0)
    s["status"].zero_()
    return s["seen"], s["counts"], s["status"]


def _reserve_own(s):
    import draft_verification_amd as sdv
    c = s["c"]
    sdv.sd_slot_reserve(s["seq"], s["ell"], s["table"], s["free_list"], s["free_count"], c["bs"], c["q_max"],
                        padded=c["padded"], x0=s["x0"], tokens=s["tokens"], out=s["out"], workspace=s["ws"])
    return dict(s["out"], table=s["table"])


def _reserve_plain(s):
    c, o = s["c"], s["out"]
    R, q, bs, mb, rows = c["R"], c["q_max"], c["bs"], c["max_blocks"], s["rows"]
    seq, P = s["seq"], s["free_list"].numel()
    F = s["free_count"].long()
    asked = s["ell"].long().clamp(max=q - 1) + 1
    want = torch.minimum(asked, bs * mb - seq)
    if not c["padded"]:
        want = torch.minimum(want, (rows - (torch.cumsum(want, 0) - want)).clamp(min=0))
    h0 = _held(seq, bs)
    need = _held(seq + want, bs) - h0
    d = torch.cumsum(need, 0) - need
    got = torch.minimum(need, (F - d).clamp(min=0))
    n = torch.minimum(want, (h0 + got) * bs - seq)
    cu = torch.cumsum(n, 0)
    o["cu_rows"][0] = 0
    o["cu_rows"][1:] = cu
    o["ell"].copy_(n - 1)
    o["ctx_len"].copy_(seq + n)
    o["batch"].copy_(cu[-1:])
    o["free_count"].copy_(F - got.sum())
    o["status"].copy_(torch.where(n < asked, NO_SLOT, 0))
    # the new blocks, from the end of the free list
    i = torch.arange(mb, device=DEV)[None, :] - h0[:, None]
    k = (F - 1 - d[:, None] - i).clamp(0, P - 1)
    s["table"].copy_(torch.where((i >= 0) & (i < got[:, None]), s["free_list"][k], s["table"]))
    e = torch.arange(rows, device=DEV)
    if c["padded"]:
        first = torch.arange(R, device=DEV) * q
        r = torch.div(e, q, rounding_mode="floor")
    else:
        first = cu - n
        r = torch.searchsorted(cu, e, right=True).clamp(max=R - 1)
    o["row0"].copy_(first.clamp(max=rows - 1))
    at = e - first[r]
    live = at < n[r]
    pos = (seq[r] + at).clamp(max=bs * mb - 1)
    block = s["table"][r, torch.div(pos, bs, rounding_mode="floor")].long()
    tok = torch.where(at == 0, s["x0"][r], s["tokens"][r, (at - 1).clamp(0, q - 1)])
    o["row_req"].copy_(torch.where(live, r, -1))
    o["row_pos"].copy_(torch.where(live, pos, -1))
    o["row_slot"].copy_(torch.where(live, block * bs + pos % bs, -1))
    o["row_token"].copy_(torch.where(live, tok, -1))
    return dict(o, table=s["table"])


def _commit_own(s):
    import draft_verification_amd as sdv
    sdv.sd_slot_commit(s["seq"], s["ell"], s["n_acc"], s["table"], s["free_list"], s["free_count"], s["c"]["bs"],
                       out_tokens=s["tokens"], x0=s["x0"], status=s["status"], release=s["release"],
                       keep=s["keep"], out=s["out"], workspace=s["ws"])
    return dict(s["out"], free_list=s["free_list"])


def _commit_plain(s):
    c, o = s["c"], s["out"]
    bs, mb = c["bs"], c["max_blocks"]
    seq, ell, P = s["seq"], s["ell"].long(), s["free_list"].numel()
    F = s["free_count"].long()
    ok = (ell >= 0) & ((s["status"] & 6) == 0)
    acc = torch.minimum(s["n_acc"].long().clamp(min=0), ell.clamp(min=0))
    adv = torch.where(ok, acc + 1, 0)
    free = s["release"] != 0
    new = torch.where(free, 0, seq + adv)
    held = _held(seq + ell + 1, bs)
    kept = torch.where(free, torch.minimum(s["keep"].long().clamp(min=0), held), _held(new, bs))
    give = held - kept
    d = torch.cumsum(give, 0) - give
    i = torch.arange(mb, device=DEV)[None, :] - kept[:, None]
    to = torch.where((i >= 0) & (i < give[:, None]), (F + d)[:, None] + i, P)
    wide = torch.cat([s["free_list"], s["free_list"][:1]])
    wide[to] = s["table"]
    s["free_list"].copy_(wide[:P])
    o["seq_len"].copy_(new)
    o["free_count"].copy_(F + give.sum())
    nxt = torch.gather(s["tokens"], 1, acc[:, None])[:, 0]
    o["x0"].copy_(torch.where(adv > 0, nxt, s["x0"]))
    o["n_new"].copy_(adv)
    return dict(o, free_list=s["free_list"])


_RUN = {"shape": (_shape_plain, _shape_own), "counts": (_counts_plain, _counts_own),
        "reserve": (_reserve_plain, _reserve_own), "commit": (_commit_plain, _commit_own)}


def run(state):
    return _RUN[state["c"]["op"]][1 if own else 0](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without

def work(case):
    c = case
    R = c["R"]
    if c["op"] == "shape":
        n = R * (c["gmax"] / 2 + 1 if c["ragged"] else c["gmax"] + 1)
        es = 4 if c["dtype"] == "fp32" else 2
        V = c["V"]
        mask = 0.6 * n * V / 8 if c["mask"] else 0
        state = R * (V / 8 + 8 * 0.5 * c["hist"]) if c["penalties"] else 0
        # in place only what changes is written: the masked share of the masked rows
        rows = 0.6 * 0.68 * n * V * es if c["in_place"] else 2 * n * V * es
        return dict(bytes=rows + mask + state + 0.25 * R * c["bias"] * 8, flops=n * V)
    if c["op"] == "counts":
        lo, hi = c["lo"] + 1, c["hi"] + 1
        mean = (hi - lo) / math.log(hi / lo) if hi > lo else lo
        # the row of a request that starts anew is written whole
        return dict(bytes=R * (4 * mean + c["V"] / 8 + 4 * c["V"]), flops=R * mean)
    if c["op"] == "reserve":
        n = R * (c["q_max"] / 2 if c["q_max"] <= 64 else c["q_max"] / 4)
        rows = R * c["q_max"] if c["padded"] else _packed_rows(c)
        return dict(bytes=rows * 20 + n * 4 + R * 60 + 8 * n / c["bs"], flops=10 * n)
    give = R * (c["q_max"] / 4 / c["bs"] + c["release"] * c["max_blocks"] / 2)
    return dict(bytes=R * 60 + 8 * give, flops=10 * R)


# ---------------------------------------------------------------------------
# The definition in 64 bits: request by request, token by token that a term touches

def exact(case, seed):
    if case["op"] != "shape":
        return None   # whole numbers: compared for equality
    s = prepare(case, seed)
    c = s["c"]
    V = c["V"]
    out = torch.zeros((s["logits"].shape[0], s["logits"].shape[1]), dtype=torch.float64, device=DEV)
    if c["in_place"]:
        out.copy_(s["logits"])
    row0, ell, slot = s["row0"].tolist(), s["ell"].tolist(), s["slot"].tolist()
    draft = s["draft"].tolist() if s["draft"] is not None else None
    off = s["bias"][0].tolist() if s["bias"] is not None else None
    m0 = s["mask_row0"].tolist() if s["mask"] is not None else None
    word, bit = torch.arange(V, device=DEV) // 32, torch.arange(V, device=DEV) % 32
    for r in range(c["R"]):
        n = ell[r] + 1
        x = s["logits"][row0[r]:row0[r] + n, :V].double()
        if c["penalties"]:
            rep, freq, pres = (float(s[k][r]) for k in ("rep", "freq", "pres"))
            base = s["counts"][slot[r]].double()
            old = (s["seen"][slot[r]][word] >> bit) & 1
            more = torch.zeros((n, V), dtype=torch.float64, device=DEV)
            for i in range(1, n):
                if draft is not None:
                    more[i:, draft[r][i - 1]] += 1.0
            met = (old != 0)[None, :] | (more > 0)
            total = base[None, :] + more
            x = torch.where(met & (x > 0), x / rep, torch.where(met, x * rep, x))
            x = x - freq * total - pres * total.clamp(max=1.0)
        if off is not None and off[r + 1] > off[r]:
            at = s["bias"][1][off[r]:off[r + 1]].long()
            x[:, at] += s["bias"][2][off[r]:off[r + 1]].double()
        if m0 is not None and m0[r] >= 0:
            for i in range(n):
                x[i][((s["mask"][m0[r] + i][word] >> bit) & 1) == 0] = -math.inf
        out[row0[r]:row0[r] + n, :V] = x
    return dict(logits=out, status=None)
