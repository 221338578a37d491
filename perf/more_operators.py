"""Cases of the operators between a step's slots and its logits: norms and
position rotation of queries and keys, keys and values appended to the paged
cache (in bf16 or in 4 bits) and read back, and attention of a step's rows over
that cache.

``run`` computes each operator in its plain form (elementary torch operations)
or, where ``own`` is true, through the library's entry points.

A cache of 4 bits holds, per token and head, 32 channels at a time: values of
{0, .5, 1, 1.5, 2, 3, 4, 6} and a sign (two to a byte, the even channel in the
low half) times one power of two 2^(byte - 127), the smallest for which the
group's largest magnitude is at most 7.
"""

import math

import torch

own = False

DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6
BASE = 10000.0
UNUSED = 2.0 ** -12   # what rows of no request hold


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # a few rows in fp32, pairs next to each other: the latency of a call
        dict(name="rope_tiny_fp32", op="rope", rows=4, n_q=8, n_kv=2, D=64, rot=64, dtype="fp32", interleaved=True,
             norm=True, far=2000, skip=0.0),
        # the rows of many long prompt pieces, cut from the fused projection; a quarter of the row buffer unused
        dict(name="rope_pieces", op="rope", rows=16384, n_q=32, n_kv=8, D=128, rot=128, dtype="bf16",
             interleaved=False, norm=True, far=131072, skip=0.25),
        # 64 requests decoding a token each: queries turned, keys and values into their slots
        dict(name="append_tokens", op="append", rows=64, n_q=32, n_kv=8, D=128, rot=128, dtype="bf16",
             interleaved=False, norm=True, cache="bf16", bs=16, blocks=4096, far=8192, skip=0.0),
        # prompt pieces entering the cache, part of each head rotated, no norms
        dict(name="append_pieces", op="append", rows=8192, n_q=64, n_kv=8, D=128, rot=64, dtype="bf16",
             interleaved=False, norm=False, cache="bf16", bs=64, blocks=600, far=32768, skip=0.1),
        # a verify batch's keys and values into 4 bits, and back
        dict(name="append_verify_4bit", op="append", rows=768, n_q=0, n_kv=8, D=128, rot=128, dtype="bf16",
             interleaved=False, norm=True, cache="fp4", bs=16, blocks=2048, far=8192, skip=0.3),
        # prompt pieces into 4 bits, and back
        dict(name="append_pieces_4bit", op="append", rows=8192, n_q=0, n_kv=8, D=128, rot=128, dtype="bf16",
             interleaved=False, norm=True, cache="fp4", bs=64, blocks=600, far=131072, skip=0.1),
        # one small batch, a token each: the latency of a call
        dict(name="attn_tiny", op="attn", R=4, q_max=1, n_q=8, n_kv=2, D=64, cache="bf16", bs=16, lo=20, hi=300,
             window=0, causal=True, many=1.0),
        # decoding without drafts over contexts of very different lengths
        dict(name="attn_tokens", op="attn", R=128, q_max=1, n_q=32, n_kv=8, D=128, cache="bf16", bs=16, lo=1024,
             hi=16384, window=0, causal=True, many=1.0),
        # the same over a cache in 4 bits
        dict(name="attn_tokens_4bit", op="attn", R=128, q_max=1, n_q=32, n_kv=8, D=128, cache="fp4", bs=64, lo=1024,
             hi=16384, window=0, causal=True, many=1.0),
        # the rows of a verify batch: an anchor and up to 11 drafts each
        dict(name="attn_verify", op="attn", R=128, q_max=12, n_q=32, n_kv=8, D=128, cache="bf16", bs=64, lo=512,
             hi=8192, window=0, causal=True, many=1.0),
        # two very long contexts in 4 bits, a few drafts
        dict(name="attn_long_4bit", op="attn", R=2, q_max=5, n_q=64, n_kv=8, D=128, cache="fp4", bs=256, lo=100000,
             hi=131072, window=0, causal=True, many=1.0),
        # pieces of prompts beside decoding requests
        dict(name="attn_pieces", op="attn", R=16, q_max=512, n_q=32, n_kv=8, D=128, cache="bf16", bs=64, lo=600,
             hi=8192, window=0, causal=True, many=0.6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "append", "attn", "attn", "attn"))
    n_kv = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 4, 5, 7, 8))
    D = rng.choice((64, 96, 128, 128, 192, 256))
    if op == "attn":
        while True:
            c = dict(op=op, R=_log_int(rng, 1, 200), q_max=rng.choice((1, 1, rng.randint(2, 17), rng.randint(2, 17),
                                                                       _log_int(rng, 18, 500))),
                     n_q=n_kv * group, n_kv=n_kv, D=D, cache=rng.choice(("bf16", "fp4")),
                     bs=rng.choice((16, 32, 64, 128, 256, rng.randint(1, 100))), lo=0, hi=0,
                     window=rng.choice((0, 0, 0, _log_int(rng, 30, 4000))), causal=rng.random() < 0.85,
                     many=rng.choice((1.0, 0.5)))
            c["hi"] = c["q_max"] + _log_int(rng, 16, 60000)
            c["lo"] = c["q_max"] + _log_int(rng, 8, c["hi"] - c["q_max"])
            w = work(c)
            plain = c["R"] * c["hi"] * c["n_kv"] * D
            scores = c["R"] * c["hi"] * c["n_q"] * c["q_max"]
            if w["bytes"] < 2e9 and w["flops"] < 2e11 and plain < 1.5e9 and scores < 1.5e9:
                return c
    rows = _log_int(rng, 1, 8192)
    c = dict(op=op, rows=rows, n_q=n_kv * group, n_kv=n_kv, D=D, rot=rng.choice((D, D, D // 2, 32)),
             dtype=rng.choice(("bf16", "bf16", "fp32")), interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
             far=_log_int(rng, 64, 1000000), skip=rng.choice((0.0, 0.2)))
    if op == "append":
        c["cache"] = rng.choice(("bf16", "fp4"))
        c["bs"] = rng.choice((16, 32, 64, 128, 256, rng.randint(1, 100)))
        c["blocks"] = -(-rows // c["bs"]) + _log_int(rng, 1, 200)
        if c["cache"] == "fp4":
            c["n_q"] = 0
    return c


# ---------------------------------------------------------------------------
# Inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32)


def _type(c):
    return torch.float32 if c["dtype"] == "fp32" else torch.bfloat16


def _to_4bit(x):
    """(codes, scale bytes) of x [..., D] (fp32 or fp64, finite)."""
    D = x.shape[-1]
    grp = x.unflatten(-1, (D // 32, 32))
    top = grp.abs().amax(-1)
    m, e = torch.frexp(top)                              # top = m 2^e, m in [.5, 1)
    e = torch.where(m > 0.875, e - 2, e - 3)             # top <= 7 2^e
    e = torch.where(top > 0, e, -126).clamp(min=-126)
    a = torch.ldexp(grp.abs(), -e[..., None])
    # nearest level, ties to the even code
    lev = torch.full(a.shape, 0, dtype=torch.uint8, device=x.device)
    for k, (mid, up) in enumerate(((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                                   (3.5, True), (5.0, False))):
        lev = lev + ((a >= mid) if up else (a > mid)).to(torch.uint8)
    lev = lev | (torch.signbit(grp).to(torch.uint8) << 3)
    lev = lev.flatten(-2)
    return lev[..., 0::2] | (lev[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _pairs():
    """[256][2]: the two values of a byte of codes, without the scale."""
    one = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=DEV)
    b = torch.arange(256, device=DEV)
    return torch.stack([one[b & 15], one[b >> 4]], 1)


def _from_4bit(codes, scale, pairs):
    """fp32 values [..., D] of codes [..., D/2] and scale bytes [..., D/32]."""
    v = pairs[codes.long()].flatten(-2)
    s = torch.ldexp(torch.ones((), device=DEV), scale.int() - 127)
    return (v.unflatten(-1, (scale.shape[-1], 32)) * s[..., None]).flatten(-2)


def _cut_heads(g, c):
    """q, k, v as parts of the rows of one fused projection."""
    n, D, nq, nk = c["rows"], c["D"], c["n_q"], c["n_kv"]
    y = _normal(g, (n, nq + 2 * nk, D)) * (0.5 + 2 * _rand(g, 1, nq + 2 * nk, 1))
    y[:, nq:nq + nk] *= torch.where(_rand(g, 1, nk, D) < 0.03, 6.0, 1.0)      # a few large channels of the keys
    y = y.to(_type(c))
    return y[:, :nq], y[:, nq:nq + nk], y[:, nq + nk:]


def _prepare_heads(c, seed):
    g = _gen(seed)
    n, D = c["rows"], c["D"]
    q, k, v = _cut_heads(g, c)
    pos = (_rand(g, n) * c["far"]).to(torch.int32)
    pos = torch.where(_rand(g, n) < c["skip"], -1, pos)      # rows that are no request's
    s = dict(c=c, q=q, k=k, v=v, pos=pos, wq=None, wk=None,
             inv_freq=(BASE ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])).float())
    if c["norm"]:
        s["wq"], s["wk"] = 1.0 + 0.2 * _normal(g, (D,)), 1.0 + 0.2 * _normal(g, (D,))
    s["q_out"] = torch.full((n, c["n_q"], D), 0.5, dtype=q.dtype, device=DEV)
    if c["op"] == "rope":
        s["k_out"] = torch.full((n, c["n_kv"], D), 0.5, dtype=q.dtype, device=DEV)
        return s
    slots = c["blocks"] * c["bs"]
    at = torch.randperm(c["blocks"], generator=g, device=DEV)     # runs of slots in scattered blocks
    i = torch.arange(n, device=DEV)
    slot = at[torch.div(i, c["bs"], rounding_mode="floor")] * c["bs"] + i % c["bs"]
    s["slot"] = torch.where(pos < 0, -1, slot)
    shape = (c["blocks"] + 1, c["n_kv"], c["bs"], D)              # and a spare block behind the pool
    if c["cache"] == "bf16":
        full = tuple(torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    else:
        half = shape[:3] + (D // 2,)
        full = tuple(torch.zeros(half, dtype=torch.uint8, device=DEV) for _ in range(2)) + tuple(
            torch.full(shape[:3] + (D // 32,), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
        s["pairs"] = _pairs()
        s["values"] = torch.zeros((2, n, c["n_kv"], D), dtype=torch.bfloat16, device=DEV)
    s["full"], s["cache"] = full, tuple(t[:-1] for t in full)
    s["put"] = torch.where(s["slot"] < 0, slots, s["slot"])       # where the plain form writes
    return s


def _rows_of(c, g):
    """Rows and context of each request."""
    R, q = c["R"], c["q_max"]
    n = _randint(g, 1, q, R)
    if c["many"] < 1.0:
        n = torch.where(_rand(g, R) < c["many"], n, 1)
    if q > 17:
        n[0] = q
    if R > 2 and q > 1:
        n[1] = 0                       # a request that sits this step out
    ctx = torch.exp(math.log(c["lo"]) + _rand(g, R) * (math.log(c["hi"]) - math.log(c["lo"]))).round().to(torch.int32)
    if R > 1:
        ctx[0], ctx[-1] = c["hi"], c["lo"]
    return n, torch.maximum(ctx.clamp(c["lo"], c["hi"]), n)


def _prepare_attn(c, seed):
    g = _gen(seed)
    R, D, bs, nk = c["R"], c["D"], c["bs"], c["n_kv"]
    n, ctx = _rows_of(c, g)
    mb = -(-c["hi"] // bs) + 1
    held = torch.div(ctx + bs - 1, bs, rounding_mode="floor").long()
    first = torch.cumsum(held, 0) - held
    used = int(held.sum())
    perm = torch.randperm(used + 3, generator=g, device=DEV).to(torch.int32)
    i = torch.arange(mb, device=DEV)
    table = torch.where(i[None] < held[:, None], perm[(first[:, None] + i[None]).clamp(max=used)], -1)
    rows = R * c["q_max"] + 5              # a packed batch in the row buffers of the largest one
    s = dict(c=c, table=table.to(torch.int32).contiguous(), ctx=ctx, ell=(n - 1).to(torch.int32),
             row0=(torch.cumsum(n, 0) - n).to(torch.int32), rows=rows, pairs=_pairs(),
             q=(2.0 * _normal(g, (rows, c["n_q"], D))).to(torch.bfloat16),
             scale=D ** -0.5)
    shape = (used + 3, nk, bs, D)
    cache = []
    for part in range(2):
        if c["cache"] == "bf16":
            t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
            for b in range(0, used + 3, 1 + (1 << 28) // (nk * bs * D)):
                e = min(used + 3, b + 1 + (1 << 28) // (nk * bs * D))
                t[b:e] = _normal(g, (e - b,) + shape[1:], torch.bfloat16)
            cache.append((t,))
        else:
            t = torch.empty(shape[:3] + (D // 2,), dtype=torch.uint8, device=DEV)
            sc = torch.empty(shape[:3] + (D // 32,), dtype=torch.uint8, device=DEV)
            for b in range(0, used + 3, 1 + (1 << 27) // (nk * bs * D)):
                e = min(used + 3, b + 1 + (1 << 27) // (nk * bs * D))
                t[b:e], sc[b:e] = _to_4bit(_normal(g, (e - b,) + shape[1:]))
            cache.append((t, sc))
    s["cache"] = tuple(cache[k][p] for p in range(len(cache[0])) for k in range(2))
    s["out_full"] = torch.full((rows + 1, c["n_q"], D), UNUSED, dtype=torch.bfloat16, device=DEV)
    s["lse_full"] = torch.full((rows + 1, c["n_q"]), UNUSED, device=DEV)
    s["out"], s["lse"] = s["out_full"][:-1], s["lse_full"][:-1]
    if own:      # a step's plan, which every layer's call takes
        import draft_verification_amd as sdv
        s["plan"] = sdv.sd_attn_plan(s["row0"], s["ell"], ctx, c["q_max"], c["n_q"], s["cache"],
                                     causal=c["causal"], window=c["window"])
    return s


def prepare(case, seed):
    return (_prepare_attn if case["op"] == "attn" else _prepare_heads)(case, seed)


# ---------------------------------------------------------------------------
# One pass

def _angles(pos, inv_freq):
    a = pos.double()[:, None] * inv_freq.double()[None, :]
    return a.cos(), a.sin()


def _turn(x, w, cos, sin, interleaved):
    """Norm of every head, then the rotation of its first channels; x [n][H][D] fp32 or fp64."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)
    r = 2 * cos.shape[1]
    cos, sin = cos.to(x.dtype)[:, None], sin.to(x.dtype)[:, None]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _rope_own(s):
    import draft_verification_amd as sdv
    r = sdv.sd_qk_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                       interleaved=s["c"]["interleaved"], out=dict(q=s["q_out"], k=s["k_out"]))
    return r["q"], r["k"]


def _rope_plain(s):
    cos, sin = _angles(s["pos"], s["inv_freq"])
    live = (s["pos"] >= 0)[:, None, None]
    for x, w, o in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
        o.copy_(torch.where(live, _turn(x.float(), w, cos, sin, s["c"]["interleaved"]).to(o.dtype), o))
    return s["q_out"], s["k_out"]


def _append_own(s):
    import draft_verification_amd as sdv
    c = s["c"]
    sdv.sd_cache_append(s["k"], s["v"], s["cache"], s["slot"], row_pos=s["pos"], inv_freq=s["inv_freq"],
                        q=s["q"] if c["n_q"] else None, q_weight=s["wq"] if c["n_q"] else None, k_weight=s["wk"],
                        eps=EPS, interleaved=c["interleaved"], out=dict(q=s["q_out"]) if c["n_q"] else None)
    if c["cache"] == "bf16":
        return s["q_out"], s["cache"]
    sdv.sd_cache_read(s["slot"], s["cache"], out=dict(k=s["values"][0], v=s["values"][1]))
    # 4 bits times a power of two: exact in e5m2
    return s["values"].to(torch.float8_e5m2)


def _append_plain(s):
    c = s["c"]
    cos, sin = _angles(s["pos"], s["inv_freq"])
    live = (s["pos"] >= 0)[:, None, None]
    put, bs = s["put"], c["bs"]
    block, off = torch.div(put, bs, rounding_mode="floor"), put % bs
    if c["n_q"]:
        q = _turn(s["q"].float(), s["wq"], cos, sin, c["interleaved"])
        s["q_out"].copy_(torch.where(live, q.to(s["q_out"].dtype), s["q_out"]))
    if c["cache"] == "bf16":
        k = _turn(s["k"].float(), s["wk"], cos, sin, c["interleaved"])
        s["full"][0][block, :, off] = k.bfloat16()
        s["full"][1][block, :, off] = s["v"].bfloat16()
        return s["q_out"], s["cache"]
    # in 64 bits: the values next to a level's border
    k = _turn(s["k"].double(), s["wk"], cos, sin, c["interleaved"])
    for part, x in enumerate((k, s["v"].double())):
        codes, scale = _to_4bit(x)
        s["full"][part][block, :, off] = codes
        s["full"][2 + part][block, :, off] = scale
        back = _from_4bit(s["full"][part][block, :, off], s["full"][2 + part][block, :, off], s["pairs"])
        s["values"][part].copy_(torch.where(live, back.bfloat16(), s["values"][part]))
    return s["values"].to(torch.float8_e5m2)


def _attn_own(s):
    import draft_verification_amd as sdv
    r = sdv.sd_cache_attn(s["q"], s["cache"], s["table"], s["plan"], scale=s["scale"],
                          out=dict(out=s["out"], lse=s["lse"]))
    return r["out"], r["lse"]


def _attn_plain(s):
    c = s["c"]
    R, qm, nq, nk, D, bs = (c[k] for k in ("R", "q_max", "n_q", "n_kv", "D", "bs"))
    G = nq // nk
    nb = -(-c["hi"] // bs)
    T = nb * bs
    at = s["table"][:, :nb].long().clamp(min=0)

    def side(part):
        if c["cache"] == "bf16":
            x = s["cache"][part][at].float()
        else:
            x = _from_4bit(s["cache"][part][at], s["cache"][2 + part][at], s["pairs"])
        return x.permute(0, 2, 1, 3, 4).reshape(R * nk, T, D)

    n = s["ell"].long() + 1
    i = torch.arange(qm, device=DEV)
    row = torch.where(i[None] < n[:, None], s["row0"].long()[:, None] + i[None], s["rows"])
    q = s["q"][row.clamp(max=s["rows"] - 1)].float()                     # [R][qm][nq][D]
    q = q.view(R, qm, nk, G, D).permute(0, 2, 3, 1, 4).reshape(R * nk, G * qm, D)
    x = torch.matmul(q, side(0).transpose(1, 2).contiguous()) * s["scale"]
    pos = (s["ctx"].long() - n)[:, None] + i[None]                       # [R][qm]
    t = torch.arange(T, device=DEV)
    see = (t[None, None] < s["ctx"][:, None, None]).expand(R, qm, T)
    if c["causal"]:
        see = see & (t[None, None] <= pos[..., None])
    if c["window"]:
        see = see & (t[None, None] > pos[..., None] - c["window"])
    x = x.view(R, nk, G, qm, T).masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(R * nk, G * qm, T), side(1)).view(R, nk, G, qm, D) / torch.where(z > 0, z, 1.0)
    s["out_full"][row] = o.permute(0, 3, 1, 2, 4).reshape(R, qm, nq, D).bfloat16()
    s["lse_full"][row] = (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).reshape(R, qm, nq)
    return s["out"], s["lse"]


_RUN = {"rope": (_rope_plain, _rope_own), "append": (_append_plain, _append_own), "attn": (_attn_plain, _attn_own)}


def run(state):
    return _RUN[state["c"]["op"]][1 if own else 0](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without

def work(case):
    c = case
    D, nq, nk = c["D"], c["n_q"], c["n_kv"]
    if c["op"] == "attn":
        R, q = c["R"], c["q_max"]
        lo, hi = c["lo"], c["hi"]
        ctx = (hi - lo) / math.log(hi / lo) if hi > lo else lo
        n = c["many"] * (q + 1) / 2 + 1 - c["many"]
        keys = min(ctx, c["window"] + n) if c["window"] else ctx
        side = 2 if c["cache"] == "bf16" else 0.5 + 1 / 32
        seen = min(ctx, c["window"]) if c["window"] else ctx - (n / 2 if c["causal"] else 0)
        return dict(bytes=R * (keys * nk * D * 2 * side + n * nq * (D * 4 + 4)), flops=4 * R * n * seen * nq * D)
    n = c["rows"] * (1 - c["skip"])
    es = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "rope":
        return dict(bytes=2 * n * (nq + nk) * D * es, flops=8 * n * (nq + nk) * D)
    side = 2 if c["cache"] == "bf16" else 0.5 + 1 / 32
    moved = n * D * (2 * nq * es + 2 * nk * (es + side))
    if c["cache"] == "fp4":                          # and read back
        moved += n * D * 2 * nk * (side + 2)
    return dict(bytes=moved, flops=8 * n * (nq + nk) * D)


# ---------------------------------------------------------------------------
# The definition in 64 bits: heads as complex numbers, requests one by one

def _exact_turn(x, w, pos, inv_freq, interleaved):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) * w.double()
    a = torch.outer(pos.double(), inv_freq.double())
    r = 2 * inv_freq.numel()
    head, tail = x[..., :r], x[..., r:]
    pair = head.unflatten(-1, (r // 2, 2)) if interleaved else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(a), a)[:, None]
    z = torch.view_as_real(z)
    y = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([y, tail], -1)


def _exact_4bit(x):
    """The values that x [..., D] becomes in 4 bits."""
    lev = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
    grp = x.unflatten(-1, (-1, 32))
    top = grp.abs().amax(-1, keepdim=True)
    step = torch.exp2(torch.ceil(torch.log2(top / 7.0)))
    step = torch.where(top > 7.0 * step, 2 * step, torch.where(top <= 3.5 * step, step / 2, step))
    step = torch.where(top > 0, step, 2.0 ** -126)
    a = (grp.abs() / step).contiguous()
    hi = torch.searchsorted(lev, a.clamp(max=6.0)).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up, down = lev[hi] - a, a - lev[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), lev[hi], lev[lo])
    return (torch.copysign(pick, grp) * step).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] != "attn":
        live = (s["pos"] >= 0)[:, None, None]
        turn = lambda x, w: _exact_turn(x, w, s["pos"], s["inv_freq"], c["interleaved"])  # noqa: E731
        q = torch.where(live, turn(s["q"], s["wq"]), 0.5) if c["n_q"] else None
        k = turn(s["k"], s["wk"])
        if c["op"] == "rope":
            return q, torch.where(live, k, 0.5)
        v = s["v"].double()
        if c["cache"] == "fp4":
            return torch.where(live[None], torch.stack([_exact_4bit(k), _exact_4bit(v)]), 0.0)
        caches = []
        for x in (k, v):
            t = torch.zeros(s["cache"][0].shape, dtype=torch.float64, device=DEV)
            at = s["slot"][s["slot"] >= 0]
            t.transpose(1, 2)[torch.div(at, c["bs"], rounding_mode="floor"), at % c["bs"]] = x[s["slot"] >= 0]
            caches.append(t)
        return q, tuple(caches)
    out = torch.full(s["out"].shape, UNUSED, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, UNUSED, dtype=torch.float64, device=DEV)
    lev = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device=DEV)
    nk, G, D = c["n_kv"], c["n_q"] // c["n_kv"], c["D"]
    ctx, ell, row0 = s["ctx"].tolist(), s["ell"].tolist(), s["row0"].tolist()
    for r in range(c["R"]):
        n, T = ell[r] + 1, ctx[r]
        if n < 1:
            continue
        at = s["table"][r, :-(-T // c["bs"])].long()
        side = []
        for part in range(2):
            x = s["cache"][part][at]
            if c["cache"] == "fp4":
                x = torch.stack([lev[(x & 15).long()], lev[(x >> 4).long()]], -1).flatten(-2)
                e = torch.exp2(s["cache"][2 + part][at].double() - 127.0)
                x = x * e.repeat_interleave(32, -1)
            side.append(x.double().transpose(0, 1).reshape(nk, -1, D)[:, :T])
        q = s["q"][row0[r]:row0[r] + n].double().view(n, nk, G, D).permute(1, 2, 0, 3).reshape(nk, G * n, D)
        x = (torch.matmul(q, side[0].transpose(1, 2).contiguous()) * s["scale"]).view(nk, G, n, T)
        pos = T - n + torch.arange(n, device=DEV)[:, None]
        t = torch.arange(T, device=DEV)[None]
        see = torch.ones((n, T), dtype=torch.bool, device=DEV)
        if c["causal"]:
            see &= t <= pos
        if c["window"]:
            see &= t > pos - c["window"]
        x = torch.where(see, x, -math.inf)
        z = torch.logsumexp(x, -1)
        p = torch.exp(x - z[..., None])
        o = torch.matmul(p.view(nk, G * n, T), side[1].contiguous()).view(nk, G, n, D)
        out[row0[r]:row0[r] + n] = o.permute(2, 0, 1, 3).reshape(n, nk * G, D)
        lse[row0[r]:row0[r] + n] = z.permute(2, 0, 1).reshape(n, nk * G)
    return out, lse
