"""The paged cache's calls as a step makes them: sd_slot_reserve, for each layer
sd_cache_append and sd_cache_attn with one sd_attn_plan, sd_slot_commit; in
graphs, on side streams and two at once."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from oracle import heads as OH
from tests.attn_util import DEV, U, check, gen, np64, random_batch, random_cache, tokens_of, visible

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _t(x, dt=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dt).to(DEV)


class Layers:
    """A pool's state and the caches of a few layers."""

    def __init__(self, seed, kind, R, q_max, n_q, n_kv, D, bs, mb, pool, padded, layers=2):
        self.g = gen(seed)
        self.kind, self.R, self.q_max, self.n_q, self.n_kv, self.D = kind, R, q_max, n_q, n_kv, D
        self.bs, self.padded, self.pool = bs, padded, pool
        self.rows = R * q_max if padded else R * q_max - 3
        self.seq, self.table = _t(np.zeros(R), torch.int64), _t(np.full((R, mb), -1))
        self.free, self.F = torch.randperm(pool, generator=self.g).to(torch.int32).to(DEV), _t([pool])
        self.cache = [random_cache(self.g, kind, pool, n_kv, bs, D)[0] for _ in range(layers)]   # what was there before
        self.freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(DEV)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=self.g)).to(DEV) for _ in range(2))

    def projected(self):
        """A projection's rows: queries, keys and values side by side."""
        x = torch.randn((self.rows, self.n_q + 2 * self.n_kv, self.D), generator=self.g).to(torch.bfloat16).to(DEV)
        return x[:, :self.n_q], x[:, self.n_q:self.n_q + self.n_kv], x[:, self.n_q + self.n_kv:]

    def reserve(self, ell, **kw):
        return sdv.sd_slot_reserve(self.seq, ell, self.table, self.free, self.F, self.bs, self.q_max,
                                   max_rows=self.rows, padded=self.padded, **kw)

    def append(self, l, s, x, **kw):
        q, k, v = x
        sdv.sd_cache_append(k, v, self.cache[l], s["row_slot"], s["row_pos"], self.freq, q=q, q_weight=self.wq,
                            k_weight=self.wk, eps=EPS, out=dict(q=q), **kw)

    def plan(self, s, **kw):
        return sdv.sd_attn_plan(s["row0"], s["ell"], s["ctx_len"], self.q_max, self.n_q, self.cache[0], **kw)


def _stored(L, y, size):
    """How far a stored key may be from y, which is known within 24u of size
    (norm and rotation in fp32): half a step of bf16; in 4 bits half the
    distance of two levels, at most one scale (between 4 and 6, or 7 and 6), and
    at a border between two scales as much."""
    if L.kind == "bf16":
        return 24 * U * size + 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -16)
    top = np.repeat(np.exp2(OH.scale_exponent(y).astype(float)), 32, -1)
    return 24 * U * size.max(-1, keepdims=True) + top * (1 + 2.0 ** -16)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("kind,n_q,n_kv,D,bs", [("bf16", 8, 2, 128, 16), ("bf16", 4, 4, 64, 5), ("fp4", 8, 2, 128, 16),
                                                ("fp4", 6, 1, 96, 7), ("fp4", 4, 2, 256, 32)])
def test_steps(kind, n_q, n_kv, D, bs, padded):
    R, q_max, mb = 5, 40, -(-200 // bs)
    L = Layers(11, kind, R, q_max, n_q, n_kv, D, bs, mb, -(-360 // bs), padded)
    hist = [[[] for _ in range(R)] for _ in L.cache]
    asked = [[39, 20, -1, 0, 38], [4, 4, 39, 4, 4], [4, 3, 2, -1, 0], [39, 39, 0, 39, 39], [39, 39, 4, 39, 39],
             [39, 39, 4, 39, 39]]
    kept = [[39, 20, 0, 0, 38], [0, 4, 39, 2, 1], [4, 0, 1, 0, 0], [39, 39, 0, 39, 39], [3, 39, 2, 39, 0],
            [39, 39, 4, 39, 39]]
    seen = 0
    for step, (ell, n_acc) in enumerate(zip(asked, kept)):
        seq = L.seq.cpu().numpy()
        if step == 2:                                   # a request whose length is no length
            L.seq[3] = -5
        s = L.reserve(_t(ell))
        xs = [L.projected() for _ in L.cache]
        raw = [[np64(t) for t in x] for x in xs]
        plan = L.plan(s)
        outs = []
        for l, x in enumerate(xs):
            L.append(l, s, x)
            outs.append(sdv.sd_cache_attn(x[0], L.cache[l], L.table, plan, lse=True, out=dict(
                out=torch.full((L.rows, n_q, D), 77.0, dtype=torch.bfloat16, device=DEV),
                lse=torch.full((L.rows, n_q), 77.0, device=DEV))))
        read = [sdv.sd_cache_read(s["row_slot"], c, dtype=torch.float32) for c in L.cache]
        torch.cuda.synchronize()
        status = s["status"] | plan["status"]
        assert not (plan["status"] != 0).any()
        seen |= int(np.bitwise_or.reduce(s["status"].cpu().numpy()))
        got, row0, pos = (s[k].cpu().numpy() for k in ("ell", "row0", "row_pos"))
        live = np.zeros(L.rows, bool)
        for r in range(R):
            n, r0 = int(got[r]) + 1, int(row0[r])
            if n == 0:
                continue
            at = slice(r0, r0 + n)
            live[at] = True
            assert np.array_equal(pos[at], seq[r] + np.arange(n))
            for l, (x, (q0, k0, v0)) in enumerate(zip(xs, raw)):
                k, v = np64(read[l]["k"])[at], np64(read[l]["v"])[at]
                freq = np64(L.freq)
                y, size = OH.turn(k0[at], np64(L.wk), pos[at], freq, EPS, False)
                assert (np.abs(k - y) <= _stored(L, y, size)).all()
                assert np.array_equal(v, v0[at] if kind == "bf16" else OH.nearest(v0[at], OH.scale_exponent(v0[at])))
                y, size = OH.turn(q0[at], np64(L.wq), pos[at], freq, EPS, False)
                q = np64(x[0])[at]
                assert (np.abs(q - y) <= 24 * U * size + 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -16)).all()
                h = hist[l][r]
                h += list(zip(k, v))
                T = int(seq[r]) + n
                assert len(h) == T
                check(np64(outs[l]["out"])[at], np64(outs[l]["lse"])[at], q, np.stack([e[0] for e in h]),
                      np.stack([e[1] for e in h]), visible(n, T, True, 0), float(np.float32(D ** -0.5)), (step, r, l))
        for l, x in enumerate(xs):                      # rows of no request stay as they are
            assert (np64(outs[l]["out"])[~live] == 77.0).all() and (np64(outs[l]["lse"])[~live] == 77.0).all()
            assert np.array_equal(np64(x[0])[~live], raw[l][0][~live])
        if step == 2:
            assert int(s["status"][3]) & sdv.SD_ST_BAD_INPUT and got[3] == -1
            L.seq[3] = int(seq[3])
        c = sdv.sd_slot_commit(L.seq, s["ell"], _t(n_acc), L.table, L.free, s["free_count"], bs, q_max=q_max,
                               status=status)
        L.seq, L.F = c["seq_len"], c["free_count"]
        for l in hist:
            for r, n in enumerate(L.seq.tolist()):
                del l[r][n:]
    assert seen & sdv.SD_ST_NO_SLOT                     # the pool ran out on the way


def _same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("kind,bs", [("bf16", 16), ("fp4", 16), ("fp4", 9)])
def test_a_captured_step_replays(kind, bs):
    """A step is captured once; each replay, with eager work in between, begins
    from the same state and gives what the eager step gave.  Then the lengths
    are changed in place: the captured step follows them."""
    R, q_max, n_q, n_kv, D = 4, 6, 8, 2, 128
    L = Layers(5, kind, R, q_max, n_q, n_kv, D, bs, 100, 420, False)
    held = 40
    L.table[:, :held] = L.free[:R * held].reshape(R, held)
    L.free[:L.pool - R * held] = L.free[R * held:].clone()
    L.F -= R * held
    L.seq.copy_(_t([bs * held - 3, bs * held, bs * held - 1, bs * (held - 1) + 1], torch.int64))
    ell, acc = _t([5, 0, -1, 3]), _t([2, 0, 0, 3])
    xs = [L.projected() for _ in L.cache]
    first = {k: v.clone() for k, v in dict(table=L.table, free=L.free, F=L.F, seq=L.seq).items()}
    caches = [[t.clone() for t in c] for c in L.cache]
    raw = [[t.clone() for t in x] for x in xs]
    outs = [dict(out=torch.zeros((L.rows, n_q, D), dtype=torch.bfloat16, device=DEV),
                 lse=torch.zeros((L.rows, n_q), device=DEV)) for _ in xs]
    new = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device=DEV)  # noqa: E731
    sb = dict(ell=new(R), row0=new(R), cu_rows=new(R + 1), ctx_len=new(R), batch=new(1), free_count=new(1),
              row_req=new(L.rows), row_pos=new(L.rows), row_slot=new(L.rows, torch.int64), status=new(R))
    cb = dict(seq_len=new(R, torch.int64), n_new=new(R), free_count=new(1))
    status = new(R)
    sws, cws = (new(max(f(R), 256), torch.uint8) for f in (sdv.sd_slot_reserve_workspace_size,
                                                           sdv.sd_slot_commit_workspace_size))
    aws = new(sdv.sd_attn_workspace_size(R, q_max, n_q, n_kv, D), torch.uint8)

    def step():
        s = L.reserve(ell, out=sb, workspace=sws)
        plan = L.plan(s, out=dict(status=status), workspace=aws)
        for l, x in enumerate(xs):
            L.append(l, s, x)
            sdv.sd_cache_attn(x[0], L.cache[l], L.table, plan, out=outs[l])
        sdv.sd_slot_commit(L.seq, s["ell"], acc, L.table, L.free, s["free_count"], bs, q_max=q_max, out=cb,
                           workspace=cws)

    def reset(seq=None):
        for k, v in first.items():
            getattr(L, k).copy_(v)
        if seq is not None:
            L.seq.copy_(seq)
        for to, frm in zip(L.cache + xs, caches + raw):
            for a, b in zip(to, frm):
                a.copy_(b)
        for o in outs:
            o["out"].fill_(9.0), o["lse"].fill_(9.0)
        aws.fill_(0xA5)

    def state():
        torch.cuda.synchronize()
        all_of = [L.table, L.free, status] + list(sb.values()) + list(cb.values())
        for l, x in enumerate(xs):
            all_of += list(L.cache[l]) + [x[0].contiguous()] + list(outs[l].values())
        return [t.clone() for t in all_of]

    other = _t([bs * (held - 1) + 2, bs * held, bs * held - 2, bs * (held - 1) + 5], torch.int64)
    want = []
    for seq in (None, other):
        reset(seq)
        step()
        want.append(state())
    reset()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for which in (0, 1, 0, 0, 1):
        reset(other if which else None)
        torch.cuda.synchronize()
        graph.replay()
        _same(state(), want[which])
        sdv.sd_qk_rope(xs[0][0], xs[0][1], sb["row_pos"], L.freq)   # eager work in between


def _batch(seed, kind, R, q_max, n_q, n_kv, D, bs, lo, hi):
    g = gen(seed)
    n, ctx, row0, table, blocks = random_batch(g, R, q_max, lo, hi, bs)
    cache, sides = random_cache(g, kind, blocks, n_kv, bs, D)
    rows = int(n.sum()) + 3
    q = torch.randn((rows, n_q, D), generator=g).to(torch.bfloat16).to(DEV)
    return dict(n=n, ctx=ctx, row0=row0, table=table, cache=cache, sides=sides, q=q, rows=rows, q_max=q_max, n_q=n_q,
                D=D, bs=bs, args=(_t(row0), _t(n - 1), _t(ctx)), dev_table=table.to(DEV))


def _attend(b, plan=None, stream=None, out=None, **mask):
    plan = plan or sdv.sd_attn_plan(*b["args"], b["q_max"], b["n_q"], b["cache"], stream=stream, **mask)
    out = out or dict(out=torch.zeros_like(b["q"]), lse=torch.zeros(b["q"].shape[:2], device=DEV))
    r = sdv.sd_cache_attn(b["q"], b["cache"], b["dev_table"], plan, out=out, stream=stream)
    return [r["out"], r["lse"], r["status"]]


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_two_at_once(kind):
    """Two plans over one cache, on two streams at the same time, several times
    over: each gives what it gives alone."""
    b = _batch(21, kind, 6, 7, 8, 2, 128, 16, 1, 3000)
    alone = _attend(b), _attend(b, causal=False, window=100)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    rounds = []
    for _ in range(4):
        rounds.append((_attend(b, stream=streams[0]), _attend(b, stream=streams[1], causal=False, window=100)))
    for s in streams:
        s.synchronize()
    for pair in rounds:
        for got, want in zip(pair, alone):
            _same(got, want)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_one_plan_serves_layers_and_repeats(kind):
    """Calls with one plan follow each other, here with other queries in
    between, and leave the plan as it was."""
    b = _batch(22, kind, 5, 9, 6, 3, 64, 16, 200, 4000)
    plan = sdv.sd_attn_plan(*b["args"], b["q_max"], b["n_q"], b["cache"])
    first = [t.clone() for t in _attend(b, plan)]
    other = dict(b, q=(b["q"] * 3).contiguous())
    loud = [t.clone() for t in _attend(other, plan)]
    assert not torch.equal(first[0], loud[0])
    for _ in range(3):
        _same(_attend(b, plan), first)
        _same(_attend(other, plan), loud)


def test_on_a_side_stream():
    """Outputs and workspaces of calls on a side stream are that stream's, while
    the default stream allocates, fills and frees memory."""
    b = _batch(23, "bf16", 4, 5, 8, 2, 128, 16, 1, 2000)
    slot = torch.randperm(b["cache"][0].shape[0] * 16, generator=gen(1))[:300].to(DEV)
    k, v = (torch.randn((300, 2, 128), generator=gen(i)).to(DEV) for i in (2, 3))
    pos, freq = _t(np.arange(300)), torch.full((64,), 0.01, device=DEV)

    def run(cache, **kw):
        r = sdv.sd_qk_rope(k, v, pos, freq, **kw)
        q = sdv.sd_cache_append(k, v, cache, slot, pos, freq, q=v, **kw)["q"]
        back = sdv.sd_cache_read(slot, cache, **kw)
        plan = sdv.sd_attn_plan(*b["args"], b["q_max"], b["n_q"], cache, **kw)
        o = sdv.sd_cache_attn(b["q"], cache, b["dev_table"], plan, lse=True, **kw)
        return [r["q"], r["k"], q, back["k"], back["v"], o["out"], o["lse"], o["status"]]

    caches = [tuple(t.clone() for t in b["cache"]) for _ in range(2)]
    want = run(caches[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(caches[1], stream=side)
    for i in range(8):
        t = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
        t.fill_(i)
        del t
    side.synchronize()
    torch.cuda.synchronize()
    live = torch.cat([torch.arange(int(r0), int(r0) + int(n)) for r0, n in zip(b["row0"], b["n"])]).to(DEV)
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x[live], y[live]) if i in (5, 6) else torch.equal(x, y), i


# D, query heads, key heads, rows of a request: queries of a tile from 1 to past
# the widest one; block sizes that 16 divides, that it does not, and 1
@pytest.mark.parametrize("kind", ["fp4", "bf16"])
@pytest.mark.parametrize("bs", [16, 48, 9, 1])
@pytest.mark.parametrize("D,n_q,n_kv,q_max", [(64, 1, 1, 1), (64, 8, 1, 4), (64, 12, 2, 8), (64, 8, 2, 15),
                                              (64, 8, 1, 40), (128, 16, 2, 2), (128, 4, 1, 8), (128, 10, 2, 9),
                                              (128, 4, 1, 30), (256, 4, 2, 8), (256, 4, 1, 9), (96, 4, 4, 3),
                                              (192, 3, 1, 11)])
def test_forms(kind, bs, D, n_q, n_kv, q_max):
    b = _batch(31, kind, 4, q_max, n_q, n_kv, D, bs, 1, 700)
    for mask in (dict(), dict(window=33)):
        got = [np64(t) for t in _attend(b, **mask)]
        assert not got[2].any()
        for r in range(4):
            n, T, r0 = int(b["n"][r]), int(b["ctx"][r]), int(b["row0"][r])
            if n == 0:
                continue
            k, v = (tokens_of(x, b["table"], r, T, bs) for x in b["sides"])
            check(got[0][r0:r0 + n], got[1][r0:r0 + n], np64(b["q"])[r0:r0 + n], k, v,
                  visible(n, T, True, mask.get("window", 0)), float(np.float32(D ** -0.5)), (r, mask))


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
def test_many_requests(kind):
    """More requests than the plan has threads, and than there are runs."""
    b = _batch(71, kind, 2600, 2, 2, 1, 64, 16, 1, 40)
    got = [np64(t) for t in _attend(b)]
    assert not got[2].any()
    for r in range(2600):
        n, T, r0 = int(b["n"][r]), int(b["ctx"][r]), int(b["row0"][r])
        if n:
            k, v = (tokens_of(x, b["table"], r, T, 16) for x in b["sides"])
            check(got[0][r0:r0 + n], got[1][r0:r0 + n], np64(b["q"][r0:r0 + n]), k, v, visible(n, T, True, 0), 0.125, r)


@pytest.mark.parametrize("kind", ["fp4", "bf16"])
@pytest.mark.parametrize("n_q,n_kv,q_max", [(130, 1, 2), (1024, 2, 1), (200, 200, 1)])
def test_many_heads(kind, n_q, n_kv, q_max):
    """Groups of more heads than a tile has queries, and a head to each."""
    b = _batch(61, kind, 3, q_max, n_q, n_kv, 64, 16, 1, 150)
    got = [np64(t) for t in _attend(b)]
    assert not got[2].any()
    for r in range(3):
        n, T, r0 = int(b["n"][r]), int(b["ctx"][r]), int(b["row0"][r])
        if n:
            k, v = (tokens_of(x, b["table"], r, T, 16) for x in b["sides"])
            check(got[0][r0:r0 + n], got[1][r0:r0 + n], np64(b["q"])[r0:r0 + n], k, v, visible(n, T, True, 0), 0.125, r)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("q_max", [3, 40])
def test_many_units_to_a_run(kind, q_max):
    """Enough work for long runs of the 512 workgroups, in tiles of one unit and
    of a hundred: requests share the pool's blocks, each in an order of its own."""
    g = gen(51)
    R, n_q, n_kv, D, bs, blocks = 160, 16, 8, 64, 16, 420
    n = torch.randint(1, q_max + 1, (R,), generator=g)
    ctx = torch.maximum(torch.exp(torch.rand(R, generator=g) * 8.8).long(), n)
    n[0], ctx[0], n[5], ctx[7] = q_max, bs * blocks, 0, 6000
    row0 = torch.cumsum(n, 0) - n
    table = torch.stack([torch.randperm(blocks, generator=g) for _ in range(R)]).to(torch.int32)
    cache, sides = random_cache(g, kind, blocks, n_kv, bs, D)
    q = torch.randn((int(n.sum()), n_q, D), generator=g).to(torch.bfloat16).to(DEV)
    assert int(((ctx + 127) // 128)[n > 0].sum()) * n_kv > 16 * 512
    b = dict(q=q, cache=cache, dev_table=table.to(DEV), args=(_t(row0), _t(n - 1), _t(ctx)), q_max=q_max, n_q=n_q)
    got = [np64(t) for t in _attend(b)]
    assert not got[2].any()
    for r in range(R):
        m, T, r0 = int(n[r]), int(ctx[r]), int(row0[r])
        if m:
            k, v = (tokens_of(x, table, r, T, bs) for x in sides)
            check(got[0][r0:r0 + m], got[1][r0:r0 + m], np64(q)[r0:r0 + m], k, v, visible(m, T, True, 0), 0.125, r)


def test_single_rows_no_rows_and_refusals():
    """A single row's stride says nothing, and an empty step is no error."""
    b = _batch(41, "bf16", 1, 1, 4, 2, 64, 16, 50, 50)
    wide = torch.zeros((1, 5, 64), dtype=torch.bfloat16, device=DEV)
    wide[:, :4] = b["q"][1:2]
    b["row0"][0], b["args"] = 0, (_t([0]),) + b["args"][1:]
    plan = sdv.sd_attn_plan(*b["args"], 1, 4, b["cache"])
    o = sdv.sd_cache_attn(wide[:, :4], b["cache"], b["dev_table"], plan)
    k, v = (tokens_of(x, b["table"], 0, 50, 16) for x in b["sides"])
    check(np64(o["out"]), None, np64(wide[:, :4]), k, v, visible(1, 50, True, 0), 0.125)
    none = sdv.sd_cache_attn(wide[:0, :4], b["cache"], b["dev_table"], plan)
    assert none["out"].shape == (0, 4, 64)
    with pytest.raises(ValueError, match="plan is for"):
        sdv.sd_cache_attn(wide, b["cache"], b["dev_table"], plan)
    with pytest.raises(ValueError, match="lie together"):
        sdv.sd_qk_rope(torch.zeros((3, 4, 64), device=DEV).transpose(0, 1), None, None)
    with pytest.raises(sdv.SdvError):
        sdv.sd_cache_attn(wide[:, :4], b["cache"], b["dev_table"], plan, scale=0.0)
    with pytest.raises(sdv.SdvError):
        sdv.sd_cache_attn(wide[:, :4], b["cache"], b["dev_table"], plan, out=dict(out=wide[:, :4]))
    with pytest.raises(TypeError):
        sdv.sd_cache_attn(wide[:, :4].float(), b["cache"], b["dev_table"], plan)
    with pytest.raises(ValueError, match="n_blocks"):
        sdv.sd_cache_read(_t([0], torch.int64), (b["cache"][0], b["cache"][1][:1]))
