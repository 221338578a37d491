"""The operators around a verification step run together, as a serving loop
runs them: schedule, slots, the target's rows, their shaping, verification,
the committed slots and token counts; eagerly on the default and a side
stream, and captured in a graph."""

import numpy as np
import pytest
import torch

import draft_verification_amd as sdv
from oracle import shape as OS
from oracle import slots as OL
from oracle import verify as OV
from tests.parity_util import to_np
from workloads import sps_table

pytestmark = pytest.mark.gpu

DEV = "cuda"
R, G, V, BS, MB = 6, 4, 512, 8, 12
Q = G + 1
WORDS = V // 32


class Loop:
    """R requests, all state on the device; `logits` stands for the target:
    rows of a step are a fixed table's rows by (token, position)."""

    def __init__(self, seed=0, pool=R * MB - 20):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *k: torch.rand(k, generator=g, device=DEV)  # noqa: E731
        i32 = lambda *k: torch.zeros(k, dtype=torch.int32, device=DEV)  # noqa: E731
        ints = lambda hi, *k: torch.randint(0, hi, k, generator=g, device=DEV, dtype=torch.int32)  # noqa: E731
        self.model = torch.randn((V, V), generator=g, device=DEV) * 2.0
        self.seq = torch.zeros(R, dtype=torch.int64, device=DEV)
        self.table, self.F = i32(R, MB) - 1, i32(1) + pool
        self.free = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
        self.x0, self.seen, self.counts = ints(V, R), i32(R, WORDS), i32(R, V)
        self.rep, self.freq, self.pres = 1.0 + rand(R), 0.5 * rand(R), 0.5 * rand(R)
        self.mask = torch.where(rand(R * Q, V) < 0.7, 1, 0)
        self.mask_w = torch.as_tensor(OS.pack_bits(to_np(self.mask))).to(DEV)
        self.m0 = torch.tensor([0, -1, 2 * Q, -1, 4 * Q, 5 * Q], dtype=torch.int32, device=DEV)
        self.conf, self.drafts = 0.3 + 0.7 * rand(R, G), ints(V, R, G)
        self.drf = torch.randn((R * G, V), generator=g, device=DEV) * 2.0
        self.drf_row0 = torch.arange(R, dtype=torch.int32, device=DEV) * G
        self.sps = sps_table(R * Q, 8, 0.05, 8).to(DEV)
        self.release = i32(R)
        self.rows = torch.zeros((R * Q, V), device=DEV)
        self.buf = dict(sched=dict(ell=i32(R), batch=i32(1), n_sel=i32(1),
                                   theta=torch.zeros(1, dtype=torch.float64, device=DEV), surv=rand(R, G)),
                        slots=dict(ell=i32(R), row0=i32(R), cu_rows=i32(R + 1), ctx_len=i32(R), batch=i32(1),
                                   free_count=i32(1), row_req=i32(R * Q), row_pos=i32(R * Q),
                                   row_slot=torch.zeros(R * Q, dtype=torch.int64, device=DEV), row_token=i32(R * Q),
                                   status=i32(R)),
                        shape=dict(logits=self.rows, status=i32(R)),
                        verify=dict(n_acc=i32(R), tokens=i32(R, Q), status=i32(R)),
                        commit=dict(seq_len=self.seq, x0=self.x0, free_count=self.F, n_new=i32(R)),
                        counts=dict(status=i32(R)))
        u8 = lambda n: torch.empty(max(int(n), 256), dtype=torch.uint8, device=DEV)  # noqa: E731
        self.ws = dict(sched=u8(sdv.sd_schedule_workspace_size(R, G)),
                       slots=u8(sdv.sd_slot_reserve_workspace_size(R)),
                       verify=u8(sdv.sd_verify_workspace_size(R, G, V)),
                       commit=u8(sdv.sd_slot_commit_workspace_size(R)))

    def step(self, stream=None):
        b, w, kw = self.buf, self.ws, dict(stream=stream)
        sdv.sd_schedule(self.conf, self.sps, sdv.SD_SCHED_GLOBAL_ARGMAX, out=b["sched"], workspace=w["sched"], **kw)
        s = sdv.sd_slot_reserve(self.seq, b["sched"]["ell"], self.table, self.free, self.F, BS, Q, x0=self.x0,
                                tokens=self.drafts, out=b["slots"], workspace=w["slots"], **kw)
        torch.index_select(self.model, 0, s["row_token"].clamp(min=0), out=self.rows)   # the target's pass
        sdv.sd_logit_shape(self.rows, s["row0"], s["ell"], V, draft_tokens=self.drafts, repetition=self.rep,
                           frequency=self.freq, presence=self.pres, seen=self.seen, counts=self.counts,
                           mask=self.mask_w, mask_row0=self.m0, out=b["shape"], **kw)
        v = sdv.sd_verify(self.rows, s["row0"], self.drf, self.drf_row0, self.drafts, s["ell"], V, 1.0, 77,
                          pos0=self.seq, workspace=w["verify"], out=b["verify"], **kw)
        c = sdv.sd_slot_commit(self.seq, s["ell"], v["n_acc"], self.table, self.free, s["free_count"], BS,
                               out_tokens=v["tokens"], x0=self.x0, status=v["status"], release=self.release,
                               out=b["commit"], workspace=w["commit"], **kw)
        sdv.sd_token_counts(v["tokens"], self.seen, self.counts, V, length=c["n_new"], out=b["counts"], **kw)

    def state(self):
        return {k: getattr(self, k).clone() for k in ("seq", "table", "F", "free", "x0", "seen", "counts", "rows")} | \
            {f"{n}.{k}": t.clone() for n, d in self.buf.items() for k, t in d.items()}

    def restore(self, s):
        for k in ("seq", "table", "F", "free", "x0", "seen", "counts", "rows"):
            getattr(self, k).copy_(s[k])


@pytest.mark.parametrize("pool", [R * MB - 20, 14])
def test_loop_against_the_oracle(pool):
    """With few blocks requests go short, and some sit steps out."""
    L = Loop(pool=pool)
    n = lambda t: to_np(t).copy()  # noqa: E731
    seen, counts = np.zeros((R, V), bool), np.zeros((R, V), int)
    model, drafts, mask = n(L.model).astype(np.float64), n(L.drafts), n(L.mask).astype(bool)
    m0, rep, freq, pres = n(L.m0), n(L.rep), n(L.freq), n(L.pres)
    table, free, F = n(L.table), n(L.free), int(L.F[0])
    seq, x0 = n(L.seq), n(L.x0)
    released, short, none = 0, 0, 0
    for step in range(25):
        L.release.copy_(torch.tensor([(step + r) % 9 == 8 for r in range(R)]).to(torch.int32))
        L.drafts.copy_(torch.as_tensor((drafts * (step + 1) + 7 * step) % V, dtype=torch.int32))
        L.step()
        torch.cuda.synchronize()
        d = n(L.drafts)
        ell = n(L.buf["sched"]["ell"])
        want = OL.reserve(seq, ell, table, free, F, BS, Q, R * Q, False, x0, d)
        for k, v in want.items():
            assert np.array_equal(n(L.buf["slots"][k]), v), (step, k)
        short += int((want["status"] == OL.NO_SLOT).sum())
        none += int((want["ell"] < 0).sum())
        rows = n(L.rows).astype(np.float64)
        shaped = rows.copy()
        for r in range(R):
            for i in range(want["ell"][r] + 1):
                e = want["row0"][r] + i
                row, mag = OS.shape_row(model[want["row_token"][e]], d[r][:i], seen[r], counts[r], float(rep[r]),
                                        float(freq[r]), float(pres[r]), (), mask[m0[r] + i] if m0[r] >= 0 else None)
                fin = np.isfinite(row)
                assert np.array_equal(fin, np.isfinite(rows[e]))
                # half a step of each intermediate and of the result, itself the last of them
                assert (np.abs(rows[e][fin] - row[fin]) <= 2.0 ** -23 * mag[fin]).all(), (step, r, i)
                shaped[e] = rows[e]   # verified as they are
        ora = OV.verify(shaped, want["row0"], n(L.drf).astype(np.float64), n(L.drf_row0), d,
                        np.maximum(want["ell"], 0), V, 1.0, 77, seq)
        live = want["ell"] >= 0
        got = {k: n(t) for k, t in L.buf["verify"].items()}
        same = np.array_equal(got["tokens"][live], ora["tokens"][live])
        assert same or min(x[3] for x in ora["decisions"]) < 1e-6, step   # else a draw on a boundary
        c = OL.commit(seq, want["ell"], got["n_acc"], table, free, int(want["free_count"][0]), BS, Q, got["tokens"], x0,
                      got["status"].copy(), n(L.release))
        seq, x0, F = c["seq_len"], c["x0"], int(c["free_count"][0])
        released += int(n(L.release).sum())
        for k, v in c.items():
            assert np.array_equal(n(L.buf["commit"][k]), v), (step, k)
        assert np.array_equal(n(L.free)[:F], free[:F]) and np.array_equal(n(L.table), table)
        for r in range(R):
            OS.enter_tokens(seen[r], counts[r], got["tokens"][r][:c["n_new"][r]])
        assert np.array_equal(n(L.seen), OS.pack_bits(seen)) and np.array_equal(n(L.counts), counts)
    assert released and counts.sum() > 25
    assert (short > 0) == (none > 0) == (pool == 14)
    blocks = sum((table[r, :-(-int(seq[r]) // BS)].tolist() for r in range(R)), []) + free[:F].tolist()
    assert sorted(blocks) == list(range(len(free)))


def _same(a, b):
    for k, v in a.items():
        assert torch.equal(v.nan_to_num(), b[k].nan_to_num()), k


def test_loop_on_a_side_stream():
    a, b = Loop(3), Loop(3)
    for _ in range(4):
        a.step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        with torch.cuda.stream(side):   # the stand-in for the target runs there too
            b.step(stream=side)
        junk = torch.empty(1 << 22, dtype=torch.uint8, device=DEV).fill_(7)
        del junk
    side.synchronize()
    _same(a.state(), b.state())


def test_loop_replays_from_a_graph():
    """A captured step, replayed with eager work in between, does what eager
    steps do; a second graph of another loop runs between the replays."""
    a, b, other = Loop(5), Loop(5), Loop(6)
    b.step()
    other.step()
    a.step()
    torch.cuda.synchronize()
    s0, s1 = b.state(), other.state()

    def capture(L):
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                L.step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        return graph

    gb, go = capture(b), capture(other)
    b.restore(s0)
    other.restore(s1)
    for i in range(4):
        a.step()
        gb.replay()
        go.replay()
        for w in b.ws.values():
            w.fill_(i)     # nothing is kept in a workspace from one step to the next
        torch.cuda.synchronize()
        _same(a.state(), b.state())


def test_parts_replay_from_a_graph():
    """Lists entered through LDS, slots and their commit with outputs of their
    own, captured once and replayed with eager work in between."""
    g = torch.Generator(device=DEV).manual_seed(9)
    ints = lambda hi, *k: torch.randint(0, hi, k, generator=g, device=DEV, dtype=torch.int32)  # noqa: E731
    V1, n, r = 40000, 9000, 40
    toks, seen, counts = ints(V1, 3, n), ints(9, 3, 1250), ints(9, 3, V1)
    reset = torch.ones(3, dtype=torch.int32, device=DEV)
    seq, ell = ints(50, r).long(), ints(9, r)
    table, free = ints(500, r, 16), torch.randperm(500, generator=g, device=DEV).to(torch.int32)
    F = torch.full((1,), 300, dtype=torch.int32, device=DEV)
    e32 = lambda *k: torch.empty(k, dtype=torch.int32, device=DEV)  # noqa: E731
    so = dict(ell=e32(r), row0=e32(r), cu_rows=e32(r + 1), ctx_len=e32(r), batch=e32(1), free_count=e32(1),
              row_req=e32(300), row_pos=e32(300), row_slot=e32(300).long(), row_token=e32(300), status=e32(r))
    co = dict(seq_len=e32(r).long(), x0=e32(r), n_new=e32(r), free_count=e32(1))
    st = e32(3)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    x0, drafts, acc, rel = ints(99, r), ints(99, r, 9), ints(9, r), ints(2, r)

    def call():
        sdv.sd_token_counts(toks, seen, counts, V1, reset=reset, out=dict(status=st))
        sdv.sd_slot_reserve(seq, ell, table, free, F, 8, 9, x0=x0, tokens=drafts, out=so, workspace=ws)
        sdv.sd_slot_commit(seq, so["ell"], acc, table, free, so["free_count"], 8, out_tokens=drafts, x0=x0,
                           release=rel, out=co, workspace=ws)

    outs = {**so, **{"c_" + k: v for k, v in co.items()}, "st": st, "seen": seen, "counts": counts, "free": free,
            "table": table}
    before = {k: outs[k].clone() for k in ("free", "table")}   # a step changes them: each begins from here
    call()
    torch.cuda.synchronize()
    ref = {k: v.clone() for k, v in outs.items()}
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for i in range(3):
        for k, v in outs.items():
            if k in before:
                v.copy_(before[k])
            else:
                v.fill_(-3)
        ws.fill_(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in ref.items():
            assert torch.equal(outs[k], v), (i, k)


def test_two_loops_at_once():
    """Two loops on two streams, nothing shared, give what each gives alone."""
    alone, both = [Loop(11), Loop(12)], [Loop(11), Loop(12)]
    for L in alone:
        for _ in range(5):
            L.step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for L, s in zip(both, streams):
            with torch.cuda.stream(s):
                L.step()
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        _same(a.state(), b.state())


def test_parts_allocate_what_they_are_not_given():
    """The binding's own outputs and workspaces, on a side stream."""
    L, M = Loop(8), Loop(8)
    M.step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sch = sdv.sd_schedule(L.conf, L.sps, sdv.SD_SCHED_GLOBAL_ARGMAX, stream=side)
    s = sdv.sd_slot_reserve(L.seq, sch["ell"], L.table, L.free, L.F, BS, Q, x0=L.x0, tokens=L.drafts, stream=side)
    with torch.cuda.stream(side):
        rows = torch.index_select(L.model, 0, s["row_token"].clamp(min=0))
    z = sdv.sd_logit_shape(rows, s["row0"], s["ell"], V, draft_tokens=L.drafts, repetition=L.rep, frequency=L.freq,
                           presence=L.pres, seen=L.seen, counts=L.counts, mask=L.mask_w, mask_row0=L.m0, stream=side)
    v = sdv.sd_verify(z["logits"], s["row0"], L.drf, L.drf_row0, L.drafts, s["ell"], V, 1.0, 77, pos0=L.seq, stream=side)
    c = sdv.sd_slot_commit(L.seq, s["ell"], v["n_acc"], L.table, L.free, s["free_count"], BS, out_tokens=v["tokens"],
                           x0=L.x0, status=v["status"], release=L.release, stream=side)
    sdv.sd_token_counts(v["tokens"], L.seen, L.counts, V, length=c["n_new"], stream=side)
    side.synchronize()
    for k in c:
        assert torch.equal(c[k], M.buf["commit"][k]), k
    assert torch.equal(L.seen, M.seen) and torch.equal(L.counts, M.counts) and torch.equal(L.free, M.free)
