"""ctypes binding of libsdv (include/sdv.h).

Argument marshalling only: torch tensors supply device pointers and the
current HIP stream; every step of the path runs in the library's kernels.
The functions carry the C names.  A missing library is an error, never a
fallback.
"""

import ctypes
import functools
import inspect
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsdv.so")
_lib = None

SD_OK = 0
SD_EINVAL = -1
SD_ERANGE = -2
SD_EUNSUPPORTED = -3
SD_ELAUNCH = -4

SD_DTYPE_F32 = 0
SD_DTYPE_BF16 = 1

SD_VERIFY_STOP_AT_REJECTION = 1

SD_SCHED_EARLY_STOP = 0
SD_SCHED_GLOBAL_ARGMAX = 1
SD_SCHED_CAPPED_TOPK = 2
SD_SCHED_THRESHOLD = 3

SD_ST_BAD_TOKEN = 1
SD_ST_NONFINITE = 2
SD_ST_ZERO_Z = 4
SD_ST_ZERO_RESIDUAL = 8
SD_ST_ZERO_Q = 16
SD_ST_BAD_INPUT = 32
SD_ST_NO_SLOT = 64

SD_CACHE_BF16 = 0
SD_CACHE_FP4 = 1

EXPORTS = (
    "sd_abi_version", "sd_status_string", "sd_schedule_workspace_size", "sd_schedule",
    "sd_verify_workspace_size",
    "sd_verify", "sd_markov_draft_workspace_size", "sd_markov_draft",
    "sd_rnn_draft_workspace_size", "sd_rnn_draft",
    "sd_lightspec_update", "sd_lightspec_plan_workspace_size", "sd_lightspec_plan",
    "sd_uniforms", "sd_verify_noalloc",
    "sd_logit_shape", "sd_token_counts", "sd_slot_reserve_workspace_size", "sd_slot_reserve",
    "sd_slot_commit_workspace_size", "sd_slot_commit",
    "sd_qk_rope", "sd_cache_append", "sd_cache_read",
    "sd_attn_workspace_size", "sd_attn_plan", "sd_cache_attn",
)


class SdvError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {code} ({status_string(code)})")
        self.code = code


_P = ctypes.c_void_p
_I = ctypes.c_int
_U64 = ctypes.c_uint64
_SZ = ctypes.c_size_t


def lib():
    """Load libsdv.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build()")
    L = ctypes.CDLL(_LIB_PATH)
    L.sd_abi_version.restype = _I
    L.sd_abi_version.argtypes = []
    L.sd_status_string.restype = ctypes.c_char_p
    L.sd_status_string.argtypes = [_I]
    L.sd_schedule.restype = _I
    L.sd_schedule_workspace_size.restype = _SZ
    L.sd_schedule_workspace_size.argtypes = [_I, _I]
    L.sd_schedule.argtypes = [_P, _I, _I, _P, _P, _P, _P, _I, _I, _P, ctypes.c_float, _P, _P, _P,
                              _P, _P, _P, _SZ]
    L.sd_verify_workspace_size.restype = _SZ
    L.sd_verify_workspace_size.argtypes = [_I, _I, _I]
    L.sd_verify.restype = _I
    L.sd_verify.argtypes = [_P, _I, _I, _I, _I, _I, ctypes.c_float, _U64, _P, _P, _P, _P, _P, _P,
                            _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _SZ, _P, _P]
    L.sd_markov_draft_workspace_size.restype = _SZ
    L.sd_markov_draft_workspace_size.argtypes = [_I, _I, _I, _I]
    L.sd_markov_draft.restype = _I
    L.sd_markov_draft.argtypes = [_P, _I, _I, _I, _I, ctypes.c_float, _U64, _P, _P, _P, _P, _P,
                                  _P, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _SZ]
    L.sd_rnn_draft_workspace_size.restype = _SZ
    L.sd_rnn_draft_workspace_size.argtypes = [_I, _I, _I, _I]
    L.sd_rnn_draft.restype = _I
    L.sd_rnn_draft.argtypes = [_P, _I, _I, _I, _I, ctypes.c_float, _U64, _P, _P, _P, _P, _P, _P, _P,
                               _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _SZ]
    L.sd_lightspec_update.restype = _I
    L.sd_lightspec_update.argtypes = [_P, _I, _I, _P, _P, _P, ctypes.c_double, _P, _P]
    L.sd_lightspec_plan_workspace_size.restype = _SZ
    L.sd_lightspec_plan_workspace_size.argtypes = [_I, _I]
    L.sd_lightspec_plan.restype = _I
    L.sd_lightspec_plan.argtypes = [_P, _I, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _P, _SZ]
    L.sd_verify_noalloc.restype = _I
    L.sd_verify_noalloc.argtypes = [_P, _I, _I, _I, _I, _I, ctypes.c_float, _U64, _P, _P, _P, _P, _P,
                                    _P, _P, _P, _P, _P, _P, _P, _P, _P, _I]
    L.sd_uniforms.restype = _I
    L.sd_uniforms.argtypes = [_P, _U64, ctypes.c_longlong, _P, _P, _I, _P]
    L.sd_logit_shape.restype = _I
    L.sd_logit_shape.argtypes = [_P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I,
                                 _I, _P, _P, _P, _P, ctypes.c_longlong, _P, _I, _I, _P, _P]
    L.sd_token_counts.restype = _I
    L.sd_token_counts.argtypes = [_P, _I, _I, _P, ctypes.c_longlong, _I, _P, _P, _P, _P, _P, _P, _I, _P, _I,
                                  _I, _P]
    L.sd_slot_reserve_workspace_size.restype = _SZ
    L.sd_slot_reserve_workspace_size.argtypes = [_I]
    L.sd_slot_reserve.restype = _I
    L.sd_slot_reserve.argtypes = [_P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P,
                                  _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ]
    L.sd_slot_commit_workspace_size.restype = _SZ
    L.sd_slot_commit_workspace_size.argtypes = [_I]
    L.sd_slot_commit.restype = _I
    L.sd_slot_commit.argtypes = [_P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                 _P, _P, _P, _SZ]
    _F, _L = ctypes.c_float, ctypes.c_longlong
    L.sd_qk_rope.restype = _I
    L.sd_qk_rope.argtypes = [_P, _I, _I, _I, _P, _I, _L, _P, _I, _L, _P, _P, _P, _F, _P, _I, _I, _P, _L, _P, _L]
    L.sd_cache_append.restype = _I
    L.sd_cache_append.argtypes = [_P, _I, _I, _I, _P, _I, _L, _P, _L, _P, _L, _I, _P, _P, _P, _P, _F, _P, _I, _I, _P,
                                  _L, _I, _I, _I, _P, _P, _P, _P]
    L.sd_cache_read.restype = _I
    L.sd_cache_read.argtypes = [_P, _I, _I, _P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _L, _P, _L]
    L.sd_attn_workspace_size.restype = _SZ
    L.sd_attn_workspace_size.argtypes = [_I, _I, _I, _I, _I]
    L.sd_attn_plan.restype = _I
    L.sd_attn_plan.argtypes = [_P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _I, _I, _P, _P, _SZ]
    L.sd_cache_attn.restype = _I
    L.sd_cache_attn.argtypes = [_P, _I, _I, _I, _I, _I, _I, _P, _L, _I, _I, _I, _P, _P, _P, _P, _P, _I, _F, _P, _L, _P,
                                _P, _P, _SZ]
    _lib = L
    return L


def sd_abi_version():
    return lib().sd_abi_version()


def status_string(code):
    return lib().sd_status_string(int(code)).decode()


sd_status_string = status_string


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _on_stream(fn):
    """Run fn with its `stream` argument as torch's current stream, so the
    outputs and the temporary workspace it allocates belong to the stream the
    kernels are enqueued on: when the workspace is freed on return, the
    caching allocator hands that block only to later work of the same stream,
    never to another stream while these kernels may still use it.  Outputs
    and workspaces the caller passes in are the caller's to keep alive on
    that stream."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def wrapper(*args, **kw):
        stream = kw.get("stream") if "stream" in kw else (args[at] if len(args) > at else None)
        if stream is None:  # torch's current stream already
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return wrapper


def _out(o, key, make):
    """The caller's output `key` from `o` when present, else a new tensor
    from make() (made only then)."""
    return o[key] if key in o else make()


def _check(fn, code):
    if code != SD_OK:
        raise SdvError(fn, code)


def _workspace(nbytes, device):
    # 256-byte aligned by torch's caching allocator
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def sd_schedule_workspace_size(R, gmax):
    return lib().sd_schedule_workspace_size(R, gmax)


@_on_stream
def sd_schedule(conf, sps, mode, gamma_r=None, cap_k=None, out=None, surv=True, workspace=None,
                stream=None, sts_temp=None, threshold=0.0):
    """Run the scheduler.  conf [R][gmax] fp32, sps fp32, gamma_r [R] int32 or
    None, cap_k a 1-element int32 device tensor (CAPPED_TOPK), sts_temp
    [gmax] fp32 per-position temperatures or None, threshold the survival
    threshold (THRESHOLD mode).  Returns a dict of device tensors: ell, batch,
    n_sel, theta, surv."""
    R, gmax = conf.shape
    dev = conf.device
    o = out or {}
    ell = _out(o, "ell", lambda: torch.empty(R, dtype=torch.int32, device=dev))
    batch = _out(o, "batch", lambda: torch.empty(1, dtype=torch.int32, device=dev))
    n_sel = _out(o, "n_sel", lambda: torch.empty(1, dtype=torch.int32, device=dev))
    theta = _out(o, "theta", lambda: torch.empty(1, dtype=torch.float64, device=dev))
    sv = _out(o, "surv", lambda: torch.empty((R, gmax), dtype=torch.float32, device=dev)) if surv else None
    ws = workspace if workspace is not None else _workspace(sd_schedule_workspace_size(R, gmax), dev)
    code = lib().sd_schedule(
        _stream(stream), R, gmax, _ptr(gamma_r, torch.int32, "gamma_r"),
        _ptr(conf, torch.float32, "conf"), _ptr(sts_temp, torch.float32, "sts_temp"),
        _ptr(sps, torch.float32, "sps"), sps.numel(), int(mode), _ptr(cap_k, torch.int32, "cap_k"),
        float(threshold), _ptr(ell, torch.int32), _ptr(batch, torch.int32),
        _ptr(n_sel, torch.int32), _ptr(theta, torch.float64), _ptr(sv, torch.float32),
        ws.data_ptr(), ws.numel())
    _check("sd_schedule", code)
    return dict(ell=ell, batch=batch, n_sel=n_sel, theta=theta, surv=sv)


def sd_verify_workspace_size(R, gmax, V):
    return lib().sd_verify_workspace_size(R, gmax, V)


@_on_stream
def sd_verify(tgt, tgt_row0, drf, drf_row0, draft_tokens, ell, V, temperature=1.0, seed=0,
              pos0=None, probe=False, stats=False, alpha=False, workspace=None, out=None,
              stream=None, prof_events=None, drf_stats=None, stop_at_rejection=False):
    """Run verification.  tgt / drf: 2-D logit tensors (bf16 or fp32, ld =
    shape[1]); the rest int32 device tensors.  Returns a dict of device
    tensors: n_acc, tokens, status (and probe, row_stats, alpha if asked).
    prof_events: optional pair of raw hipEvent_t handles (ints) recorded
    around the row-statistics pass.  drf_stats: optional [R][gamma_max][2]
    fp32 (m, Z) of the draft rows (a drafting head's q_stats); the draft rows
    are then read only where needed.  stop_at_rejection: read each request's
    rows in rounds of positions and stop at its first rejection
    (SD_VERIFY_STOP_AT_REJECTION; alpha must be off)."""
    R, gmax = draft_tokens.shape
    if drf_stats is not None and drf_stats.numel() != R * gmax * 2:
        raise ValueError("drf_stats must hold R * gamma_max (m, Z) pairs")
    dev = tgt.device
    if tgt.dtype == torch.bfloat16:
        dt = SD_DTYPE_BF16
    elif tgt.dtype == torch.float32:
        dt = SD_DTYPE_F32
    else:
        raise TypeError("logits must be bf16 or fp32")
    if drf.dtype != tgt.dtype or drf.shape[1] != tgt.shape[1]:
        raise ValueError("target and draft rows must share dtype and leading dimension")
    ld = tgt.shape[1]
    o = out or {}
    n_acc = _out(o, "n_acc", lambda: torch.empty(R, dtype=torch.int32, device=dev))
    toks = _out(o, "tokens", lambda: torch.empty((R, gmax + 1), dtype=torch.int32, device=dev))
    status = _out(o, "status", lambda: torch.empty(R, dtype=torch.int32, device=dev))
    pp = _out(o, "probe", lambda: torch.zeros((R, gmax, 2), dtype=torch.float32, device=dev)) if probe else None
    rs = _out(o, "row_stats", lambda: torch.zeros((R, 2 * gmax + 1, 2), dtype=torch.float32, device=dev)) if stats else None
    al = _out(o, "alpha", lambda: torch.zeros((R, gmax), dtype=torch.float32, device=dev)) if alpha else None
    ws = workspace if workspace is not None else _workspace(sd_verify_workspace_size(R, gmax, V), dev)
    code = lib().sd_verify(
        _stream(stream), R, gmax, int(V), ld, dt, float(temperature), int(seed) & (2**64 - 1),
        _ptr(pos0, torch.int64, "pos0"), _ptr(tgt, None, "tgt"), _ptr(tgt_row0, torch.int32, "tgt_row0"),
        _ptr(drf, None, "drf"), _ptr(drf_row0, torch.int32, "drf_row0"),
        _ptr(drf_stats, torch.float32, "drf_stats"),
        _ptr(draft_tokens, torch.int32, "draft_tokens"), _ptr(ell, torch.int32, "ell"),
        _ptr(n_acc, torch.int32), _ptr(toks, torch.int32), _ptr(status, torch.int32),
        _ptr(pp, torch.float32), _ptr(rs, torch.float32), _ptr(al, torch.float32),
        SD_VERIFY_STOP_AT_REJECTION if stop_at_rejection else 0, ws.data_ptr(), ws.numel(),
        *(prof_events if prof_events else (None, None)))
    _check("sd_verify", code)
    return dict(n_acc=n_acc, tokens=toks, status=status, probe=pp, row_stats=rs, alpha=al)


@_on_stream
def sd_verify_noalloc(tgt, tgt_row0, drf, drf_row0, draft_tokens, ell, V, temperature=1.0, seed=0,
                      pos0=None, drf_stats=None, stop_at_rejection=False, out=None, stream=None):
    """sd_verify through the entry point that allocates nothing: the library
    holds the workspace.  The caller passes every output in `out` (n_acc,
    tokens, status, and optionally probe, row_stats, alpha), as a caller
    that cannot allocate would; returns `out`."""
    R, gmax = draft_tokens.shape
    if tgt.dtype == torch.bfloat16:
        dt = SD_DTYPE_BF16
    elif tgt.dtype == torch.float32:
        dt = SD_DTYPE_F32
    else:
        raise TypeError("logits must be bf16 or fp32")
    if drf.dtype != tgt.dtype or drf.shape[1] != tgt.shape[1]:
        raise ValueError("target and draft rows must share dtype and leading dimension")
    o = out
    code = lib().sd_verify_noalloc(
        _stream(stream), R, gmax, int(V), tgt.shape[1], dt, float(temperature), int(seed) & (2**64 - 1),
        _ptr(pos0, torch.int64, "pos0"), _ptr(tgt, None, "tgt"), _ptr(tgt_row0, torch.int32, "tgt_row0"),
        _ptr(drf, None, "drf"), _ptr(drf_row0, torch.int32, "drf_row0"),
        _ptr(drf_stats, torch.float32, "drf_stats"),
        _ptr(draft_tokens, torch.int32, "draft_tokens"), _ptr(ell, torch.int32, "ell"),
        _ptr(o["n_acc"], torch.int32, "n_acc"), _ptr(o["tokens"], torch.int32, "tokens"),
        _ptr(o["status"], torch.int32, "status"), _ptr(o.get("probe"), torch.float32, "probe"),
        _ptr(o.get("row_stats"), torch.float32, "row_stats"), _ptr(o.get("alpha"), torch.float32, "alpha"),
        SD_VERIFY_STOP_AT_REJECTION if stop_at_rejection else 0)
    _check("sd_verify_noalloc", code)
    return o


def sd_markov_draft_workspace_size(R, gamma, V, rank):
    return lib().sd_markov_draft_workspace_size(R, gamma, V, rank)


@_on_stream
def sd_markov_draft(U, A, Ct, x0, h, E, w, temperature=1.0, seed=0, pos0=None, workspace=None,
                    out=None, stream=None, stats=False):
    """Run the Markov drafting head.  Returns a dict of device tensors:
    tokens [R][gamma], q_logits [R][gamma][V] bf16, conf [R][gamma], status [R],
    and q_stats [R][gamma][2] ((m, Z) of each drafted row) if stats."""
    R, gamma, V = U.shape
    rank = A.shape[2]
    H = h.shape[2]
    rank_e = E.shape[1]
    dev = U.device
    bf = torch.bfloat16
    o = out or {}
    tokens = _out(o, "tokens", lambda: torch.empty((R, gamma), dtype=torch.int32, device=dev))
    ql = _out(o, "q_logits", lambda: torch.empty((R, gamma, V), dtype=bf, device=dev))
    conf = _out(o, "conf", lambda: torch.empty((R, gamma), dtype=torch.float32, device=dev))
    status = _out(o, "status", lambda: torch.empty(R, dtype=torch.int32, device=dev))
    qs = _out(o, "q_stats", lambda: torch.empty((R, gamma, 2), dtype=torch.float32, device=dev)) if stats else None
    ws = workspace if workspace is not None else _workspace(sd_markov_draft_workspace_size(R, gamma, V, rank), dev)
    code = lib().sd_markov_draft(
        _stream(stream), R, gamma, V, rank, float(temperature), int(seed) & (2**64 - 1),
        _ptr(pos0, torch.int64, "pos0"), _ptr(U, bf, "U"), _ptr(A, bf, "A"), _ptr(Ct, bf, "Ct"),
        _ptr(x0, torch.int32, "x0"), _ptr(h, bf, "h"), H, _ptr(E, bf, "E"), rank_e,
        _ptr(w, torch.float32, "w"), _ptr(tokens, torch.int32), _ptr(ql, bf),
        _ptr(qs, torch.float32, "q_stats"), _ptr(conf, torch.float32), _ptr(status, torch.int32),
        ws.data_ptr(), ws.numel())
    _check("sd_markov_draft", code)
    return dict(tokens=tokens, q_logits=ql, conf=conf, status=status, q_stats=qs)


def sd_rnn_draft_workspace_size(R, gamma, V, d):
    return lib().sd_rnn_draft_workspace_size(R, gamma, V, d)


@_on_stream
def sd_rnn_draft(U, W, Es, Ct, x0, h, E, w, temperature=1.0, seed=0, pos0=None, workspace=None,
                 out=None, stream=None, stats=False):
    """Run the RNN drafting head.  Returns a dict of device tensors:
    tokens [R][gamma], q_logits [R][gamma][V] bf16, conf [R][gamma], status [R],
    and q_stats [R][gamma][2] ((m, Z) of each drafted row) if stats."""
    R, gamma, V = U.shape
    d = W.shape[0]
    H = h.shape[2]
    rank_e = E.shape[1]
    dev = U.device
    bf = torch.bfloat16
    o = out or {}
    tokens = _out(o, "tokens", lambda: torch.empty((R, gamma), dtype=torch.int32, device=dev))
    ql = _out(o, "q_logits", lambda: torch.empty((R, gamma, V), dtype=bf, device=dev))
    conf = _out(o, "conf", lambda: torch.empty((R, gamma), dtype=torch.float32, device=dev))
    status = _out(o, "status", lambda: torch.empty(R, dtype=torch.int32, device=dev))
    qs = _out(o, "q_stats", lambda: torch.empty((R, gamma, 2), dtype=torch.float32, device=dev)) if stats else None
    ws = workspace if workspace is not None else _workspace(sd_rnn_draft_workspace_size(R, gamma, V, d),
                                                            dev)
    code = lib().sd_rnn_draft(
        _stream(stream), R, gamma, V, d, float(temperature), int(seed) & (2**64 - 1),
        _ptr(pos0, torch.int64, "pos0"), _ptr(U, bf, "U"), _ptr(W, bf, "W"), _ptr(Es, bf, "Es"),
        _ptr(Ct, bf, "Ct"), _ptr(x0, torch.int32, "x0"), _ptr(h, bf, "h"), H, _ptr(E, bf, "E"), rank_e,
        _ptr(w, torch.float32, "w"), _ptr(tokens, torch.int32), _ptr(ql, bf),
        _ptr(qs, torch.float32, "q_stats"), _ptr(conf, torch.float32), _ptr(status, torch.int32),
        ws.data_ptr(), ws.numel())
    _check("sd_rnn_draft", code)
    return dict(tokens=tokens, q_logits=ql, conf=conf, status=status, q_stats=qs)


@_on_stream
def sd_uniforms(seed, req, pos, draw, out=None, stream=None):
    """The uniforms u(seed, req[i], pos[i], draw) the library's decisions
    draw (req, pos int64 device tensors of one length).  Returns fp32."""
    n = req.numel()
    if pos.numel() != n:
        raise ValueError("req and pos must have the same length")
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=req.device)
    _check("sd_uniforms", lib().sd_uniforms(_stream(stream), int(seed) & (2**64 - 1), n,
                                            _ptr(req, torch.int64, "req"), _ptr(pos, torch.int64, "pos"),
                                            int(draw), _ptr(out, torch.float32, "out")))
    return out


@_on_stream
def sd_lightspec_update(alpha, ell, status, lam, ema, count, stream=None):
    """Fold one verify step's acceptance probabilities alpha [R][gmax] fp32
    into the per-position EMA state ema [gmax] fp64 / count [gmax] int64
    (updated in place on the device)."""
    R, gmax = alpha.shape
    _check("sd_lightspec_update", lib().sd_lightspec_update(
        _stream(stream), R, gmax, _ptr(alpha, torch.float32, "alpha"), _ptr(ell, torch.int32, "ell"),
        _ptr(status, torch.int32, "status"), float(lam), _ptr(ema, torch.float64, "ema"),
        _ptr(count, torch.int64, "count")))


@_on_stream
def sd_lightspec_plan(ema, count, d_prev, sps, draft_cost, out=None, workspace=None, stream=None):
    """Both planning stages.  d_prev [R] int32 (the previous round's draft
    lengths).  Returns a dict of device tensors: conf (planning confidences),
    ell, batch, n_sel, theta (stage 1), d_next, b_next, phi (stage 2)."""
    gmax = ema.shape[0]
    R = d_prev.shape[0]
    dev = ema.device
    o = out or {}
    conf = _out(o, "conf", lambda: torch.empty(gmax, dtype=torch.float32, device=dev))
    ell = _out(o, "ell", lambda: torch.empty(R, dtype=torch.int32, device=dev))
    batch = _out(o, "batch", lambda: torch.empty(1, dtype=torch.int32, device=dev))
    n_sel = _out(o, "n_sel", lambda: torch.empty(1, dtype=torch.int32, device=dev))
    theta = _out(o, "theta", lambda: torch.empty(1, dtype=torch.float64, device=dev))
    d_next = _out(o, "d_next", lambda: torch.empty(1, dtype=torch.int32, device=dev))
    b_next = _out(o, "b_next", lambda: torch.empty(1, dtype=torch.int32, device=dev))
    phi = _out(o, "phi", lambda: torch.empty(gmax, dtype=torch.float64, device=dev))
    ws = workspace if workspace is not None else _workspace(lib().sd_lightspec_plan_workspace_size(R, gmax), dev)
    _check("sd_lightspec_plan", lib().sd_lightspec_plan(
        _stream(stream), R, gmax, _ptr(ema, torch.float64, "ema"), _ptr(count, torch.int64, "count"),
        _ptr(d_prev, torch.int32, "d_prev"), _ptr(sps, torch.float32, "sps"), sps.numel(),
        _ptr(draft_cost, torch.float32, "draft_cost"), _ptr(conf, torch.float32),
        _ptr(ell, torch.int32), _ptr(batch, torch.int32), _ptr(n_sel, torch.int32),
        _ptr(theta, torch.float64), _ptr(d_next, torch.int32), _ptr(b_next, torch.int32),
        _ptr(phi, torch.float64), ws.data_ptr(), ws.numel()))
    return dict(conf=conf, ell=ell, batch=batch, n_sel=n_sel, theta=theta, d_next=d_next,
                b_next=b_next, phi=phi)


# The handle of a device's current stream, without a stream object in between.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_device(fn):
    """Run fn with the device of its first argument as torch's current one and
    its `stream` argument, where given, as the current stream (see _on_stream),
    so that the kernels are launched, and outputs made, where the tensors live.
    The stream has to be that device's."""
    name = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def wrapper(*args, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        index = first.get_device()
        if index < 0:
            raise ValueError(f"{name} must live on the GPU")
        stream = kw.get("stream")
        if stream is None:
            if index == torch.cuda.current_device():
                return fn(*args, **kw)
            with torch.cuda.device(index):
                return fn(*args, **kw)
        if stream.device_index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {first.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return wrapper


_Tensor = torch.Tensor


def _arg(t, dtype, name, index, n=None):
    """The address of tensor t (None: NULL) after checking its type, that it
    is contiguous and on device `index`, and its number of elements where
    given."""
    if t is None:
        return None
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous() and (n is None or t.numel() == n):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must live on cuda:{index}, not {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must hold {n} elements, got shape {list(t.shape)}")


def _fits(fn, sizes):
    """Refuse sizes that the C interface's int does not hold, which ctypes
    would cut to their low 32 bits.  `sizes`: all of them, OR-ed together (a
    negative one is refused there)."""
    if sizes >> 31 not in (0, -1):
        raise SdvError(fn, SD_EUNSUPPORTED)


def _state_rows(seen, counts, V):
    """(n_slots, ld_seen, ld_counts) of a token state; 0 where there is none."""
    if seen is None:
        if counts is not None:
            raise ValueError("counts need seen")
        return 0, 0, 0
    if seen.dim() != 2 or (counts is not None and (counts.dim() != 2 or counts.shape[0] != seen.shape[0])):
        raise ValueError("seen and counts must be 2-D with one row per slot")
    return seen.shape[0], seen.shape[1], 0 if counts is None else counts.shape[1]


@_on_device
def sd_logit_shape(logits, row0, ell, V, gamma_max=None, draft_tokens=None, repetition=None, frequency=None,
                   presence=None, seen=None, counts=None, slot=None, bias=None, mask=None, mask_row0=None,
                   out=None, *, stream=None):
    """Apply penalties, biases and grammar masks to the rows of a verify batch.
    logits: 2-D rows (bf16 or fp32, ld = shape[1]); row0, ell [R] int32 as for
    sd_verify (ell < 0: no rows); draft_tokens [R][gamma_max] int32, or None
    with gamma_max given.  repetition, frequency, presence [R] fp32; seen
    [n_slots][words] int32 and counts [n_slots][ld] int32 as sd_token_counts
    keeps them; slot [R] int32.  bias: (offsets [R + 1] int64, tokens int32,
    values fp32).  mask [rows][words] int32 with mask_row0 [R] int32.
    out["logits"] may be logits itself (in place); without it new rows are
    made, whose parts outside the batch are undefined.  Returns a dict of
    device tensors: logits, status."""
    dev = logits.get_device()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    n_rows, ld = logits.shape
    R = row0.numel()
    if draft_tokens is not None:
        if draft_tokens.dim() != 2 or gamma_max not in (None, draft_tokens.shape[1]):
            raise ValueError("draft_tokens must be [R][gamma_max]")
        gamma_max = draft_tokens.shape[1]
    elif gamma_max is None:
        raise ValueError("gamma_max is needed without draft_tokens")
    if logits.dtype is torch.bfloat16:
        dt = SD_DTYPE_BF16
    elif logits.dtype is torch.float32:
        dt = SD_DTYPE_F32
    else:
        raise TypeError("logits must be bf16 or fp32")
    n_slots, ld_seen, ld_counts = _state_rows(seen, counts, V)
    b_off, b_tok, b_val = (None, None, None) if bias is None else bias
    n_bias = 0 if b_tok is None else b_tok.numel()
    if (mask is None) != (mask_row0 is None):
        raise ValueError("mask and mask_row0 go together")
    if mask is not None and mask.dim() != 2:
        raise ValueError("mask must be 2-D")
    o = out or {}
    dst = o["logits"] if "logits" in o else torch.empty_like(logits)
    status = o["status"] if "status" in o else torch.empty(R, dtype=torch.int32, device=logits.device)
    if dst.shape != logits.shape:
        raise ValueError(f"out must have the logits' shape {list(logits.shape)}, got {list(dst.shape)}")
    i32, f32, ldt = torch.int32, torch.float32, logits.dtype
    V, gamma_max = int(V), int(gamma_max)
    m_rows, m_ld = (0, 0) if mask is None else mask.shape
    _fits("sd_logit_shape", R | gamma_max | V | ld | n_rows | n_slots | ld_seen | ld_counts | m_rows | m_ld)
    code = lib().sd_logit_shape(
        _raw_stream(dev), R, gamma_max, V, ld, dt, _arg(logits, ldt, "logits", dev),
        _arg(dst, ldt, "out", dev), n_rows, _arg(row0, i32, "row0", dev), _arg(ell, i32, "ell", dev, R),
        _arg(draft_tokens, i32, "draft_tokens", dev, R * gamma_max), _arg(repetition, f32, "repetition", dev, R),
        _arg(frequency, f32, "frequency", dev, R), _arg(presence, f32, "presence", dev, R),
        _arg(seen, i32, "seen", dev), ld_seen, _arg(counts, i32, "counts", dev), ld_counts, n_slots,
        _arg(slot, i32, "slot", dev, R), _arg(b_off, torch.int64, "bias offsets", dev, R + 1),
        _arg(b_tok, i32, "bias tokens", dev), _arg(b_val, f32, "bias values", dev, n_bias), n_bias,
        _arg(mask, i32, "mask", dev), m_ld, m_rows, _arg(mask_row0, i32, "mask_row0", dev, R),
        _arg(status, i32, "status", dev, R))
    _check("sd_logit_shape", code)
    return dict(logits=dst, status=status)


@_on_device
def sd_token_counts(tokens, seen, counts, V, start=None, length=None, prompt_len=None, slot=None, reset=None,
                    out=None, max_length=0, *, stream=None):
    """Enter token lists into the state behind the penalties, in place: seen
    [n_slots][words] int32 (bits), counts [n_slots][ld] int32 or None.
    tokens: [R][width] int32 (entries outside [0, V) are skipped, such as the
    -1 behind sd_verify's tokens), with length [R] int32 or None; or any shape
    with start [R] int64 (into all of it) and length, of at most max_length
    where that is given: do so for short lists in a large buffer.  prompt_len [R] int32: how many leading tokens
    of each list are prompt; reset [R] int32: clear the state row first (for
    calls that start requests: with it short lists take many times as long).
    Returns a dict: status."""
    dev = tokens.get_device()
    if start is not None:
        R, width = start.numel(), int(max_length)
        if length is None:
            raise ValueError("start needs length")
    else:
        if tokens.dim() != 2:
            raise ValueError("tokens must be [R][width] without start")
        if max_length:
            raise ValueError("max_length goes with start")
        R, width = tokens.shape
    if seen is None:
        raise ValueError("seen is needed")
    n_slots, ld_seen, ld_counts = _state_rows(seen, counts, V)
    status = out["status"] if out and "status" in out else torch.empty(R, dtype=torch.int32, device=tokens.device)
    i32, V = torch.int32, int(V)
    _fits("sd_token_counts", R | V | width | n_slots | ld_seen | ld_counts)
    code = lib().sd_token_counts(
        _raw_stream(dev), R, V, _arg(tokens, i32, "tokens", dev), tokens.numel(), width,
        _arg(start, torch.int64, "start", dev), _arg(length, i32, "length", dev, R),
        _arg(prompt_len, i32, "prompt_len", dev, R), _arg(slot, i32, "slot", dev, R),
        _arg(reset, i32, "reset", dev, R), _arg(seen, i32, "seen", dev), ld_seen,
        _arg(counts, i32, "counts", dev), ld_counts, n_slots, _arg(status, i32, "status", dev, R))
    _check("sd_token_counts", code)
    return dict(status=status)


def sd_slot_reserve_workspace_size(R):
    return lib().sd_slot_reserve_workspace_size(R)


@_on_device
def sd_slot_reserve(seq_len, ell, block_table, free_list, free_count, block_size, q_max, max_rows=None,
                    padded=False, x0=None, tokens=None, out=None, workspace=None, *, stream=None):
    """Rows and cache slots of a step.  seq_len [R] int64, ell [R] int32
    (rows - 1 asked for; -1: none), block_table [R][max_blocks] int32 (new
    blocks are entered in place), free_list [n_blocks] int32, free_count [1]
    int32.  x0 [R] and / or tokens [R][n] int32 give the rows' tokens.
    max_rows: rows of the buffers (default R * q_max, or those of
    out["row_req"]).  Returns a dict of device tensors: ell, row0, cu_rows,
    ctx_len, batch, free_count, row_req, row_pos, row_slot, row_token (None
    without tokens), status."""
    dev, device = seq_len.get_device(), seq_len.device
    R = seq_len.numel()
    if block_table.dim() != 2 or (tokens is not None and tokens.dim() != 2):
        raise ValueError("block_table and tokens must be 2-D")
    mb, n_blocks, ld_tokens = block_table.shape[1], free_list.numel(), 0 if tokens is None else tokens.shape[1]
    o = out or {}
    i32, q_max, block_size = torch.int32, int(q_max), int(block_size)
    if max_rows is None:
        max_rows = o["row_req"].numel() if "row_req" in o else R * q_max
    _fits("sd_slot_reserve", R | q_max | block_size | mb | n_blocks | max_rows | ld_tokens)
    i64 = torch.int64
    make = lambda k, n, dt=i32: o[k] if k in o else torch.empty(n, dtype=dt, device=device)  # noqa: E731
    res = dict(ell=make("ell", R), row0=make("row0", R), cu_rows=make("cu_rows", R + 1), ctx_len=make("ctx_len", R),
               batch=make("batch", 1), free_count=make("free_count", 1), row_req=make("row_req", max_rows),
               row_pos=make("row_pos", max_rows), row_slot=make("row_slot", max_rows, i64),
               row_token=None if x0 is None and tokens is None else make("row_token", max_rows),
               status=make("status", R))
    ws = workspace if workspace is not None else _workspace(sd_slot_reserve_workspace_size(R), device)
    code = lib().sd_slot_reserve(
        _raw_stream(dev), R, q_max, block_size, mb, n_blocks, max_rows, 1 if padded else 0,
        _arg(seq_len, i64, "seq_len", dev), _arg(ell, i32, "ell", dev, R), _arg(x0, i32, "x0", dev, R),
        _arg(tokens, i32, "tokens", dev, R * ld_tokens), ld_tokens, _arg(block_table, i32, "block_table", dev, R * mb),
        _arg(free_list, i32, "free_list", dev), _arg(free_count, i32, "free_count", dev, 1),
        _arg(res["ell"], i32, "out ell", dev, R), _arg(res["row0"], i32, "row0", dev, R),
        _arg(res["cu_rows"], i32, "cu_rows", dev, R + 1), _arg(res["ctx_len"], i32, "ctx_len", dev, R),
        _arg(res["batch"], i32, "batch", dev, 1), _arg(res["free_count"], i32, "out free_count", dev, 1),
        _arg(res["row_req"], i32, "row_req", dev, max_rows), _arg(res["row_pos"], i32, "row_pos", dev, max_rows),
        _arg(res["row_slot"], i64, "row_slot", dev, max_rows),
        _arg(res["row_token"], i32, "row_token", dev, max_rows), _arg(res["status"], i32, "status", dev, R),
        _arg(ws, torch.uint8, "workspace", dev), ws.numel())
    _check("sd_slot_reserve", code)
    return res


def sd_slot_commit_workspace_size(R):
    return lib().sd_slot_commit_workspace_size(R)


@_on_device
def sd_slot_commit(seq_len, ell, n_acc, block_table, free_list, free_count, block_size, q_max=None,
                   out_tokens=None, x0=None, status=None, release=None, keep=None, out=None, workspace=None,
                   *, stream=None):
    """Keep what verification accepted of a step and give the other blocks
    back.  seq_len [R] int64, ell [R] int32 and free_count [1] int32 as
    sd_slot_reserve left them, n_acc, out_tokens [R][q_max] sd_verify's,
    status [R] int32 the statuses of the step's calls OR-ed (slots, shaping
    and verification: a request that one of them refused keeps nothing of the
    step), x0 [R] int32 the step's anchors (with out_tokens: the next ones are
    returned); release, keep [R] int32.  free_list is updated in place, and
    status where a request is refused.  Returns a dict of device tensors:
    seq_len, n_new, free_count, x0 (None without out_tokens)."""
    dev, device = seq_len.get_device(), seq_len.device
    R = seq_len.numel()
    if block_table.dim() != 2:
        raise ValueError("block_table must be 2-D")
    mb = block_table.shape[1]
    if out_tokens is not None:
        if out_tokens.dim() != 2 or q_max not in (None, out_tokens.shape[1]):
            raise ValueError("out_tokens must be [R][q_max]")
        q_max = out_tokens.shape[1]
    elif q_max is None:
        raise ValueError("q_max is needed without out_tokens")
    n_blocks, q_max, block_size = free_list.numel(), int(q_max), int(block_size)
    _fits("sd_slot_commit", R | q_max | block_size | mb | n_blocks)
    o = out or {}
    i32 = torch.int32
    i64 = torch.int64
    make = lambda k, n, dt=i32: o[k] if k in o else torch.empty(n, dtype=dt, device=device)  # noqa: E731
    res = dict(seq_len=make("seq_len", R, i64), n_new=make("n_new", R), free_count=make("free_count", 1),
               x0=None if out_tokens is None else make("x0", R))
    ws = workspace if workspace is not None else _workspace(sd_slot_commit_workspace_size(R), device)
    code = lib().sd_slot_commit(
        _raw_stream(dev), R, q_max, block_size, mb, n_blocks,
        _arg(seq_len, i64, "seq_len", dev), _arg(ell, i32, "ell", dev, R), _arg(n_acc, i32, "n_acc", dev, R),
        _arg(out_tokens, i32, "out_tokens", dev, R * q_max), _arg(x0, i32, "x0", dev, R),
        _arg(release, i32, "release", dev, R), _arg(keep, i32, "keep", dev, R),
        _arg(block_table, i32, "block_table", dev, R * mb), _arg(free_list, i32, "free_list", dev),
        _arg(free_count, i32, "free_count", dev, 1), _arg(status, i32, "status", dev, R),
        _arg(res["seq_len"], i64, "out seq_len", dev, R), _arg(res["x0"], i32, "out x0", dev, R),
        _arg(res["n_new"], i32, "n_new", dev, R), _arg(res["free_count"], i32, "out free_count", dev, 1),
        _arg(ws, torch.uint8, "workspace", dev), ws.numel())
    _check("sd_slot_commit", code)
    return res


def _heads(t, dtype, name, index, shape=None):
    """(address, leading dimension) of rows of heads [rows][heads][D] whose
    heads and channels lie together (None: (NULL, 0)), such as a part of a
    projection's rows."""
    if t is None:
        return None, 0
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must live on cuda:{index}, not {t.device}")
    got = t.shape
    if len(got) != 3 or (shape is not None and got != shape):
        raise ValueError(f"{name} must be [rows][heads][D]{'' if shape is None else f' {list(shape)}'}, "
                         f"got shape {list(got)}")
    n, h, d = got
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        raise ValueError(f"{name}: the heads of a row must lie together, got strides {[s0, s1, s2]}")
    # a single row's stride says nothing
    return t.data_ptr(), s0 if n > 1 else -(-h * d // 8) * 8


_ROW_TYPES = {torch.bfloat16: SD_DTYPE_BF16, torch.float32: SD_DTYPE_F32}


def _row_type(t, name):
    dt = _ROW_TYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be bf16 or fp32")
    return dt


def _rotation(inv_freq, pos, D, what):
    """rot_dim of the frequencies, checked against the heads."""
    if inv_freq is None:
        return 0
    if pos is None:
        raise ValueError(f"inv_freq needs {what}")
    pairs = inv_freq.numel()
    if 2 * pairs > D:
        raise ValueError(f"inv_freq holds {pairs} pairs, a head {D} channels")
    return 2 * pairs


def _cache_args(cache, index):
    """(type, n_blocks, n_kv, block_size, D, addresses) of a cache: (k, v) in
    bf16, or (k, v, k_scale, v_scale) uint8 in 4 bits."""
    if not isinstance(cache, (tuple, list)) or len(cache) not in (2, 4):
        raise ValueError("cache must be (k, v) or (k, v, k_scale, v_scale)")
    if len(cache) == 2:
        (k, v), dt, ctype = cache, torch.bfloat16, SD_CACHE_BF16
    else:
        (k, v, k_scale, v_scale), dt, ctype = cache, torch.uint8, SD_CACHE_FP4
    at_k, at_v = _arg(k, dt, "k cache", index), _arg(v, dt, "v cache", index)
    shape = None if k is None or v is None else k.shape
    if shape is None or len(shape) != 4 or v.shape != shape:
        raise ValueError("the caches must be [n_blocks][n_kv][block_size][channels] and alike")
    n_blocks, n_kv, bs, D = shape
    if ctype == SD_CACHE_BF16:
        return ctype, n_blocks, n_kv, bs, D, (at_k, at_v, None, None)
    D *= 2
    at_ks, at_vs = _arg(k_scale, dt, "k_scale", index), _arg(v_scale, dt, "v_scale", index)
    groups = (n_blocks, n_kv, bs, D // 32)
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t is None or t.shape != groups:
            raise ValueError(f"{name} must be [n_blocks][n_kv][block_size][D / 32]")
    return ctype, n_blocks, n_kv, bs, D, (at_k, at_v, at_ks, at_vs)


@_on_device
def sd_qk_rope(q, k, pos, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, out=None, *,
               stream=None):
    """Norm and rotate the heads of queries and keys.  q [rows][n_q][D], k
    [rows][n_kv][D] (or None) in bf16 or fp32, each row's heads together;
    pos [rows] int32 (< 0: the row is left out; None without inv_freq);
    inv_freq fp32, one frequency per pair of channels; q_weight, k_weight [D]
    fp32 or None (no norm).  out["q"], out["k"] may be q and k themselves (in
    place); without them new tensors are made, whose left-out rows are
    undefined.  Returns a dict of device tensors: q, k."""
    dev = q.get_device()
    dt = _row_type(q, "q")
    at_q, ld_q = _heads(q, q.dtype, "q", dev)
    n, n_q, D = q.shape
    n_k = 0 if k is None else k.shape[1] if k.dim() == 3 else -1
    at_k, ld_k = _heads(k, q.dtype, "k", dev, None if k is None else (n, n_k, D))
    o = out or {}
    empty = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
    qo = o["q"] if "q" in o else empty(q)
    ko = o["k"] if "k" in o else empty(k)
    at_qo, ld_qo = _heads(qo, q.dtype, "out q", dev, q.shape)
    at_ko, ld_ko = (None, 0) if k is None else _heads(ko, q.dtype, "out k", dev, k.shape)
    rot = _rotation(inv_freq, pos, D, "pos")
    _fits("sd_qk_rope", n | n_q | n_k | D)
    f32 = torch.float32
    code = lib().sd_qk_rope(
        _raw_stream(dev), n, D, dt, at_q, n_q, ld_q, at_k, n_k, ld_k, _arg(pos, torch.int32, "pos", dev, n),
        _arg(q_weight, f32, "q_weight", dev, D), _arg(k_weight, f32, "k_weight", dev, D), float(eps),
        _arg(inv_freq, f32, "inv_freq", dev), rot, 1 if interleaved else 0, at_qo, ld_qo, at_ko, ld_ko)
    _check("sd_qk_rope", code)
    return dict(q=qo, k=None if k is None else ko)


@_on_device
def sd_cache_append(k, v, cache, row_slot, row_pos=None, inv_freq=None, q=None, q_weight=None, k_weight=None, eps=1e-6,
                    interleaved=False, out=None, *, stream=None):
    """Put keys and values of a step's rows into their slots of a paged cache.
    k, v [rows][n_kv][D] in bf16 or fp32, each row's heads together; cache:
    (k, v) bf16 [n_blocks][n_kv][block_size][D], or (k, v, k_scale, v_scale)
    uint8 [...][D / 2] and [...][D / 32] (4 bits), written in place; row_slot
    [rows] int64 and row_pos [rows] int32 sd_slot_reserve's.  The keys are
    normed and rotated as by sd_qk_rope on the way; with q [rows][n_q][D] so
    are the queries, into out["q"] (which may be q) or a new tensor.  Returns
    a dict: q (None without q)."""
    dev = k.get_device()
    dt = _row_type(k, "k")
    at_k, ld_k = _heads(k, k.dtype, "k", dev)
    n, n_kv, D = k.shape
    at_v, ld_v = _heads(v, k.dtype, "v", dev, k.shape)
    if v is None:
        raise ValueError("v is needed")
    n_q = 0 if q is None else q.shape[1] if q.dim() == 3 else -1
    at_q, ld_q = _heads(q, k.dtype, "q", dev, None if q is None else (n, n_q, D))
    qo = None
    if q is not None:
        qo = out["q"] if out and "q" in out else torch.empty(q.shape, dtype=q.dtype, device=q.device)
    at_qo, ld_qo = _heads(qo, k.dtype, "out q", dev, None if q is None else q.shape)
    ctype, n_blocks, c_kv, bs, c_D, at = _cache_args(cache, dev)
    if (c_kv, c_D) != (n_kv, D):
        raise ValueError(f"the cache holds {c_kv} heads of {c_D} channels, k {n_kv} of {D}")
    rot = _rotation(inv_freq, row_pos, D, "row_pos")
    _fits("sd_cache_append", n | n_q | n_kv | D | n_blocks | bs)
    f32 = torch.float32
    code = lib().sd_cache_append(
        _raw_stream(dev), n, D, dt, at_q, n_q, ld_q, at_k, ld_k, at_v, ld_v, n_kv,
        _arg(row_pos, torch.int32, "row_pos", dev, n), _arg(row_slot, torch.int64, "row_slot", dev, n),
        _arg(q_weight, f32, "q_weight", dev, D), _arg(k_weight, f32, "k_weight", dev, D), float(eps),
        _arg(inv_freq, f32, "inv_freq", dev), rot, 1 if interleaved else 0, at_qo, ld_qo, ctype, bs, n_blocks, *at)
    _check("sd_cache_append", code)
    return dict(q=qo)


@_on_device
def sd_cache_read(row_slot, cache, out=None, dtype=torch.bfloat16, *, stream=None):
    """Keys and values at slots of a paged cache as rows [rows][n_kv][D], in
    bf16 or fp32 (out's type where given).  row_slot [rows] int64 (outside the
    cache: the row is left as it is, undefined in new tensors), cache as for
    sd_cache_append.  Returns a dict of device tensors: k, v."""
    dev, device = row_slot.get_device(), row_slot.device
    ctype, n_blocks, n_kv, bs, D, at = _cache_args(cache, dev)
    n, o = row_slot.numel(), out or {}
    if o:
        dtype = next(iter(o.values())).dtype
    make = lambda key: o[key] if key in o else torch.empty((n, n_kv, D), dtype=dtype, device=device)  # noqa: E731
    ko, vo = make("k"), make("v")
    at_k, ld_k = _heads(ko, dtype, "out k", dev, (n, n_kv, D))
    at_v, ld_v = _heads(vo, dtype, "out v", dev, (n, n_kv, D))
    _fits("sd_cache_read", n | n_kv | D | n_blocks | bs)
    code = lib().sd_cache_read(
        _raw_stream(dev), n, D, _arg(row_slot, torch.int64, "row_slot", dev), ctype, n_kv, bs, n_blocks, *at,
        _row_type(ko, "out"), at_k, ld_k, at_v, ld_v)
    _check("sd_cache_read", code)
    return dict(k=ko, v=vo)


def sd_attn_workspace_size(R, q_max, n_q, n_kv, D):
    return lib().sd_attn_workspace_size(R, q_max, n_q, n_kv, D)


@_on_device
def sd_attn_plan(row0, ell, ctx_len, q_max, n_q, cache, causal=True, window=0, out=None, workspace=None, *,
                 stream=None):
    """Cut a step's attention into equal parts, once for all its layers.  row0,
    ell, ctx_len [R] int32 as sd_slot_reserve leaves them, q_max its bound on
    a request's rows, n_q query heads; cache: one layer's, for its type and
    sizes (layers that differ in the type or the block size need plans of their
    own).  causal: a row sees the tokens up to its own, else all of its
    request's; window > 0: only the last so many up to its own.  Returns a dict
    that sd_cache_attn takes: workspace and status (device tensors) and what
    they are for."""
    dev, device = row0.get_device(), row0.device
    R = row0.numel()
    ctype, _, n_kv, bs, D, _ = _cache_args(cache, dev)
    q_max, n_q, window = int(q_max), int(n_q), int(window)
    _fits("sd_attn_plan", R | q_max | n_q | n_kv | D | bs | window)
    status = out["status"] if out and "status" in out else torch.empty(R, dtype=torch.int32, device=device)
    ws = workspace if workspace is not None else _workspace(sd_attn_workspace_size(R, q_max, n_q, n_kv, D), device)
    i32 = torch.int32
    code = lib().sd_attn_plan(
        _raw_stream(dev), R, q_max, n_q, n_kv, D, ctype, bs, _arg(row0, i32, "row0", dev), _arg(ell, i32, "ell", dev, R),
        _arg(ctx_len, i32, "ctx_len", dev, R), 1 if causal else 0, window, _arg(status, i32, "status", dev, R),
        _arg(ws, torch.uint8, "workspace", dev), ws.numel())
    _check("sd_attn_plan", code)
    return dict(workspace=ws, status=status, R=R, q_max=q_max, n_q=n_q, n_kv=n_kv, D=D, cache_type=ctype,
                block_size=bs)


@_on_device
def sd_cache_attn(q, cache, block_table, plan, scale=None, lse=False, out=None, *, stream=None):
    """Attention of a step's rows over a paged cache.  q [rows][n_q][D] bf16,
    each row's heads together; cache as for sd_cache_append; block_table
    [R][max_blocks] int32; plan: sd_attn_plan's for this step.  scale: 1 /
    sqrt(D) if None.  lse: also return the log of each softmax's sum (or give
    out["lse"], [rows][n_q] fp32).  Rows of no request are left as they are,
    undefined in new tensors.  Returns a dict of device tensors: out, lse (or
    None), status (the plan's, OR-ed into)."""
    dev = q.get_device()
    if q.dim() != 3:
        raise ValueError("q must be [rows][n_q][D]")
    n, n_q, D = q.shape
    bf = torch.bfloat16
    at_q, ld_q = _heads(q, bf, "q", dev)
    ctype, n_blocks, n_kv, bs, c_D, at = _cache_args(cache, dev)
    if (n_q, n_kv, D, D) != (plan["n_q"], plan["n_kv"], plan["D"], c_D):
        raise ValueError(f"the plan is for {plan['n_q']} and {plan['n_kv']} heads of {plan['D']} channels, got "
                         f"{n_q} and {n_kv} of {D} and {c_D}")
    if (ctype, bs) != (plan["cache_type"], plan["block_size"]):
        kinds = {SD_CACHE_BF16: "bf16", SD_CACHE_FP4: "4 bits"}
        raise ValueError(f"the plan is for a cache in {kinds[plan['cache_type']]} with blocks of {plan['block_size']}, "
                         f"got {kinds[ctype]} and {bs}")
    R = plan["R"]
    if block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError(f"block_table must be [R][max_blocks] with R = {R}")
    mb = block_table.shape[1]
    o = out or {}
    dst = o["out"] if "out" in o else torch.empty(q.shape, dtype=bf, device=q.device)
    at_out, ld_out = _heads(dst, bf, "out", dev, q.shape)
    z = o["lse"] if "lse" in o else torch.empty((n, n_q), dtype=torch.float32, device=q.device) if lse else None
    _fits("sd_cache_attn", n | n_q | n_blocks | bs | mb)
    ws = plan["workspace"]
    code = lib().sd_cache_attn(
        _raw_stream(dev), R, plan["q_max"], n_q, n_kv, D, n, at_q, ld_q, ctype, bs, n_blocks, *at,
        _arg(block_table, torch.int32, "block_table", dev), mb, float(D ** -0.5 if scale is None else scale), at_out,
        ld_out, _arg(z, torch.float32, "lse", dev, n * n_q), _arg(plan["status"], torch.int32, "status", dev, R),
        _arg(ws, torch.uint8, "workspace", dev), ws.numel())
    _check("sd_cache_attn", code)
    return dict(out=dst, lse=z, status=plan["status"])
