"""Focus centroid-gated sparse attention for GB300 (sm_103a): routing, the forward
pass (exact-set segments or group lists), decode, and the backward pass with the
group masks held fixed; rotary positions, and a key/value cache in bf16 or 8 bits with
the decode step of one or many drafted tokens over it, for a batch behind one prefix too;
sampling from logits, and the acceptance of drafted tokens.

Thin ctypes binding over the C ABI in ``include/focus.h`` (``libfocus.so``, built
in-tree by ``learned_centroid_gated_gb300.build``). This module only marshals
arguments: every step of the computation runs in the library's CUDA kernels.
PyTorch supplies device memory and streams. There is no CPU fallback: importing
this package fails if the library is missing.

Method: "Why Attend to Everything? Focus is the Key" -- gist.science technical
summary, section 2 "Core Architecture" and "Inference Efficiency (Top-k)".
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# FOCUS_DEBUG_BOUNDS=1: the debug build (index checks raise FOCUS_ERR_BOUNDS; build it
# with the same variable set), else the default build
LIB_PATH = os.path.join(_HERE, "libfocus_debug.so" if os.environ.get("FOCUS_DEBUG_BOUNDS", "")
                        not in ("", "0") else "libfocus.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "focus.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"Focus CUDA library not built ({LIB_PATH} missing); run "
        "`python learned_centroid_gated_gb300/build.py` on a machine with nvcc")

_lib = ctypes.CDLL(LIB_PATH)

FOCUS_OK = 0
ERRORS = {
    -1: "FOCUS_ERR_INVALID_ARG", -2: "FOCUS_ERR_UNSUPPORTED", -3: "FOCUS_ERR_WORKSPACE",
    -4: "FOCUS_ERR_CUDA", -5: "FOCUS_ERR_TIMEOUT", -6: "FOCUS_ERR_BOUNDS", -7: "FOCUS_ERR_ALIGNMENT",
    -8: "FOCUS_ERR_NONFINITE",
}


class FocusError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        detail = strerror(code)
        if code == -4:  # FOCUS_ERR_CUDA: name the CUDA error behind it
            detail += ": " + _lib.focus_cuda_error_string().decode()
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({detail})")


class _Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "N", "H", "H_kv", "d_head", "R", "K", "top_k", "w", "sinkhorn_iters")] + \
               [("sinkhorn_eps", ctypes.c_float), ("softmax_scale", ctypes.c_float),
                ("schedule", ctypes.c_int32)]

SCHEDULE_AUTO, SCHEDULE_SEGMENTS, SCHEDULE_GROUPS = 0, 1, 2


@dataclasses.dataclass(frozen=True)
class Params:
    """Problem description (focus_params).  softmax_scale <= 0 selects 1/sqrt(d_head);
    schedule: SCHEDULE_AUTO, SCHEDULE_SEGMENTS (exact group sets) or SCHEDULE_GROUPS
    (one list per group)."""
    B: int
    N: int
    H: int
    H_kv: int
    d_head: int
    R: int
    K: int
    top_k: int
    w: int
    sinkhorn_iters: int = 0
    sinkhorn_eps: float = 1.0
    softmax_scale: float = 0.0
    schedule: int = 0

    @classmethod
    def from_workload(cls, wl, **kw) -> "Params":
        return cls(B=wl.B, N=wl.N, H=wl.H, H_kv=wl.H_kv, d_head=wl.d_head, R=wl.R, K=wl.K,
                   top_k=wl.top_k, w=wl.w, sinkhorn_iters=wl.sinkhorn_iters,
                   sinkhorn_eps=wl.sinkhorn_eps, **kw)

    def c(self) -> _Params:
        return _Params(*[getattr(self, f.name) for f in dataclasses.fields(self)])

    @property
    def nseg(self) -> int:
        """Segments of the bucketing that runs: C(K, top_k) exact sets, or K lists."""
        return self.bucket_shape()[1]

    def bucket_shape(self):
        """(schedule that runs, segments, permuted rows per (b, routing head))."""
        nseg, rows = ctypes.c_int32(), ctypes.c_int32()
        rc = _lib.focus_bucket_shape(ctypes.byref(self.c()), ctypes.byref(nseg), ctypes.byref(rows))
        _check(rc if rc < 0 else 0, "focus_bucket_shape")
        return rc, nseg.value, rows.value

    @property
    def scale(self) -> float:
        return self.softmax_scale if self.softmax_scale > 0 else 1.0 / math.sqrt(self.d_head)


_P = ctypes.c_void_p
_PP = ctypes.POINTER(_Params)
_lib.focus_workspace_size.argtypes = [_PP]
_lib.focus_workspace_size.restype = ctypes.c_size_t
_lib.focus_route.argtypes = [_PP, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.focus_route.restype = ctypes.c_int
_lib.focus_bucket_shape.argtypes = [_PP, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
_lib.focus_bucket_shape.restype = ctypes.c_int
_lib.focus_bucket.argtypes = [_PP, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.focus_bucket.restype = ctypes.c_int
_lib.focus_attn_fwd.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.focus_attn_fwd.restype = ctypes.c_int
_lib.focus_attn_fwd_ev.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P,
                                   ctypes.POINTER(ctypes.c_void_p)]
_lib.focus_attn_fwd_ev.restype = ctypes.c_int
N_STAGE_EVENTS = 6
STAGES = ("route", "bucket", "permute", "attn_window", "attn_long")
_lib.focus_route_static.argtypes = [_PP, _P, _P, _P, _P, _P]
_lib.focus_route_static.restype = ctypes.c_int
_lib.focus_route_static_limit.argtypes = []
_lib.focus_route_static_limit.restype = ctypes.c_size_t
_lib.focus_bwd_workspace_size.argtypes = [_PP]
_lib.focus_bwd_workspace_size.restype = ctypes.c_size_t
_lib.focus_attn_bwd.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.focus_attn_bwd.restype = ctypes.c_int
_lib.focus_attn_bwd_ev.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P,
                                   ctypes.POINTER(ctypes.c_void_p)]
_lib.focus_attn_bwd_ev.restype = ctypes.c_int
N_BWD_STAGE_EVENTS = 5
BWD_STAGES = ("prepare", "window", "long_dq", "long_dkdv")
_lib.focus_decode_workspace_size.argtypes = [_PP]
_lib.focus_decode_workspace_size.restype = ctypes.c_size_t
_lib.focus_decode.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.focus_decode.restype = ctypes.c_int
_lib.focus_selftest_timeout.argtypes = [_P, ctypes.c_size_t, _P]
_lib.focus_selftest_timeout.restype = ctypes.c_int
_lib.focus_selftest_timeout_decode.argtypes = [_P, ctypes.c_size_t, _P]
_lib.focus_selftest_timeout_decode.restype = ctypes.c_int
_lib.focus_selftest_timeout_shared.argtypes = [_P, ctypes.c_size_t, _P]
_lib.focus_selftest_timeout_shared.restype = ctypes.c_int
_lib.focus_get_status.argtypes = [_P, _P]
_lib.focus_get_status.restype = ctypes.c_int
_lib.focus_strerror.argtypes = [ctypes.c_int]
_lib.focus_strerror.restype = ctypes.c_char_p
_lib.focus_version.argtypes = []
_lib.focus_version.restype = ctypes.c_int
_lib.focus_cuda_error_string.argtypes = []
_lib.focus_cuda_error_string.restype = ctypes.c_char_p


def declared_symbols() -> list[str]:
    """Function names declared in include/focus.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(focus_\w+)\s*\(", text, re.M)))


def strerror(code: int) -> str:
    return _lib.focus_strerror(code).decode()


def version() -> int:
    return _lib.focus_version()


def workspace_size(p: Params) -> int:
    return int(_lib.focus_workspace_size(ctypes.byref(p.c())))


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, what: str):
    if rc != FOCUS_OK:
        raise FocusError(rc, what)


class Workspace:
    """Caller-owned device workspace (a torch uint8 buffer), grown on demand."""

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf: torch.Tensor | None = None

    def get(self, p: Params) -> torch.Tensor:
        need = workspace_size(p)
        if need == 0:
            raise FocusError(-1, "focus_workspace_size")
        if self.buf is None or self.buf.numel() < need:
            self.buf = torch.empty(need, dtype=torch.uint8, device=self.device)
        return self.buf


_default_ws: dict = {}


def _ws(p: Params, ws, device) -> torch.Tensor:
    if isinstance(ws, torch.Tensor):
        return ws
    if ws is None:
        ws = _default_ws.setdefault(str(device), Workspace(device))
    return ws.get(p)


def _bf16_bits(t: torch.Tensor) -> torch.Tensor:
    assert t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous()
    return t


def route(p: Params, r: torch.Tensor, C: torch.Tensor, *, margin: bool = False, ws=None,
          stream=None):
    """Group bitmasks [B, R, N] uint32 (as int32 tensor) and optional fp32 margins."""
    assert r.dtype == torch.float32 and C.dtype == torch.float32 and r.is_cuda and C.is_cuda
    mask = torch.empty(p.B, p.R, p.N, dtype=torch.int32, device=r.device)
    marg = torch.empty(p.B, p.R, p.N, dtype=torch.float32, device=r.device) if margin else None
    w = _ws(p, ws, r.device)
    _check(_lib.focus_route(ctypes.byref(p.c()), _ptr(r.contiguous()), _ptr(C.contiguous()),
                            _ptr(mask), _ptr(marg), _ptr(w), w.numel(), _stream(stream)),
           "focus_route")
    return mask, marg


def route_static_limit() -> int:
    """Bytes of the fixed device scratch that route_static uses for Sinkhorn."""
    return int(_lib.focus_route_static_limit())


def route_static(p: Params, r: torch.Tensor, C: torch.Tensor, *, margin: bool = False,
                 stream=None):
    """route() without a workspace: the library's fixed device scratch
    (route_static_limit() bytes, used by the Sinkhorn step only) is used instead,
    for callers that must not allocate device memory when they call in.  The
    outputs here are still torch tensors; pass preallocated ones through the C ABI
    (focus_route_static) to allocate nothing at all."""
    assert r.dtype == torch.float32 and C.dtype == torch.float32 and r.is_cuda and C.is_cuda
    mask = torch.empty(p.B, p.R, p.N, dtype=torch.int32, device=r.device)
    marg = torch.empty(p.B, p.R, p.N, dtype=torch.float32, device=r.device) if margin else None
    _check(_lib.focus_route_static(ctypes.byref(p.c()), _ptr(r.contiguous()), _ptr(C.contiguous()),
                                   _ptr(mask), _ptr(marg), _stream(stream)), "focus_route_static")
    return mask, marg


def bucket(p: Params, mask: torch.Tensor, *, ws=None, stream=None):
    """Stable bucketing: perm [B, R, rows] int32 and seg_off [B, R, nseg+1] int32, where
    (nseg, rows) = (C(K, top_k), N) for exact-set segments and (K, N * top_k) for group lists."""
    _, nseg, rows = p.bucket_shape()
    perm = torch.empty(p.B, p.R, rows, dtype=torch.int32, device=mask.device)
    seg = torch.empty(p.B, p.R, nseg + 1, dtype=torch.int32, device=mask.device)
    w = _ws(p, ws, mask.device)
    _check(_lib.focus_bucket(ctypes.byref(p.c()), _ptr(mask.contiguous()), _ptr(perm), _ptr(seg),
                             _ptr(w), w.numel(), _stream(stream)), "focus_bucket")
    return perm, seg


def attn_fwd(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, r=None, C=None,
             mask=None, *, out=None, lse=None, want_lse: bool = True, ws=None, stream=None,
             stage_events=None):
    """Focus attention forward on device tensors. Returns (o bf16 [B,N,H,d], lse fp32 [B,H,N]).

    stage_events: optional list of N_STAGE_EVENTS torch.cuda.Event(enable_timing=True),
    recorded at the stage boundaries (see focus_attn_fwd_ev)."""
    for t in (q, k, v):
        _bf16_bits(t)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(p.B, p.H, p.N, dtype=torch.float32, device=q.device)
    w = _ws(p, ws, q.device)
    args = (ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(r), _ptr(C), _ptr(mask), _ptr(out),
            _ptr(lse), _ptr(w), w.numel(), _stream(stream))
    if stage_events is None:
        _check(_lib.focus_attn_fwd(*args), "focus_attn_fwd")
    else:
        assert len(stage_events) == N_STAGE_EVENTS
        for e in stage_events:
            if e.cuda_event == 0:  # torch creates the CUDA event on its first record
                e.record(stream or torch.cuda.current_stream())
        evs = (ctypes.c_void_p * N_STAGE_EVENTS)(*[e.cuda_event for e in stage_events])
        _check(_lib.focus_attn_fwd_ev(*args, evs), "focus_attn_fwd_ev")
    return out, lse


_lib.focus_host_workspace_size.argtypes = [_PP, ctypes.c_int]
_lib.focus_host_workspace_size.restype = ctypes.c_size_t
_lib.focus_attn_fwd_host.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _P, ctypes.c_size_t,
                                     _P, _P]
_lib.focus_attn_fwd_host.restype = ctypes.c_int
_lib.focus_host_groups.argtypes = [_PP, ctypes.c_int, ctypes.POINTER(ctypes.c_int32), ctypes.c_int]
_lib.focus_host_groups.restype = ctypes.c_int


def host_groups(p: Params, n_groups: int = 0) -> list[int]:
    """KV heads of each head group focus_attn_fwd_host uses (in order)."""
    buf = (ctypes.c_int32 * 64)()
    n = _lib.focus_host_groups(ctypes.byref(p.c()), n_groups, buf, 64)
    _check(n if n < 0 else 0, "focus_host_groups")
    return list(buf[:n])


def host_workspace_size(p: Params, n_groups: int = 0) -> int:
    return int(_lib.focus_host_workspace_size(ctypes.byref(p.c()), n_groups))


class HostSession:
    """End-to-end calls on HOST tensors through focus_attn_fwd_host: the heads are
    processed in groups, copies of one group overlapping the compute of another, on
    two streams of this session.  Inputs should be pinned (tensor.pin_memory()) for
    the copies to overlap.  Each call returns pinned host tensors (o, lse) that the
    next call overwrites."""

    def __init__(self, p: Params, device="cuda", n_groups: int = 0):
        self.p = p
        self.device = torch.device(device)
        self.n_groups = n_groups
        need = host_workspace_size(p, n_groups)
        if need == 0:
            raise FocusError(-1, "focus_host_workspace_size")
        self.ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        self.compute = torch.cuda.Stream(self.device)
        self.copy = torch.cuda.Stream(self.device)
        self.o_host = torch.empty(p.B, p.N, p.H, p.d_head, dtype=torch.bfloat16, pin_memory=True)
        self.lse_host = torch.empty(p.B, p.H, p.N, dtype=torch.float32, pin_memory=True)

    def group_sizes(self) -> list[int]:
        """KV heads of each head group, in processing order."""
        return host_groups(self.p, self.n_groups)

    def h2d_bytes(self, *tensors) -> int:
        return sum(t.numel() * t.element_size() for t in tensors)

    def d2h_bytes(self) -> int:
        return self.o_host.numel() * 2 + self.lse_host.numel() * 4

    def __call__(self, q, k, v, r, C):
        for t, dt in ((q, torch.bfloat16), (k, torch.bfloat16), (v, torch.bfloat16),
                      (r, torch.float32), (C, torch.float32)):
            assert t.device.type == "cpu" and t.dtype == dt and t.is_contiguous()
        _check(_lib.focus_attn_fwd_host(ctypes.byref(self.p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(r),
                                        _ptr(C), _ptr(self.o_host), _ptr(self.lse_host), self.n_groups,
                                        _ptr(self.ws), self.ws.numel(),
                                        ctypes.c_void_p(self.compute.cuda_stream),
                                        ctypes.c_void_p(self.copy.cuda_stream)),
               "focus_attn_fwd_host")
        self.copy.synchronize()
        return self.o_host, self.lse_host


def attn_fwd_host(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, r: torch.Tensor,
                  C: torch.Tensor, *, device="cuda", n_groups: int = 0):
    """One end-to-end call on HOST tensors (see HostSession for repeated calls).
    Returns host (o, lse)."""
    o, lse = HostSession(p, device, n_groups)(q, k, v, r, C)
    return o.clone(), lse.clone()


def decode_workspace_size(p: Params) -> int:
    return int(_lib.focus_decode_workspace_size(ctypes.byref(p.c())))


def decode(p: Params, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           mask: torch.Tensor, *, out=None, lse=None, want_lse: bool = True, ws=None, stream=None):
    """Decode step for the newest token of each sequence (position p.N - 1).
    q [B, H, d] bf16; caches [B, N, H_kv, d] bf16 (newest token included); mask
    [B, R, N] (int32 view of uint32).  Returns (o [B, H, d] bf16, lse [B, H] fp32)."""
    for t in (q, k_cache, v_cache):
        _bf16_bits(t)
    if out is None:
        out = torch.empty(p.B, p.H, p.d_head, dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(p.B, p.H, dtype=torch.float32, device=q.device)
    need = decode_workspace_size(p)
    if need == 0:
        raise FocusError(-1, "focus_decode_workspace_size")
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(_lib.focus_decode(ctypes.byref(p.c()), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                             _ptr(mask.contiguous()), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                             _stream(stream)), "focus_decode")
    return out, lse


def bwd_workspace_size(p: Params) -> int:
    return int(_lib.focus_bwd_workspace_size(ctypes.byref(p.c())))


def attn_bwd(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask: torch.Tensor,
             o: torch.Tensor, lse: torch.Tensor, d_o: torch.Tensor, *, dq=None, dk=None, dv=None,
             ws=None, stream=None, stage_events=None):
    """Backward of attn_fwd with the masks held fixed.  q, o, d_o [B, N, H, d] bf16;
    k, v [B, N, H_kv, d] bf16; mask [B, R, N] (the forward's); lse [B, H, N] fp32 (the
    forward's).  Returns (dq, dk, dv) bf16 in the layouts of q, k, v.

    stage_events: optional list of N_BWD_STAGE_EVENTS torch.cuda.Event(enable_timing=True)
    recorded at the stage boundaries (see focus_attn_bwd_ev)."""
    for t in (q, k, v, o, d_o):
        _bf16_bits(t)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = bwd_workspace_size(p)
    if need == 0:
        raise FocusError(-2, "focus_bwd_workspace_size")
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    args = (ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(mask.contiguous()), _ptr(o),
            _ptr(lse.contiguous()), _ptr(d_o), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(),
            _stream(stream))
    if stage_events is None:
        _check(_lib.focus_attn_bwd(*args), "focus_attn_bwd")
    else:
        assert len(stage_events) == N_BWD_STAGE_EVENTS
        for e in stage_events:
            if e.cuda_event == 0:  # torch creates the CUDA event on its first record
                e.record(stream or torch.cuda.current_stream())
        evs = (ctypes.c_void_p * N_BWD_STAGE_EVENTS)(*[e.cuda_event for e in stage_events])
        _check(_lib.focus_attn_bwd_ev(*args, evs), "focus_attn_bwd_ev")
    return dq, dk, dv


# ---------------------------------------------------------------- rotary positions ----
class _RopeParams(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("orig_len", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("attn_factor", ctypes.c_double)]


class _RopePlan(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("attn_factor", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turn", ctypes.c_uint64 * 64)]


class _Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("n", ctypes.c_int64), ("h", ctypes.c_int64)]


class _CacheParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "cap", "T", "H", "H_kv", "d_head", "R", "K", "top_k", "w",
                                              "format")] + [("softmax_scale", ctypes.c_float)]

    @property
    def addr(self) -> int:
        """Where this struct stands: worked out anew, since a copy stands elsewhere."""
        return ctypes.addressof(self)


_I32, _I64 = ctypes.c_int32, ctypes.c_int64
_lib.focus_rope_init.argtypes = [_P, _P]
_lib.focus_rope_init.restype = ctypes.c_int
_lib.focus_rope_apply.argtypes = [_P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _I64, _I32,
                                  _P, _P, _P, _P, _P]
_lib.focus_rope_apply.restype = ctypes.c_int
_lib.focus_cache_write.argtypes = [_P] * 17
_lib.focus_cache_write.restype = ctypes.c_int
_lib.focus_cache_read.argtypes = [_P] * 11
_lib.focus_cache_read.restype = ctypes.c_int
_lib.focus_decode_tree_workspace_size.argtypes = [_P]
_lib.focus_decode_tree_workspace_size.restype = ctypes.c_size_t
_lib.focus_decode_tree.argtypes = [_P] * 12 + [ctypes.c_size_t, _P]
_lib.focus_decode_tree.restype = ctypes.c_int

_lib.focus_decode_shared_workspace_size.argtypes = [_P, _I32]
_lib.focus_decode_shared_workspace_size.restype = ctypes.c_size_t
_lib.focus_decode_shared.argtypes = [_P, _P, _I32, _I32] + [_P] * 15 + [ctypes.c_size_t, _P]
_lib.focus_decode_shared.restype = ctypes.c_int
_lib.focus_tree_accept.argtypes = [_P] * 16
_lib.focus_tree_accept.restype = ctypes.c_int
_lib.focus_sample.argtypes = [_P] * 11
_lib.focus_sample.restype = ctypes.c_int

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}
_ROPE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
CACHE_FORMATS = {"bf16": 0, "e4m3": 1, "int8": 2}
_CACHE_DTYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
MAX_DRAFT = 64


def _require(ok, what: str):
    """An argument that the C ABI cannot see to be wrong (a tensor's shape, type or device)."""
    if not ok:
        raise FocusError(-1, what)


def _made_anew(x):
    """What copy and pickle keep of a frozen parameter object: its fields.  The copy makes its
    own C structs, in its own process, with the library that is loaded there."""
    return type(x), tuple(getattr(x, f.name) for f in dataclasses.fields(x))


@dataclasses.dataclass(frozen=True)
class Rope:
    """Rotary positions (focus_rope_params): dim rotated columns of each head, pairs
    (i, i + dim / 2) ("half") or (2i, 2i + 1) ("interleaved"); scaling "none", "linear",
    "ntk" or "by_parts" stretches the positions by `factor` (by_parts: beyond orig_len
    tokens; attn_factor 0 selects 0.1 ln(factor) + 1 there, else 1).  Made once and kept:
    it holds the plan (focus_rope) that every call passes."""
    dim: int
    layout: str = "half"
    base: float = 10000.0
    scaling: str = "none"
    factor: float = 1.0
    orig_len: int = 4096
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    attn_factor: float = 0.0

    def __post_init__(self):
        _require(self.layout in ROPE_LAYOUTS and self.scaling in ROPE_SCALINGS, "focus_rope_init")
        plan = _RopePlan()
        params = _RopeParams(self.dim, ROPE_LAYOUTS[self.layout], ROPE_SCALINGS[self.scaling], self.orig_len,
                             self.base, self.factor, self.beta_fast, self.beta_slow, self.attn_factor)
        _check(_lib.focus_rope_init(ctypes.byref(params), ctypes.byref(plan)), "focus_rope_init")
        object.__setattr__(self, "_plan", plan)

    @property
    def _addr(self) -> int:
        return ctypes.addressof(self._plan)

    def __reduce__(self):
        return _made_anew(self)


# Device and stream look-ups of the serving calls, which a program makes for every token:
# the raw forms where this torch has them.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Launch:
    """Makes the device of a call's tensors current, and the stream that it runs on, so
    that what is allocated meanwhile belongs to that stream; gives the raw stream."""

    def __init__(self, index: int, stream):
        _require(stream is None or stream.device_index == index, "stream of another device than the tensors'")
        self.index = index
        self.device = None if _current_device() == index else torch.cuda.device(index)
        self.stream = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self) -> int:
        if self.device is not None:
            self.device.__enter__()
        if self.stream is not None:
            self.stream.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        if self.stream is not None:
            self.stream.__exit__(*exc)
        if self.device is not None:
            self.device.__exit__(*exc)


def _strides_of(t: torch.Tensor):
    """focus_strides of a [B, N, H, d] tensor, None where it is dense."""
    return None if t.is_contiguous() else ctypes.byref(_Strides(*t.stride()[:3]))


def _rope_call(what, rope_plan, q, k, positions, offset, out, out_k, inverse, stream):
    _require(positions is None or offset == 0, "positions and offset given together")
    dev, dtype = q.get_device(), q.dtype
    code = _ROPE_DTYPES.get(dtype)
    _require(dev >= 0 and code is not None and q.dim() == 4 and q.stride(3) == 1, what)
    B, N, H, d = q.shape
    H_kv = kp = ks = pos = kop = kos = None
    if k is not None:
        _require(k.get_device() == dev and k.dtype is dtype and k.dim() == 4 and k.stride(3) == 1, what)
        kB, kN, H_kv, kd = k.shape
        _require(kB == B and kN == N and kd == d, what)
        kp, ks = k.data_ptr(), _strides_of(k)
    if positions is not None:
        pos = _vector(positions, (B, N), dev, what)
    with _Launch(dev, stream) as s:
        qs = qos = _strides_of(q)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            qos = None
        elif out is not q:
            _require(out.shape == q.shape and out.dtype is dtype and out.get_device() == dev and
                     out.stride(3) == 1, what)
            qos = _strides_of(out)
        if k is not None:
            kos = ks
            if out_k is None:
                out_k = torch.empty_like(k, memory_format=torch.contiguous_format)
                kos = None
            elif out_k is not k:
                _require(out_k.shape == k.shape and out_k.dtype is dtype and out_k.get_device() == dev and
                         out_k.stride(3) == 1, what)
                kos = _strides_of(out_k)
            kop = out_k.data_ptr()
        if B and N:
            _check(_lib.focus_rope_apply(rope_plan._addr, code, B, N, H, H_kv or 0, d, q.data_ptr(), qs, kp, ks, pos,
                                         offset, inverse, out.data_ptr(), qos, kop, kos, s), what)
    return out if k is None else (out, out_k)


def rope(plan: Rope, q: torch.Tensor, k: torch.Tensor | None = None, *, positions=None, offset: int = 0,
         out=None, out_k=None, stream=None):
    """Rotary positions of q [B, N, H, d] and, in the same launch, k [B, N, H_kv, d] (bf16,
    fp16 or fp32; strided views with consecutive columns are fine).  Token n stands at
    offset + n, or at positions[b, n] (int32; not both).  out / out_k may be q / k themselves.
    An input may be a broadcast view, an output not.  Returns the rotated q, or (q, k)."""
    return _rope_call("focus_rope_apply", plan, q, k, positions, offset, out, out_k, 0, stream)


def rope_bwd(plan: Rope, dq: torch.Tensor, dk: torch.Tensor | None = None, *, positions=None, offset: int = 0,
             out=None, out_k=None, stream=None):
    """Backward of rope(): gradients of its inputs from those of its outputs (e.g. from
    attn_bwd), with the forward's plan and positions."""
    return _rope_call("focus_rope_apply", plan, dq, dk, positions, offset, out, out_k, 1, stream)


# ------------------------------------------------------------------ key/value cache ----
@dataclasses.dataclass(frozen=True)
class CacheParams:
    """A key/value cache and the attention over it (focus_cache_params): B sequences of
    `cap` token slots, format "bf16", "e4m3" or "int8".  K, top_k: groups and groups per
    token, as routed (they balance the work of decode_tree)."""
    B: int
    cap: int
    H: int
    H_kv: int
    d_head: int
    R: int
    K: int
    top_k: int
    w: int
    format: str = "bf16"
    softmax_scale: float = 0.0

    def __post_init__(self):
        _require(self.format in CACHE_FORMATS, "focus_cache_params")
        object.__setattr__(self, "_by_tokens", {})

    def c(self, T: int) -> _CacheParams:
        """focus_cache_params for T tokens, with its address and decode_tree's workspace size;
        kept, since a program calls with few different T for every token that it makes."""
        c = self._by_tokens.get(T)
        if c is None:
            c = _CacheParams(self.B, self.cap, T, self.H, self.H_kv, self.d_head, self.R, self.K, self.top_k, self.w,
                             CACHE_FORMATS[self.format], self.softmax_scale)
            c.shared_ws = {}
            c.tree_ws = int(_lib.focus_decode_tree_workspace_size(c.addr))
            if len(self._by_tokens) < 4096:
                self._by_tokens[T] = c
        return c

    def __reduce__(self):
        return _made_anew(self)

    @property
    def scale(self) -> float:
        return self.softmax_scale if self.softmax_scale > 0 else 1.0 / math.sqrt(self.d_head)


@dataclasses.dataclass
class KVCache:
    """The tensors of a cache: k, v [B, cap, H_kv, d] (bfloat16, float8_e4m3fn or int8),
    k_scale, v_scale [B, H_kv, cap] fp32 (None for bf16), mask [B, R, cap] int32."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None
    v_scale: torch.Tensor | None
    mask: torch.Tensor

    @classmethod
    def empty(cls, p: CacheParams, device="cuda") -> "KVCache":
        """A cache of zeros."""
        kv = [torch.zeros(p.B, p.cap, p.H_kv, p.d_head, dtype=torch.uint8 if p.format != "bf16" else torch.bfloat16,
                          device=device).view(_CACHE_DTYPES[p.format]) for _ in range(2)]
        sc = [None if p.format == "bf16" else torch.zeros(p.B, p.H_kv, p.cap, device=device) for _ in range(2)]
        return cls(*kv, *sc, torch.zeros(p.B, p.R, p.cap, dtype=torch.int32, device=device))

    def _args(self, p: CacheParams, what: str, size=None):
        """The device's index, and the addresses of k, v, their scales and the masks.  size:
        (sequences, slots) of a cache that has others than p."""
        k, v, mask, ks, vs = self.k, self.v, self.mask, self.k_scale, self.v_scale
        B, cap = size or (p.B, p.cap)
        dev, dtype, shape = k.get_device(), _CACHE_DTYPES.get(p.format), (B, cap, p.H_kv, p.d_head)
        _require(dev >= 0 and k.dtype is dtype and k.shape == shape and k.is_contiguous() and
                 v.get_device() == dev and v.dtype is dtype and v.shape == shape and v.is_contiguous(), what)
        if p.format == "bf16":
            _require(ks is None and vs is None, what)
            return dev, k.data_ptr(), v.data_ptr(), None, None, _vector(mask, (B, p.R, cap), dev, what)
        shape = (B, p.H_kv, cap)
        _require(ks is not None and vs is not None, what)
        return (dev, k.data_ptr(), v.data_ptr(), _vector(ks, shape, dev, what, torch.float32),
                _vector(vs, shape, dev, what, torch.float32), _vector(mask, (B, p.R, cap), dev, what))


def _vector(t, shape, dev: int, what: str, dtype=torch.int32):
    """The address of an optional dense tensor of the given device, shape and type."""
    if t is None:
        return None
    _require(t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous(), what)
    return t.data_ptr()


def cache_write(p: CacheParams, cache: KVCache, k: torch.Tensor, v: torch.Tensor, mask, start: torch.Tensor,
                count=None, *, rope: Rope | None = None, positions=None, status=None, stream=None) -> KVCache:
    """Append tokens to the cache: k, v [B, T, H_kv, d] bf16 (token strides free, 16-byte
    aligned rows), mask [B, R, T] int32 (e.g. from route) or None to leave the cache's masks;
    token t < count[b] goes to slot start[b] + t (int32 device tensors; count None: all T),
    its key rotated by `rope` at positions[b, t], or at its slot.  status: an int32 device
    word that get_status reads (FOCUS_ERR_BOUNDS when a token had no slot).  A tree's accepted
    path is committed by tree_accept, or by writing its tokens again from start on, in order.  k and
    v are no views of the cache."""
    what = "focus_cache_write"
    dev, kc, vc, ksc, vsc, mc = cache._args(p, what)
    _require(k.dim() == 4 and start is not None, what)
    T = k.shape[1]
    for x in (k, v):
        _require(x.get_device() == dev and x.dtype is torch.bfloat16 and x.shape == (p.B, T, p.H_kv, p.d_head) and
                 x.stride(3) == 1, what)
    if T == 0:
        return cache
    c = p.c(T)
    with _Launch(dev, stream) as s:
        _check(_lib.focus_cache_write(
            c.addr, k.data_ptr(), _strides_of(k), v.data_ptr(), _strides_of(v),
            _vector(mask, (p.B, p.R, T), dev, what), _vector(start, (p.B,), dev, what),
            _vector(count, (p.B,), dev, what), None if rope is None else rope._addr,
            _vector(positions, (p.B, T), dev, what), kc, vc, ksc, vsc, mc, _vector(status, (1,), dev, what), s), what)
    return cache


def cache_read(p: CacheParams, cache: KVCache, T: int, start=None, count=None, *, out=None, status=None,
               stream=None):
    """k, v [B, T, H_kv, d] bf16 of the tokens in slots start[b] + t (start None: 0), zeros
    for t >= count[b].  out: (k, v) to fill.  (attn_fwd takes as many queries as keys: a further
    prompt on a prefix read back needs queries for the prefix too, whose rows are left.)"""
    what = "focus_cache_read"
    dev, kc, vc, ksc, vsc, _ = cache._args(p, what)
    shape = (p.B, T, p.H_kv, p.d_head)
    with _Launch(dev, stream) as s:
        if out is None:
            at = cache.k.device
            k, v = torch.empty(shape, dtype=torch.bfloat16, device=at), torch.empty(shape, dtype=torch.bfloat16, device=at)
        else:
            k, v = out
            _vector(k, shape, dev, what, torch.bfloat16), _vector(v, shape, dev, what, torch.bfloat16)
        if T:
            c = p.c(T)
            _check(_lib.focus_cache_read(
                c.addr, kc, vc, ksc, vsc, _vector(start, (p.B,), dev, what),
                _vector(count, (p.B,), dev, what), k.data_ptr(), v.data_ptr(), _vector(status, (1,), dev, what), s), what)
    return k, v


def decode_tree_workspace_size(p: CacheParams, T: int) -> int:
    return p.c(T).tree_ws


def decode_tree(p: CacheParams, q: torch.Tensor, cache: KVCache, lens: torch.Tensor, tree=None, *, out=None,
                lse=None, want_lse: bool = True, ws=None, status=None, stream=None):
    """Decode step for T <= MAX_DRAFT drafted tokens per sequence: q [B, T, H, d] bf16, lens [B]
    int32 tokens in the cache before them; the drafted tokens' own keys, values and masks stand
    in slots lens[b] + u.  tree [B, T] int64: bit u of word t set when drafted token u is an
    ancestor of t or t itself (None: a chain; a word of 0 marks a row that is no token).
    T = 1 is the plain next token of sequences of different lengths (decode: of bf16 sequences of
    one length).  ws: a workspace of
    decode_tree_workspace_size(p, T) bytes, of one call at a time; get_status(ws) reads the
    call's status (FOCUS_ERR_BOUNDS where a length does not fit: zeros and -inf; FOCUS_ERR_TIMEOUT:
    NaN).  status: an int32 device word, as in cache_write, that keeps the lowest code of all
    calls of one stream that it was given to; without ws and status a call's code is lost.
    Returns (o [B, T, H, d] bf16, lse [B, H, T] fp32)."""
    what = "focus_decode_tree"
    dev, kc, vc, ksc, vsc, mc = cache._args(p, what)
    _require(q.dim() == 4 and lens is not None, what)
    T = q.shape[1]
    shape = (p.B, T, p.H, p.d_head)
    qp = _vector(q, shape, dev, what, torch.bfloat16)
    c = p.c(T)
    if c.tree_ws == 0:
        raise FocusError(-2 if T > MAX_DRAFT else -1, "focus_decode_tree_workspace_size")
    with _Launch(dev, stream) as s:
        out = torch.empty_like(q) if out is None else out
        if lse is None and want_lse:
            lse = torch.empty((p.B, p.H, T), dtype=torch.float32, device=q.device)
        ws = torch.empty(c.tree_ws, dtype=torch.uint8, device=q.device) if ws is None else ws
        _require(ws.get_device() == dev and ws.is_contiguous(), what)
        _vector(status, (1,), dev, what)
        _check(_lib.focus_decode_tree(
            c.addr, qp, kc, vc, ksc, vsc, mc, _vector(lens, (p.B,), dev, what),
            _vector(tree, (p.B, T), dev, what, torch.int64), _vector(out, shape, dev, what, torch.bfloat16),
            _vector(lse, (p.B, p.H, T), dev, what, torch.float32), ws.data_ptr(), ws.nbytes, s), what)
        if status is not None:
            torch.minimum(status, ws.view(-1).view(torch.uint8)[:4].view(torch.int32), out=status)
    return out, lse


def decode_shared_workspace_size(p: CacheParams, T: int, prefix_len: int) -> int:
    return int(_lib.focus_decode_shared_workspace_size(p.c(T).addr, prefix_len))


def decode_shared(p: CacheParams, q: torch.Tensor, prefix: KVCache, prefix_len: int, cache: KVCache, lens: torch.Tensor,
                  tree=None, *, out=None, lse=None, want_lse: bool = True, ws=None, status=None, stream=None):
    """decode_tree for a batch whose sequences share a prefix, held and read once: prefix is a cache
    of one sequence (B = 1, any capacity) in p's format with prefix_len tokens, p and cache are the
    sequences' own.  Slot j of a sequence's own cache is position prefix_len + j (write it with
    cache_write's positions), token t stands at prefix_len + lens[b] + depth.  All else as in
    decode_tree; ws: decode_shared_workspace_size(p, T, prefix_len) bytes.
    Returns (o [B, T, H, d] bf16, lse [B, H, T] fp32)."""
    what = "focus_decode_shared"
    dev, kc, vc, ksc, vsc, mc = cache._args(p, what)
    _require(q.dim() == 4 and lens is not None and prefix.k.dim() == 4, what)
    T, prefix_cap = q.shape[1], prefix.k.shape[1]
    pdev, pk, pv, pks, pvs, pm = prefix._args(p, what, (1, prefix_cap))
    shape = (p.B, T, p.H, p.d_head)
    qp = _vector(q, shape, dev, what, torch.bfloat16)
    c = p.c(T)
    if c.tree_ws == 0:
        raise FocusError(-2 if T > MAX_DRAFT else -1, "focus_decode_shared_workspace_size")
    _require(pdev == dev and 0 <= prefix_len <= prefix_cap, what)
    need = c.shared_ws.get(prefix_len)
    if need is None:
        need = c.shared_ws[prefix_len] = int(_lib.focus_decode_shared_workspace_size(c.addr, prefix_len))
        if len(c.shared_ws) > 64:
            c.shared_ws = {}
    with _Launch(dev, stream) as s:
        out = torch.empty_like(q) if out is None else out
        if lse is None and want_lse:
            lse = torch.empty((p.B, p.H, T), dtype=torch.float32, device=q.device)
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if ws is None else ws
        _require(ws.get_device() == dev and ws.is_contiguous(), what)
        _vector(status, (1,), dev, what)
        _check(_lib.focus_decode_shared(
            c.addr, qp, prefix_cap, prefix_len, pk, pv, pks, pvs, pm, kc, vc, ksc, vsc, mc,
            _vector(lens, (p.B,), dev, what), _vector(tree, (p.B, T), dev, what, torch.int64),
            _vector(out, shape, dev, what, torch.bfloat16), _vector(lse, (p.B, p.H, T), dev, what, torch.float32),
            ws.data_ptr(), ws.nbytes, s), what)
        if status is not None:
            torch.minimum(status, ws.view(-1).view(torch.uint8)[:4].view(torch.int32), out=status)
    return out, lse


def tree_accept(p: CacheParams, cache: KVCache, lens: torch.Tensor, draft: torch.Tensor, chosen: torch.Tensor, tree=None, *,
                out_lens=None, status=None, stream=None):
    """The path of drafted tokens that the model's choices follow, taken into the cache: draft [B, T]
    int32 (token 0 the root, which the sequence has already), chosen [B, T] int32 the token chosen
    after each (e.g. by sample), tree as in decode_tree.  From the root on, the first child whose
    token is the one chosen is accepted (a negative token is none and never is).  The accepted tokens' rows move to slots lens[b] + i.
    out_lens: where the new lengths go (lens itself is fine).  status: an int32 device word, as in
    cache_write.  Returns int32 (count [B] of accepted tokens with the root, path [B, T] of their
    indices and then -1, next [B], the token chosen after the last, or -1, and the new lens [B])."""
    what = "focus_tree_accept"
    dev, kc, vc, ksc, vsc, mc = cache._args(p, what)
    _require(draft.dim() == 2 and lens is not None and chosen is not None, what)
    T = draft.shape[1]
    c = p.c(T)
    with _Launch(dev, stream) as s:
        # count, next, the new lens and the path, as parts of one tensor
        B = p.B
        parts = torch.empty(B * (3 + T), dtype=torch.int32, device=cache.k.device)
        at = parts.data_ptr()
        op = at + 8 * B if out_lens is None else _vector(out_lens, (B,), dev, what)
        _check(_lib.focus_tree_accept(
            c.addr, _vector(draft, (B, T), dev, what), _vector(chosen, (B, T), dev, what),
            _vector(tree, (B, T), dev, what, torch.int64), kc, vc, ksc, vsc, mc, _vector(lens, (B,), dev, what), op, at,
            at + 12 * B, at + 4 * B, _vector(status, (1,), dev, what), s), what)
    count, following, new, path = parts.split_with_sizes((B, B, B, B * T))
    return count, path.view(B, T), following, new if out_lens is None else out_lens


# -------------------------------------------------------------------------- sampling ----
class _SampleParams(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("stride", ctypes.c_int64), ("temperature", ctypes.c_double), ("top_p", ctypes.c_double),
                ("min_p", ctypes.c_double)]


MAX_VOCAB = 1 << 19


def sample(logits: torch.Tensor, u: torch.Tensor, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None,
           logprob=None, want_logprob: bool = True, status=None, stream=None):
    """One token for each row of logits [..., V] (bf16, fp16 or fp32; a matrix may have strided
    rows) from random numbers u [...] fp32 in [0, 1): of the top_k largest (0: all) the fewest
    with top_p of their weight, of these those with at least min_p of the largest's weight, drawn
    by the running sum of weights exp(logit / temperature) in the order of the vocabulary.
    temperature 0: the largest logit.  Each of the four is a number, or a tensor with one for each
    row (fp32; top_k int32).  status: an int32 device word that get_status reads
    (FOCUS_ERR_NONFINITE, FOCUS_ERR_INVALID_ARG for a row's own parameters; such a row's token is -1).
    Returns (token [...] int32, logprob [...] fp32 or None: the token's share of what was left)."""
    what = "focus_sample"
    dev, shape = logits.get_device(), u.shape
    code = _ROPE_DTYPES.get(logits.dtype)
    _require(dev >= 0 and code is not None and logits.dim() >= 1 and logits.shape[:-1] == shape, what)
    V, rows = logits.shape[-1], u.numel()
    if logits.dim() == 2:
        _require(V <= 1 or logits.stride(1) == 1, what)
        stride = logits.stride(0) if rows > 1 else V
    else:
        _require(logits.is_contiguous(), what)
        stride = V
    one, each = [], []
    for x, dtype in ((temperature, torch.float32), (top_p, torch.float32), (min_p, torch.float32), (top_k, torch.int32)):
        given = isinstance(x, torch.Tensor)
        each.append(_vector(x, shape, dev, what, dtype) if given else None)
        one.append(0 if given else x)
    with _Launch(dev, stream) as s:
        out = torch.empty(shape, dtype=torch.int32, device=logits.device) if out is None else out
        if logprob is None and want_logprob:
            logprob = torch.empty(shape, dtype=torch.float32, device=logits.device)
        tp, lp = _vector(out, shape, dev, what), _vector(logprob, shape, dev, what, torch.float32)
        up, sp = _vector(u, shape, dev, what, torch.float32), _vector(status, (1,), dev, what)
        if rows:
            c = _SampleParams(rows, V, code, min(max(int(one[3]), 0), 1 << 30), stride, one[0], one[1], one[2])
            _check(_lib.focus_sample(ctypes.addressof(c), logits.data_ptr(), up, each[0], each[3], each[1], each[2], tp, lp,
                                     sp, s), what)
    return out, logprob


def selftest_timeout(device="cuda", stream=None) -> int:
    """Run the device failure-path diagnostic; returns the status (-5 = FOCUS_ERR_TIMEOUT)."""
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=device)
    return _lib.focus_selftest_timeout(_ptr(ws), ws.numel(), _stream(stream))


def selftest_timeout_decode(device="cuda", stream=None) -> int:
    """The same for decode_tree's tensor-core kernel in its four forms (bf16 and 8 bits, up to 128
    and more rows per KV head): -5 where each raised FOCUS_ERR_TIMEOUT and left NaN in every row."""
    ws = torch.empty(16 << 20, dtype=torch.uint8, device=device)
    return _lib.focus_selftest_timeout_decode(_ptr(ws), ws.numel(), _stream(stream))


def selftest_timeout_shared(device="cuda", stream=None) -> int:
    """The same for decode_shared, with the arrival kept back in the prefix's kernel or in the own part's."""
    ws = torch.empty(16 << 20, dtype=torch.uint8, device=device)
    return _lib.focus_selftest_timeout_shared(_ptr(ws), ws.numel(), _stream(stream))


def get_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronise and read the device status word of the last call on `ws`."""
    return _lib.focus_get_status(_ptr(ws), _stream(stream))
