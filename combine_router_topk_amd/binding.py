"""ctypes binding of libmoe_route.so: one Python function per C entry point,
same names, same argument order (see include/moe_route.h).

Only argument marshalling happens here: torch tensors (device memory) become
pointers, the stream becomes torch's current HIP stream unless given, and
tensor sizes are checked against the problem so the library can never be
handed a buffer shorter than the shape it is told about. Every step of the
routing path runs in the HIP library; there is no fallback. If the library is
missing, or was built from sources other than those beside it (its
moe_build_id() differs from the digest of csrc/ and include/), importing this
module raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_route.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_F16, MOE_BF16 = 1, 2
MOE_FLAG_GREEDY_ID_ORDER = 1 << 0
MOE_FLAG_OUT_F32 = 1 << 1
MOE_FLAG_EXACT_SUMS = 1 << 2
MOE_MAX_E, MOE_MAX_K, MOE_MAX_R, MOE_MAX_REP = 1024, 16, 1024, 16
MOE_MAX_ROWS = (1 << 24) - 1
MOE_NOALLOC_SCRATCH_BYTES = 2 << 20
MOE_SCALE_BLOCK, MOE_MAX_NORM_H, MOE_MAX_FEW_TOKENS = 128, 16384, 64

EXPORTED = ("moe_version", "moe_build_id", "moe_status_string", "moe_last_error", "moe_workspace_bytes",
            "moe_route", "moe_assign_replicas", "moe_layout", "moe_route_assign_layout",
            "moe_route_assign_layout_noalloc", "moe_route_assign_layout_single_send",
            "moe_layout_single_send",
            "moe_single_send_dispatch", "moe_single_send_expand", "moe_dispatch",
            "moe_expert_standin", "moe_combine", "moe_combine_backward", "moe_dispatch_backward",
            "moe_routing_stats", "moe_token_balanced_split",
           "moe_rms_norm", "moe_rms_norm_workspace_bytes", "moe_rms_norm_backward",
           "moe_expert_gemm", "moe_expert_gemm_swiglu", "moe_layer_workspace_bytes",
           "moe_layer_few_tokens")

_TORCH_ACT = {MOE_F16: torch.float16, MOE_BF16: torch.bfloat16}
E4M3 = torch.float8_e4m3fn


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({_status_string(status)}): {detail}")


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("H", ctypes.c_int32), ("R", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]

    def __repr__(self):
        return (f"Problem(T={self.T}, E={self.E}, k={self.k}, H={self.H}, R={self.R}, "
                f"act_dtype={self.act_dtype}, flags={self.flags})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python combine_router_topk_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(Problem)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    sig = {
        "moe_version": (i32, []),
        "moe_build_id": (ctypes.c_char_p, []),
        "moe_status_string": (ctypes.c_char_p, [i32]),
        "moe_last_error": (ctypes.c_char_p, []),
        "moe_workspace_bytes": (i32, [P, ctypes.POINTER(sz)]),
        "moe_route": (i32, [P, vp, vp, vp, vp, vp, sz, vp]),
        "moe_assign_replicas": (i32, [P, vp, vp, i32, vp, vp, vp]),
        "moe_layout": (i32, [P, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_route_assign_layout": (i32, [P, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                          vp, vp, sz, vp]),
        "moe_route_assign_layout_noalloc": (i32, [P, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                                  vp, vp, vp, vp]),
        "moe_route_assign_layout_single_send": (i32, [P, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                                      vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_layout_single_send": (i32, [P, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                         vp, sz, vp]),
        "moe_single_send_dispatch": (i32, [P, vp, vp, vp, i32, vp]),
        "moe_single_send_expand": (i32, [P, vp, vp, vp, vp, vp, i32, vp, vp]),
        "moe_dispatch": (i32, [P, vp, vp, vp, vp]),
        "moe_expert_standin": (i32, [P, vp, vp, vp, vp, vp]),
        "moe_combine": (i32, [P, vp, vp, vp, vp, vp]),
        "moe_combine_backward": (i32, [P, vp, vp, vp, vp, vp, vp, vp]),
        "moe_dispatch_backward": (i32, [P, vp, vp, vp, vp]),
        "moe_routing_stats": (i32, [P, vp, vp, vp, vp, vp, vp, vp]),
        "moe_token_balanced_split": (i32, [P, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp]),
        "moe_rms_norm": (i32, [P, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp, vp]),
        "moe_rms_norm_workspace_bytes": (i32, [P, ctypes.POINTER(sz)]),
        "moe_rms_norm_backward": (i32, [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_expert_gemm": (i32, [P, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_gemm_swiglu": (i32, [P, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_layer_workspace_bytes": (i32, [P, i32, ctypes.POINTER(sz)]),
        "moe_layer_few_tokens": (i32, [P, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    built, want = lib.moe_build_id().decode(), _build.source_digest()
    if built != want:
        raise ImportError(f"{LIB_PATH} was built from other sources (build id {built}, sources "
                          f"{want}); rebuild with `python combine_router_topk_amd/build.py`")
    return lib


_lib = _load()


def _status_string(status: int) -> str:
    return _lib.moe_status_string(status).decode()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where, _lib.moe_last_error().decode())


def make_problem(T: int, E: int, k: int, H: int, R: int, act_dtype: int, flags: int = 0) -> Problem:
    return Problem(T, E, k, H, R, act_dtype, flags)


def _ptr(t: torch.Tensor | None, dtype: torch.dtype | None, numel: int | None, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, need {numel}")
    return ctypes.c_void_p(t.data_ptr())


def _nbytes(t: torch.Tensor | None) -> int:
    """Byte size of a workspace tensor; 0 for None (the library then reports
    the NULL pointer)."""
    return 0 if t is None else t.numel() * t.element_size()


def _rows(t: torch.Tensor | None) -> int:
    """Row count of a single-send buffer (its capacity); 0 for None."""
    return 0 if t is None else t.shape[0]


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def moe_version() -> int:
    return _lib.moe_version()


def moe_build_id() -> str:
    return _lib.moe_build_id().decode()


def moe_status_string(status: int) -> str:
    return _status_string(status)


def moe_last_error() -> str:
    return _lib.moe_last_error().decode()


def moe_workspace_bytes(p: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_workspace_bytes(ctypes.byref(p), ctypes.byref(n)), "moe_workspace_bytes")
    return n.value


def moe_route(p: Problem, logits, idx, w, counts, ws, stream=None) -> None:
    n = p.T * p.k
    _check(_lib.moe_route(ctypes.byref(p),
                          _ptr(logits, torch.float32, p.T * p.E, "logits"),
                          _ptr(idx, torch.int32, n, "idx"), _ptr(w, torch.float32, n, "w"),
                          _ptr(counts, torch.int32, p.E, "counts"), _ptr(ws, None, None, "ws"),
                          _nbytes(ws), _stream(stream)), "moe_route")


def moe_assign_replicas(p: Problem, counts, rep, maxrep: int, assign, active, stream=None) -> None:
    _check(_lib.moe_assign_replicas(ctypes.byref(p), _ptr(counts, torch.int32, p.E, "counts"),
                                    _ptr(rep, torch.int32, p.E * maxrep if rep is not None else 0, "rep"),
                                    maxrep, _ptr(assign, torch.int32, p.E, "assign"),
                                    _ptr(active, torch.int32, p.R, "active"), _stream(stream)),
           "moe_assign_replicas")


def moe_layout(p: Problem, idx, assign, rep, maxrep: int, rank_of, expert_offsets, rank_offsets,
               pos, src, dedup, ws, stream=None) -> None:
    n = p.T * p.k
    _check(_lib.moe_layout(ctypes.byref(p), _ptr(idx, torch.int32, n, "idx"),
                           _ptr(assign, torch.int32, p.E, "assign"),
                           _ptr(rep, torch.int32, p.E * maxrep if rep is not None else 0, "rep"),
                           maxrep, _ptr(rank_of, torch.int32, p.E, "rank_of"),
                           _ptr(expert_offsets, torch.int32, p.E, "expert_offsets"),
                           _ptr(rank_offsets, torch.int32, p.R + 1, "rank_offsets"),
                           _ptr(pos, torch.int32, n, "pos"), _ptr(src, torch.int32, n, "src"),
                           _ptr(dedup, torch.int32, p.R, "dedup"), _ptr(ws, None, None, "ws"),
                           _nbytes(ws), _stream(stream)), "moe_layout")


def moe_route_assign_layout(p: Problem, logits, rep, maxrep: int, idx, w, counts, assign, active,
                            rank_of, expert_offsets, rank_offsets, pos, src, dedup, ws,
                            stream=None) -> None:
    n = p.T * p.k
    _check(_lib.moe_route_assign_layout(
        ctypes.byref(p), _ptr(logits, torch.float32, p.T * p.E, "logits"),
        _ptr(rep, torch.int32, p.E * maxrep if rep is not None else 0, "rep"), maxrep,
        _ptr(idx, torch.int32, n, "idx"), _ptr(w, torch.float32, n, "w"),
        _ptr(counts, torch.int32, p.E, "counts"), _ptr(assign, torch.int32, p.E, "assign"),
        _ptr(active, torch.int32, p.R, "active"), _ptr(rank_of, torch.int32, p.E, "rank_of"),
        _ptr(expert_offsets, torch.int32, p.E, "expert_offsets"),
        _ptr(rank_offsets, torch.int32, p.R + 1, "rank_offsets"),
        _ptr(pos, torch.int32, n, "pos"), _ptr(src, torch.int32, n, "src"),
        _ptr(dedup, torch.int32, p.R, "dedup"), _ptr(ws, None, None, "ws"), _nbytes(ws),
        _stream(stream)), "moe_route_assign_layout")


def moe_route_assign_layout_single_send(p: Problem, logits, rep, maxrep: int, idx, w, counts,
                                        assign, active, rank_of, expert_offsets, rank_offsets,
                                        pos, src, dedup, ss_rank_offsets, ss_row, ss_token, ws,
                                        stream=None) -> None:
    n = p.T * p.k
    _check(_lib.moe_route_assign_layout_single_send(
        ctypes.byref(p), _ptr(logits, torch.float32, p.T * p.E, "logits"),
        _ptr(rep, torch.int32, p.E * maxrep if rep is not None else 0, "rep"), maxrep,
        _ptr(idx, torch.int32, n, "idx"), _ptr(w, torch.float32, n, "w"),
        _ptr(counts, torch.int32, p.E, "counts"), _ptr(assign, torch.int32, p.E, "assign"),
        _ptr(active, torch.int32, p.R, "active"), _ptr(rank_of, torch.int32, p.E, "rank_of"),
        _ptr(expert_offsets, torch.int32, p.E, "expert_offsets"),
        _ptr(rank_offsets, torch.int32, p.R + 1, "rank_offsets"),
        _ptr(pos, torch.int32, n, "pos"), _ptr(src, torch.int32, n, "src"),
        _ptr(dedup, torch.int32, p.R, "dedup"),
        _ptr(ss_rank_offsets, torch.int32, p.R + 1, "ss_rank_offsets"),
        _ptr(ss_row, torch.int32, n, "ss_row"), _ptr(ss_token, torch.int32, n, "ss_token"),
        _ptr(ws, None, None, "ws"), _nbytes(ws), _stream(stream)),
        "moe_route_assign_layout_single_send")


def moe_route_assign_layout_noalloc(p: Problem, logits, rep, maxrep: int, idx, w, counts, assign,
                                    active, rank_of, expert_offsets, rank_offsets, pos, src, dedup,
                                    stream=None) -> None:
    n = p.T * p.k
    _check(_lib.moe_route_assign_layout_noalloc(
        ctypes.byref(p), _ptr(logits, torch.float32, p.T * p.E, "logits"),
        _ptr(rep, torch.int32, p.E * maxrep if rep is not None else 0, "rep"), maxrep,
        _ptr(idx, torch.int32, n, "idx"), _ptr(w, torch.float32, n, "w"),
        _ptr(counts, torch.int32, p.E, "counts"), _ptr(assign, torch.int32, p.E, "assign"),
        _ptr(active, torch.int32, p.R, "active"), _ptr(rank_of, torch.int32, p.E, "rank_of"),
        _ptr(expert_offsets, torch.int32, p.E, "expert_offsets"),
        _ptr(rank_offsets, torch.int32, p.R + 1, "rank_offsets"),
        _ptr(pos, torch.int32, n, "pos"), _ptr(src, torch.int32, n, "src"),
        _ptr(dedup, torch.int32, p.R, "dedup"), _stream(stream)),
        "moe_route_assign_layout_noalloc")


def moe_layout_single_send(p: Problem, idx, assign, rep, maxrep: int, rank_of, expert_offsets,
                           rank_offsets, pos, src, dedup, ss_rank_offsets, ss_row, ss_token, ws,
                           stream=None) -> None:
    n = p.T * p.k
    _check(_lib.moe_layout_single_send(
        ctypes.byref(p), _ptr(idx, torch.int32, n, "idx"), _ptr(assign, torch.int32, p.E, "assign"),
        _ptr(rep, torch.int32, p.E * maxrep if rep is not None else 0, "rep"), maxrep,
        _ptr(rank_of, torch.int32, p.E, "rank_of"),
        _ptr(expert_offsets, torch.int32, p.E, "expert_offsets"),
        _ptr(rank_offsets, torch.int32, p.R + 1, "rank_offsets"),
        _ptr(pos, torch.int32, n, "pos"), _ptr(src, torch.int32, n, "src"),
        _ptr(dedup, torch.int32, p.R, "dedup"),
        _ptr(ss_rank_offsets, torch.int32, p.R + 1, "ss_rank_offsets"),
        _ptr(ss_row, torch.int32, n, "ss_row"), _ptr(ss_token, torch.int32, n, "ss_token"),
        _ptr(ws, None, None, "ws"), _nbytes(ws), _stream(stream)),
        "moe_layout_single_send")


def moe_single_send_dispatch(p: Problem, x, ss_row, send_ss, stream=None) -> None:
    """send_ss holds the single-send rows; its row count is the capacity."""
    act = _TORCH_ACT.get(p.act_dtype)
    cap = _rows(send_ss)
    _check(_lib.moe_single_send_dispatch(ctypes.byref(p), _ptr(x, act, p.T * p.H, "x"),
                                         _ptr(ss_row, torch.int32, p.T * p.k, "ss_row"),
                                         _ptr(send_ss, act, cap * p.H, "send_ss"), cap,
                                         _stream(stream)), "moe_single_send_dispatch")


def moe_single_send_expand(p: Problem, send_ss, ss_rank_offsets, ss_token, ss_row, pos, send,
                           stream=None) -> None:
    """send_ss holds the single-send rows; its row count is the capacity."""
    act = _TORCH_ACT.get(p.act_dtype)
    n = p.T * p.k
    cap = _rows(send_ss)
    _check(_lib.moe_single_send_expand(ctypes.byref(p), _ptr(send_ss, act, cap * p.H, "send_ss"),
                                       _ptr(ss_rank_offsets, torch.int32, p.R + 1, "ss_rank_offsets"),
                                       _ptr(ss_token, torch.int32, min(cap, n), "ss_token"),
                                       _ptr(ss_row, torch.int32, n, "ss_row"),
                                       _ptr(pos, torch.int32, n, "pos"), cap,
                                       _ptr(send, act, n * p.H, "send"), _stream(stream)),
           "moe_single_send_expand")


def moe_dispatch(p: Problem, x, pos, send, stream=None) -> None:
    act = _TORCH_ACT.get(p.act_dtype)
    _check(_lib.moe_dispatch(ctypes.byref(p), _ptr(x, act, p.T * p.H, "x"),
                             _ptr(pos, torch.int32, p.T * p.k, "pos"),
                             _ptr(send, act, p.T * p.k * p.H, "send"), _stream(stream)),
           "moe_dispatch")


def moe_expert_standin(p: Problem, send, src, idx, y, stream=None) -> None:
    act = _TORCH_ACT.get(p.act_dtype)
    n = p.T * p.k
    _check(_lib.moe_expert_standin(ctypes.byref(p), _ptr(send, act, n * p.H, "send"),
                                   _ptr(src, torch.int32, n, "src"), _ptr(idx, torch.int32, n, "idx"),
                                   _ptr(y, act, n * p.H, "y"), _stream(stream)),
           "moe_expert_standin")


def moe_combine(p: Problem, y, pos, w, out, stream=None) -> None:
    act = _TORCH_ACT.get(p.act_dtype)
    out_dt = torch.float32 if p.flags & MOE_FLAG_OUT_F32 else act
    n = p.T * p.k
    _check(_lib.moe_combine(ctypes.byref(p), _ptr(y, act, n * p.H, "y"),
                            _ptr(pos, torch.int32, n, "pos"), _ptr(w, torch.float32, n, "w"),
                            _ptr(out, out_dt, p.T * p.H, "out"), _stream(stream)), "moe_combine")


def moe_combine_backward(p: Problem, dout, y, pos, w, dy, dw, stream=None) -> None:
    """dy and/or dw (either may be None); y may be None without dw and w
    without dy."""
    act = _TORCH_ACT.get(p.act_dtype)
    n = p.T * p.k
    _check(_lib.moe_combine_backward(ctypes.byref(p), _ptr(dout, act, p.T * p.H, "dout"),
                                     _ptr(y, act, n * p.H, "y"), _ptr(pos, torch.int32, n, "pos"),
                                     _ptr(w, torch.float32, n, "w"), _ptr(dy, act, n * p.H, "dy"),
                                     _ptr(dw, torch.float32, n, "dw"), _stream(stream)),
           "moe_combine_backward")


def moe_dispatch_backward(p: Problem, dsend, pos, dx, stream=None) -> None:
    act = _TORCH_ACT.get(p.act_dtype)
    out_dt = torch.float32 if p.flags & MOE_FLAG_OUT_F32 else act
    n = p.T * p.k
    _check(_lib.moe_dispatch_backward(ctypes.byref(p), _ptr(dsend, act, n * p.H, "dsend"),
                                      _ptr(pos, torch.int32, n, "pos"),
                                      _ptr(dx, out_dt, p.T * p.H, "dx"), _stream(stream)),
           "moe_dispatch_backward")


def moe_routing_stats(p: Problem, idx, counts, rank_of, send_counts, coselect, stats,
                      stream=None) -> None:
    """coselect may be None; stats is a float64 tensor of 4."""
    _check(_lib.moe_routing_stats(ctypes.byref(p), _ptr(idx, torch.int32, p.T * p.k, "idx"),
                                  _ptr(counts, torch.int32, p.E, "counts"),
                                  _ptr(rank_of, torch.int32, p.E, "rank_of"),
                                  _ptr(send_counts, torch.int32, p.R * p.R, "send_counts"),
                                  _ptr(coselect, torch.int32, p.E * p.E, "coselect"),
                                  _ptr(stats, torch.float64, 4, "stats"), _stream(stream)),
           "moe_routing_stats")


def moe_token_balanced_split(p: Problem, idx, counts, pos, expert_offsets, rep, maxrep: int,
                             gpu_of_pair, active, tokens, stream=None) -> None:
    n = p.T * p.k
    _check(_lib.moe_token_balanced_split(
        ctypes.byref(p), _ptr(idx, torch.int32, n, "idx"), _ptr(counts, torch.int32, p.E, "counts"),
        _ptr(pos, torch.int32, n, "pos"), _ptr(expert_offsets, torch.int32, p.E, "expert_offsets"),
        _ptr(rep, torch.int32, p.E * maxrep if rep is not None else 0, "rep"), maxrep,
        _ptr(gpu_of_pair, torch.int32, n, "gpu_of_pair"), _ptr(active, torch.int32, p.R, "active"),
        _ptr(tokens, torch.int32, p.R, "tokens"), _stream(stream)), "moe_token_balanced_split")


def scale_blocks(cols: int) -> int:
    """Scales of an 8-bit row of `cols` columns."""
    return -(-cols // MOE_SCALE_BLOCK)


class _Args:
    """Tensor arguments of one call: each checked as _ptr checks it, and that
    all live on one device."""
    __slots__ = ("name", "dev")

    def __init__(self, name: str):
        self.name, self.dev = name, None

    def __call__(self, t, dtype, numel, name):
        if t is None:
            return None
        dev = t.get_device() if isinstance(t, torch.Tensor) else -1
        if dev < 0 or not t.is_contiguous() or (dtype is not None and t.dtype is not dtype) \
                or (numel is not None and t.numel() < numel):
            _ptr(t, dtype, numel, name)  # raises
        if dev != self.dev:
            if self.dev is not None:
                raise ValueError(f"{self.name}: {name} is on device {dev}, others on {self.dev}")
            self.dev = dev
        return t.data_ptr()

    def call(self, f, stream, *args) -> None:
        """The library's function on the tensors' device, on that device's
        current stream unless one is given."""
        if self.dev is None or self.dev == torch.cuda.current_device():
            _check(f(*args, _raw_stream(stream, self.dev)), self.name)
        else:
            with torch.cuda.device(self.dev):
                _check(f(*args, _raw_stream(stream, self.dev)), self.name)


# The current stream's handle without a Stream object around it (2.9 us).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, dev) -> int:
    if stream is None:
        if _current_raw_stream is not None and dev is not None:
            return _current_raw_stream(dev)
        return torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def moe_rms_norm(p: Problem, x, residual, gamma, eps: float, h, y, q, q_scale, rstd, stream=None) -> None:
    """residual and h go together, q and q_scale too (None to leave them out);
    y may be None beside q, rstd too. q holds float8_e4m3fn."""
    act, T, H = _TORCH_ACT.get(p.act_dtype), p.T, p.H
    n, a = T * H, _Args("moe_rms_norm")
    a.call(_lib.moe_rms_norm, stream, ctypes.byref(p), a(x, act, n, "x"), a(residual, act, n, "residual"),
           a(gamma, act, H, "gamma"), eps, a(h, act, n, "h"), a(y, act, n, "y"), a(q, E4M3, n, "q"),
           a(q_scale, torch.float32, T * scale_blocks(H), "q_scale"), a(rstd, torch.float32, T, "rstd"))


def moe_rms_norm_workspace_bytes(p: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_rms_norm_workspace_bytes(ctypes.byref(p), ctypes.byref(n)),
           "moe_rms_norm_workspace_bytes")
    return n.value


def moe_rms_norm_backward(p: Problem, dy, dh, h, gamma, rstd, dx, dgamma, ws, stream=None) -> None:
    """dh may be None (no gradient along the residual stream)."""
    act, T, H = _TORCH_ACT.get(p.act_dtype), p.T, p.H
    n, a = T * H, _Args("moe_rms_norm_backward")
    a.call(_lib.moe_rms_norm_backward, stream, ctypes.byref(p), a(dy, act, n, "dy"), a(dh, act, n, "dh"),
           a(h, act, n, "h"), a(gamma, act, H, "gamma"), a(rstd, torch.float32, T, "rstd"), a(dx, act, n, "dx"),
           a(dgamma, torch.float32, H, "dgamma"), a(ws, None, None, "ws"), _nbytes(ws))


def _gemm_args(arg: _Args, p: Problem, K: int, rows: int, a, a_scale, src, w, w_scale, counts, expert_offsets):
    """The arguments that both experts' products share; `rows` of weights."""
    n, E = p.T * p.k, p.E
    a_rows = n if src is None else p.T
    nb = scale_blocks(K)
    return (arg(a, E4M3, a_rows * K, "a"), arg(a_scale, torch.float32, a_rows * nb, "a_scale"),
            arg(src, torch.int32, n, "src"), arg(w, E4M3, E * rows * K, "w"),
            arg(w_scale, torch.float32, E * scale_blocks(rows) * nb, "w_scale"),
            arg(counts, torch.int32, E, "counts"), arg(expert_offsets, torch.int32, E, "expert_offsets"))


def moe_expert_gemm(p: Problem, K: int, N: int, a, a_scale, src, w, w_scale, counts, expert_offsets,
                    y, stream=None) -> None:
    """src None: a holds the T k rows in send order; given: the T token rows."""
    out_dt = torch.float32 if p.flags & MOE_FLAG_OUT_F32 else _TORCH_ACT.get(p.act_dtype)
    arg = _Args("moe_expert_gemm")
    arg.call(_lib.moe_expert_gemm, stream, ctypes.byref(p), K, N,
             *_gemm_args(arg, p, K, N, a, a_scale, src, w, w_scale, counts, expert_offsets),
             arg(y, out_dt, p.T * p.k * N, "y"))


def moe_expert_gemm_swiglu(p: Problem, K: int, I: int, a, a_scale, src, w, w_scale, counts,
                           expert_offsets, q, q_scale, stream=None) -> None:
    """w holds 2 I rows an expert, the gate's first; src as in moe_expert_gemm."""
    n, arg = p.T * p.k, _Args("moe_expert_gemm_swiglu")
    arg.call(_lib.moe_expert_gemm_swiglu, stream, ctypes.byref(p), K, I,
             *_gemm_args(arg, p, K, 2 * I, a, a_scale, src, w, w_scale, counts, expert_offsets),
             arg(q, E4M3, n * I, "q"), arg(q_scale, torch.float32, n * scale_blocks(I), "q_scale"))


def moe_layer_workspace_bytes(p: Problem, I: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_layer_workspace_bytes(ctypes.byref(p), I, ctypes.byref(n)), "moe_layer_workspace_bytes")
    return n.value


def moe_layer_few_tokens(p: Problem, I: int, logits, x, w_up, s_up, w_down, s_down, idx, w, out, ws,
                         stream=None) -> None:
    """s_up and s_down None: weights in the activation format; given: e4m3."""
    act, T, E, H, n = _TORCH_ACT.get(p.act_dtype), p.T, p.E, p.H, p.T * p.k
    out_dt = torch.float32 if p.flags & MOE_FLAG_OUT_F32 else act
    f32, w_dt = torch.float32, act if s_up is None else E4M3
    nh, ni = scale_blocks(H), scale_blocks(I)
    a = _Args("moe_layer_few_tokens")
    a.call(_lib.moe_layer_few_tokens, stream, ctypes.byref(p), I, a(logits, f32, T * E, "logits"),
           a(x, act, T * H, "x"), a(w_up, w_dt, E * 2 * I * H, "w_up"),
           a(s_up, f32, E * scale_blocks(2 * I) * nh, "s_up"), a(w_down, w_dt, E * H * I, "w_down"),
           a(s_down, f32, E * nh * ni, "s_down"), a(idx, torch.int32, n, "idx"), a(w, f32, n, "w"),
           a(out, out_dt, T * H, "out"), a(ws, None, None, "ws"), _nbytes(ws))
