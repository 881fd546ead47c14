"""Python binding of libspecverify (ctypes): argument marshalling only.

Each function takes torch tensors that already live on the GPU, checks their
shapes and layouts, allocates the outputs, and calls the C entry point of the
same name on torch's current stream.  Every step of the computation runs in
the HIP kernels of libspecverify.so; if that library is not built, importing
this module fails.

Layout rules (the C ABI's): logit tensors are [..., V] with a unit stride
along V and evenly spaced rows whose start addresses are 16-byte aligned
(row stride * element size a multiple of 16).  dtype bfloat16 or float32.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# SV_LIBRARY selects another build of the library (the timeline build), by path
_LIB_PATH = os.environ.get("SV_LIBRARY") or os.path.join(_HERE, "libspecverify.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is not built; build it with `python -m lossless_draft_verification_04_amd.build` "
        "(hipcc, gfx950)")

_lib = ctypes.CDLL(_LIB_PATH)

SV_OK, SV_EINVAL, SV_EDTYPE, SV_EALIGN, SV_EWORKSPACE, SV_EUNSUPPORTED, SV_EHIP = range(7)
SV_F32, SV_BF16 = 0, 1
(SV_OP_CHAIN, SV_OP_GREEDY, SV_OP_MULTI, SV_OP_TREE, SV_OP_FANOUT, SV_OP_CHAIN_PM, SV_OP_TREE_PM,
 SV_OP_CACHE, SV_OP_PRESTO, SV_OP_BRANCH) = range(10)
DERR_TOKEN, DERR_TREE, DERR_FANOUT, DERR_ROW, DERR_TIMEOUT = 1, 2, 4, 8, 16
# the drafter's side (specverify_draft.h)
SV_DRAFT_TEACHER, SV_DRAFT_DISTILL, SV_DRAFT_BEAM, SV_DRAFT_REORDER = range(4)
DERR_RANGE = 32
# the verifier's pass (specverify_pass.h)
SV_F16 = 2
SV_PASS_ROPE, SV_PASS_WRITE, SV_PASS_READ, SV_PASS_ATTENTION, SV_PASS_COMMIT = range(5)
SV_ROPE_KINDS = {"plain": 0, "linear": 1, "base": 2, "parts": 3}

_P = ctypes.c_void_p
_i32, _i64, _u32, _u64, _f32, _f64, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64,
                                           ctypes.c_float, ctypes.c_double, ctypes.c_size_t)

_SIGS = {
    "sv_version": ([], _i32),
    "sv_status_string": ([_i32], ctypes.c_char_p),
    "sv_workspace_size": ([_i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_sz)], _i32),
    "sv_workspace_init": ([_P, _sz, _P], _i32),
    "sv_get_device_error": ([_P, ctypes.POINTER(_i32), _P], _i32),
    "sv_verify_chain": ([_P, _P, _i32, _i64, _i64, _P, _i32, _i32, _i32, _f32, _u64, _u32, _P, _P, _P, _P, _P,
                         _sz, _P], _i32),
    "sv_verify_greedy": ([_P, _i32, _i64, _P, _i32, _i32, _i32, _P, _P, _P, _P, _sz, _P], _i32),
    "sv_verify_multi": ([_P, _P, _i32, _i64, _i64, _P, _i32, _i32, _i32, _i32, _f32, _u64, _u32, _P, _P, _P, _P,
                         _P, _P, _P, _sz, _P], _i32),
    "sv_verify_tree": ([_P, _P, _i32, _i64, _i64, _P, _P, _i32, _i32, _i32, _i32, _f32, _u64, _u32, _P, _P, _P,
                        _P, _P, _P, _sz, _P], _i32),
    "sv_verify_chain_noalloc": ([_P, _P, _i32, _i64, _i64, _P, _i32, _i32, _i32, _f32, _u64, _u32, _P, _P, _P, _P,
                                 _P, _P], _i32),
    "sv_verify_chain_pm": ([_P, _i32, _i64, _P, _i32, _i32, _i32, _f32, _u64, _u32, _P, _P, _P, _P, _sz, _P], _i32),
    "sv_verify_tree_pm": ([_P, _i32, _i64, _P, _P, _i32, _i32, _i32, _i32, _f32, _u64, _u32, _P, _P, _P, _P, _P,
                           _sz, _P], _i32),
    "sv_fanout_topk": ([_P, _i32, _i64, _i32, _i32, _P, _i32, _P, _P, _P, _sz, _P], _i32),
    "sv_cache_hit_test": ([_P, _i32, _i64, _i32, _i32, _i32, _P, _P, _P, _P, _P, _P, _sz, _P], _i32),
    "sv_presto_score": ([_P, _P, _i32, _i64, _i64, _P, _P, _i32, _i32, _i32, _f32, _P, _i32, _i32, _i32, _P, _P,
                         _P, _P, _P, _P, _sz, _P], _i32),
    "sv_branch_fork": ([_P, _i32, _i64, _P, _P, _i32, _i32, _i32, _f32, _f32, _i32, _P, _P, _P, _P, _P, _sz, _P],
                       _i32),
    "sv_geometric_fanout": ([_i32, _f64, _f64, _i32, _i32, ctypes.POINTER(_i32)], _i32),
    "sv_read_probe": ([_P, _sz, _i32, _i32, _i32, _sz, _P, _P], _i32),
    "sv_timeline_set": ([_P, ctypes.c_uint64], _i32),
}
# entry points of specverify_draft.h
_DRAFT_SIGS = {
    "sv_draft_workspace_size": ([_i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_sz)], _i32),
    "sv_teacher_topk": ([_P, _i32, _i64, _i32, _i32, _i32, _f32, _P, _P, _P, _P, _sz, _P], _i32),
    "sv_distill_topk": ([_P, _i32, _i64, _i32, _i32, _P, _P, _P, _i32, _f32, _P, _P, _P, _P, _i64, _P, _sz, _P],
                        _i32),
    "sv_distill_topk_backward": ([_P, _i32, _i64, _i32, _i32, _P, _P, _P, _i32, _f32, _P, _P, _P, _i64, _P, _sz, _P],
                                 _i32),
    "sv_beam_select": ([_P, _i32, _i64, _P, _P, _i32, _i32, _i32, _f32, _i32, _i32, _P, _P, _P, _P, _sz, _P], _i32),
    "sv_beam_reorder": ([_P, ctypes.POINTER(_i64), _P, ctypes.POINTER(_i64), _P, _P, _i32, _i32, _i32, _i32, _i32,
                         _i64, _i64, _P, _sz, _P], _i32),
}


class _CCache(ctypes.Structure):
    """sv_kv_cache"""
    _fields_ = [("pool", _P), ("pages", _P), ("page_stride", _i64), ("layer_stride", _i64), ("num_pages", _i32),
                ("max_pages", _i32), ("page_tokens", _i32), ("H", _i32), ("D", _i32), ("layers", _i32)]


# entry points of specverify_pass.h
_S, _C = ctypes.POINTER(_i64), ctypes.POINTER(_CCache)
_PASS_SIGS = {
    "sv_kv_page_bytes": ([_i32, _i32, _i32, _S], _i32),
    "sv_pass_workspace_size": ([_i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_sz)], _i32),
    "sv_rope": ([_P, _S, _P, _S, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _P, _f32, _i32, _i32, _P, _P, _P, _P, _S, _P, _S,
                 _P, _sz, _P], _i32),
    "sv_rope_frequencies": ([_i32, _i32, _f64, _f64, _i32, _f64, _f64, ctypes.POINTER(_f64), ctypes.POINTER(_f32)], _i32),
    "sv_kv_write": ([_P, _S, _P, _S, _i32, _C, _P, _P, _i32, _i32, _P, _sz, _P], _i32),
    "sv_kv_read": ([_C, _P, _P, _i32, _i32, _i32, _P, _S, _P, _S, _P, _sz, _P], _i32),
    "sv_kv_attention": ([_P, _S, _i32, _C, _P, _P, _P, _i32, _i32, _i32, _f32, _f32, _P, _i32, _P, _S, _P, _P, _sz, _P],
                        _i32),
    "sv_kv_commit": ([_C, _P, _P, _P, _i32, _i32, _P, _P, _sz, _P], _i32),
}
for _name, (_args, _res) in (*_SIGS.items(), *_DRAFT_SIGS.items(), *_PASS_SIGS.items()):
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_SIGS)
DRAFT_EXPORTED = tuple(_DRAFT_SIGS)
PASS_EXPORTED = tuple(_PASS_SIGS)


class SpecVerifyError(RuntimeError):
    def __init__(self, status, what):
        super().__init__(f"{what}: {_lib.sv_status_string(status).decode()} (status {status})")
        self.status = status


def _check(status, what):
    if status != SV_OK:
        raise SpecVerifyError(status, what)


class DeviceError(RuntimeError):
    """Device-side input error bits (DERR_*) reported by a call in checked mode."""

    def __init__(self, flags, what):
        names = [n for n, b in (("token", DERR_TOKEN), ("tree", DERR_TREE), ("fanout", DERR_FANOUT),
                                ("row", DERR_ROW), ("timeout", DERR_TIMEOUT),
                                ("range", DERR_RANGE)) if flags & b]
        super().__init__(f"{what}: device error word {flags} ({', '.join(names)}); outputs of the call are invalid")
        self.flags = flags


_CHECKED = False


def set_checked(on: bool = True) -> None:
    """Checked mode: after every call, synchronise its stream and raise DeviceError if the workspace's device
    error word is set (and clear it).  Off by default: a call is then asynchronous and the word is read only
    through sv_get_device_error."""
    global _CHECKED
    _CHECKED = bool(on)


def _checked(device, what, workspace=None):
    if not _CHECKED:
        return
    ws = workspace if workspace is not None else Workspace.get(device, 0)
    flags = _i32(0)
    _check(_lib.sv_get_device_error(_ptr(ws), ctypes.byref(flags), _stream(device)), "sv_get_device_error")
    if flags.value:
        raise DeviceError(flags.value, what)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise SpecVerifyError(SV_EDTYPE, f"logits dtype {t.dtype}")


def _row_stride(t: torch.Tensor, what: str) -> int:
    """Row stride (elements) of a [..., V] logit tensor with evenly spaced rows."""
    if t.stride(-1) != 1:
        raise SpecVerifyError(SV_EINVAL, f"{what}: vocabulary axis must have unit stride")
    if t.dim() < 2:
        return t.shape[-1]
    rs = t.stride(-2)
    step = rs
    for ax in range(t.dim() - 2, 0, -1):
        step *= t.shape[ax]
        if t.shape[ax - 1] > 1 and t.stride(ax - 1) != step:
            raise SpecVerifyError(SV_EINVAL, f"{what}: rows must be evenly spaced")
    return rs


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _i32_tensor(t: torch.Tensor, shape, what):
    if t.dtype != torch.int32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise SpecVerifyError(SV_EINVAL, f"{what}: want contiguous int32 {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t


def _capturing(index) -> bool:
    """Whether the device's current stream is being captured into a graph."""
    if index == torch.cuda.current_device():
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(index):
        return torch.cuda.is_current_stream_capturing()


class Workspace:
    """Per-device scratch for the kernels (zero-filled on creation, grown on demand).

    A buffer that a larger one replaces is kept: graphs captured with it go on using it, and calls of other streams may
    still be running in it.  Sizes double, so that the replaced ones together take less than the one in use.  A buffer
    made while a graph is being captured lies in the graph's memory and its zero fill runs with the graph, so it serves
    that one call and is never handed to another; its error word means something once the graph has run."""

    _lock = threading.Lock()
    _cache = {}
    _replaced = {}  # by device: buffers replaced, and those of captured calls

    @classmethod
    def get(cls, device, nbytes: int, in_capture=True) -> torch.Tensor:
        """The device's buffer, of nbytes at least.  in_capture: what to do where that takes a new one while a graph is
        being captured: give the call one of its own, or (False) raise."""
        dev = torch.device(device)
        key = dev.index if dev.index is not None else torch.cuda.current_device()
        with cls._lock:
            ws = cls._cache.get(key)
            if ws is None or ws.numel() < nbytes:
                capturing = _capturing(key)
                if capturing and not in_capture:
                    raise SpecVerifyError(SV_EWORKSPACE, f"default workspace of {nbytes} bytes while a graph is being "
                                          "captured: make a call of this size before the capture, or hand over workspace=")
                least = 2 * ws.numel() if ws is not None and not capturing else 1 << 20
                new = torch.zeros(max(nbytes, least), dtype=torch.uint8, device=dev)
                if new.data_ptr() % 256:
                    raise SpecVerifyError(SV_EALIGN, "workspace allocation not 256-byte aligned")
                other = new if capturing else ws
                if other is not None:
                    cls._replaced.setdefault(key, []).append(other)
                if not capturing:
                    cls._cache[key] = new
                return new
            return ws

    @classmethod
    def every(cls, device):
        """All of the device's buffers (at least the one in use)."""
        first = cls.get(device, 0)
        dev = torch.device(device)
        key = dev.index if dev.index is not None else torch.cuda.current_device()
        with cls._lock:
            return [first, *cls._replaced.get(key, ())]


def workspace_size(op, dt, B, K, gamma_or_N, V, F_max=1) -> int:
    n = _sz(0)
    _check(_lib.sv_workspace_size(op, dt, B, K, gamma_or_N, V, F_max, ctypes.byref(n)), "sv_workspace_size")
    return n.value


def sv_get_device_error(device=None) -> int:
    """Synchronise and read (and clear) the device error word of this device's workspace; graphs that keep an earlier
    one report there."""
    device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    found = 0
    for ws in Workspace.every(device):
        flags = _i32(0)
        _check(_lib.sv_get_device_error(_ptr(ws), ctypes.byref(flags), _stream(device)), "sv_get_device_error")
        found |= flags.value
    return found


def sv_verify_chain(tgt, drf, tok, T, seed=0, round_=0, want_pq=True, workspace=None):
    """tgt [B, gamma+1, V], drf [B, gamma, V], tok [B, gamma] int32 -> dict(n, tok, p, q)."""
    B, g1, V = tgt.shape
    gamma = g1 - 1
    if tuple(drf.shape) != (B, gamma, V) or drf.dtype != tgt.dtype:
        raise SpecVerifyError(SV_EINVAL, f"drf shape {tuple(drf.shape)} / dtype does not match tgt")
    _i32_tensor(tok, (B, gamma), "tok")
    dt = _dtype_code(tgt)
    dev = tgt.device
    ws = workspace if workspace is not None else Workspace.get(dev, workspace_size(SV_OP_CHAIN, dt, B, 1, gamma, V))
    out_n = torch.empty(B, dtype=torch.int32, device=dev)
    out_tok = torch.empty(B, dtype=torch.int32, device=dev)
    p = torch.empty(B, gamma, dtype=torch.float32, device=dev) if want_pq else None
    q = torch.empty(B, gamma, dtype=torch.float32, device=dev) if want_pq else None
    _check(_lib.sv_verify_chain(_ptr(tgt), _ptr(drf), dt, _row_stride(tgt, "tgt"), _row_stride(drf, "drf"),
                                _ptr(tok), B, gamma, V, float(T), int(seed), int(round_), _ptr(out_n), _ptr(out_tok),
                                _ptr(p), _ptr(q), _ptr(ws), ws.numel(), _stream(dev)), "sv_verify_chain")
    _checked(dev, "sv_verify_chain", workspace)
    return dict(n=out_n, tok=out_tok, p=p, q=q)


NOALLOC_SCRATCH_BYTES = 8 << 20


def sv_verify_chain_noalloc(tgt, drf, tok, T, seed=0, round_=0, want_pq=True, out_err=None):
    """sv_verify_chain through the allocation-free entry point: the library's own per-GPU scratch array, no
    workspace.  out_err: optional zeroed device int32 tensor [1] that receives the device error bits."""
    B, g1, V = tgt.shape
    gamma = g1 - 1
    if tuple(drf.shape) != (B, gamma, V) or drf.dtype != tgt.dtype:
        raise SpecVerifyError(SV_EINVAL, f"drf shape {tuple(drf.shape)} / dtype does not match tgt")
    _i32_tensor(tok, (B, gamma), "tok")
    if out_err is not None:
        _i32_tensor(out_err, (1,), "out_err")
    dt = _dtype_code(tgt)
    dev = tgt.device
    out_n = torch.empty(B, dtype=torch.int32, device=dev)
    out_tok = torch.empty(B, dtype=torch.int32, device=dev)
    p = torch.empty(B, gamma, dtype=torch.float32, device=dev) if want_pq else None
    q = torch.empty(B, gamma, dtype=torch.float32, device=dev) if want_pq else None
    _check(_lib.sv_verify_chain_noalloc(_ptr(tgt), _ptr(drf), dt, _row_stride(tgt, "tgt"), _row_stride(drf, "drf"),
                                        _ptr(tok), B, gamma, V, float(T), int(seed), int(round_), _ptr(out_n),
                                        _ptr(out_tok), _ptr(p), _ptr(q), _ptr(out_err), _stream(dev)),
           "sv_verify_chain_noalloc")
    return dict(n=out_n, tok=out_tok, p=p, q=q)


def sv_verify_chain_pm(tgt, tok, T, seed=0, round_=0, want_p=True, workspace=None):
    """Point-mass acceptance. tgt [B, gamma+1, V], tok [B, gamma] int32 -> dict(n, tok, p)."""
    B, g1, V = tgt.shape
    gamma = g1 - 1
    _i32_tensor(tok, (B, gamma), "tok")
    dt = _dtype_code(tgt)
    dev = tgt.device
    ws = workspace if workspace is not None else Workspace.get(
        dev, workspace_size(SV_OP_CHAIN_PM, dt, B, 1, gamma, V))
    out_n = torch.empty(B, dtype=torch.int32, device=dev)
    out_tok = torch.empty(B, dtype=torch.int32, device=dev)
    p = torch.empty(B, gamma, dtype=torch.float32, device=dev) if want_p else None
    _check(_lib.sv_verify_chain_pm(_ptr(tgt), dt, _row_stride(tgt, "tgt"), _ptr(tok), B, gamma, V, float(T),
                                   int(seed), int(round_), _ptr(out_n), _ptr(out_tok), _ptr(p), _ptr(ws),
                                   ws.numel(), _stream(dev)), "sv_verify_chain_pm")
    _checked(dev, "sv_verify_chain_pm", workspace)
    return dict(n=out_n, tok=out_tok, p=p)


def sv_verify_greedy(tgt, tok, want_argmax=True, workspace=None):
    """tgt [B, gamma+1, V], tok [B, gamma] -> dict(n, tok, argmax [B, gamma+1])."""
    B, g1, V = tgt.shape
    gamma = g1 - 1
    _i32_tensor(tok, (B, gamma), "tok")
    dt = _dtype_code(tgt)
    dev = tgt.device
    ws = workspace if workspace is not None else Workspace.get(dev, workspace_size(SV_OP_GREEDY, dt, B, 1, gamma, V))
    out_n = torch.empty(B, dtype=torch.int32, device=dev)
    out_tok = torch.empty(B, dtype=torch.int32, device=dev)
    am = torch.empty(B, g1, dtype=torch.int32, device=dev) if want_argmax else None
    _check(_lib.sv_verify_greedy(_ptr(tgt), dt, _row_stride(tgt, "tgt"), _ptr(tok), B, gamma, V, _ptr(out_n),
                                 _ptr(out_tok), _ptr(am), _ptr(ws), ws.numel(), _stream(dev)), "sv_verify_greedy")
    _checked(dev, "sv_verify_greedy", workspace)
    return dict(n=out_n, tok=out_tok, argmax=am)


def sv_verify_multi(tgt, drf, tok, T, seed=0, round_=0, want_pq=True, workspace=None):
    """tgt [B, K, gamma+1, V], drf [B, gamma, V], tok [B, K, gamma] -> dict(k, n, tok, n_cand, p, q)."""
    B, K, g1, V = tgt.shape
    gamma = g1 - 1
    if tuple(drf.shape) != (B, gamma, V) or drf.dtype != tgt.dtype:
        raise SpecVerifyError(SV_EINVAL, f"drf shape {tuple(drf.shape)} / dtype does not match tgt")
    _i32_tensor(tok, (B, K, gamma), "tok")
    dt = _dtype_code(tgt)
    dev = tgt.device
    ws = workspace if workspace is not None else Workspace.get(dev, workspace_size(SV_OP_MULTI, dt, B, K, gamma, V))
    out = dict(k=torch.empty(B, dtype=torch.int32, device=dev), n=torch.empty(B, dtype=torch.int32, device=dev),
               tok=torch.empty(B, dtype=torch.int32, device=dev),
               n_cand=torch.empty(B, K, dtype=torch.int32, device=dev),
               p=torch.empty(B, K, gamma, dtype=torch.float32, device=dev) if want_pq else None,
               q=torch.empty(B, K, gamma, dtype=torch.float32, device=dev) if want_pq else None)
    _check(_lib.sv_verify_multi(_ptr(tgt), _ptr(drf), dt, _row_stride(tgt, "tgt"), _row_stride(drf, "drf"),
                                _ptr(tok), B, K, gamma, V, float(T), int(seed), int(round_), _ptr(out["k"]),
                                _ptr(out["n"]), _ptr(out["tok"]), _ptr(out["n_cand"]), _ptr(out["p"]),
                                _ptr(out["q"]), _ptr(ws), ws.numel(), _stream(dev)), "sv_verify_multi")
    _checked(dev, "sv_verify_multi", workspace)
    return out


def sv_verify_tree(tgt, drf, node_tok, parent, max_depth, T, seed=0, round_=0, want_pq=True, workspace=None):
    """tgt, drf [B, N, V]; node_tok, parent [B, N] -> dict(len, path [B, max_depth], tok, p, q)."""
    B, N, V = tgt.shape
    if tuple(drf.shape) != (B, N, V) or drf.dtype != tgt.dtype:
        raise SpecVerifyError(SV_EINVAL, f"drf shape {tuple(drf.shape)} / dtype does not match tgt")
    _i32_tensor(node_tok, (B, N), "node_tok")
    _i32_tensor(parent, (B, N), "parent")
    dt = _dtype_code(tgt)
    dev = tgt.device
    ws = workspace if workspace is not None else Workspace.get(dev, workspace_size(SV_OP_TREE, dt, B, 1, N, V))
    out = dict(len=torch.empty(B, dtype=torch.int32, device=dev),
               path=torch.empty(B, max_depth, dtype=torch.int32, device=dev),
               tok=torch.empty(B, dtype=torch.int32, device=dev),
               p=torch.full((B, N), float("nan"), dtype=torch.float32, device=dev) if want_pq else None,
               q=torch.full((B, N), float("nan"), dtype=torch.float32, device=dev) if want_pq else None)
    _check(_lib.sv_verify_tree(_ptr(tgt), _ptr(drf), dt, _row_stride(tgt, "tgt"), _row_stride(drf, "drf"),
                               _ptr(node_tok), _ptr(parent), B, N, int(max_depth), V, float(T), int(seed),
                               int(round_), _ptr(out["len"]), _ptr(out["path"]), _ptr(out["tok"]), _ptr(out["p"]),
                               _ptr(out["q"]), _ptr(ws), ws.numel(), _stream(dev)), "sv_verify_tree")
    _checked(dev, "sv_verify_tree", workspace)
    return out


def sv_verify_tree_pm(tgt, node_tok, parent, max_depth, T, seed=0, round_=0, want_p=True, workspace=None):
    """Point-mass acceptance. tgt [B, N, V]; node_tok, parent [B, N] -> dict(len, path, tok, p)."""
    B, N, V = tgt.shape
    _i32_tensor(node_tok, (B, N), "node_tok")
    _i32_tensor(parent, (B, N), "parent")
    dt = _dtype_code(tgt)
    dev = tgt.device
    ws = workspace if workspace is not None else Workspace.get(dev, workspace_size(SV_OP_TREE_PM, dt, B, 1, N, V))
    out = dict(len=torch.empty(B, dtype=torch.int32, device=dev),
               path=torch.empty(B, max_depth, dtype=torch.int32, device=dev),
               tok=torch.empty(B, dtype=torch.int32, device=dev),
               p=torch.full((B, N), float("nan"), dtype=torch.float32, device=dev) if want_p else None)
    _check(_lib.sv_verify_tree_pm(_ptr(tgt), dt, _row_stride(tgt, "tgt"), _ptr(node_tok), _ptr(parent), B, N,
                                  int(max_depth), V, float(T), int(seed), int(round_), _ptr(out["len"]),
                                  _ptr(out["path"]), _ptr(out["tok"]), _ptr(out["p"]), _ptr(ws), ws.numel(),
                                  _stream(dev)), "sv_verify_tree_pm")
    _checked(dev, "sv_verify_tree_pm", workspace)
    return out


def sv_fanout_topk(logits, F, F_max, want_vals=True, workspace=None):
    """logits [R, V], F [R] int32 (device) -> (ids [R, F_max], vals [R, F_max] or None)."""
    R, V = logits.shape
    _i32_tensor(F, (R,), "F")
    dt = _dtype_code(logits)
    dev = logits.device
    ws = workspace if workspace is not None else Workspace.get(
        dev, workspace_size(SV_OP_FANOUT, dt, R, 1, 1, V, F_max))
    ids = torch.empty(R, F_max, dtype=torch.int32, device=dev)
    vals = torch.empty(R, F_max, dtype=torch.float32, device=dev) if want_vals else None
    _check(_lib.sv_fanout_topk(_ptr(logits), dt, _row_stride(logits, "logits"), R, V, _ptr(F), int(F_max), _ptr(ids),
                               _ptr(vals), _ptr(ws), ws.numel(), _stream(dev)), "sv_fanout_topk")
    _checked(dev, "sv_fanout_topk", workspace)
    return ids, vals


def sv_cache_hit_test(drf, n, t, F=None, workspace=None):
    """drf [B, K+1, V]; outcome n, t [B] int32 (device); F [K+1] int32 (device) or None
    -> dict(rank [B], hit [B] or None)."""
    B, K1, V = drf.shape
    _i32_tensor(n, (B,), "n")
    _i32_tensor(t, (B,), "t")
    if F is not None:
        _i32_tensor(F, (K1,), "F")
    dt = _dtype_code(drf)
    dev = drf.device
    ws = workspace if workspace is not None else Workspace.get(dev, workspace_size(SV_OP_CACHE, dt, B, 1, K1 - 1, V))
    rank = torch.empty(B, dtype=torch.int32, device=dev)
    hit = torch.empty(B, dtype=torch.int32, device=dev) if F is not None else None
    _check(_lib.sv_cache_hit_test(_ptr(drf), dt, _row_stride(drf, "drf"), B, K1 - 1, V, _ptr(n), _ptr(t), _ptr(F),
                                  _ptr(rank), _ptr(hit), _ptr(ws), ws.numel(), _stream(dev)), "sv_cache_hit_test")
    _checked(dev, "sv_cache_hit_test", workspace)
    return dict(rank=rank, hit=hit)


def sv_presto_score(tgt, drf, node_tok, parent, T, lam, k, b_top, want_scores=True, workspace=None):
    """tgt, drf [B, N, V]; node_tok, parent [B, N] int32; lam [D] float32 (device)
    -> dict(s, S [B, N] float or None, node, tok [B, b_top] int32, score [B, b_top] float)."""
    B, N, V = tgt.shape
    if tuple(drf.shape) != (B, N, V) or drf.dtype != tgt.dtype:
        raise SpecVerifyError(SV_EINVAL, f"drf shape {tuple(drf.shape)} / dtype does not match tgt")
    _i32_tensor(node_tok, (B, N), "node_tok")
    _i32_tensor(parent, (B, N), "parent")
    if lam.dtype != torch.float32 or lam.dim() != 1 or not lam.is_contiguous():
        raise SpecVerifyError(SV_EINVAL, "lam: want a contiguous float32 vector")
    dt = _dtype_code(tgt)
    dev = tgt.device
    ws = workspace if workspace is not None else Workspace.get(
        dev, workspace_size(SV_OP_PRESTO, dt, B, 1, N, V, int(k)))
    f = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=dev)
    out = dict(s=f(B, N) if want_scores else None, S=f(B, N) if want_scores else None,
               node=torch.empty(B, b_top, dtype=torch.int32, device=dev),
               tok=torch.empty(B, b_top, dtype=torch.int32, device=dev), score=f(B, b_top))
    _check(_lib.sv_presto_score(_ptr(tgt), _ptr(drf), dt, _row_stride(tgt, "tgt"), _row_stride(drf, "drf"),
                                _ptr(node_tok), _ptr(parent), B, N, V, float(T), _ptr(lam), lam.numel(), int(k),
                                int(b_top), _ptr(out["s"]), _ptr(out["S"]), _ptr(out["node"]), _ptr(out["tok"]),
                                _ptr(out["score"]), _ptr(ws), ws.numel(), _stream(dev)), "sv_presto_score")
    _checked(dev, "sv_presto_score", workspace)
    return out


def sv_branch_fork(drf, tok, T, eps, k_max, cls=None, workspace=None):
    """drf [B, gamma+1, V] draft rows q_1..q_{gamma+1}; tok [B, gamma]; cls [B] int32 or None
    -> dict(pos, qb, k [B], ids [B, k_max])."""
    B, g1, V = drf.shape
    gamma = g1 - 1
    _i32_tensor(tok, (B, gamma), "tok")
    if cls is not None:
        _i32_tensor(cls, (B,), "cls")
    dt = _dtype_code(drf)
    dev = drf.device
    ws = workspace if workspace is not None else Workspace.get(
        dev, workspace_size(SV_OP_BRANCH, dt, B, 1, gamma, V, int(k_max)))
    out = dict(pos=torch.empty(B, dtype=torch.int32, device=dev), qb=torch.empty(B, dtype=torch.float32, device=dev),
               k=torch.empty(B, dtype=torch.int32, device=dev),
               ids=torch.empty(B, k_max, dtype=torch.int32, device=dev))
    _check(_lib.sv_branch_fork(_ptr(drf), dt, _row_stride(drf, "drf"), _ptr(tok), _ptr(cls), B, gamma, V, float(T),
                               float(eps), int(k_max), _ptr(out["pos"]), _ptr(out["qb"]), _ptr(out["k"]),
                               _ptr(out["ids"]), _ptr(ws), ws.numel(), _stream(dev)), "sv_branch_fork")
    _checked(dev, "sv_branch_fork", workspace)
    return out


def sv_read_probe(buf: torch.Tensor, sink: torch.Tensor, blocks=1024, mode=0, unroll=4, chunk_bytes=1 << 16):
    """Read every 16-byte vector of buf in the statistics kernels' load pattern (a bandwidth probe).  sink: int32
    [>= 3] on the device, zero before the first call (mode 2's counters; the kernel leaves them at zero)."""
    assert sink.numel() >= 3 and sink.element_size() == 4 and sink.device == buf.device
    _check(_lib.sv_read_probe(_ptr(buf), buf.numel() * buf.element_size(), int(blocks), int(mode), int(unroll),
                              int(chunk_bytes), _ptr(sink), _stream(buf.device)), "sv_read_probe")


def sv_timeline_set(buf):
    """Register a device buffer (uint64 [records, 16], zero-filled) for the timeline build's per-block stamps,
    or None to stop.  Raises on a library built without timelines (SV_EUNSUPPORTED)."""
    if buf is None:
        _check(_lib.sv_timeline_set(None, 0), "sv_timeline_set")
        return
    assert buf.dtype == torch.int64 and buf.is_contiguous() and buf.numel() % 16 == 0
    torch.cuda.synchronize(buf.device)
    _check(_lib.sv_timeline_set(_ptr(buf), buf.numel() // 16), "sv_timeline_set")


def sv_geometric_fanout(F0, a_p, r, K, capped_last=False):
    out = (_i32 * (K + 1))()
    s = _lib.sv_geometric_fanout(int(F0), float(a_p), float(r), int(K), int(bool(capped_last)), out)
    if s < 0:
        raise SpecVerifyError(SV_EINVAL, "sv_geometric_fanout")
    return list(out)


# ---------------------------------------------------------------------------
# The drafter's side (specverify_draft.h).  Tensors of one call are on one
# device, which need not be the current one; the call runs on that device's
# current stream.  The default workspace is the device's: calls that overlap
# in time on several streams, and graphs that may be replayed together, take a
# zero-filled one each (workspace=, a uint8 tensor of draft_workspace_size
# bytes).  A captured graph keeps the workspace of its capture.  The default
# one lives as long as the process, but is not made or grown in a capture:
# call once with the same sizes before, or hand over a workspace.
# ---------------------------------------------------------------------------


@functools.lru_cache(maxsize=1024)
def draft_workspace_size(op, dt, rows, W, V, k) -> int:
    n = _sz(0)
    _check(_lib.sv_draft_workspace_size(op, dt, rows, W, V, k, ctypes.byref(n)), "sv_draft_workspace_size")
    return n.value


def _draft_workspace(dev, *shape):
    need = draft_workspace_size(*shape)
    ws = Workspace._cache.get(dev.index)
    return ws if ws is not None and ws.numel() >= need else Workspace.get(dev, need, in_capture=False)


# The small calls of decoding take about as long on the host as on the GPU, so
# these bindings pass addresses as plain integers and ask for the stream's
# handle without building a Stream object (1.8 us).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _at(t):
    return None if t is None else t.data_ptr()


def _one_device(what, first, *others):
    if not first.is_cuda:
        raise SpecVerifyError(SV_EINVAL, f"{what}: want tensors on the GPU, got {first.device}")
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise SpecVerifyError(SV_EINVAL, f"{what}: tensors on {first.device} and {t.device}")
    return first.device


def _call(dev, fn, what, *args):
    """One launch with `dev` current, on its current stream."""
    if dev.index == _current_device():  # tensors on a GPU: torch has been initialised
        status = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev.index))
    if status != SV_OK:
        raise SpecVerifyError(status, what)


def _want(t, dtype, shape, what):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise SpecVerifyError(SV_EINVAL, f"{what}: want contiguous {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")


def _rows_2d(t, what):
    """R, V and the row stride of a [R, V] tensor."""
    if t.dim() != 2:
        raise SpecVerifyError(SV_EINVAL, f"{what}: want [rows, V], got {tuple(t.shape)}")
    R, V = t.shape
    stride, unit = t.stride()
    if unit != 1 and V > 1:
        raise SpecVerifyError(SV_EINVAL, f"{what}: vocabulary axis must have unit stride")
    return R, V, stride if R > 1 else _one_row(V, t)


def _one_row(V, t):
    """A stride for a single row, whatever the tensor says of it."""
    return V + -V % (16 // t.element_size())


def _rows_3d(t, what):
    """B, W, V and the row stride of a [B, W, V] tensor of evenly spaced rows."""
    if t.dim() != 3:
        raise SpecVerifyError(SV_EINVAL, f"{what}: want [B, W, V], got {tuple(t.shape)}")
    B, W, V = t.shape
    outer, stride, unit = t.stride()
    if unit != 1 and V > 1:
        raise SpecVerifyError(SV_EINVAL, f"{what}: vocabulary axis must have unit stride")
    if B > 1 and W > 1 and outer != W * stride:
        raise SpecVerifyError(SV_EINVAL, f"{what}: rows must be evenly spaced")
    return B, W, V, stride if W > 1 else outer if B > 1 else _one_row(V, t)


def sv_teacher_topk(logits, k, T, workspace=None):
    """The k largest logits of each row and the logarithm of the mass outside them at temperature T.
    logits [R, V] -> dict(ids [R, k] int32, vals [R, k], rest [R])."""
    R, V, stride = _rows_2d(logits, "logits")
    dt, k = _dtype_code(logits), int(k)
    dev = _one_device("sv_teacher_topk", logits, workspace)
    ws = workspace if workspace is not None else _draft_workspace(dev, SV_DRAFT_TEACHER, dt, R, 1, V, k)
    out = dict(ids=torch.empty(R, k, dtype=torch.int32, device=dev),
               vals=torch.empty(R, k, dtype=torch.float32, device=dev),
               rest=torch.empty(R, dtype=torch.float32, device=dev))
    _call(dev, _lib.sv_teacher_topk, "sv_teacher_topk", logits.data_ptr(), dt, stride, R, V, k,
          float(T), out["ids"].data_ptr(), out["vals"].data_ptr(), out["rest"].data_ptr(), ws.data_ptr(), ws.numel())
    _checked(dev, "sv_teacher_topk", workspace)
    return out


def _distill_args(what, z, ids, vals, rest, grad_loss, grad, workspace):
    R, V, stride = _rows_2d(z, "z")
    if ids.dim() != 2 or ids.shape[0] != R:
        raise SpecVerifyError(SV_EINVAL, f"ids: want [{R}, k], got {tuple(ids.shape)}")
    k = ids.shape[1]
    _want(ids, torch.int32, (R, k), "ids")
    _want(vals, torch.float32, (R, k), "vals")
    if rest is not None:
        _want(rest, torch.float32, (R,), "rest")
    if grad_loss is not None:
        _want(grad_loss, torch.float32, (R,), "grad_loss")
    if grad is not None and (grad.shape != (R, V) or grad.dtype is not z.dtype):
        raise SpecVerifyError(SV_EINVAL, f"grad: want {z.dtype} {(R, V)}, got {grad.dtype} {tuple(grad.shape)}")
    dt = _dtype_code(z)
    dev = _one_device(what, z, ids, vals, rest, grad_loss, grad, workspace)
    ws = workspace if workspace is not None else _draft_workspace(dev, SV_DRAFT_DISTILL, dt, R, 1, V, k)
    return R, V, stride, k, dt, dev, ws


def _grad_rows(z, R, V):
    """Gradient rows beside z, 16-byte aligned (a view of padded rows where V needs it)."""
    pad = -V % (16 // z.element_size())
    rows = torch.empty(R, V + pad, dtype=z.dtype, device=z.device)
    return rows[:, :V] if pad else rows


def sv_distill_topk(z, ids, vals, T, rest=None, grad_loss=None, want_grad=False, grad=None, workspace=None):
    """KL divergence of a drafter's rows from a teacher's top logits (sv_teacher_topk's ids, vals and rest; rest None:
    renormalised over the ids), and with want_grad its gradient, times grad_loss [R] (None: 1).
    z [R, V], ids, vals [R, k] -> dict(loss [R], stat [R, 4] for the backward pass, grad [R, V] or None).
    grad: where to write the gradient (z itself: in place); hand it on with z.backward(out["grad"])."""
    R, V, stride, k, dt, dev, ws = _distill_args("sv_distill_topk", z, ids, vals, rest, grad_loss, grad, workspace)
    if grad is None and want_grad:
        grad = _grad_rows(z, R, V)
    out = dict(loss=torch.empty(R, dtype=torch.float32, device=dev),
               stat=torch.empty(R, 4, dtype=torch.float32, device=dev), grad=grad)
    _call(dev, _lib.sv_distill_topk, "sv_distill_topk", z.data_ptr(), dt, stride, R, V, ids.data_ptr(), vals.data_ptr(),
          _at(rest), k, float(T), _at(grad_loss), out["loss"].data_ptr(), out["stat"].data_ptr(), _at(grad),
          _rows_2d(grad, "grad")[2] if grad is not None else 0, ws.data_ptr(), ws.numel())
    _checked(dev, "sv_distill_topk", workspace)
    return out


def sv_distill_topk_backward(z, ids, vals, stat, T, rest=None, grad_loss=None, grad=None, workspace=None):
    """The gradient of sv_distill_topk from its stat: [R, V] of z's type (grad: where to write it; z itself: in place)."""
    R, V, stride, k, dt, dev, ws = _distill_args("sv_distill_topk_backward", z, ids, vals, rest, grad_loss, grad, workspace)
    _want(stat, torch.float32, (R, 4), "stat")
    _one_device("sv_distill_topk_backward", z, stat)
    if grad is None:
        grad = _grad_rows(z, R, V)
    _call(dev, _lib.sv_distill_topk_backward, "sv_distill_topk_backward", z.data_ptr(), dt, stride, R, V,
          ids.data_ptr(), vals.data_ptr(), _at(rest), k, float(T), stat.data_ptr(), _at(grad_loss), _at(grad),
          _rows_2d(grad, "grad")[2], ws.data_ptr(), ws.numel())
    _checked(dev, "sv_distill_topk_backward", workspace)
    return grad


def sv_beam_select(logits, scores, N, T=1.0, finished=None, pad_tok=0, workspace=None):
    """One step of beam search.  logits [B, W, V], scores [B, W] float32, finished [B, W] int32 or None
    -> dict(beam, tok [B, N] int32, score [B, N])."""
    B, W, V, stride = _rows_3d(logits, "logits")
    _want(scores, torch.float32, (B, W), "scores")
    if finished is not None:
        _want(finished, torch.int32, (B, W), "finished")
    dt, N, pad = _dtype_code(logits), int(N), int(pad_tok)
    if not -(1 << 31) <= pad < 1 << 31:
        raise SpecVerifyError(SV_EINVAL, f"pad_tok {pad} outside int32")
    dev = _one_device("sv_beam_select", logits, scores, finished, workspace)
    ws = workspace if workspace is not None else _draft_workspace(dev, SV_DRAFT_BEAM, dt, B, W, V, N)
    out = dict(beam=torch.empty(B, N, dtype=torch.int32, device=dev),
               tok=torch.empty(B, N, dtype=torch.int32, device=dev),
               score=torch.empty(B, N, dtype=torch.float32, device=dev))
    _call(dev, _lib.sv_beam_select, "sv_beam_select", logits.data_ptr(), dt, stride, scores.data_ptr(),
          _at(finished), B, W, V, float(T), pad, N, out["beam"].data_ptr(), out["tok"].data_ptr(), out["score"].data_ptr(), ws.data_ptr(),
          ws.numel())
    _checked(dev, "sv_beam_select", workspace)
    return out


def _state_layout(t, pos_dim, what):
    return _state_layout_of(t.shape, t.stride(), t.element_size(), pos_dim, what)


@functools.lru_cache(maxsize=1024)
def _state_layout_of(shape, st, es, pos_dim, what):
    """(L, B, beams, H, S, position bytes) and the strides in bytes of a state [L, B, beams, ...]."""
    dims = len(shape)
    if dims < 3:
        raise SpecVerifyError(SV_EINVAL, f"{what}: want [L, B, beams, ...], got {tuple(shape)}")
    p = dims if pos_dim is None else int(pos_dim)
    if pos_dim is not None and not 3 <= p < dims:
        raise SpecVerifyError(SV_EINVAL, f"{what}: pos_dim {pos_dim} of a state of {dims} dimensions")
    first = 3 if pos_dim is None else p  # dimensions from here on are adjacent in memory
    run = 1
    for ax in range(dims - 1, first - 1, -1):
        if shape[ax] > 1 and st[ax] != run:
            raise SpecVerifyError(SV_EINVAL, f"{what}: the values of a position and the positions must be adjacent")
        run *= shape[ax]
    S = 1 if pos_dim is None else shape[p]
    H, sh = 1, 0
    for ax in range(first - 1, 2, -1):  # segments: evenly spaced
        if shape[ax] == 1:
            continue
        if H > 1 and st[ax] != sh * H:
            raise SpecVerifyError(SV_EINVAL, f"{what}: the dimensions between beams and positions must be evenly spaced")
        sh = st[ax] if H == 1 else sh
        H *= shape[ax]
    pos = (run // S if S else 1) * es
    return (shape[0], shape[1], shape[2], H, S, pos), (_i64 * 4)(st[0] * es, st[1] * es, st[2] * es, sh * es)


def sv_beam_reorder(state, parent, pos_dim=None, lens=None, out=None, workspace=None):
    """The beams' states after a selection: out[l, b, n] = state[l, b, parent[b, n]] (parent -1: left as it is).
    state [L, B, W, ...] of any type, parent [B, N] int32; pos_dim names the dimension of the positions, of which only
    the first lens[b] ([B] int32) move; between the beams and the positions may stand heads, after them a position's
    values.  out [L, B, N, ...] apart from state, or None: in place (N <= W).  Returns out, or state."""
    if lens is not None and pos_dim is None:
        raise SpecVerifyError(SV_EINVAL, "lens: want pos_dim with it")
    dst = state if out is None else out
    if dst.dim() != state.dim() or dst.dtype != state.dtype:
        raise SpecVerifyError(SV_EINVAL, f"out: want {state.dtype} of {state.dim()} dimensions")
    (L, B, W, H, S, pos), ss = _state_layout(state, pos_dim, "state")
    (_, _, Nd, Hd, Sd, posd), ds = _state_layout(dst, pos_dim, "out")
    if parent.dim() != 2:
        raise SpecVerifyError(SV_EINVAL, f"parent: want [B, N], got {tuple(parent.shape)}")
    N = parent.shape[1]
    _want(parent, torch.int32, (B, N), "parent")
    if lens is not None:
        _want(lens, torch.int32, (B,), "lens")
    if out is None:
        if N > W:
            raise SpecVerifyError(SV_EINVAL, f"parent: {N} beams in place of {W}")
    elif Nd != N or dst.shape[:2] != state.shape[:2] or dst.shape[3:] != state.shape[3:]:
        raise SpecVerifyError(SV_EINVAL, f"out: shape {tuple(dst.shape)} for {N} beams of {tuple(state.shape)}")
    dev = _one_device("sv_beam_reorder", state, dst, parent, lens, workspace)
    ws = workspace if workspace is not None else _draft_workspace(dev, SV_DRAFT_REORDER, 0, 0, 0, 0, 0)
    _call(dev, _lib.sv_beam_reorder, "sv_beam_reorder", state.data_ptr(), ss, dst.data_ptr(), ds, parent.data_ptr(), _at(lens), L, B,
          W, N, H, S, pos, ws.data_ptr(), ws.numel())
    _checked(dev, "sv_beam_reorder", workspace)
    return dst


# ---------------------------------------------------------------------------
# The verifier's pass (specverify_pass.h): the same rules as the drafter's
# side.  Tensors of a window are [B, N, heads, D] with a unit stride along D.
# ---------------------------------------------------------------------------
_PASS_TYPES = {torch.bfloat16: SV_BF16, torch.float16: SV_F16, torch.float32: SV_F32}


@functools.lru_cache(maxsize=1024)
def pass_workspace_size(op, B=0, N=0, Hq=0, H=0, D=0) -> int:
    n = _sz(0)
    _check(_lib.sv_pass_workspace_size(op, B, N, Hq, H, D, ctypes.byref(n)), "sv_pass_workspace_size")
    return n.value


def _pass_workspace(dev, *shape):
    need = pass_workspace_size(*shape)
    ws = Workspace._cache.get(dev.index)
    return ws if ws is not None and ws.numel() >= need else Workspace.get(dev, need, in_capture=False)


def _window(t, what):
    """The type's code and the strides of a [B, N, heads, D] tensor."""
    dt = _PASS_TYPES.get(t.dtype)
    if dt is None:
        raise SpecVerifyError(SV_EDTYPE, f"{what}: {t.dtype}")
    return dt, _window_strides(t.shape, t.stride(), what)


@functools.lru_cache(maxsize=1024)
def _window_strides(shape, st, what):
    if len(shape) != 4:
        raise SpecVerifyError(SV_EINVAL, f"{what}: want [B, N, heads, D], got {tuple(shape)}")
    if st[3] != 1 and shape[3] > 1:
        raise SpecVerifyError(SV_EINVAL, f"{what}: a head's values must have unit stride")
    return (_i64 * 3)(*st[:3])


def _int32(t, shape, what):
    if t is not None:
        _want(t, torch.int32, shape, what)


def kv_page_bytes(H, D, page_tokens) -> int:
    """Bytes of a page of the 4-bit cache."""
    n = _i64(0)
    _check(_lib.sv_kv_page_bytes(int(H), int(D), int(page_tokens), ctypes.byref(n)), "sv_kv_page_bytes")
    return n.value


class KvCache:
    """A paged 4-bit cache: pool uint8 [pages, bytes] of one layer or [L, pages, bytes] of several (bytes at least
    kv_page_bytes(H, D, page_tokens), unit stride), pages int32 [B, max_pages] on the same device: sequence b's tokens t lie in page
    pages[b, t // page_tokens].  The entry points read and write one layer's cache (layer(l) of a pool of several),
    sv_kv_commit all layers of its pool.  Holds the tensors; what they contain may change between calls."""

    def __init__(self, pool, pages, H, D, page_tokens):
        H, D, page_tokens = int(H), int(D), int(page_tokens)
        need = kv_page_bytes(H, D, page_tokens)
        if pool.dtype is not torch.uint8 or pool.dim() not in (2, 3) or pool.shape[-1] < need or pool.stride(-1) != 1:
            raise SpecVerifyError(SV_EINVAL, f"pool: want uint8 [pages, {need}] or [L, pages, {need}], got {pool.dtype} "
                                  f"{tuple(pool.shape)}")
        if pages.dim() != 2:
            raise SpecVerifyError(SV_EINVAL, f"pages: want [B, max_pages], got {tuple(pages.shape)}")
        _want(pages, torch.int32, tuple(pages.shape), "pages")
        if pages.get_device() != pool.get_device():
            raise SpecVerifyError(SV_EINVAL, f"KvCache: pool on {pool.device}, pages on {pages.device}")
        self.pool, self.pages, self.H, self.D, self.page_tokens = pool, pages, H, D, page_tokens
        self.device = pool.device
        n, layers = pool.shape[-2], pool.shape[0] if pool.dim() == 3 else 1
        # a single page or layer has no stride of its own
        page = pool.stride(-2) if n > 1 else need + -need % 16
        self._c = _CCache(pool.data_ptr(), pages.data_ptr(), page, pool.stride(0) if layers > 1 and pool.dim() == 3 else 0, n,
                          pages.shape[1], page_tokens, H, D, layers)
        self._ref = ctypes.byref(self._c)

    def layer(self, l):
        """The cache of one layer: a handle to keep (making one takes about as long as a small call)."""
        return KvCache(self.pool[l], self.pages, self.H, self.D, self.page_tokens)

    def _one(self, what):
        if self._c.layers != 1:
            raise SpecVerifyError(SV_EINVAL, f"{what}: a cache of one layer, not of {self._c.layers} (KvCache.layer)")
        return self._ref


def sv_rope_frequencies(R, theta=10000.0, kind="plain", scale=1.0, original=0, fast=32.0, slow=1.0):
    """Angles a position of R/2 pairs, float64 [R/2] on the CPU, and the factor for sv_rope.  kind: plain, linear, base or
    parts (specverify_pass.h)."""
    if kind not in SV_ROPE_KINDS:
        raise SpecVerifyError(SV_EINVAL, f"kind {kind!r}: one of {', '.join(SV_ROPE_KINDS)}")
    R = int(R)
    out, factor = (_f64 * max(1, R // 2))(), _f32(0)
    _check(_lib.sv_rope_frequencies(SV_ROPE_KINDS[kind], R, float(theta), float(scale), int(original), float(fast),
                                    float(slow), out, ctypes.byref(factor)), "sv_rope_frequencies")
    return torch.tensor(list(out), dtype=torch.float64), factor.value


@functools.lru_cache(maxsize=1024)
def _rope_layout(q, qst, out_q, out_qst, k=None, kst=None, out_k=None, out_kst=None):
    """(B, N, Hq, D, Hk) and the strides of q, out_q, k, out_k."""
    sq, soq, sk, sok = _window_strides(q, qst, "q"), _window_strides(out_q, out_qst, "out_q"), None, None
    if out_q != q:
        raise SpecVerifyError(SV_EINVAL, f"out_q: want {tuple(q)}, got {tuple(out_q)}")
    if k is not None:
        sk, sok = _window_strides(k, kst, "k"), _window_strides(out_k, out_kst, "out_k")
        if k[:2] != q[:2] or k[3] != q[3] or out_k != k:
            raise SpecVerifyError(SV_EINVAL, f"k: want {(*q[:2], 'heads', q[3])} twice, got {tuple(k)} and {tuple(out_k)}")
    return (*q, 0 if k is None else k[2]), (sq, soq, sk, sok)


def sv_rope(q, freq, k=None, positions=None, lens=None, parent=None, interleaved=False, factor=1.0, inverse=False,
            out_q=None, out_k=None, workspace=None):
    """Rotary positions of q [B, N, Hq, D] and k [B, N, Hk, D] (or None) over the first 2 * len(freq) values of each head;
    freq float64 on the device.  positions [B, N] int32, or lens [B] int32 (None: 0) + the node's depth in parent [B, N] int32
    (None: its number).  inverse: the transposed rotation, the gradient.  out_q, out_k: where to write (q, k themselves:
    in place).  Returns dict(q, k)."""
    dt = _PASS_TYPES.get(q.dtype)
    if dt is None:
        raise SpecVerifyError(SV_EDTYPE, f"q: {q.dtype}")
    if out_q is None:
        out_q = torch.empty_like(q)
    if k is None:
        if out_k is not None:
            raise SpecVerifyError(SV_EINVAL, "out_k: want k with it")
        layout = _rope_layout(q.shape, q.stride(), out_q.shape, out_q.stride())
    else:
        if out_k is None:
            out_k = torch.empty_like(k)
        if k.dtype is not q.dtype or out_k.dtype is not q.dtype:
            raise SpecVerifyError(SV_EINVAL, f"k: want {q.dtype}, got {k.dtype} and {out_k.dtype}")
        layout = _rope_layout(q.shape, q.stride(), out_q.shape, out_q.stride(), k.shape, k.stride(), out_k.shape,
                              out_k.stride())
    if out_q.dtype is not q.dtype:
        raise SpecVerifyError(SV_EINVAL, f"out_q: want {q.dtype}, got {out_q.dtype}")
    (B, N, Hq, D, Hk), (sq, soq, sk, sok) = layout
    if freq.dim() != 1:
        raise SpecVerifyError(SV_EINVAL, f"freq: want [R/2], got {tuple(freq.shape)}")
    _want(freq, torch.float64, freq.shape, "freq")
    if positions is not None:
        _want(positions, torch.int32, (B, N), "positions")
    if lens is not None:
        _want(lens, torch.int32, (B,), "lens")
    if parent is not None:
        _want(parent, torch.int32, (B, N), "parent")
    dev = _one_device("sv_rope", q, freq, k, positions, lens, parent, out_q, out_k, workspace)
    ws = workspace if workspace is not None else _pass_workspace(dev, SV_PASS_ROPE)
    _call(dev, _lib.sv_rope, "sv_rope", q.data_ptr(), sq, _at(k), sk, dt, B, N, Hq, Hk, D, 2 * freq.shape[0], freq.data_ptr(),
          float(factor), bool(interleaved), bool(inverse), _at(positions), _at(lens), _at(parent), out_q.data_ptr(), soq,
          _at(out_k), sok, ws.data_ptr(), ws.numel())
    _checked(dev, "sv_rope", workspace)
    return dict(q=out_q, k=out_k)


@functools.lru_cache(maxsize=1024)
def _kv_layout(shape, kst, vshape, vst, want, what):
    """The strides of keys and values [B, N, H, D] that go with a cache."""
    sk, sv = _window_strides(shape, kst, "k"), _window_strides(vshape, vst, "v")
    if vshape != shape:
        raise SpecVerifyError(SV_EINVAL, f"v: want {tuple(shape)}, got {tuple(vshape)}")
    if (shape[0], *shape[2:]) != want:
        raise SpecVerifyError(SV_EINVAL, f"{what}: want [{want[0]}, N, {want[1]}, {want[2]}], got {tuple(shape)}")
    return sk, sv


def _kv_rows(what, cache, k, v, B):
    """The type's code and the strides of the keys and values [B, N, H, D] that go with a cache."""
    dt = _PASS_TYPES.get(k.dtype)
    if dt is None:
        raise SpecVerifyError(SV_EDTYPE, f"{what}: {k.dtype}")
    if v.dtype is not k.dtype:
        raise SpecVerifyError(SV_EINVAL, f"v: want {k.dtype}, got {v.dtype}")
    return dt, *_kv_layout(k.shape, k.stride(), v.shape, v.stride(), (B, cache.H, cache.D), what)


def sv_kv_write(cache, k, v, lens, news=None, workspace=None):
    """Keys and values [B, N, H, D] into the cache: token n of sequence b to place lens[b] + n, for n < news[b] (None: N)."""
    B = cache.pages.shape[0]
    dt, sk, sv = _kv_rows("k", cache, k, v, B)
    _int32(lens, (B,), "lens")
    _int32(news, (B,), "news")
    dev = _one_device("sv_kv_write", cache.pool, k, v, lens, news, workspace)
    ws = workspace if workspace is not None else _pass_workspace(dev, SV_PASS_WRITE)
    _call(dev, _lib.sv_kv_write, "sv_kv_write", k.data_ptr(), sk, v.data_ptr(), sv, dt, cache._one("sv_kv_write"),
          lens.data_ptr(), _at(news), B, k.shape[1], ws.data_ptr(), ws.numel())
    _checked(dev, "sv_kv_write", workspace)


def sv_kv_read(cache, start, count, k, v, workspace=None):
    """What the cache holds: tokens start[b] (None: 0) .. + count[b] (None: N) into the first rows of k, v [B, N, H, D] of
    any type; the others are left as they were.  Returns dict(k, v)."""
    B = cache.pages.shape[0]
    dt, sk, sv = _kv_rows("k", cache, k, v, B)
    _int32(start, (B,), "start")
    _int32(count, (B,), "count")
    dev = _one_device("sv_kv_read", cache.pool, k, v, start, count, workspace)
    ws = workspace if workspace is not None else _pass_workspace(dev, SV_PASS_READ)
    _call(dev, _lib.sv_kv_read, "sv_kv_read", cache._one("sv_kv_read"), _at(start), _at(count), B, k.shape[1], dt,
          k.data_ptr(), sk, v.data_ptr(), sv, ws.data_ptr(), ws.numel())
    _checked(dev, "sv_kv_read", workspace)
    return dict(k=k, v=v)


def sv_kv_attention(cache, q, lens, news=None, parent=None, scale=None, cap=0.0, slopes=None, reach=0, out=None,
                    want_lse=False, workspace=None):
    """Attention of a window's nodes q [B, N, Hq, D] (bfloat16 or float16), already written to the cache at places lens[b] + n,
    over the tokens before the window and each node's ancestors (parent [B, N] int32; None: a chain).  scale None:
    D^-0.5; cap: scores go through cap * tanh(s / cap); slopes [Hq] float32: minus slope * distance; reach: only keys nearer
    than that.  Rows from news[b] on are left as they were.  Returns dict(out [B, N, Hq, D], lse [B, N, Hq] or None)."""
    dt, sq = _window(q, "q")
    B, N, Hq, D = q.shape
    if B != cache.pages.shape[0] or D != cache.D:
        raise SpecVerifyError(SV_EINVAL, f"q: want [{cache.pages.shape[0]}, N, heads, {cache.D}], got {tuple(q.shape)}")
    _int32(lens, (B,), "lens")
    _int32(news, (B,), "news")
    _int32(parent, (B, N), "parent")
    if slopes is not None:
        _want(slopes, torch.float32, (Hq,), "slopes")
    out = torch.empty_like(q) if out is None else out
    if out.dtype is not q.dtype or out.shape != q.shape:
        raise SpecVerifyError(SV_EINVAL, f"out: want {q.dtype} {tuple(q.shape)}, got {out.dtype} {tuple(out.shape)}")
    dev = _one_device("sv_kv_attention", q, cache.pool, lens, news, parent, slopes, out, workspace)
    ws = workspace if workspace is not None else _pass_workspace(dev, SV_PASS_ATTENTION, B, N, Hq, cache.H, D)
    lse = torch.empty(B, N, Hq, dtype=torch.float32, device=dev) if want_lse else None
    _call(dev, _lib.sv_kv_attention, "sv_kv_attention", q.data_ptr(), sq, dt, cache._one("sv_kv_attention"), lens.data_ptr(),
          _at(news), _at(parent), B, N, Hq, float(D ** -0.5 if scale is None else scale), float(cap), _at(slopes),
          max(-1, min(int(reach), 2 ** 31 - 1)), out.data_ptr(), _window(out, "out")[1], _at(lse), ws.data_ptr(), ws.numel())
    _checked(dev, "sv_kv_attention", workspace)
    return dict(out=out, lse=lse)


def sv_kv_commit(cache, lens, n, path=None, out_lens=None, workspace=None):
    """After a verification, in all layers of the cache's pool: the root and the accepted path (n [B], path [B, M] int32:
    sv_verify_tree's len and path; path None: a chain) stay, the path's tokens move next to the root.  n -1 leaves a sequence as
    it was.  Returns the new lengths lens + 1 + n [B] (out_lens: where to write them, not lens itself)."""
    B = cache.pages.shape[0]
    _int32(lens, (B,), "lens")
    _int32(n, (B,), "n")
    if path is not None:
        if path.dim() != 2:
            raise SpecVerifyError(SV_EINVAL, f"path: want [{B}, M], got {tuple(path.shape)}")
        _int32(path, (B, path.shape[1]), "path")
    if out_lens is None:
        out_lens = torch.empty_like(lens)
    _int32(out_lens, (B,), "out_lens")
    dev = _one_device("sv_kv_commit", cache.pool, lens, n, path, out_lens, workspace)
    ws = workspace if workspace is not None else _pass_workspace(dev, SV_PASS_COMMIT)
    # a path without places has no address, and none would say a chain: any other will do, nothing of it is read
    M, at = (0, None) if path is None else (path.shape[1], path.data_ptr() or lens.data_ptr())
    _call(dev, _lib.sv_kv_commit, "sv_kv_commit", cache._ref, lens.data_ptr(), n.data_ptr(), at, B, M, out_lens.data_ptr(),
          ws.data_ptr(), ws.numel())
    _checked(dev, "sv_kv_commit", workspace)
    return out_lens
