"""Python binding of liblizard.so: argument marshalling only.

Every function here checks tensor shapes, dtypes and contiguity, then calls the
C entry point of the same name with raw device pointers and the current CUDA
stream.  All arithmetic runs in the library's CUDA kernels; there is no CPU
path.  If the library has not been built, loading it raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import numpy as np

import torch

from . import _build

LIZARD_OK = 0
LIZARD_ERR_INVALID_ARG = 1
LIZARD_ERR_UNSUPPORTED = 2
LIZARD_ERR_WORKSPACE = 3
LIZARD_ERR_CUDA = 4
LIZARD_ERR_TIMEOUT = 5
LIZARD_F32 = 0
LIZARD_BF16 = 1
# decay readings (include/lizard.h, lizard_decay)
LIZARD_DECAY_DELAYED = 0
LIZARD_DECAY_MASKED = 1
LIZARD_DECAY_LAGGED = 2
# lizard_act
LIZARD_ACT_NONE = 0
LIZARD_ACT_SILU = 1
LIZARD_ACT_SIGMOID = 2

EXPORTED = ["lizard_attn_fwd_workspace", "lizard_workspace_init", "lizard_attn_fwd",
            "lizard_attn_bwd_workspace", "lizard_attn_bwd", "lizard_decode_workspace",
            "lizard_decode_step", "lizard_decode_step_positions", "lizard_read_device_status",
            "lizard_status_string",
            "lizard_profile_events", "lizard_version", "lizard_attn_fwd_noalloc",
            "lizard_attn_fwd_kernel", "lizard_selftest_wait_timeout", "lizard_attn_fwd_varlen",
            "lizard_attn_fwd_varlen_workspace",
            "lizard_attn_bwd_varlen_workspace", "lizard_attn_bwd_varlen",
            "lizard_attn_fwd_noalloc_scratch", "lizard_read_noalloc_status",
            "lizard_qkvg_proj", "lizard_qkvg_proj_bwd", "lizard_gate_cache_fill",
            "lizard_conv_fwd", "lizard_conv_bwd_workspace", "lizard_conv_bwd", "lizard_conv_step",
            "lizard_scan_fwd_workspace", "lizard_scan_states_bytes", "lizard_scan_fwd",
            "lizard_scan_bwd_workspace", "lizard_scan_bwd", "lizard_scan_step",
            "lizard_block_norm_fwd", "lizard_block_norm_bwd_workspace", "lizard_block_norm_bwd"]


class lizard_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("L", ctypes.c_int64), ("Hq", ctypes.c_int64),
                ("Hkv", ctypes.c_int64), ("d", ctypes.c_int64), ("D", ctypes.c_int64),
                ("w", ctypes.c_int64), ("M", ctypes.c_int64), ("chunk", ctypes.c_int64),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("decay", ctypes.c_int32)]


def _fields(int64s: str, floats: str, int32s: str):
    return [(n, t) for names, t in ((int64s, ctypes.c_int64), (floats, ctypes.c_float),
                                    (int32s, ctypes.c_int32)) for n in names.split()]


class lizard_conv_dims(ctypes.Structure):
    _fields_ = _fields("B L C K nseq ldx ldy lddx", "", "dtype act")


class lizard_scan_dims(ctypes.Structure):
    _fields_ = _fields("B L C N G nseq ldx lddt ldz ldb ldc ldy lddx ldddt lddz lddb lddc", "",
                       "dtype softplus")


class lizard_norm_dims(ctypes.Structure):
    _fields_ = _fields("T D groups ldo ldg ldr ldro ldn lddo lddg lddr", "eps_post eps_pre",
                       "dtype res_dtype act gate_first")


class LizardError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None
_VP = ctypes.c_void_p
_DP = ctypes.POINTER(lizard_dims)


def load(path: str | None = None) -> ctypes.CDLL:
    """Load liblizard.so; raises if it is missing (build it with __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: the CUDA library must be built first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    lib.lizard_attn_fwd_workspace.argtypes = [_DP]
    lib.lizard_attn_fwd_workspace.restype = ctypes.c_size_t
    lib.lizard_attn_bwd_workspace.argtypes = [_DP]
    lib.lizard_attn_bwd_workspace.restype = ctypes.c_size_t
    lib.lizard_decode_workspace.argtypes = [_DP]
    lib.lizard_decode_workspace.restype = ctypes.c_size_t
    lib.lizard_selftest_wait_timeout.argtypes = [_VP, ctypes.c_size_t, ctypes.c_longlong, _VP]
    lib.lizard_selftest_wait_timeout.restype = ctypes.c_int
    lib.lizard_attn_fwd_kernel.argtypes = [_DP]
    lib.lizard_attn_fwd_kernel.restype = ctypes.c_int
    lib.lizard_workspace_init.argtypes = [_VP, ctypes.c_size_t, _VP]
    lib.lizard_workspace_init.restype = ctypes.c_int
    lib.lizard_attn_fwd.argtypes = [_DP] + [_VP] * 13 + [ctypes.c_size_t, _VP]
    lib.lizard_attn_fwd.restype = ctypes.c_int
    lib.lizard_attn_fwd_varlen_workspace.argtypes = [_DP, _VP]
    lib.lizard_attn_fwd_varlen_workspace.restype = ctypes.c_size_t
    lib.lizard_attn_fwd_varlen.argtypes = [_DP, _VP] + [_VP] * 13 + [ctypes.c_size_t, _VP]
    lib.lizard_attn_fwd_varlen.restype = ctypes.c_int
    lib.lizard_attn_bwd_varlen_workspace.argtypes = [_DP, _VP]
    lib.lizard_attn_bwd_varlen_workspace.restype = ctypes.c_size_t
    lib.lizard_attn_bwd_varlen.argtypes = [_DP, _VP] + [_VP] * 16 + [ctypes.c_size_t, _VP]
    lib.lizard_attn_bwd_varlen.restype = ctypes.c_int
    lib.lizard_attn_fwd_noalloc.argtypes = [_DP] + [_VP] * 13
    lib.lizard_attn_fwd_noalloc.restype = ctypes.c_int
    lib.lizard_attn_fwd_noalloc_scratch.argtypes = [_DP]
    lib.lizard_attn_fwd_noalloc_scratch.restype = ctypes.c_size_t
    lib.lizard_read_noalloc_status.argtypes = [_VP]
    lib.lizard_read_noalloc_status.restype = ctypes.c_int
    lib.lizard_qkvg_proj.argtypes = [_DP, ctypes.c_int64] + [_VP] * 7 + [ctypes.c_size_t, _VP]
    lib.lizard_qkvg_proj.restype = ctypes.c_int
    lib.lizard_qkvg_proj_bwd.argtypes = [_DP, ctypes.c_int64] + [_VP] * 9 + [ctypes.c_size_t, _VP]
    lib.lizard_qkvg_proj_bwd.restype = ctypes.c_int
    lib.lizard_attn_bwd.argtypes = [_DP] + [_VP] * 16 + [ctypes.c_size_t, _VP]
    lib.lizard_attn_bwd.restype = ctypes.c_int
    lib.lizard_decode_step.argtypes = [_DP, ctypes.c_int64] + [_VP] * 13 + [ctypes.c_size_t, _VP]
    lib.lizard_decode_step.restype = ctypes.c_int
    lib.lizard_decode_step_positions.argtypes = [_DP] + [_VP] * 14 + [ctypes.c_size_t, _VP]
    lib.lizard_decode_step_positions.restype = ctypes.c_int
    lib.lizard_gate_cache_fill.argtypes = [_DP, _VP, _VP, _VP]
    lib.lizard_gate_cache_fill.restype = ctypes.c_int
    lib.lizard_read_device_status.argtypes = [_VP, _VP]
    lib.lizard_read_device_status.restype = ctypes.c_int
    lib.lizard_status_string.argtypes = [ctypes.c_int]
    lib.lizard_status_string.restype = ctypes.c_char_p
    lib.lizard_profile_events.argtypes = [_VP, _VP]
    lib.lizard_profile_events.restype = ctypes.c_int
    dims_of_call = {"conv": ctypes.POINTER(lizard_conv_dims),
                    "scan": ctypes.POINTER(lizard_scan_dims),
                    "block": ctypes.POINTER(lizard_norm_dims)}
    sz = ctypes.c_size_t
    for name, rest in (("lizard_conv_fwd", [_VP] * 8 + [sz, _VP]),
                       ("lizard_conv_bwd", [_VP] * 12 + [sz, _VP]),
                       ("lizard_conv_step", [_VP] * 4 + [ctypes.c_int64] + [_VP] * 3 + [sz, _VP]),
                       ("lizard_scan_fwd", [_VP] * 14 + [sz, _VP]),
                       ("lizard_scan_bwd", [_VP] * 23 + [sz, _VP]),
                       ("lizard_scan_step", [_VP] * 9 + [ctypes.c_int64] + [_VP] * 3 + [sz, _VP]),
                       ("lizard_block_norm_fwd", [_VP] * 9),
                       ("lizard_block_norm_bwd", [_VP] * 15 + [sz, _VP]),
                       ("lizard_conv_bwd_workspace", None), ("lizard_scan_fwd_workspace", None),
                       ("lizard_scan_states_bytes", None), ("lizard_scan_bwd_workspace", None),
                       ("lizard_block_norm_bwd_workspace", None)):
        fn = getattr(lib, name)
        fn.argtypes = [dims_of_call[name.split("_")[1]]] + (rest or [])
        fn.restype = sz if rest is None else ctypes.c_int
    lib.lizard_version.argtypes = []
    lib.lizard_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().lizard_status_string(status).decode()


def lizard_version() -> str:
    return load().lizard_version().decode()


def _check(status: int, where: str):
    if status != LIZARD_OK:
        raise LizardError(status, where)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None or stream is _HERE:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _under(stream):
    """Context in which `stream` (None: the current one) is the current stream."""
    if stream is None or stream is _HERE:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


@functools.cache
def _gpus() -> int:
    return torch.cuda.device_count()


def _one_device(args):
    """Launches go to the current device: tensors of another one are refused."""
    here = torch.cuda.current_device()
    for t in args:
        if getattr(t, "is_cuda", False) and t.device.index != here:
            raise ValueError(f"a tensor is on device {t.device}, the current device is cuda:{here}")


_HERE = object()  # for `stream`: the current stream, everything has been looked at


def _placed(fn, given):
    """Runs a call, given its arguments by name, under the stream it is given, so that what it
    allocates (workspaces, copies of offsets, outputs) belongs to that stream: memory of the current
    stream's pool may still be in use there, and goes back to it while the kernels on the other stream
    run."""
    with _under(given["stream"]):
        if _gpus() > 1:
            _one_device(given.values())
        return fn(**dict(given, stream=_HERE))


def _ws(workspace):
    """Address and bytes of an optional workspace."""
    if workspace is None:
        return None, 0
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LIZARD_F32
    if t.dtype == torch.bfloat16:
        return LIZARD_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def make_dims(B, L, Hq, Hkv, d, D, w, M, dtype, scale: float = 0.0, chunk: int = 0,
              decay: int = LIZARD_DECAY_DELAYED) -> lizard_dims:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return lizard_dims(B, L, Hq, Hkv, d, D, w, M, chunk, float(scale), code, int(decay))


def dims_of(q, k, g, sinks, w: int, scale: float = 0.0,
            decay: int = LIZARD_DECAY_DELAYED) -> lizard_dims:
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    D = g.shape[-1]
    M = sinks.shape[1]
    return lizard_dims(B, L, Hq, Hkv, d, D, w, M, 0, float(scale), _dtype_code(q), int(decay))


def _need(t, name, shape, dtype):
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {dtype}")
    if not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def lizard_attn_fwd_workspace(dims: lizard_dims) -> int:
    return int(load().lizard_attn_fwd_workspace(ctypes.byref(dims)))


def lizard_attn_fwd_kernel(dims: lizard_dims) -> int:
    """1 if the tensor-core chunk walk serves these sizes, 0 for the SIMT walk, -1 invalid."""
    return int(load().lizard_attn_fwd_kernel(ctypes.byref(dims)))


def lizard_attn_bwd_workspace(dims: lizard_dims) -> int:
    return int(load().lizard_attn_bwd_workspace(ctypes.byref(dims)))


def lizard_decode_workspace(dims: lizard_dims) -> int:
    return int(load().lizard_decode_workspace(ctypes.byref(dims)))


def new_workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """Allocate a workspace (torch owns the memory, which belongs to the stream) and zero its status
    word."""
    with _under(stream):
        ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    _check(load().lizard_workspace_init(_p(ws), ws.numel(), _stream(stream)),
           "lizard_workspace_init")
    return ws


def lizard_profile_events(before=None, after=None):
    """Bracket the dominant kernel of later forward/backward calls with two
    torch.cuda.Event objects (None, None turns it off)."""
    handles = []
    for ev in (before, after):
        if ev is None:
            handles.append(None)
            continue
        if not ev.cuda_event:
            ev.record()  # torch creates the underlying cudaEvent_t on first record
        handles.append(ctypes.c_void_p(ev.cuda_event))
    _check(load().lizard_profile_events(*handles), "lizard_profile_events")


def lizard_selftest_wait_timeout(workspace, limit_cycles: int, stream=None):
    """Run the bounded-wait failure path once (see include/lizard.h).  workspace None targets
    the status word of lizard_attn_fwd_noalloc's fixed array."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().lizard_selftest_wait_timeout(_p(workspace), nbytes, int(limit_cycles),
                                               _stream(stream)), "lizard_selftest_wait_timeout")


def lizard_read_noalloc_status(stream=None) -> int:
    """Synchronise the stream, read and clear lizard_attn_fwd_noalloc's status word."""
    return int(load().lizard_read_noalloc_status(_stream(stream)))


def lizard_attn_fwd_noalloc_scratch(dims) -> int:
    return int(load().lizard_attn_fwd_noalloc_scratch(ctypes.byref(dims)))


def lizard_read_device_status(workspace: torch.Tensor, stream=None) -> int:
    return int(load().lizard_read_device_status(_p(workspace), _stream(stream)))


def lizard_attn_fwd(q, k, v, g, Wf, sinks, w: int, *, scale: float = 0.0, y=None, lse=None,
                    S_out=None, z_out=None, kcache_out=None, vcache_out=None, workspace=None,
                    stream=None, decay: int = LIZARD_DECAY_DELAYED):
    """Forward over L tokens.  Returns y [B, L, Hq, d] (allocated if not given).  `decay`
    selects the decay reading (LIZARD_DECAY_*)."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_attn_fwd, locals())
    B, L, Hq, d = q.shape
    Hkv, D, M = k.shape[2], g.shape[-1], sinks.shape[1]
    dt = q.dtype
    _need(q, "q", (B, L, Hq, d), dt)
    _need(k, "k", (B, L, Hkv, d), dt)
    _need(v, "v", (B, L, Hkv, d), dt)
    _need(g, "g", (B, L, Hkv, D), dt)
    _need(Wf, "Wf", (Hkv, d, D // 2), dt)
    _need(sinks, "sinks", (Hq, M), torch.float32)
    if y is None:
        y = torch.empty_like(q)
    _need(y, "y", (B, L, Hq, d), dt)
    if lse is not None:
        _need(lse, "lse", (B, L, Hq), torch.float32)
    if S_out is not None:
        _need(S_out, "S_out", (B, Hkv, D, d), torch.float32)
        _need(z_out, "z_out", (B, Hkv, D), torch.float32)
    if kcache_out is not None:
        _need(kcache_out, "kcache_out", (B, Hkv, w + 1, d), dt)
        _need(vcache_out, "vcache_out", (B, Hkv, w + 1, d), dt)
    dims = dims_of(q, k, g, sinks, w, scale, decay)
    if workspace is None:
        workspace = new_workspace(lizard_attn_fwd_workspace(dims), q.device, stream)
    st = load().lizard_attn_fwd(ctypes.byref(dims), _p(q), _p(k), _p(v), _p(g), _p(Wf),
                                _p(sinks), _p(y), _p(lse), _p(S_out), _p(z_out), _p(kcache_out),
                                _p(vcache_out), *_ws(workspace),
                                _stream(stream))
    _check(st, "lizard_attn_fwd")
    return y


def lizard_attn_fwd_varlen_workspace(dims, cu_seqlens) -> int:
    """Workspace bytes for one launch of lizard_attn_fwd_varlen over all sequences."""
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int64))
    return int(load().lizard_attn_fwd_varlen_workspace(ctypes.byref(dims), cu.ctypes.data))


def lizard_attn_fwd_varlen(q, k, v, g, Wf, sinks, w: int, cu_seqlens, *, scale: float = 0.0,
                           y=None, lse=None, S_out=None, z_out=None, kcache_out=None,
                           vcache_out=None, workspace=None, stream=None,
                           decay: int = LIZARD_DECAY_DELAYED):
    """Forward over a packed batch: q [T, Hq, d], k, v [T, Hkv, d], g [T, Hkv, D], and
    cu_seqlens (host integers, B + 1 offsets) delimiting B sequences.  Returns y [T, Hq, d];
    S_out, z_out, kcache_out, vcache_out hold one entry per sequence."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_attn_fwd_varlen, locals())
    T, Hq, d = q.shape
    Hkv, D, M = k.shape[1], g.shape[-1], sinks.shape[1]
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int64))
    nseq = cu.shape[0] - 1
    dt = q.dtype
    _need(q, "q", (T, Hq, d), dt)
    _need(k, "k", (T, Hkv, d), dt)
    _need(v, "v", (T, Hkv, d), dt)
    _need(g, "g", (T, Hkv, D), dt)
    _need(Wf, "Wf", (Hkv, d, D // 2), dt)
    _need(sinks, "sinks", (Hq, M), torch.float32)
    if y is None:
        y = torch.empty_like(q)
    _need(y, "y", (T, Hq, d), dt)
    if lse is not None:
        _need(lse, "lse", (T, Hq), torch.float32)
    if S_out is not None:
        _need(S_out, "S_out", (nseq, Hkv, D, d), torch.float32)
        _need(z_out, "z_out", (nseq, Hkv, D), torch.float32)
    if kcache_out is not None:
        _need(kcache_out, "kcache_out", (nseq, Hkv, w + 1, d), dt)
        _need(vcache_out, "vcache_out", (nseq, Hkv, w + 1, d), dt)
    dims = lizard_dims(nseq, T, Hq, Hkv, d, D, w, M, 0, float(scale), _dtype_code(q), int(decay))
    if workspace is None:  # the size of one launch over all sequences
        workspace = new_workspace(lizard_attn_fwd_varlen_workspace(dims, cu), q.device, stream)
    st = load().lizard_attn_fwd_varlen(ctypes.byref(dims), cu.ctypes.data, _p(q), _p(k), _p(v),
                                       _p(g), _p(Wf), _p(sinks), _p(y), _p(lse), _p(S_out),
                                       _p(z_out), _p(kcache_out), _p(vcache_out), *_ws(workspace), _stream(stream))
    _check(st, "lizard_attn_fwd_varlen")
    return y


def lizard_attn_fwd_noalloc(q, k, v, g, Wf, sinks, w: int, *, scale: float = 0.0, y=None,
                            lse=None, S_out=None, z_out=None, kcache_out=None, vcache_out=None,
                            stream=None, decay: int = LIZARD_DECAY_DELAYED):
    """The forward without a workspace, for callers that cannot allocate device memory.

    Same arguments and result as lizard_attn_fwd; the library keeps the scratch in a
    fixed 32 MiB device array (see include/lizard.h for the limit and the sharing rules).
    `y` is allocated here only for the Python caller's convenience when not given."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_attn_fwd_noalloc, locals())
    B, L, Hq, d = q.shape
    Hkv, D, M = k.shape[2], g.shape[-1], sinks.shape[1]
    dt = q.dtype
    _need(q, "q", (B, L, Hq, d), dt)
    _need(k, "k", (B, L, Hkv, d), dt)
    _need(v, "v", (B, L, Hkv, d), dt)
    _need(g, "g", (B, L, Hkv, D), dt)
    _need(Wf, "Wf", (Hkv, d, D // 2), dt)
    _need(sinks, "sinks", (Hq, M), torch.float32)
    if y is None:
        y = torch.empty_like(q)
    _need(y, "y", (B, L, Hq, d), dt)
    dims = dims_of(q, k, g, sinks, w, scale, decay)
    st = load().lizard_attn_fwd_noalloc(ctypes.byref(dims), _p(q), _p(k), _p(v), _p(g), _p(Wf),
                                        _p(sinks), _p(y), _p(lse), _p(S_out), _p(z_out),
                                        _p(kcache_out), _p(vcache_out), _stream(stream))
    _check(st, "lizard_attn_fwd_noalloc")
    return y


def lizard_attn_bwd(q, k, v, g, Wf, sinks, y, lse, dy, w: int, *, scale: float = 0.0,
                    dq=None, dk=None, dv=None, dg=None, dWf=None, dsinks=None, workspace=None,
                    stream=None, decay: int = LIZARD_DECAY_DELAYED):
    """Gradients (dq, dk, dv, dg, dWf, dsinks) of y against dy (same decay reading as the
    forward that made y)."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_attn_bwd, locals())
    B, L, Hq, d = q.shape
    Hkv, D, M = k.shape[2], g.shape[-1], sinks.shape[1]
    dt = q.dtype
    for t, n, shp in ((q, "q", (B, L, Hq, d)), (k, "k", (B, L, Hkv, d)), (v, "v", (B, L, Hkv, d)),
                      (g, "g", (B, L, Hkv, D)), (Wf, "Wf", (Hkv, d, D // 2)),
                      (y, "y", (B, L, Hq, d)), (dy, "dy", (B, L, Hq, d))):
        _need(t, n, shp, dt)
    _need(sinks, "sinks", (Hq, M), torch.float32)
    _need(lse, "lse", (B, L, Hq), torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dg = torch.empty_like(g) if dg is None else dg
    dWf = torch.empty(Hkv, d, D // 2, dtype=torch.float32, device=q.device) if dWf is None else dWf
    dsinks = torch.empty(Hq, M, dtype=torch.float32, device=q.device) if dsinks is None else dsinks
    dims = dims_of(q, k, g, sinks, w, scale, decay)
    if workspace is None:
        workspace = new_workspace(lizard_attn_bwd_workspace(dims), q.device, stream)
    st = load().lizard_attn_bwd(ctypes.byref(dims), _p(q), _p(k), _p(v), _p(g), _p(Wf),
                                _p(sinks), _p(y), _p(lse), _p(dy), _p(dq), _p(dk), _p(dv),
                                _p(dg), _p(dWf), _p(dsinks), *_ws(workspace),
                                _stream(stream))
    _check(st, "lizard_attn_bwd")
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dWf=dWf, dsinks=dsinks)


def lizard_attn_bwd_varlen_workspace(dims, cu_seqlens) -> int:
    """Workspace bytes of lizard_attn_bwd_varlen for this packed batch (0: bad offsets)."""
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int64))
    return int(load().lizard_attn_bwd_varlen_workspace(ctypes.byref(dims), cu.ctypes.data))


def lizard_attn_bwd_varlen(q, k, v, g, Wf, sinks, y, lse, dy, w: int, cu_seqlens, *,
                           scale: float = 0.0, workspace=None, stream=None,
                           decay: int = LIZARD_DECAY_DELAYED):
    """Gradients of lizard_attn_fwd_varlen's y against dy for a packed batch: dq, dk, dv,
    dg packed like the inputs; dWf and dsinks summed over the sequences."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_attn_bwd_varlen, locals())
    T, Hq, d = q.shape
    Hkv, D, M = k.shape[1], g.shape[-1], sinks.shape[1]
    cu = np.asarray(cu_seqlens, dtype=np.int64)
    nseq = cu.shape[0] - 1
    dt = q.dtype
    for t, n, shp in ((q, "q", (T, Hq, d)), (k, "k", (T, Hkv, d)), (v, "v", (T, Hkv, d)),
                      (g, "g", (T, Hkv, D)), (Wf, "Wf", (Hkv, d, D // 2)),
                      (y, "y", (T, Hq, d)), (dy, "dy", (T, Hq, d))):
        _need(t, n, shp, dt)
    _need(sinks, "sinks", (Hq, M), torch.float32)
    _need(lse, "lse", (T, Hq), torch.float32)
    dq, dk, dv, dg = (torch.empty_like(x) for x in (q, k, v, g))
    dWf = torch.empty(Hkv, d, D // 2, dtype=torch.float32, device=q.device)
    dsinks = torch.empty(Hq, M, dtype=torch.float32, device=q.device)
    dims = lizard_dims(nseq, T, Hq, Hkv, d, D, w, M, 0, float(scale), _dtype_code(q), int(decay))
    if workspace is None:
        nbytes = int(load().lizard_attn_bwd_varlen_workspace(ctypes.byref(dims), cu.ctypes.data))
        if nbytes == 0:
            raise ValueError("cu_seqlens: inconsistent offsets")
        workspace = new_workspace(nbytes, q.device, stream)
    st = load().lizard_attn_bwd_varlen(ctypes.byref(dims), cu.ctypes.data, _p(q), _p(k), _p(v),
                                       _p(g), _p(Wf), _p(sinks), _p(y), _p(lse), _p(dy),
                                       _p(dq), _p(dk), _p(dv), _p(dg), _p(dWf), _p(dsinks),
                                       *_ws(workspace), _stream(stream))
    _check(st, "lizard_attn_bwd_varlen")
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dWf=dWf, dsinks=dsinks)


def _decode_common(q, k, v, g, Wf, sinks, S, z, kcache, vcache, gcache, w, decay):
    B, Hq, d = q.shape
    Hkv, D, M = k.shape[1], g.shape[-1], sinks.shape[1]
    dt = q.dtype
    _need(k, "k", (B, Hkv, d), dt)
    _need(v, "v", (B, Hkv, d), dt)
    _need(g, "g", (B, Hkv, D), dt)
    _need(Wf, "Wf", (Hkv, d, D // 2), dt)
    _need(sinks, "sinks", (Hq, M), torch.float32)
    _need(S, "S", (B, Hkv, D, d), torch.float32)
    _need(z, "z", (B, Hkv, D), torch.float32)
    _need(kcache, "kcache", (B, Hkv, w + 1, d), dt)
    _need(vcache, "vcache", (B, Hkv, w + 1, d), dt)
    if decay != LIZARD_DECAY_DELAYED or gcache is not None:
        _need(gcache, "gcache", (B, Hkv, w + 1, D), dt)
    return B, Hq, Hkv, d, D, M


def lizard_decode_step(pos: int, q, k, v, g, Wf, sinks, S, z, kcache, vcache, w: int, *,
                       scale: float = 0.0, y=None, workspace=None, stream=None, gcache=None,
                       decay: int = LIZARD_DECAY_DELAYED):
    """One decode step at position pos; S, z, kcache, vcache (and gcache, the gate ring the
    MASKED and LAGGED readings need) are updated in place."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_decode_step, locals())
    B, Hq, Hkv, d, D, M = _decode_common(q, k, v, g, Wf, sinks, S, z, kcache, vcache, gcache,
                                         w, decay)
    y = torch.empty_like(q) if y is None else y
    dims = lizard_dims(B, 1, Hq, Hkv, d, D, w, M, 0, float(scale), _dtype_code(q), int(decay))
    if workspace is None:
        workspace = new_workspace(lizard_decode_workspace(dims), q.device, stream)
    st = load().lizard_decode_step(ctypes.byref(dims), int(pos), _p(q), _p(k), _p(v), _p(g),
                                   _p(Wf), _p(sinks), _p(y), _p(S), _p(z), _p(kcache),
                                   _p(vcache), _p(gcache), *_ws(workspace),
                                   _stream(stream))
    _check(st, "lizard_decode_step")
    return y


def lizard_decode_step_positions(pos, q, k, v, g, Wf, sinks, S, z, kcache, vcache, w: int, *,
                                 scale: float = 0.0, y=None, workspace=None, stream=None,
                                 gcache=None, decay: int = LIZARD_DECAY_DELAYED):
    """One decode step with a position per sequence: pos is an int64 device tensor [B],
    read when the kernel runs.  A negative entry is reported through the workspace status
    (lizard_read_device_status) and leaves that sequence untouched."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_decode_step_positions, locals())
    B = q.shape[0]
    _need(pos, "pos", (B,), torch.int64)
    B, Hq, Hkv, d, D, M = _decode_common(q, k, v, g, Wf, sinks, S, z, kcache, vcache, gcache,
                                         w, decay)
    y = torch.empty_like(q) if y is None else y
    dims = lizard_dims(B, 1, Hq, Hkv, d, D, w, M, 0, float(scale), _dtype_code(q), int(decay))
    if workspace is None:
        workspace = new_workspace(lizard_decode_workspace(dims), q.device, stream)
    st = load().lizard_decode_step_positions(ctypes.byref(dims), _p(pos), _p(q), _p(k), _p(v),
                                             _p(g), _p(Wf), _p(sinks), _p(y), _p(S), _p(z),
                                             _p(kcache), _p(vcache), _p(gcache), *_ws(workspace), _stream(stream))
    _check(st, "lizard_decode_step_positions")
    return y


def lizard_gate_cache_fill(g, gcache, w: int, *, stream=None):
    """Gate ring of a prefill: the gate rows of the last min(L, w) tokens of g [B, L, Hkv, D]
    go to slot t mod (w+1) of gcache [B, Hkv, w+1, D] (same dtype)."""
    B, L, Hkv, D = g.shape
    _need(g, "g", (B, L, Hkv, D), g.dtype)
    _need(gcache, "gcache", (B, Hkv, w + 1, D), g.dtype)
    dims = lizard_dims(B, L, Hkv, Hkv, D, D, w, 0, 0, 0.0, _dtype_code(g))
    _check(load().lizard_gate_cache_fill(ctypes.byref(dims), _p(g), _p(gcache), _stream(stream)),
           "lizard_gate_cache_fill")


def lizard_qkvg_proj(x, W, Hq: int, Hkv: int, d: int, D: int, *, q=None, k=None, v=None,
                     g=None, workspace=None, stream=None):
    """[q | k | v | g] = x W^T on the tensor cores.  x [B, L, dm], W [N, dm] (bf16).
    Returns (q, k, v, g) in the mixer's layouts (allocated if not given)."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_qkvg_proj, locals())
    B, L, dm = x.shape
    N = Hq * d + 2 * Hkv * d + Hkv * D
    _need(x, "x", (B, L, dm), torch.bfloat16)
    _need(W, "W", (N, dm), torch.bfloat16)
    outs = []
    for t, name, shape in ((q, "q", (B, L, Hq, d)), (k, "k", (B, L, Hkv, d)),
                           (v, "v", (B, L, Hkv, d)), (g, "g", (B, L, Hkv, D))):
        if t is None:
            t = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
        _need(t, name, shape, torch.bfloat16)
        outs.append(t)
    dims = make_dims(B, L, Hq, Hkv, d, D, 1, 0, LIZARD_BF16)
    st = load().lizard_qkvg_proj(ctypes.byref(dims), dm, _p(x), _p(W), *[_p(t) for t in outs],
                                 *_ws(workspace), _stream(stream))
    _check(st, "lizard_qkvg_proj")
    return tuple(outs)


def lizard_qkvg_proj_bwd(x, W, dq, dk, dv, dg, *, dx=None, dW=None, workspace=None,
                         stream=None):
    """dx = dY W (bf16) and dW = dY^T x (fp32) for dY = [dq | dk | dv | dg]."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_qkvg_proj_bwd, locals())
    B, L, dm = x.shape
    Hq, d = dq.shape[2], dq.shape[3]
    Hkv, D = dg.shape[2], dg.shape[3]
    N = Hq * d + 2 * Hkv * d + Hkv * D
    _need(x, "x", (B, L, dm), torch.bfloat16)
    _need(W, "W", (N, dm), torch.bfloat16)
    _need(dq, "dq", (B, L, Hq, d), torch.bfloat16)
    _need(dk, "dk", (B, L, Hkv, d), torch.bfloat16)
    _need(dv, "dv", (B, L, Hkv, d), torch.bfloat16)
    _need(dg, "dg", (B, L, Hkv, D), torch.bfloat16)
    if dx is None:
        dx = torch.empty_like(x)
    if dW is None:
        dW = torch.empty(N, dm, dtype=torch.float32, device=x.device)
    _need(dx, "dx", (B, L, dm), torch.bfloat16)
    _need(dW, "dW", (N, dm), torch.float32)
    dims = make_dims(B, L, Hq, Hkv, d, D, 1, 0, LIZARD_BF16)
    st = load().lizard_qkvg_proj_bwd(ctypes.byref(dims), dm, _p(x), _p(W), _p(dq), _p(dk),
                                     _p(dv), _p(dg), _p(dx), _p(dW), *_ws(workspace),
                                     _stream(stream))
    _check(st, "lizard_qkvg_proj_bwd")
    return dx, dW


# ---- the selective state space block -----------------------------------------------------
#
# Activations are [B, L, width] (dtype fp32 or bf16) and may be column ranges of wider rows: the
# last axes contiguous, every token the same distance after the one before.  Parameters, scan
# states and parameter gradients are fp32 and contiguous.  cu_seqlens packs sequences into one row
# (B = 1): int64 offsets on the device, read when the kernels run, or host integers, which are
# checked and copied (the host waits for the copy).  What a call allocates belongs to the stream it
# runs on: `stream`, or the current one.


def _ld(t, name, shape, dtype, lead=2):
    """Distance between the token rows of t (0 when dense); the first `lead` axes of `shape`
    count tokens."""
    if t.shape == shape and t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return 0
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {shape}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    st, width = t.stride(), 1
    for size, stride in zip(reversed(shape[lead:]), reversed(st[lead:])):
        if size > 1 and stride != width:
            raise ValueError(f"{name}: the values of a token must be contiguous")
        width *= size
    if lead == 1:
        ld, even = st[0], True
    else:
        ld = st[1] if shape[1] > 1 else st[0]
        even = shape[0] == 1 or shape[1] == 1 or st[0] == shape[1] * st[1]
    if not even or ld < width:
        raise ValueError(f"{name}: token rows must be evenly spaced and not overlap")
    return ld


def _need_f32(t, name, shape):
    """An optional fp32 parameter or state; its address (None when absent)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not torch.float32 or not t.is_cuda or not t.is_contiguous():
        _need(t, name, shape, torch.float32)
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(t):
    """Handle of the current stream of t's device (without making the Stream object, which costs
    as much as a launch)."""
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _packed(cu_seqlens, B, L, device):
    """(number of packed sequences, device offsets or None)."""
    if cu_seqlens is None:
        return 0, None
    if B != 1:
        raise ValueError("cu_seqlens packs sequences into one row: B must be 1")
    if not (isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.is_cuda):
        cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int64))
        if cu.ndim != 1 or cu.size < 2 or cu[0] != 0 or cu[-1] != L or (np.diff(cu) < 0).any():
            raise ValueError("cu_seqlens: inconsistent offsets")
        cu_seqlens = torch.from_numpy(cu).to(device)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens: at least two offsets in one axis")
    _need(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int64)
    return cu_seqlens.numel() - 1, cu_seqlens


def _scratch(workspace, nbytes, device):
    """A workspace of the call's own (its status word is not read by anyone) where none is
    given."""
    if workspace is not None:
        return workspace
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _slots(slots, B):
    if slots is None:
        return None
    if slots.shape != (B,) or slots.dtype is not torch.int64 or not slots.is_cuda or not slots.is_contiguous():
        _need(slots, "slots", (B,), torch.int64)
    return slots.data_ptr()


def lizard_conv_fwd(x, w, bias=None, *, act: int = LIZARD_ACT_NONE, state_in=None, state_out=None,
                    cu_seqlens=None, y=None, workspace=None, stream=None):
    """Short causal depthwise convolution of x [B, L, C] with w [C, K]; returns y [B, L, C].
    state_in, state_out [B or sequences, K-1, C]: the inputs before each sequence's first token
    and its last ones (state_out may be state_in)."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_conv_fwd, locals())
    B, L, C = x.shape
    K, dt = w.shape[1], x.dtype
    nseq, cu = _packed(cu_seqlens, B, L, x.device)
    n = nseq or B
    if y is None:
        y = x.new_empty((B, L, C))
    for t, name in ((state_in, "state_in"), (state_out, "state_out")):
        if t is not None:
            _need(t, name, (n, K - 1, C), dt)
    dims = lizard_conv_dims(B, L, C, K, nseq, _ld(x, "x", (B, L, C), dt),
                            _ld(y, "y", (B, L, C), dt), 0, _dtype_code(x), act)
    st = load().lizard_conv_fwd(ctypes.byref(dims), x.data_ptr(), _need_f32(w, "w", (C, K)),
                                _need_f32(bias, "bias", (C,)), _ptr(state_in), _ptr(cu),
                                y.data_ptr(), _ptr(state_out), *_ws(workspace),
                                _stream_of(x))
    _check(st, "lizard_conv_fwd")
    return y


def lizard_conv_bwd_workspace(dims) -> int:
    return int(load().lizard_conv_bwd_workspace(ctypes.byref(dims)))


def lizard_conv_bwd(x, w, bias, dy, *, act: int = LIZARD_ACT_NONE, state_in=None,
                    dstate_out=None, dstate_in=None, cu_seqlens=None, dx=None, workspace=None,
                    stream=None):
    """Gradients dx, dw, dbias of lizard_conv_fwd's y against dy (bias and dbias may be None);
    dstate_out is the gradient of state_out, dstate_in (if given) receives that of state_in."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_conv_bwd, locals())
    B, L, C = x.shape
    K, dt = w.shape[1], x.dtype
    nseq, cu = _packed(cu_seqlens, B, L, x.device)
    n = nseq or B
    if dx is None:
        dx = x.new_empty((B, L, C))
    for t, name in ((state_in, "state_in"), (dstate_out, "dstate_out"), (dstate_in, "dstate_in")):
        if t is not None:
            _need(t, name, (n, K - 1, C), dt)
    dw = torch.empty((C, K), dtype=torch.float32, device=x.device)
    dbias = None if bias is None else torch.empty_like(bias)
    dims = lizard_conv_dims(B, L, C, K, nseq, _ld(x, "x", (B, L, C), dt),
                            _ld(dy, "dy", (B, L, C), dt), _ld(dx, "dx", (B, L, C), dt),
                            _dtype_code(x), act)
    workspace = _scratch(workspace, lizard_conv_bwd_workspace(dims), x.device)
    st = load().lizard_conv_bwd(ctypes.byref(dims), x.data_ptr(), _need_f32(w, "w", (C, K)),
                                _need_f32(bias, "bias", (C,)), _ptr(state_in), _ptr(cu),
                                dy.data_ptr(), _ptr(dstate_out), dx.data_ptr(), dw.data_ptr(),
                                _ptr(dbias), _ptr(dstate_in), *_ws(workspace),
                                _stream_of(x))
    _check(st, "lizard_conv_bwd")
    return dict(dx=dx, dw=dw, dbias=dbias, dstate_in=dstate_in)


def lizard_conv_step(x, w, bias, state, *, slots=None, act: int = LIZARD_ACT_NONE, y=None,
                     workspace=None, stream=None):
    """One token for each of B sequences: y [B, C] from x [B, C]; state [slots, K-1, C] is moved
    on IN PLACE.  slots: int64 device tensor [B] naming each row's state (negative: an idle row),
    or None (row b uses entry b)."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_conv_step, locals())
    B, C = x.shape
    K, dt = w.shape[1], x.dtype
    ldy = 0
    if y is None:
        y = x.new_empty((B, C))
    else:
        ldy = _ld(y, "y", (B, C), dt, 1)
    if _ld(state, "state", (state.shape[0], K - 1, C), dt, 1):
        raise ValueError("state must be a contiguous CUDA tensor")
    dims = lizard_conv_dims(B, 1, C, K, 0, _ld(x, "x", (B, C), dt, 1), ldy, 0, _dtype_code(x), act)
    st = load().lizard_conv_step(ctypes.byref(dims), x.data_ptr(), _need_f32(w, "w", (C, K)),
                                 _need_f32(bias, "bias", (C,)), state.data_ptr(), state.shape[0],
                                 _slots(slots, B), y.data_ptr(), *_ws(workspace),
                                 _stream_of(x))
    _check(st, "lizard_conv_step")
    return y


def _scan_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, nseq):
    """lizard_scan_dims of the inputs, and the addresses of x, dt, A, Bm, Cm, D, z, dt_bias."""
    tp, lead = x.dtype, tuple(x.shape[:-1])
    n = len(lead)
    C, N = A.shape
    G = Bm.shape[-2]
    wide, group = lead + (C,), lead + (G, N)
    dims = lizard_scan_dims(lead[0], lead[1] if n == 2 else 1, C, N, G, nseq,
                            _ld(x, "x", wide, tp, n), _ld(dt, "dt", wide, tp, n),
                            0 if z is None else _ld(z, "z", wide, tp, n),
                            _ld(Bm, "Bm", group, tp, n), _ld(Cm, "Cm", group, tp, n), 0, 0, 0, 0, 0, 0,
                            _dtype_code(x), 1 if softplus else 0)
    return dims, (x.data_ptr(), dt.data_ptr(), _need_f32(A, "A", (C, N)), Bm.data_ptr(),
                  Cm.data_ptr(), _need_f32(D, "D", (C,)), _ptr(z),
                  _need_f32(dt_bias, "dt_bias", (C,)))


def lizard_scan_fwd_workspace(dims) -> int:
    return int(load().lizard_scan_fwd_workspace(ctypes.byref(dims)))


def lizard_scan_bwd_workspace(dims) -> int:
    return int(load().lizard_scan_bwd_workspace(ctypes.byref(dims)))


def lizard_scan_states_bytes(dims) -> int:
    return int(load().lizard_scan_states_bytes(ctypes.byref(dims)))


def lizard_scan_fwd(x, dt, A, Bm, Cm, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                    h0=None, h_out=None, cu_seqlens=None, y=None, save_states: bool = False,
                    workspace=None, stream=None):
    """Selective scan of x [B, L, C] with step sizes dt [B, L, C], rates A [C, N], input and
    output vectors Bm, Cm [B, L, G, N], skip D [C] and output gate z [B, L, C]; returns y, or
    (y, states) with save_states, which lizard_scan_bwd takes.  h0, h_out [B or sequences, C, N]
    fp32: the states before and after (h_out may be h0)."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_scan_fwd, locals())
    B, L, C = x.shape
    nseq, cu = _packed(cu_seqlens, B, L, x.device)
    dims, ptrs = _scan_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, nseq)
    if y is None:
        y = x.new_empty((B, L, C))
    else:
        dims.ldy = _ld(y, "y", (B, L, C), x.dtype)
    shape = (nseq or B, C, A.shape[1])
    lib = load()
    states = None
    if save_states:
        states = torch.empty(lizard_scan_states_bytes(dims), dtype=torch.uint8, device=x.device)
    workspace = _scratch(workspace, lib.lizard_scan_fwd_workspace(ctypes.byref(dims)), x.device)
    st = lib.lizard_scan_fwd(ctypes.byref(dims), *ptrs, _need_f32(h0, "h0", shape), _ptr(cu),
                             y.data_ptr(), _need_f32(h_out, "h_out", shape), _ptr(states),
                             *_ws(workspace), _stream_of(x))
    _check(st, "lizard_scan_fwd")
    return (y, states) if save_states else y


def lizard_scan_bwd(x, dt, A, Bm, Cm, dy, states, *, D=None, z=None, dt_bias=None,
                    softplus: bool = True, h0=None, dh_out=None, dh0=None, cu_seqlens=None,
                    dx=None, ddt=None, dz=None, dBm=None, dCm=None, workspace=None, stream=None):
    """Gradients dx, ddt, dA, dBm, dCm, dD, dz, ddt_bias of lizard_scan_fwd's y against dy, from
    the same inputs and the states that call returned (None for an absent D, z, dt_bias).
    dh_out is the gradient of h_out; dh0 (if given) receives that of h0."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_scan_bwd, locals())
    B, L, C = x.shape
    nseq, cu = _packed(cu_seqlens, B, L, x.device)
    dims, ptrs = _scan_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, nseq)
    tp, N, wide = x.dtype, A.shape[1], (B, L, C)
    group = (B, L, dims.G, N)
    dims.ldy = _ld(dy, "dy", wide, tp)

    def out(t, name, shape):
        return (x.new_empty(shape), 0) if t is None else (t, _ld(t, name, shape, tp))

    dx, dims.lddx = out(dx, "dx", wide)
    ddt, dims.ldddt = out(ddt, "ddt", wide)
    dBm, dims.lddb = out(dBm, "dBm", group)
    dCm, dims.lddc = out(dCm, "dCm", group)
    if z is None:
        dz = None
    else:
        dz, dims.lddz = out(dz, "dz", wide)
    dA = torch.empty_like(A)
    dD = None if D is None else torch.empty_like(D)
    ddt_bias = None if dt_bias is None else torch.empty_like(dt_bias)
    _need(states, "states", (lizard_scan_states_bytes(dims),), torch.uint8)
    shape = (nseq or B, C, N)
    lib = load()
    workspace = _scratch(workspace, lib.lizard_scan_bwd_workspace(ctypes.byref(dims)), x.device)
    st = lib.lizard_scan_bwd(ctypes.byref(dims), *ptrs, _need_f32(h0, "h0", shape), _ptr(cu),
                             states.data_ptr(), dy.data_ptr(),
                             _need_f32(dh_out, "dh_out", shape), dx.data_ptr(), ddt.data_ptr(),
                             _ptr(dz), dBm.data_ptr(), dCm.data_ptr(), dA.data_ptr(), _ptr(dD),
                             _ptr(ddt_bias), _need_f32(dh0, "dh0", shape), *_ws(workspace), _stream_of(x))
    _check(st, "lizard_scan_bwd")
    return dict(dx=dx, ddt=ddt, dA=dA, dBm=dBm, dCm=dCm, dD=dD, dz=dz, ddt_bias=ddt_bias, dh0=dh0)


def lizard_scan_step(x, dt, A, Bm, Cm, state, *, D=None, z=None, dt_bias=None,
                     softplus: bool = True, slots=None, y=None, workspace=None, stream=None):
    """One token for each of B sequences: y [B, C] from x, dt, z [B, C] and Bm, Cm [B, G, N];
    state [slots, C, N] fp32 is moved on IN PLACE.  slots as for lizard_conv_step."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_scan_step, locals())
    dims, ptrs = _scan_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, 0)
    B, C = x.shape
    if y is None:
        y = x.new_empty((B, C))
    else:
        dims.ldy = _ld(y, "y", (B, C), x.dtype, 1)
    nslots = state.shape[0]
    st = load().lizard_scan_step(ctypes.byref(dims), *ptrs,
                                 _need_f32(state, "state", (nslots, C, dims.N)), nslots,
                                 _slots(slots, B), y.data_ptr(), *_ws(workspace),
                                 _stream_of(x))
    _check(st, "lizard_scan_step")
    return y


def _norm_inputs(o, gate, r, w_post, scale, w_pre, res_dtype, groups, act, gate_first, eps,
                 eps_pre):
    """lizard_norm_dims of the inputs, and the addresses of o, gate, r, w_post, scale, w_pre."""
    shape, tp = tuple(o.shape), o.dtype
    if len(shape) != 2:
        raise ValueError("o must be [T, D]")
    if res_dtype not in (tp, torch.float32):
        raise ValueError(f"residual stream: dtype {res_dtype} is neither o's ({tp}) nor float32")
    D = shape[1]
    dims = lizard_norm_dims(shape[0], D, groups, _ld(o, "o", shape, tp, 1),
                            0 if gate is None else _ld(gate, "gate", shape, tp, 1),
                            0 if r is None else _ld(r, "r", shape, res_dtype, 1), 0, 0, 0, 0, 0,
                            eps, eps if eps_pre is None else eps_pre, _dtype_code(o),
                            LIZARD_F32 if res_dtype is torch.float32 else LIZARD_BF16, act,
                            1 if gate_first else 0)
    return dims, (o.data_ptr(), _ptr(gate), _ptr(r), _need_f32(w_post, "w_post", (D,)),
                  _need_f32(scale, "scale", (D,)), _need_f32(w_pre, "w_pre", (D,)))


def lizard_block_norm_fwd(o, *, gate=None, r=None, w_post=None, scale=None, w_pre=None,
                          groups: int = 1, act: int = LIZARD_ACT_SILU, gate_first: bool = False,
                          eps: float = 1e-5, eps_pre=None, r_out=None, n_out=None, stream=None):
    """Norm after a block with its gate, residual scale and add, and the norm before the next
    block: o [T, D] is the block's output, r [T, D] the residual stream (its dtype or fp32).
    Returns (r_out, n_out); n_out is None without w_pre.  r_out takes r's dtype, or o's."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_block_norm_fwd, locals())
    shape = tuple(o.shape)
    rtp = r.dtype if r is not None else r_out.dtype if r_out is not None else o.dtype
    dims, ptrs = _norm_inputs(o, gate, r, w_post, scale, w_pre, rtp, groups, act, gate_first, eps,
                              eps_pre)
    if r_out is None:
        r_out = o.new_empty(shape, dtype=rtp)
    else:
        dims.ldro = _ld(r_out, "r_out", shape, rtp, 1)
    if w_pre is None:
        if n_out is not None:
            raise ValueError("n_out needs w_pre")
    elif n_out is None:
        n_out = o.new_empty(shape)
    else:
        dims.ldn = _ld(n_out, "n_out", shape, o.dtype, 1)
    st = load().lizard_block_norm_fwd(ctypes.byref(dims), *ptrs, r_out.data_ptr(), _ptr(n_out),
                                      _stream_of(o))
    _check(st, "lizard_block_norm_fwd")
    return r_out, n_out


def lizard_block_norm_bwd_workspace(dims) -> int:
    return int(load().lizard_block_norm_bwd_workspace(ctypes.byref(dims)))


def lizard_block_norm_bwd(o, *, dr_out=None, dn_out=None, gate=None, r=None, w_post=None,
                          scale=None, w_pre=None, groups: int = 1, act: int = LIZARD_ACT_SILU,
                          gate_first: bool = False, eps: float = 1e-5, eps_pre=None,
                          workspace=None, stream=None):
    """Gradients do, dgate, dr, dw_post, dscale, dw_pre of lizard_block_norm_fwd against dr_out
    and dn_out (one may be None; dn_out goes with w_pre), from the forward's inputs; None for an
    absent input."""
    if stream is not _HERE and (stream is not None or _gpus() > 1):
        return _placed(lizard_block_norm_bwd, locals())
    shape = tuple(o.shape)
    rtp = r.dtype if r is not None else dr_out.dtype if dr_out is not None else o.dtype
    dims, ptrs = _norm_inputs(o, gate, r, w_post, scale, w_pre, rtp, groups, act, gate_first, eps,
                              eps_pre)
    if dr_out is not None:
        dims.ldro = _ld(dr_out, "dr_out", shape, rtp, 1)
    if dn_out is not None:
        dims.ldn = _ld(dn_out, "dn_out", shape, o.dtype, 1)

    def like(t, dtype=None):
        return None if t is None else torch.empty(tuple(t.shape), dtype=dtype or t.dtype, device=o.device)

    do, dgate, dr = like(o), like(gate), like(r)
    dw_post, dscale, dw_pre = like(w_post), like(scale), like(w_pre)
    workspace = _scratch(workspace, lizard_block_norm_bwd_workspace(dims), o.device)
    st = load().lizard_block_norm_bwd(ctypes.byref(dims), *ptrs, _ptr(dr_out), _ptr(dn_out),
                                      do.data_ptr(), _ptr(dgate), _ptr(dr), _ptr(dw_post),
                                      _ptr(dscale), _ptr(dw_pre), *_ws(workspace), _stream_of(o))
    _check(st, "lizard_block_norm_bwd")
    return dict(do=do, dgate=dgate, dr=dr, dw_post=dw_post, dscale=dscale, dw_pre=dw_pre)
