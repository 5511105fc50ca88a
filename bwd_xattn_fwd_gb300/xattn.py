"""ctypes binding of libxattn (include/xattn.h).

Argument marshalling only: tensors become device pointers, the current torch CUDA
stream becomes the ``stream`` argument, and a non-OK status raises ``XattnError``.
Every step of the attention runs in libxattn's kernels; there is no fallback. If
the library has not been built, importing this module raises at once.

The functions named like the C entry points (``xattn_fwd``, ``xattn_bwd``, ...)
take the same arguments in the same order; tensor arguments may be torch tensors
or raw integer addresses. ``attention_fwd`` / ``attention_bwd`` allocate the
outputs with torch and call them. The C-level functions take raw addresses and stream handles
without torch.
"""
from __future__ import annotations

import ctypes
import enum
import importlib.util
import os

from . import build as _build

# XATTN_LIBRARY may name another build of libxattn (for example an instrumented one).
_LIB_PATH = os.environ.get("XATTN_LIBRARY") or _build.LIB

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"libxattn is not built ({_LIB_PATH} missing): run "
        "`python -c 'import __graft_entry__ as g; g.build()'` or "
        "`python bwd_xattn_fwd_gb300/build.py` first")

_lib = ctypes.CDLL(_LIB_PATH)


class Status(enum.IntEnum):
    OK = 0
    ERR_NULL_PTR = 1
    ERR_BAD_SHAPE = 2
    ERR_GROUP = 3
    ERR_UNSUPPORTED_HD = 4
    ERR_MISALIGNED = 5
    ERR_CUDA = 6
    ERR_NO_DEVICE_SUPPORT = 7
    ERR_DEVICE_TIMEOUT = 8
    ERR_BAD_SCALE = 9
    ERR_WORKSPACE = 10
    ERR_SCRATCH_LIMIT = 11
    ERR_DEVICE_BOUNDS = 12
    ERR_WINDOW = 13
    ERR_PAGES = 14


class XattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = Status(status)
        super().__init__(f"{where}: {self.status.name} ({status_string(status)})")


_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t

_SIGS = {
    "xattn_fwd": [_vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp],
    "xattn_bwd": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp],
    "xattn_bwd_noalloc": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp],
    "xattn_bwd_preprocess": [_vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _sz, _vp],
    "xattn_bwd_main": [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _sz, _vp],
    "xattn_bwd_dq_convert": [_i, _i, _i, _i, _f, _vp, _vp, _sz, _vp],
    "xattn_bwd_deterministic": [_vp] * 5 + [_vp] + [_i] * 5 + [_f] + [_vp] * 4,
    "xattn_fwd_f32": [_vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp],
    "xattn_bwd_f32": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp],
    "xattn_decode": [_vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp],
    "xattn_window_fwd": [_vp] * 3 + [_i] * 7 + [_f] + [_vp] * 3,
    "xattn_window_bwd": [_vp] * 6 + [_i] * 7 + [_f, _i] + [_vp] * 4,
    "xattn_window_fwd_f32": [_vp] * 3 + [_i] * 7 + [_f] + [_vp] * 3,
    "xattn_window_bwd_f32": [_vp] * 6 + [_i] * 7 + [_f] + [_vp] * 4,
    "xattn_tree_decode": [_vp] * 6 + [_i] * 10 + [_f] + [_vp] * 3,
    "xattn_cache_append": [_vp] * 6 + [_i] * 7 + [_vp],
    "xattn_cache_compact": [_vp] * 6 + [_i] * 7 + [_vp],
    "xattn_latent_fwd": [_vp] * 3 + [_i] * 6 + [_f] + [_vp] * 3,
    "xattn_latent_bwd": [_vp] * 6 + [_i] * 6 + [_f] + [_vp] * 4,
    "xattn_latent_decode": [_vp] * 4 + [_i] * 8 + [_f] + [_vp] * 3,
    "xattn_cache_reserve": [_vp] * 5 + [_i] * 5 + [_vp] * 4,
    "xattn_cache_release": [_vp] * 5 + [_i] * 4 + [_vp],
    "xattn_cache_write": [_vp] * 5 + [_i] * 5 + [_vp],
    "xattn_latent_write": [_vp] * 4 + [_i] * 5 + [_vp],
    "xattn_trim_scratch": [_sz],
    "xattn_check_device_status": [_vp],
}
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int
_lib.xattn_status_string.argtypes = [ctypes.c_int]
_lib.xattn_status_string.restype = ctypes.c_char_p
_lib.xattn_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i]
_lib.xattn_bwd_workspace_bytes.restype = ctypes.c_size_t
_lib.xattn_bwd_dq_mode.argtypes = [_i, _i, _i, _i, _i]
_lib.xattn_bwd_dq_mode.restype = ctypes.c_int
_lib.xattn_decode_runs.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.xattn_decode_runs.restype = ctypes.c_int
_lib.xattn_build_flags.argtypes = []
_lib.xattn_build_flags.restype = ctypes.c_int
_lib.xattn_selftest_bounds_check.argtypes = [_vp]
_lib.xattn_selftest_bounds_check.restype = ctypes.c_int

TREE_MAX = 64                       # XATTN_TREE_MAX in xattn.h
NO_WINDOW = 0x7FFFFFFF              # XATTN_NO_WINDOW in xattn.h
BWD_FUSED_DQ, BWD_RESIDENT_DQ, BWD_QUERY_DQ = 0, 1, 2
BUILD_DEVICE_CHECKS = 1             # xattn_build_flags bit: on-device bounds checks compiled in
ERR_DEVICE_TIMEOUT, ERR_DEVICE_BOUNDS = 8, 12


def lib_path() -> str:
    return _LIB_PATH


def status_string(status: int) -> str:
    return _lib.xattn_status_string(int(status)).decode()


def _addr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(name, *args):
    rc = getattr(_lib, name)(*args)
    if rc != 0:
        raise XattnError(rc, name)


# ---- the C entry points, same names and argument order -------------------------------

def xattn_fwd(q, k, v, B, S, nh, nkv, hd, scale, o, lse, stream=None):
    _call("xattn_fwd", _addr(q), _addr(k), _addr(v), B, S, nh, nkv, hd, scale, _addr(o),
          _addr(lse), _stream(stream))


def xattn_bwd(q, k, v, o, dO, lse, B, S, nh, nkv, hd, scale, dq, dk, dv, stream=None):
    _call("xattn_bwd", _addr(q), _addr(k), _addr(v), _addr(o), _addr(dO), _addr(lse), B, S, nh,
          nkv, hd, scale, _addr(dq), _addr(dk), _addr(dv), _stream(stream))


def xattn_bwd_deterministic(q, k, v, o, dO, lse, B, S, nh, nkv, hd, scale, dq, dk, dv, stream=None):
    """xattn_bwd with a bit-reproducible dQ (query-stationary dQ recompute, no atomics)."""
    _call("xattn_bwd_deterministic", _addr(q), _addr(k), _addr(v), _addr(o), _addr(dO), _addr(lse),
          B, S, nh, nkv, hd, scale, _addr(dq), _addr(dk), _addr(dv), _stream(stream))


def xattn_bwd_noalloc(q, k, v, o, dO, lse, B, S, nh, nkv, hd, scale, dq, dk, dv, stream=None):
    """xattn_bwd using the library's fixed device scratch array instead of allocating
    (for callers that may not allocate device memory). Sizes whose scratch exceeds
    NOALLOC_SCRATCH_BYTES raise ERR_SCRATCH_LIMIT; overlapping calls race on the array."""
    _call("xattn_bwd_noalloc", _addr(q), _addr(k), _addr(v), _addr(o), _addr(dO), _addr(lse), B,
          S, nh, nkv, hd, scale, _addr(dq), _addr(dk), _addr(dv), _stream(stream))


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024   # XATTN_NOALLOC_SCRATCH_BYTES in xattn.h


def xattn_bwd_workspace_bytes(B, S, nh, hd) -> int:
    return int(_lib.xattn_bwd_workspace_bytes(B, S, nh, hd))


def xattn_decode_runs(B, T, nh, nkv, hd, num_sms) -> int:
    """Key runs per (sequence, kv head) that xattn_decode uses on num_sms SMs (-1: rejected)."""
    return int(_lib.xattn_decode_runs(B, T, nh, nkv, hd, num_sms))


def xattn_bwd_dq_mode(S, nh, nkv, hd, deterministic=False) -> int:
    """Which backward xattn_bwd (or, with deterministic, xattn_bwd_deterministic) runs for
    these sizes (BWD_FUSED_DQ, BWD_RESIDENT_DQ, BWD_QUERY_DQ), or -1 for sizes it rejects."""
    return int(_lib.xattn_bwd_dq_mode(S, nh, nkv, hd, int(bool(deterministic))))


def xattn_bwd_preprocess(o, dO, lse, B, S, nh, hd, scale, workspace, workspace_bytes, stream=None):
    _call("xattn_bwd_preprocess", _addr(o), _addr(dO), _addr(lse), B, S, nh, hd, scale,
          _addr(workspace), workspace_bytes, _stream(stream))


def xattn_bwd_main(q, k, v, dO, B, S, nh, nkv, hd, scale, dk, dv, workspace, workspace_bytes,
                   stream=None):
    _call("xattn_bwd_main", _addr(q), _addr(k), _addr(v), _addr(dO), B, S, nh, nkv, hd, scale,
          _addr(dk), _addr(dv), _addr(workspace), workspace_bytes, _stream(stream))


def xattn_bwd_dq_convert(B, S, nh, hd, scale, dq, workspace, workspace_bytes, stream=None):
    _call("xattn_bwd_dq_convert", B, S, nh, hd, scale, _addr(dq), _addr(workspace), workspace_bytes,
          _stream(stream))


def xattn_fwd_f32(q, k, v, B, S, nh, nkv, hd, scale, o, lse, stream=None):
    _call("xattn_fwd_f32", _addr(q), _addr(k), _addr(v), B, S, nh, nkv, hd, scale, _addr(o),
          _addr(lse), _stream(stream))


def xattn_bwd_f32(q, k, v, o, dO, lse, B, S, nh, nkv, hd, scale, dq, dk, dv, stream=None):
    _call("xattn_bwd_f32", _addr(q), _addr(k), _addr(v), _addr(o), _addr(dO), _addr(lse), B, S,
          nh, nkv, hd, scale, _addr(dq), _addr(dk), _addr(dv), _stream(stream))


def xattn_decode(q, k_cache, v_cache, B, T, nh, nkv, hd, scale, o, lse, stream=None):
    _call("xattn_decode", _addr(q), _addr(k_cache), _addr(v_cache), B, T, nh, nkv, hd, scale, _addr(o),
          _addr(lse), _stream(stream))


def xattn_window_fwd(q, k, v, B, S, nh, nkv, hd, window, sinks, scale, o, lse, stream=None):
    _call("xattn_window_fwd", _addr(q), _addr(k), _addr(v), B, S, nh, nkv, hd, window, sinks, scale, _addr(o),
          _addr(lse), _stream(stream))


def xattn_window_bwd(q, k, v, o, dO, lse, B, S, nh, nkv, hd, window, sinks, scale, deterministic, dq, dk, dv,
                     stream=None):
    _call("xattn_window_bwd", _addr(q), _addr(k), _addr(v), _addr(o), _addr(dO), _addr(lse), B, S, nh, nkv, hd,
          window, sinks, scale, int(bool(deterministic)), _addr(dq), _addr(dk), _addr(dv), _stream(stream))


def xattn_window_fwd_f32(q, k, v, B, S, nh, nkv, hd, window, sinks, scale, o, lse, stream=None):
    _call("xattn_window_fwd_f32", _addr(q), _addr(k), _addr(v), B, S, nh, nkv, hd, window, sinks, scale, _addr(o),
          _addr(lse), _stream(stream))


def xattn_window_bwd_f32(q, k, v, o, dO, lse, B, S, nh, nkv, hd, window, sinks, scale, dq, dk, dv, stream=None):
    _call("xattn_window_bwd_f32", _addr(q), _addr(k), _addr(v), _addr(o), _addr(dO), _addr(lse), B, S, nh, nkv, hd,
          window, sinks, scale, _addr(dq), _addr(dk), _addr(dv), _stream(stream))


def xattn_tree_decode(q, k_pages, v_pages, page_table, ctx_lens, tree, B, n, nh, nkv, hd, num_pages, page_size,
                      max_pages, window, sinks, scale, o, lse, stream=None):
    _call("xattn_tree_decode", _addr(q), _addr(k_pages), _addr(v_pages), _addr(page_table), _addr(ctx_lens),
          _addr(tree), B, n, nh, nkv, hd, num_pages, page_size, max_pages, window, sinks, scale, _addr(o), _addr(lse),
          _stream(stream))


def xattn_cache_append(k_new, v_new, k_pages, v_pages, page_table, ctx_lens, B, n, nkv, hd, num_pages, page_size,
                       max_pages, stream=None):
    _call("xattn_cache_append", _addr(k_new), _addr(v_new), _addr(k_pages), _addr(v_pages), _addr(page_table),
          _addr(ctx_lens), B, n, nkv, hd, num_pages, page_size, max_pages, _stream(stream))


def xattn_cache_compact(k_pages, v_pages, page_table, ctx_lens, path, accepted, B, n, nkv, hd, num_pages, page_size,
                        max_pages, stream=None):
    _call("xattn_cache_compact", _addr(k_pages), _addr(v_pages), _addr(page_table), _addr(ctx_lens), _addr(path),
          _addr(accepted), B, n, nkv, hd, num_pages, page_size, max_pages, _stream(stream))


def xattn_latent_fwd(q, kv, k_rope, B, S, nh, dn, dr, dv, scale, o, lse, stream=None):
    _call("xattn_latent_fwd", _addr(q), _addr(kv), _addr(k_rope), B, S, nh, dn, dr, dv, scale, _addr(o), _addr(lse),
          _stream(stream))


def xattn_latent_bwd(q, kv, k_rope, o, dO, lse, B, S, nh, dn, dr, dv, scale, dq, dkv, dk_rope, stream=None):
    _call("xattn_latent_bwd", _addr(q), _addr(kv), _addr(k_rope), _addr(o), _addr(dO), _addr(lse), B, S, nh, dn, dr, dv,
          scale, _addr(dq), _addr(dkv), _addr(dk_rope), _stream(stream))


def xattn_latent_decode(q, pages, page_table, ctx_lens, B, n, nh, dc, dr, num_pages, page_size, max_pages, scale, o, lse,
                        stream=None):
    _call("xattn_latent_decode", _addr(q), _addr(pages), _addr(page_table), _addr(ctx_lens), B, n, nh, dc, dr, num_pages,
          page_size, max_pages, scale, _addr(o), _addr(lse), _stream(stream))


def xattn_cache_reserve(page_table, ctx_lens, new_lens, free_pages, free_count, B, num_pages, page_size, max_pages, tokens,
                        slots, offsets, granted, stream=None):
    _call("xattn_cache_reserve", _addr(page_table), _addr(ctx_lens), _addr(new_lens), _addr(free_pages),
          _addr(free_count), B, num_pages, page_size, max_pages, tokens, _addr(slots), _addr(offsets), _addr(granted),
          _stream(stream))


def xattn_cache_release(page_table, held_lens, keep_lens, free_pages, free_count, B, num_pages, page_size, max_pages,
                        stream=None):
    _call("xattn_cache_release", _addr(page_table), _addr(held_lens), _addr(keep_lens), _addr(free_pages),
          _addr(free_count), B, num_pages, page_size, max_pages, _stream(stream))


def xattn_cache_write(k_new, v_new, k_pages, v_pages, slots, rows, nkv, hd, num_pages, page_size, stream=None):
    _call("xattn_cache_write", _addr(k_new), _addr(v_new), _addr(k_pages), _addr(v_pages), _addr(slots), rows, nkv, hd,
          num_pages, page_size, _stream(stream))


def xattn_latent_write(c, k_rope, pages, slots, rows, dc, dr, num_pages, page_size, stream=None):
    _call("xattn_latent_write", _addr(c), _addr(k_rope), _addr(pages), _addr(slots), rows, dc, dr, num_pages, page_size,
          _stream(stream))


def xattn_trim_scratch(keep_bytes=0):
    """Gives back what the current device's scratch pool holds beyond keep_bytes and no call still
    uses."""
    _call("xattn_trim_scratch", keep_bytes)


def xattn_selftest_wait_timeout(limit_ns, stream=None):
    fn = _lib.xattn_selftest_wait_timeout
    fn.argtypes = [ctypes.c_ulonglong, _vp]
    fn.restype = ctypes.c_int
    st = fn(int(limit_ns), _stream(stream))
    if st != 0:
        raise XattnError(st, "xattn_selftest_wait_timeout")


def xattn_build_flags() -> int:
    """Bit BUILD_DEVICE_CHECKS is set in a debug build (on-device bounds checks)."""
    return int(_lib.xattn_build_flags())


def xattn_selftest_bounds_check(stream=None):
    st = _lib.xattn_selftest_bounds_check(_stream(stream))
    if st != 0:
        raise XattnError(st, "xattn_selftest_bounds_check")


def xattn_status_string(status: int) -> str:
    return status_string(status)


def xattn_check_device_status(stream=None) -> int:
    """Synchronises the stream; returns the device status (0 = OK) and clears it."""
    return int(_lib.xattn_check_device_status(_stream(stream)))


# ---- tensor-level helpers ---------------------------------------------------------------

def _dims(q, k):
    B, S, nh, hd = q.shape
    nkv = k.shape[2]
    return int(B), int(S), int(nh), int(nkv), int(hd)


def attention_fwd(q, k, v, scale=None, stream=None):
    """(o, lse) for contiguous CUDA tensors q [B,S,nh,hd], k/v [B,S,nkv,hd] (bf16 or fp32)."""
    import torch
    B, S, nh, nkv, hd = _dims(q, k)
    scale = float(hd ** -0.5 if scale is None else scale)
    o = torch.empty_like(q)
    lse = torch.empty((B, S, nh), dtype=torch.float32, device=q.device)
    if q.dtype == torch.bfloat16:
        xattn_fwd(q, k, v, B, S, nh, nkv, hd, scale, o, lse, stream)
    elif q.dtype == torch.float32:
        xattn_fwd_f32(q, k, v, B, S, nh, nkv, hd, scale, o, lse, stream)
    else:
        raise TypeError(f"unsupported dtype {q.dtype}")
    return o, lse


def attention_bwd(q, k, v, o, dO, lse, scale=None, stream=None, deterministic=False):
    """(dq, dk, dv) for the tensors of attention_fwd and the output gradient dO.
    deterministic (bf16): dQ bit-reproducible as well, at the cost of a second recompute."""
    import torch
    B, S, nh, nkv, hd = _dims(q, k)
    scale = float(hd ** -0.5 if scale is None else scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if q.dtype == torch.bfloat16:
        fn = xattn_bwd_deterministic if deterministic else xattn_bwd
        fn(q, k, v, o, dO, lse, B, S, nh, nkv, hd, scale, dq, dk, dv, stream)
    elif q.dtype == torch.float32:
        xattn_bwd_f32(q, k, v, o, dO, lse, B, S, nh, nkv, hd, scale, dq, dk, dv, stream)
    else:
        raise TypeError(f"unsupported dtype {q.dtype}")
    return dq, dk, dv


def attention_decode(q, k_cache, v_cache, scale=None, stream=None):
    """(o [B,nh,hd], lse [B,nh]) for one new query per sequence: q [B,nh,hd] against the
    cached k/v [B,T,nkv,hd] (bf16, contiguous CUDA tensors)."""
    import torch
    B, nh, hd = (int(x) for x in q.shape)
    T, nkv = int(k_cache.shape[1]), int(k_cache.shape[2])
    scale = float(hd ** -0.5 if scale is None else scale)
    o = torch.empty_like(q)
    lse = torch.empty((B, nh), dtype=torch.float32, device=q.device)
    xattn_decode(q, k_cache, v_cache, B, T, nh, nkv, hd, scale, o, lse, stream)
    return o, lse


# ---- tensor-level calls that check their tensors (csrc/xattn_torch.cpp) ------------------
# A stream given to one of them is as torch.cuda.stream(stream) around the call: the outputs
# belong to it, and tensors of another stream are the caller's to order and to keep.

def _load_calls():
    """The native part of the calls below, bound to this library's entry points."""
    import torch  # noqa: F401  (its libraries)
    path = _build.torch_lib()
    if not path:
        raise ImportError("the tensor-level calls need a torch built for CUDA")
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built: run `python bwd_xattn_fwd_gb300/build.py` first")
    spec = importlib.util.spec_from_file_location("xattn_torch", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.bind(*(ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in
                  ("xattn_window_fwd", "xattn_window_fwd_f32", "xattn_window_bwd", "xattn_window_bwd_f32",
                   "xattn_tree_decode", "xattn_cache_append", "xattn_cache_compact", "xattn_latent_fwd", "xattn_latent_bwd",
                   "xattn_latent_decode", "xattn_cache_reserve", "xattn_cache_release", "xattn_cache_write",
                   "xattn_latent_write")))
    return module


class _Unloaded:
    """Stands for the native part until the first of the calls below; nothing else needs it."""

    def __getattr__(self, name):
        global _calls
        _calls = _load_calls()
        return getattr(_calls, name)


_calls = _Unloaded()


class _Elsewhere:
    """Makes a tensor's device current, and the given stream (a torch stream, a raw handle, or
    None: the device's current one) the one that torch allocates on and that calls launch on."""

    def __init__(self, t, stream):
        import torch
        device = t.device
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        self._guards = [torch.cuda.device(device)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for g in self._guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False


def _again(name, status, call, where, stream, tensors):
    """What a native call that returned no outputs asks for: raises its status; or, when the
    tensors do not fit, says what is wrong with the first that does not; or, when they are
    all on another device than the current one, makes that one current and calls again."""
    import torch
    if status is not None:
        raise XattnError(status, name)
    device = None
    for label, t, shape, dtype in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: {label} must be a tensor, not {type(t).__name__}")
        device = device or t.device
        if t.dtype != dtype:
            raise TypeError(f"{name}: {label}: expected {dtype}, got {t.dtype}")
        if t.device.type != "cuda":
            raise ValueError(f"{name}: {label} must be a CUDA tensor, not on {t.device}")
        if t.device != device:
            raise ValueError(f"{name}: {label} is on {t.device}, {tensors[0][0]} on {device}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: {label}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: {label} must be contiguous")
    if torch.cuda.current_device() == device.index:
        raise ValueError(f"{name}: a dimension is beyond 2^31 - 1")
    with _Elsewhere(where, stream):
        return call()


def _need_dims(name, **tensors):
    import torch
    for label, (t, dims) in tensors.items():
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name}: {label} must be a tensor of {dims} dimensions")


def attention_window_fwd(q, k, v, window, sinks=0, scale=None, stream=None):
    """(o, lse) of causal attention in which query i sees key j only if i - j < window or
    j < sinks; tensors as for attention_fwd (bf16 or fp32)."""
    if stream is not None:
        with _Elsewhere(q, stream):
            return attention_window_fwd(q, k, v, window, sinks, scale)
    out = _calls.window_fwd(q, k, v, window, sinks, scale)
    if type(out) is tuple:
        return out
    import torch
    name = "attention_window_fwd"
    _need_dims(name, q=(q, 4), k=(k, 4))
    kv, dtype = (*q.shape[:2], k.shape[2], q.shape[3]), q.dtype if q.dtype == torch.float32 else torch.bfloat16
    return _again(name, out, lambda: attention_window_fwd(q, k, v, window, sinks, scale), q, None,
                  (("q", q, q.shape, dtype), ("k", k, kv, dtype), ("v", v, kv, dtype)))


def attention_window_bwd(q, k, v, o, dO, lse, window, sinks=0, scale=None, stream=None, deterministic=False):
    """(dq, dk, dv) for the tensors of attention_window_fwd and the output gradient dO.
    deterministic (bf16): dQ bit-reproducible as well, from a second recompute."""
    if stream is not None:
        with _Elsewhere(q, stream):
            return attention_window_bwd(q, k, v, o, dO, lse, window, sinks, scale, deterministic=deterministic)
    out = _calls.window_bwd(q, k, v, o, dO, lse, window, sinks, scale, deterministic)
    if type(out) is tuple:
        return out
    import torch
    name = "attention_window_bwd"
    _need_dims(name, q=(q, 4), k=(k, 4))
    kv, dtype = (*q.shape[:2], k.shape[2], q.shape[3]), q.dtype if q.dtype == torch.float32 else torch.bfloat16
    return _again(name, out, lambda: attention_window_bwd(q, k, v, o, dO, lse, window, sinks, scale,
                                                          deterministic=deterministic), q, None,
                  (("q", q, q.shape, dtype), ("k", k, kv, dtype), ("v", v, kv, dtype), ("o", o, q.shape, dtype),
                   ("dO", dO, q.shape, dtype), ("lse", lse, q.shape[:3], torch.float32)))


def _pool(name, k_pages, v_pages, page_table, ctx_lens):
    import torch
    _need_dims(name, k_pages=(k_pages, 4), page_table=(page_table, 2))
    return (("k_pages", k_pages, k_pages.shape, torch.bfloat16), ("v_pages", v_pages, k_pages.shape, torch.bfloat16),
            ("page_table", page_table, page_table.shape, torch.int32),
            ("ctx_lens", ctx_lens, page_table.shape[:1], torch.int32))


def attention_tree_decode(q, k_pages, v_pages, page_table, ctx_lens, tree=None, window=None, sinks=0, scale=None,
                          stream=None):
    """(o [B,n,nh,hd], lse [B,n,nh]) of n <= 64 new tokens a sequence over a paged cache: q
    [B,n,nh,hd] against the pools [num_pages,page_size,nkv,hd] (bf16), through page_table
    [B,max_pages] and ctx_lens [B] (int32); the new tokens' K and V are already at positions
    ctx_lens .. ctx_lens + n - 1 (cache_append). tree [B,n] (int64): bit j of word i lets token
    i see new token j; None: token i sees new tokens 0 .. i (n = 1: the decode step). window
    (None: no window) and sinks as in attention_window_fwd."""
    if stream is not None:
        with _Elsewhere(q, stream):
            return attention_tree_decode(q, k_pages, v_pages, page_table, ctx_lens, tree, window, sinks, scale)
    out = _calls.tree_decode(q, k_pages, v_pages, page_table, ctx_lens, tree, window, sinks, scale)
    if type(out) is tuple:
        return out
    import torch
    name = "attention_tree_decode"
    tensors = _pool(name, k_pages, v_pages, page_table, ctx_lens)
    _need_dims(name, q=(q, 4))
    B, n = page_table.shape[0], q.shape[1]
    return _again(name, out, lambda: attention_tree_decode(q, k_pages, v_pages, page_table, ctx_lens, tree, window,
                                                           sinks, scale), q, None,
                  (*tensors, ("q", q, (B, n, q.shape[2], k_pages.shape[3]), torch.bfloat16),
                   *([] if tree is None else [("tree", tree, (B, n), torch.int64)])))


def cache_append(k_new, v_new, k_pages, v_pages, page_table, ctx_lens, stream=None):
    """Writes the rows k_new, v_new [B,n,nkv,hd] to positions ctx_lens .. ctx_lens + n - 1 of each
    sequence's pages (in place)."""
    if stream is not None:
        with _Elsewhere(k_pages, stream):
            return cache_append(k_new, v_new, k_pages, v_pages, page_table, ctx_lens)
    out = _calls.cache_append(k_new, v_new, k_pages, v_pages, page_table, ctx_lens)
    if out is True:
        return None
    import torch
    name = "cache_append"
    tensors = _pool(name, k_pages, v_pages, page_table, ctx_lens)
    _need_dims(name, k_new=(k_new, 4))
    rows = (page_table.shape[0], k_new.shape[1], *k_pages.shape[2:])
    return _again(name, out, lambda: cache_append(k_new, v_new, k_pages, v_pages, page_table, ctx_lens), k_pages, None,
                  (*tensors, ("k_new", k_new, rows, torch.bfloat16), ("v_new", v_new, rows, torch.bfloat16)))


def cache_compact(k_pages, v_pages, page_table, ctx_lens, path, accepted, stream=None):
    """Moves the rows of positions ctx_lens + path[:, i], i < accepted, down to ctx_lens + i (in
    place): path [B,n] (int32, ascending over its accepted entries), accepted [B] (int32)."""
    if stream is not None:
        with _Elsewhere(k_pages, stream):
            return cache_compact(k_pages, v_pages, page_table, ctx_lens, path, accepted)
    out = _calls.cache_compact(k_pages, v_pages, page_table, ctx_lens, path, accepted)
    if out is True:
        return None
    import torch
    name = "cache_compact"
    tensors = _pool(name, k_pages, v_pages, page_table, ctx_lens)
    _need_dims(name, path=(path, 2))
    B = page_table.shape[0]
    return _again(name, out, lambda: cache_compact(k_pages, v_pages, page_table, ctx_lens, path, accepted), k_pages,
                  None, (*tensors, ("path", path, (B, path.shape[1]), torch.int32),
                         ("accepted", accepted, (B,), torch.int32)))


def attention_latent_fwd(q, kv, k_rope, scale=None, stream=None):
    """(o [B,S,nh,dv], lse [B,S,nh]) of latent attention in its expanded form, causal: q [B,S,nh,dn+dr], kv
    [B,S,nh,dn+dv] (each head's key part, then its value), k_rope [B,S,dr], the part of the keys that
    the heads share (bf16). scale: (dn + dr) ** -0.5 unless given."""
    if stream is not None:
        with _Elsewhere(q, stream):
            return attention_latent_fwd(q, kv, k_rope, scale)
    out = _calls.latent_fwd(q, kv, k_rope, scale)
    if type(out) is tuple:
        return out
    name = "attention_latent_fwd"
    return _again(name, out, lambda: attention_latent_fwd(q, kv, k_rope, scale), q, None, _latent(name, q, kv, k_rope))


def attention_latent_bwd(q, kv, k_rope, o, dO, lse, scale=None, stream=None):
    """(dq, dkv, dk_rope) for the tensors of attention_latent_fwd and the output gradient dO; k_rope's is
    the sum over the heads."""
    if stream is not None:
        with _Elsewhere(q, stream):
            return attention_latent_bwd(q, kv, k_rope, o, dO, lse, scale)
    out = _calls.latent_bwd(q, kv, k_rope, o, dO, lse, scale)
    if type(out) is tuple:
        return out
    import torch
    name = "attention_latent_bwd"
    tensors = _latent(name, q, kv, k_rope)
    outs = (*q.shape[:3], kv.shape[3] - q.shape[3] + k_rope.shape[2])
    return _again(name, out, lambda: attention_latent_bwd(q, kv, k_rope, o, dO, lse, scale), q, None,
                  (*tensors, ("o", o, outs, torch.bfloat16), ("dO", dO, outs, torch.bfloat16),
                   ("lse", lse, q.shape[:3], torch.float32)))


def _latent(name, q, kv, k_rope):
    import torch
    _need_dims(name, q=(q, 4), kv=(kv, 4), k_rope=(k_rope, 3))
    dn, dr = q.shape[3] - k_rope.shape[2], k_rope.shape[2]
    if dn < 1 or kv.shape[3] <= dn:
        raise ValueError(f"{name}: q has dn + dr numbers a head, kv dn + dv and k_rope dr: dn, dv >= 1 do not fit "
                         f"{q.shape[3]}, {kv.shape[3]} and {dr}")
    return (("q", q, q.shape, torch.bfloat16), ("kv", kv, (*q.shape[:3], kv.shape[3]), torch.bfloat16),
            ("k_rope", k_rope, (*q.shape[:2], dr), torch.bfloat16))


def attention_latent_decode(q, pages, page_table, ctx_lens, dc, scale, stream=None):
    """(o [B,n,nh,dc], lse [B,n,nh]) of latent attention in its absorbed form, n <= 64 new tokens a sequence over
    a paged cache: q [B,n,nh,dc+dr] against the rows of pages [num_pages,page_size,dc+dr] (bf16), whose first dc
    numbers are the values too, through page_table [B,max_pages] and ctx_lens [B] (int32). The new tokens' rows
    are already at positions ctx_lens .. ctx_lens + n - 1 (latent_write; of a sequence that got no places for them
    the outputs mean nothing); token i sees positions 0 .. ctx_lens + i.
    scale: that of the expanded heads."""
    if stream is not None:
        with _Elsewhere(q, stream):
            return attention_latent_decode(q, pages, page_table, ctx_lens, dc, scale)
    out = _calls.latent_decode(q, pages, page_table, ctx_lens, dc, scale)
    if type(out) is tuple:
        return out
    import torch
    name = "attention_latent_decode"
    _need_dims(name, q=(q, 4), pages=(pages, 3), page_table=(page_table, 2))
    if not 0 < dc < pages.shape[2]:
        raise ValueError(f"{name}: dc = {dc} does not fit rows of {pages.shape[2]}")
    B = page_table.shape[0]
    return _again(name, out, lambda: attention_latent_decode(q, pages, page_table, ctx_lens, dc, scale), q, None,
                  (("q", q, (B, *q.shape[1:3], pages.shape[2]), torch.bfloat16),
                   ("pages", pages, pages.shape, torch.bfloat16), ("page_table", page_table, page_table.shape, torch.int32),
                   ("ctx_lens", ctx_lens, (B,), torch.int32)))


def cache_reserve(page_table, ctx_lens, new_lens, free_pages, free_count, page_size, tokens, stream=None):
    """Takes the pages for new_lens positions a sequence, from ctx_lens on, from the stack of free pages
    (free_pages [num_pages], free_count [1]) into page_table [B,max_pages] (all int32; table and count in place).
    Returns (slots [tokens] int64, offsets [B+1], granted [B]): the pool rows of a ragged batch's tokens (-1:
    none), where each sequence's tokens begin, and the positions that it got (0 when the pages or `tokens` do
    not reach). What an attention call gives for a sequence that got less than it asked for means nothing: it sees rows
    that were not written."""
    if stream is not None:
        with _Elsewhere(page_table, stream):
            return cache_reserve(page_table, ctx_lens, new_lens, free_pages, free_count, page_size, tokens)
    out = _calls.cache_reserve(page_table, ctx_lens, new_lens, free_pages, free_count, page_size, tokens)
    if type(out) is tuple:
        return out
    name = "cache_reserve"
    return _again(name, out, lambda: cache_reserve(page_table, ctx_lens, new_lens, free_pages, free_count, page_size,
                                                   tokens), page_table, None,
                  _tables(name, page_table, ctx_lens=ctx_lens, new_lens=new_lens, free_pages=free_pages,
                          free_count=free_count))


def cache_release(page_table, held_lens, keep_lens, free_pages, free_count, page_size, stream=None):
    """Gives the pages that hold only positions from keep_lens to held_lens - 1 back to the stack, and sets
    their entries of page_table to -1 (table, stack and count in place; tensors as for cache_reserve)."""
    if stream is not None:
        with _Elsewhere(page_table, stream):
            return cache_release(page_table, held_lens, keep_lens, free_pages, free_count, page_size)
    out = _calls.cache_release(page_table, held_lens, keep_lens, free_pages, free_count, page_size)
    if out is True:
        return None
    name = "cache_release"
    return _again(name, out, lambda: cache_release(page_table, held_lens, keep_lens, free_pages, free_count, page_size),
                  page_table, None, _tables(name, page_table, held_lens=held_lens, keep_lens=keep_lens,
                                            free_pages=free_pages, free_count=free_count))


def _tables(name, page_table, free_pages, free_count, **lens):
    import torch
    _need_dims(name, page_table=(page_table, 2), free_pages=(free_pages, 1))
    return (("page_table", page_table, page_table.shape, torch.int32),
            *((label, t, page_table.shape[:1], torch.int32) for label, t in lens.items()),
            ("free_pages", free_pages, free_pages.shape, torch.int32), ("free_count", free_count, (1,), torch.int32))


def cache_write(k_new, v_new, k_pages, v_pages, slots, stream=None):
    """Writes the rows k_new, v_new [rows,nkv,hd] to the pool rows that slots [rows] (int64) names, in place
    (the slots of cache_reserve; a slot outside the pool drops its row)."""
    if stream is not None:
        with _Elsewhere(k_pages, stream):
            return cache_write(k_new, v_new, k_pages, v_pages, slots)
    out = _calls.cache_write(k_new, v_new, k_pages, v_pages, slots)
    if out is True:
        return None
    import torch
    name = "cache_write"
    _need_dims(name, k_pages=(k_pages, 4), slots=(slots, 1))
    rows = (slots.shape[0], *k_pages.shape[2:])
    return _again(name, out, lambda: cache_write(k_new, v_new, k_pages, v_pages, slots), k_pages, None,
                  (("k_pages", k_pages, k_pages.shape, torch.bfloat16), ("v_pages", v_pages, k_pages.shape, torch.bfloat16),
                   ("slots", slots, slots.shape, torch.int64), ("k_new", k_new, rows, torch.bfloat16),
                   ("v_new", v_new, rows, torch.bfloat16)))


def latent_write(c, k_rope, pages, slots, stream=None):
    """Writes the rows (c, k_rope) [rows,dc], [rows,dr] to the rows of pages [num_pages,page_size,dc+dr] that
    slots [rows] (int64) names, in place (the slots of cache_reserve; a slot outside the pool drops its row)."""
    if stream is not None:
        with _Elsewhere(pages, stream):
            return latent_write(c, k_rope, pages, slots)
    out = _calls.latent_write(c, k_rope, pages, slots)
    if out is True:
        return None
    import torch
    name = "latent_write"
    _need_dims(name, c=(c, 2), k_rope=(k_rope, 2), pages=(pages, 3), slots=(slots, 1))
    return _again(name, out, lambda: latent_write(c, k_rope, pages, slots), pages, None,
                  (("pages", pages, (*pages.shape[:2], c.shape[1] + k_rope.shape[1]), torch.bfloat16),
                   ("slots", slots, slots.shape, torch.int64), ("c", c, (slots.shape[0], c.shape[1]), torch.bfloat16),
                   ("k_rope", k_rope, (slots.shape[0], k_rope.shape[1]), torch.bfloat16)))
