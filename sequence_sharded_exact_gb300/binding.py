"""ctypes binding of libringattn.so (include/ringattn.h).  Argument marshalling only: every step of
the computation runs in the library's CUDA kernels.  torch is used for device memory and streams.

The library is loaded on first use from this package's directory; if it has not been built the
call raises RingAttnError (there is no fallback of any kind).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import operator
import os
import threading
import warnings
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libringattn.so")

RA_OK, RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED, RA_ERR_CUDA, RA_ERR_NO_DEVICE, RA_ERR_TIMEOUT = range(6)
SPECTRA = {"whole": 0, "axis": 1}
LAYOUTS = {"contiguous": 0, "zigzag": 1, "striped": 2}
PATHS = {1: "simt", 2: "tcgen05"}
RA_DEVICE_TIMEOUT = 1
RA_DEVICE_LAYOUT = 2
RA_DEVICE_RANGE = 4
RA_E4M3 = 2

_lock = threading.Lock()
_lib = None
_calls = None

EXPORTS = (
    "ring_attn_fwd", "ring_attn_ring_step_fwd", "ring_attn_lse_merge", "ring_attn_fwd_stepwise",
    "ring_attn_fwd_stepwise_workspace_size", "ring_attn_bwd", "ring_attn_bwd_workspace_size",
    "ring_attn_shard_tiles", "ring_attn_fwd_path", "ring_attn_bwd_path", "ring_attn_device_status",
    "ring_attn_last_error", "ring_attn_abi_version", "ring_attn_bwd_static_scratch",
    "ring_attn_bwd_static_scratch_capacity", "ring_attn_fwd_tile_visits", "ring_attn_bwd_tile_visits",
    "ring_attn_rope", "ring_attn_ulysses_a2a", "ring_attn_ulysses_fwd", "ring_attn_ulysses_workspace_size",
    "ring_attn_ulysses_bwd", "ring_attn_ulysses_bwd_workspace_size", "ring_attn_fwd_host",
    "ring_attn_ring_step_fwd_accumulate",
    "ring_attn_fwd_host_workspace_size", "ring_attn_selftest_bounded_wait", "ring_attn_device_check",
    "ring_attn_block_fwd", "ring_attn_block_bwd", "ring_attn_bwd_preprocess", "ring_attn_f32_zero",
    "ring_attn_f32_add", "ring_attn_f32_convert", "ring_attn_block_rope", "ring_attn_fwd_f32out",
    "ring_attn_bwd_f32out", "ring_attn_bwd_preprocess_f32out", "ring_attn_qk_norm_rope",
    "ring_attn_qk_norm_rope_bwd", "ring_attn_qk_norm_rope_bwd_workspace_size", "ring_attn_cache_write",
    "ring_attn_cache_read", "ring_attn_tree_fwd", "ring_attn_tree_fwd_workspace_size",
    "ring_attn_window_fwd", "ring_attn_window_fwd_workspace_size", "ring_attn_window_bwd",
    "ring_attn_window_bwd_workspace_size", "ring_attn_qk_rope_axes", "ring_attn_qk_rope_axes_bwd",
    "ring_attn_tree_window_fwd",
)


class RingAttnError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"libringattn status {status}: {msg}")
        self.status = status


def library():
    """The loaded ctypes library (raises RingAttnError if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RingAttnError(-1, f"{LIB_PATH} is missing: build it with "
                                    "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, LL, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
        lib.ring_attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, P]
        lib.ring_attn_fwd_f32out.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, P]
        lib.ring_attn_ring_step_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, P]
        lib.ring_attn_lse_merge.argtypes = [P, P, P, P, LL, I, P]
        lib.ring_attn_fwd_stepwise.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, SZ, P]
        lib.ring_attn_fwd_stepwise_workspace_size.argtypes = [I, I, I, I]
        lib.ring_attn_fwd_stepwise_workspace_size.restype = SZ
        lib.ring_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, P, SZ, I, I, I, I, I, I, I, I,
                                      I, P]
        lib.ring_attn_bwd_f32out.argtypes = lib.ring_attn_bwd.argtypes
        lib.ring_attn_bwd_preprocess_f32out.argtypes = [P, P, P, LL, I, I, P]
        lib.ring_attn_bwd_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.ring_attn_bwd_workspace_size.restype = SZ
        lib.ring_attn_shard_tiles.argtypes = [I, I, I, I, I, P]
        lib.ring_attn_fwd_path.argtypes = [I, I, I, I, I, I, I, I, I, P]
        lib.ring_attn_bwd_path.argtypes = [I, I, I, I, I, I, I, I, I, P]
        lib.ring_attn_device_status.argtypes = [P, P]
        lib.ring_attn_device_check.argtypes = [P]
        lib.ring_attn_device_check.restype = ctypes.c_int
        lib.ring_attn_block_fwd.argtypes = [P, P, P, P, P] + [I] * 12 + [P]
        lib.ring_attn_block_fwd.restype = ctypes.c_int
        lib.ring_attn_block_bwd.argtypes = [P] * 9 + [I] * 12 + [P]
        lib.ring_attn_block_bwd.restype = ctypes.c_int
        lib.ring_attn_bwd_preprocess.argtypes = [P, P, P, LL, I, I, P]
        lib.ring_attn_bwd_preprocess.restype = ctypes.c_int
        lib.ring_attn_f32_zero.argtypes = [P, LL, P]
        lib.ring_attn_f32_zero.restype = ctypes.c_int
        lib.ring_attn_f32_add.argtypes = [P, P, LL, P]
        lib.ring_attn_f32_add.restype = ctypes.c_int
        lib.ring_attn_f32_convert.argtypes = [P, P, LL, I, P]
        lib.ring_attn_f32_convert.restype = ctypes.c_int
        lib.ring_attn_block_rope.argtypes = [P, I, I, I, I, I, I, I, I, ctypes.c_double, I, P]
        lib.ring_attn_block_rope.restype = ctypes.c_int
        lib.ring_attn_last_error.argtypes = []
        lib.ring_attn_last_error.restype = ctypes.c_char_p
        lib.ring_attn_abi_version.argtypes = []
        lib.ring_attn_bwd_static_scratch.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I,
                                                     I, I, I, P]
        lib.ring_attn_bwd_static_scratch.restype = ctypes.c_int
        lib.ring_attn_fwd_tile_visits.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, P]
        lib.ring_attn_fwd_tile_visits.restype = ctypes.c_int
        lib.ring_attn_bwd_tile_visits.argtypes = [P, P, P, P, P, P, P, P, P, I, P, SZ, I, I, I, I, I,
                                                  I, I, I, I, P, P]
        lib.ring_attn_bwd_tile_visits.restype = ctypes.c_int
        lib.ring_attn_rope.argtypes = [P, I, I, I, I, I, I, I, ctypes.c_double, I, P]
        lib.ring_attn_rope.restype = ctypes.c_int
        lib.ring_attn_ulysses_a2a.argtypes = [P, P, I, I, I, I, I, I, I, I, P]
        lib.ring_attn_ulysses_a2a.restype = ctypes.c_int
        lib.ring_attn_ulysses_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, SZ, P]
        lib.ring_attn_ulysses_fwd.restype = ctypes.c_int
        lib.ring_attn_ulysses_workspace_size.argtypes = [I, I, I, I, I, I]
        lib.ring_attn_ulysses_workspace_size.restype = SZ
        lib.ring_attn_ulysses_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, P, SZ, I, I, I, I, I, I, I, I, I, P]
        lib.ring_attn_ulysses_bwd.restype = ctypes.c_int
        lib.ring_attn_ulysses_bwd_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
        lib.ring_attn_ulysses_bwd_workspace_size.restype = SZ
        lib.ring_attn_fwd_host.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, SZ, P]
        lib.ring_attn_fwd_host.restype = ctypes.c_int
        lib.ring_attn_fwd_host_workspace_size.argtypes = [I, I, I, I, I]
        lib.ring_attn_fwd_host_workspace_size.restype = SZ
        lib.ring_attn_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, P, P]
        lib.ring_attn_selftest_bounded_wait.restype = ctypes.c_int
        lib.ring_attn_ring_step_fwd_accumulate.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, P]
        lib.ring_attn_ring_step_fwd_accumulate.restype = ctypes.c_int
        lib.ring_attn_bwd_static_scratch_capacity.argtypes = []
        lib.ring_attn_bwd_static_scratch_capacity.restype = SZ
        D = ctypes.c_double
        lib.ring_attn_qk_norm_rope.argtypes = [P] * 8 + [I] * 9 + [D, D, P, P]
        lib.ring_attn_qk_norm_rope.restype = ctypes.c_int
        lib.ring_attn_qk_norm_rope_bwd.argtypes = [P] * 13 + [SZ] + [I] * 9 + [D, D, P, P]
        lib.ring_attn_qk_norm_rope_bwd.restype = ctypes.c_int
        lib.ring_attn_qk_norm_rope_bwd_workspace_size.argtypes = [I]
        lib.ring_attn_qk_norm_rope_bwd_workspace_size.restype = SZ
        lib.ring_attn_cache_write.argtypes = [P] * 10 + [I] * 7 + [P]
        lib.ring_attn_cache_write.restype = ctypes.c_int
        lib.ring_attn_cache_read.argtypes = [P] * 6 + [I] * 8 + [P]
        lib.ring_attn_cache_read.restype = ctypes.c_int
        lib.ring_attn_tree_fwd.argtypes = [P] * 8 + [I] + [P] * 3 + [SZ] + [I] * 9 + [P]
        lib.ring_attn_tree_fwd.restype = ctypes.c_int
        lib.ring_attn_tree_fwd_workspace_size.argtypes = [I] * 8
        lib.ring_attn_tree_fwd_workspace_size.restype = SZ
        lib.ring_attn_tree_window_fwd.argtypes = [P] * 8 + [I] + [P] * 4 + [SZ] + [I] * 11 + [P]
        lib.ring_attn_tree_window_fwd.restype = ctypes.c_int
        lib.ring_attn_qk_rope_axes.argtypes = [P] * 8 + [I] * 6 + [P, I, I, D, D, P, P]
        lib.ring_attn_qk_rope_axes.restype = ctypes.c_int
        lib.ring_attn_qk_rope_axes_bwd.argtypes = [P] * 13 + [SZ] + [I] * 6 + [P, I, I, D, D, P, P]
        lib.ring_attn_qk_rope_axes_bwd.restype = ctypes.c_int
        lib.ring_attn_window_fwd.argtypes = [P] * 6 + [SZ] + [I] * 12 + [P]
        lib.ring_attn_window_fwd.restype = ctypes.c_int
        lib.ring_attn_window_fwd_workspace_size.argtypes = [I] * 8
        lib.ring_attn_window_fwd_workspace_size.restype = SZ
        lib.ring_attn_window_bwd.argtypes = [P] * 10 + [SZ] + [I] * 13 + [P]
        lib.ring_attn_window_bwd.restype = ctypes.c_int
        lib.ring_attn_window_bwd_workspace_size.argtypes = [I] * 11
        lib.ring_attn_window_bwd_workspace_size.restype = SZ
        for name in EXPORTS:
            f = getattr(lib, name)
            if f.restype is ctypes.c_int or name in ("ring_attn_fwd", "ring_attn_ring_step_fwd",
                                                     "ring_attn_lse_merge", "ring_attn_fwd_stepwise",
                                                     "ring_attn_bwd", "ring_attn_shard_tiles",
                                                     "ring_attn_fwd_path", "ring_attn_bwd_path",
                                                     "ring_attn_device_status",
                                                     "ring_attn_abi_version"):
                f.restype = ctypes.c_int
        _load_calls(lib)
        _lib = lib
        return lib


def _load_calls(lib):
    """The compiled form of the calls below that have one (csrc/calls.cpp), if it was built for this Python and torch."""
    global _calls
    from .build_lib import calls_path

    path = calls_path()
    if not os.path.exists(path):
        return
    name = __package__ + "._calls"
    try:
        loader = importlib.machinery.ExtensionFileLoader(name, path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader(name, loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, "ring_attn_" + f), ctypes.c_void_p).value for f in (
            "qk_norm_rope", "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_size", "cache_write", "cache_read", "tree_fwd",
            "tree_fwd_workspace_size", "qk_rope_axes", "tree_window_fwd", "window_fwd", "window_fwd_workspace_size",
            "window_bwd", "window_bwd_workspace_size")))
    except (ImportError, OSError, AttributeError, TypeError, ValueError) as e:
        warnings.warn(f"the compiled calls in {path} do not load, calls go through Python: {e}", RuntimeWarning)
        return
    _calls = module


def _check(status):
    if status != RA_OK:
        msg = library().ring_attn_last_error().decode(errors="replace")
        raise RingAttnError(status, msg)


def _dtype_code(dt):
    if dt == torch.float32:
        return 0
    if dt == torch.bfloat16:
        return 1
    raise ValueError(f"unsupported dtype {dt}")


def _layout(layout):
    return LAYOUTS[layout] if isinstance(layout, str) else int(layout)


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,H,L,d] and k, v [B,Hkv,L,d]")
    B, H, L, d = q.shape
    Hkv = k.shape[1]
    return int(B), int(H), int(Hkv), int(L), int(d)


def _need(t, name, device, shape=None, dtype=None):
    """The library takes raw pointers and trusts the sizes it is given: every tensor is checked here
    (device, layout, shape, dtype) before its pointer is passed."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")


def _need_qkv(q, k, v):
    """q [B,H,L,d], k and v [B,Hkv,L,d] of q's dtype, all on q's device; returns (B, H, Hkv, L, d)."""
    B, H, Hkv, L, d = _dims(q, k)
    _need(q, "q", q.device)
    _dtype_code(q.dtype)
    _need(k, "k", q.device, (B, Hkv, L, d), q.dtype)
    _need(v, "v", q.device, (B, Hkv, L, d), q.dtype)
    return B, H, Hkv, L, d


def _need_workspace(ws, need, device):
    _need(ws, "workspace", device)
    if ws.dtype != torch.uint8 or ws.numel() < need:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")


def fwd_path(B, H, Hkv, L, d, n_shards, causal, layout, dtype):
    out = ctypes.c_int(0)
    _check(library().ring_attn_fwd_path(B, H, Hkv, L, d, n_shards, int(causal), _layout(layout),
                                        _dtype_code(dtype), ctypes.byref(out)))
    return PATHS[out.value]


def bwd_path(B, H, Hkv, L, d, n_shards, causal, layout, dtype):
    out = ctypes.c_int(0)
    _check(library().ring_attn_bwd_path(B, H, Hkv, L, d, n_shards, int(causal), _layout(layout),
                                        _dtype_code(dtype), ctypes.byref(out)))
    return PATHS[out.value]


def _visits(n_shards, device):
    return torch.zeros((n_shards, n_shards), dtype=torch.int64, device=device)


def fwd(q, k, v, n_shards, causal=True, layout="zigzag", out=None, lse=None, stream=None):
    """Ring Attention forward.  Returns (out [B,H,L,d] q.dtype, lse [B,H,L] float32)."""
    return _fwd(q, k, v, n_shards, causal, layout, out, lse, None, stream)


def fwd_tile_visits(q, k, v, n_shards, causal=True, layout="zigzag", stream=None):
    """ring_attn_fwd_tile_visits: the forward plus the count of (256-row query block, 128-row K/V
    tile) pairs computed per (query shard, key shard).  Returns (out, lse, visits [n, n] int64)."""
    visits = _visits(n_shards, q.device)
    out, lse = _fwd(q, k, v, n_shards, causal, layout, None, None, visits, stream)
    return out, lse, visits


def _fwd(q, k, v, n_shards, causal, layout, out, lse, visits, stream):
    B, H, Hkv, L, d = _need_qkv(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    _need(out, "out", q.device, q.shape, q.dtype)
    _need(lse, "lse", q.device, (B, H, L), torch.float32)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, L, d, int(n_shards),
            int(causal), _layout(layout), _dtype_code(q.dtype))
    if visits is None:
        _check(library().ring_attn_fwd(*args, _stream(stream, q.device)))
    else:
        _check(library().ring_attn_fwd_tile_visits(*args, _ptr(visits), _stream(stream, q.device)))
    return out, lse


def fwd_host(q, k, v, n_shards, causal=True, layout="zigzag", out=None, lse=None, workspace=None, device=None,
             stream=None):
    """ring_attn_fwd_host: q, k, v are CPU tensors (page-locked for overlap); returns CPU (out, lse).
    The copies in and out overlap the compute of other kv-head groups."""
    B, H, Hkv, L, d = _dims(q, k)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    _dtype_code(q.dtype)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, pin_memory=True)
    for t, nm, shape, dt in ((q, "q", q.shape, q.dtype), (k, "k", (B, Hkv, L, d), q.dtype),
                             (v, "v", (B, Hkv, L, d), q.dtype), (out, "out", q.shape, q.dtype),
                             (lse, "lse", (B, H, L), torch.float32)):
        if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{nm} must be a contiguous CPU tensor")
        if tuple(t.shape) != tuple(shape) or t.dtype != dt:
            raise ValueError(f"{nm} must be {dt} of shape {tuple(shape)}")
    need = int(library().ring_attn_fwd_host_workspace_size(H, Hkv, L, d, _dtype_code(q.dtype)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need_workspace(workspace, need, dev)
    _check(library().ring_attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, L, d,
                                        int(n_shards), int(causal), _layout(layout), _dtype_code(q.dtype),
                                        _ptr(workspace), workspace.numel(), _stream(stream, dev)))
    return out, lse


def ring_step_fwd(q, k, v, n_shards, step, causal=True, layout="zigzag", o_part=None,
                  lse_part=None, stream=None):
    """One ring step for all shards.  Returns (o_part float32 [B,H,L,d], lse_part [B,H,L])."""
    B, H, Hkv, L, d = _need_qkv(q, k, v)
    if o_part is None:
        o_part = torch.empty((B, H, L, d), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    _need(o_part, "o_part", q.device, (B, H, L, d), torch.float32)
    _need(lse_part, "lse_part", q.device, (B, H, L), torch.float32)
    _check(library().ring_attn_ring_step_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o_part),
                                             _ptr(lse_part), B, H, Hkv, L, d, int(n_shards),
                                             int(step), int(causal), _layout(layout),
                                             _dtype_code(q.dtype), _stream(stream, q.device)))
    return o_part, lse_part


def ring_step_fwd_accumulate(q, k, v, n_shards, step, o_acc, lse_acc, causal=True, layout="zigzag", stream=None):
    """ring_attn_ring_step_fwd_accumulate: fold ring step `step` into (o_acc float32 [B,H,L,d],
    lse_acc [B,H,L]) in place.  Returns (o_acc, lse_acc)."""
    B, H, Hkv, L, d = _need_qkv(q, k, v)
    _need(o_acc, "o_acc", q.device, (B, H, L, d), torch.float32)
    _need(lse_acc, "lse_acc", q.device, (B, H, L), torch.float32)
    _check(library().ring_attn_ring_step_fwd_accumulate(_ptr(q), _ptr(k), _ptr(v), _ptr(o_acc), _ptr(lse_acc), B, H,
                                                        Hkv, L, d, int(n_shards), int(step), int(causal),
                                                        _layout(layout), _dtype_code(q.dtype),
                                                        _stream(stream, q.device)))
    return o_acc, lse_acc


def lse_merge(o_acc, lse_acc, o_part, lse_part, stream=None):
    """In-place merge of a partial (o_part, lse_part) into (o_acc, lse_acc); float32 tensors."""
    if o_acc.dim() < 1 or tuple(lse_acc.shape) != tuple(o_acc.shape[:-1]):
        raise ValueError("lse_acc must have the shape of o_acc without its last dimension")
    d = int(o_acc.shape[-1])
    rows = int(lse_acc.numel())
    _need(o_acc, "o_acc", o_acc.device, None, torch.float32)
    _need(lse_acc, "lse_acc", o_acc.device, None, torch.float32)
    _need(o_part, "o_part", o_acc.device, o_acc.shape, torch.float32)
    _need(lse_part, "lse_part", o_acc.device, lse_acc.shape, torch.float32)
    _check(library().ring_attn_lse_merge(_ptr(o_acc), _ptr(lse_acc), _ptr(o_part), _ptr(lse_part),
                                         rows, d, _stream(stream, o_acc.device)))
    return o_acc, lse_acc


def fwd_stepwise(q, k, v, n_shards, causal=True, layout="zigzag", out=None, lse=None,
                 workspace=None, stream=None):
    """The ring forward run as n ring-step launches, each folding its block into the running
    result (same results as fwd)."""
    B, H, Hkv, L, d = _need_qkv(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    _need(out, "out", q.device, q.shape, q.dtype)
    _need(lse, "lse", q.device, (B, H, L), torch.float32)
    need = int(library().ring_attn_fwd_stepwise_workspace_size(B, H, L, d))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _need_workspace(workspace, need, q.device)
    _check(library().ring_attn_fwd_stepwise(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H,
                                            Hkv, L, d, int(n_shards), int(causal),
                                            _layout(layout), _dtype_code(q.dtype),
                                            _ptr(workspace), workspace.numel(),
                                            _stream(stream, q.device)))
    return out, lse


def bwd_workspace_size(B, H, Hkv, L, d, grad_dtype=torch.float32):
    return int(library().ring_attn_bwd_workspace_size(B, H, Hkv, L, d, _dtype_code(grad_dtype)))


def bwd(q, k, v, out, lse, dout, n_shards, causal=True, layout="zigzag",
        grad_dtype=torch.float32, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Ring Attention backward.  Returns (dq, dk, dv) in grad_dtype."""
    return _bwd(q, k, v, out, lse, dout, n_shards, causal, layout, grad_dtype, dq, dk, dv,
                workspace, None, stream)


def bwd_tile_visits(q, k, v, out, lse, dout, n_shards, causal=True, layout="zigzag",
                    grad_dtype=torch.float32, stream=None):
    """ring_attn_bwd_tile_visits: the backward plus the count of (128-row query tile, 128-row K/V
    tile) pairs computed per (query shard, key shard).  Returns (dq, dk, dv, visits [n, n] int64)."""
    visits = _visits(n_shards, q.device)
    dq, dk, dv = _bwd(q, k, v, out, lse, dout, n_shards, causal, layout, grad_dtype, None, None,
                      None, None, visits, stream)
    return dq, dk, dv, visits


def _need_bwd_args(q, k, v, out, lse, dout, grad_dtype, out_dtype=None):
    B, H, Hkv, L, d = _need_qkv(q, k, v)
    _need(out, "out", q.device, q.shape, q.dtype if out_dtype is None else out_dtype)
    _need(lse, "lse", q.device, (B, H, L), torch.float32)
    _need(dout, "dout", q.device, q.shape, q.dtype)
    _dtype_code(grad_dtype)
    return B, H, Hkv, L, d


def _need_grads(dq, dk, dv, device, dims, grad_dtype):
    B, H, Hkv, L, d = dims
    _need(dq, "dq", device, (B, H, L, d), grad_dtype)
    _need(dk, "dk", device, (B, Hkv, L, d), grad_dtype)
    _need(dv, "dv", device, (B, Hkv, L, d), grad_dtype)


def _bwd(q, k, v, out, lse, dout, n_shards, causal, layout, grad_dtype, dq, dk, dv, workspace,
         visits, stream, out_f32=False):
    B, H, Hkv, L, d = _need_bwd_args(q, k, v, out, lse, dout, grad_dtype,
                                     torch.float32 if out_f32 else None)
    if dq is None:
        dq = torch.empty((B, H, L, d), dtype=grad_dtype, device=q.device)
    if dk is None:
        dk = torch.empty((B, Hkv, L, d), dtype=grad_dtype, device=q.device)
    if dv is None:
        dv = torch.empty((B, Hkv, L, d), dtype=grad_dtype, device=q.device)
    _need_grads(dq, dk, dv, q.device, (B, H, Hkv, L, d), grad_dtype)
    need = bwd_workspace_size(B, H, Hkv, L, d, grad_dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _need_workspace(workspace, need, q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
            _ptr(dv), _dtype_code(grad_dtype), _ptr(workspace), workspace.numel(), B, H, Hkv, L, d,
            int(n_shards), int(causal), _layout(layout), _dtype_code(q.dtype))
    if out_f32:
        _check(library().ring_attn_bwd_f32out(*args, _stream(stream, q.device)))
    elif visits is None:
        _check(library().ring_attn_bwd(*args, _stream(stream, q.device)))
    else:
        _check(library().ring_attn_bwd_tile_visits(*args, _ptr(visits), _stream(stream, q.device)))
    return dq, dk, dv


def fwd_f32out(q, k, v, n_shards, causal=True, layout="zigzag", out=None, lse=None, stream=None):
    """ring_attn_fwd_f32out: the forward with out in float32 -- the output before it is rounded to
    q's dtype.  Returns (out [B,H,L,d] float32, lse [B,H,L] float32)."""
    B, H, Hkv, L, d = _need_qkv(q, k, v)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    _need(out, "out", q.device, q.shape, torch.float32)
    _need(lse, "lse", q.device, (B, H, L), torch.float32)
    _check(library().ring_attn_fwd_f32out(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, L, d,
                                          int(n_shards), int(causal), _layout(layout), _dtype_code(q.dtype),
                                          _stream(stream, q.device)))
    return out, lse


def bwd_f32out(q, k, v, out, lse, dout, n_shards, causal=True, layout="zigzag",
               grad_dtype=torch.float32, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """ring_attn_bwd_f32out: the backward with out in float32 (from fwd_f32out), so that D is taken from
    the unrounded output.  Returns (dq, dk, dv) in grad_dtype."""
    return _bwd(q, k, v, out, lse, dout, n_shards, causal, layout, grad_dtype, dq, dk, dv,
                workspace, None, stream, out_f32=True)


def bwd_static_scratch(q, k, v, out, lse, dout, n_shards, causal=True, layout="zigzag",
                       grad_dtype=torch.float32, dq=None, dk=None, dv=None, stream=None):
    """ring_attn_bwd_static_scratch: the backward with the library's static scratch (no workspace
    argument; the C call allocates nothing).  Returns (dq, dk, dv) in grad_dtype."""
    B, H, Hkv, L, d = _need_bwd_args(q, k, v, out, lse, dout, grad_dtype)
    if dq is None:
        dq = torch.empty((B, H, L, d), dtype=grad_dtype, device=q.device)
    if dk is None:
        dk = torch.empty((B, Hkv, L, d), dtype=grad_dtype, device=q.device)
    if dv is None:
        dv = torch.empty((B, Hkv, L, d), dtype=grad_dtype, device=q.device)
    _need_grads(dq, dk, dv, q.device, (B, H, Hkv, L, d), grad_dtype)
    _check(library().ring_attn_bwd_static_scratch(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
        _dtype_code(grad_dtype), B, H, Hkv, L, d, int(n_shards), int(causal), _layout(layout),
        _dtype_code(q.dtype), _stream(stream, q.device)))
    return dq, dk, dv


def bwd_static_scratch_capacity():
    return int(library().ring_attn_bwd_static_scratch_capacity())


def shard_tiles(L, n_shards, causal=True, layout="zigzag", tile=128):
    """Host-only: per query shard, the (query tile, key tile) pairs with a visible pair."""
    arr = (ctypes.c_longlong * n_shards)()
    _check(library().ring_attn_shard_tiles(int(L), int(n_shards), int(causal), _layout(layout),
                                           int(tile), arr))
    return [int(x) for x in arr]


def rope(x, n_shards, layout="zigzag", base=10000.0, inverse=False, stream=None):
    """ring_attn_rope: rotary position embedding of x [B, H, L, d] (bf16 or float32) in place, each row
    by its natural position under the layout; inverse=True turns the other way (for gradients).
    Returns x."""
    if x.dim() != 4:
        raise ValueError("x must be [B, H, L, d]")
    _need(x, "x", x.device)
    B, H, L, d = (int(s) for s in x.shape)
    _check(library().ring_attn_rope(_ptr(x), B, H, L, d, int(n_shards), _layout(layout), _dtype_code(x.dtype),
                                    float(base), int(bool(inverse)), _stream(stream, x.device)))
    return x


def ulysses_a2a(src, n_shards, layout="contiguous", direction=0, dst=None, stream=None):
    """ring_attn_ulysses_a2a.  direction 0: src [n, B, S, H, d] (token split) -> [n, B, H/n, L, d]
    (head split); direction 1 the reverse.  A 4-D src [n, B, S, H] (lse) moves rows of one float."""
    _need(src, "src", src.device)
    if direction == 0:
        if src.dim() == 5:
            n, B, S, H, d = (int(s) for s in src.shape)
            shape = (n, B, H // n, n * S, d)
        else:
            n, B, S, H = (int(s) for s in src.shape)
            d = 1
            shape = (n, B, H // n, n * S)
    else:
        if src.dim() == 5:
            n, B, Hn, L, d = (int(s) for s in src.shape)
            S, H = L // n, Hn * n
            shape = (n, B, S, H, d)
        else:
            n, B, Hn, L = (int(s) for s in src.shape)
            S, H, d = L // n, Hn * n, 1
            shape = (n, B, S, H)
    if n != n_shards:
        raise ValueError("the leading dimension of src must be n_shards")
    if dst is None:
        dst = torch.empty(shape, dtype=src.dtype, device=src.device)
    _need(dst, "dst", src.device, shape, src.dtype)
    _check(library().ring_attn_ulysses_a2a(_ptr(src), _ptr(dst), B, H, n * S, d, n, _layout(layout),
                                           _dtype_code(src.dtype), int(direction), _stream(stream, src.device)))
    return dst


def _need_ulysses_qkv(q, k, v, n_shards):
    """q [n, B, S, H, d], k and v [n, B, S, Hkv, d] of q's dtype; returns (n, B, S, H, Hkv, d)."""
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != 5:
            raise ValueError(f"{nm} must be [n, B, S, heads, d]")
    n, B, S, H, d = (int(s) for s in q.shape)
    Hkv = int(k.shape[3])
    if n != n_shards:
        raise ValueError("the leading dimension of q must be n_shards")
    _need(q, "q", q.device)
    _dtype_code(q.dtype)
    _need(k, "k", q.device, (n, B, S, Hkv, d), q.dtype)
    _need(v, "v", q.device, (n, B, S, Hkv, d), q.dtype)
    return n, B, S, H, Hkv, d


def ulysses_fwd(q, k, v, n_shards, causal=True, layout="contiguous", out=None, lse=None, workspace=None,
                stream=None):
    """ring_attn_ulysses_fwd: q [n, B, S, H, d], k and v [n, B, S, Hkv, d] (token split).  Returns
    (out [n, B, S, H, d], lse [n, B, S, H] float32)."""
    n, B, S, H, Hkv, d = _need_ulysses_qkv(q, k, v, n_shards)
    L = n * S
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((n, B, S, H), dtype=torch.float32, device=q.device)
    _need(out, "out", q.device, q.shape, q.dtype)
    _need(lse, "lse", q.device, (n, B, S, H), torch.float32)
    need = int(library().ring_attn_ulysses_workspace_size(B, H, Hkv, L, d, _dtype_code(q.dtype)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _need_workspace(workspace, need, q.device)
    _check(library().ring_attn_ulysses_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv, L, d, n,
                                           int(causal), _layout(layout), _dtype_code(q.dtype), _ptr(workspace),
                                           workspace.numel(), _stream(stream, q.device)))
    return out, lse


def ulysses_bwd(q, k, v, out, lse, dout, n_shards, causal=True, layout="contiguous", grad_dtype=torch.float32,
                workspace=None, stream=None):
    """ring_attn_ulysses_bwd: token-split inputs as for ulysses_fwd (plus out, lse from it and dout
    [n, B, S, H, d]).  Returns (dq, dk, dv) in the token split, grad_dtype."""
    n, B, S, H, Hkv, d = _need_ulysses_qkv(q, k, v, n_shards)
    L = n * S
    _need(out, "out", q.device, q.shape, q.dtype)
    _need(lse, "lse", q.device, (n, B, S, H), torch.float32)
    _need(dout, "dout", q.device, q.shape, q.dtype)
    _dtype_code(grad_dtype)
    dq = torch.empty(q.shape, dtype=grad_dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=grad_dtype, device=q.device)
    dv = torch.empty(v.shape, dtype=grad_dtype, device=q.device)
    need = int(library().ring_attn_ulysses_bwd_workspace_size(B, H, Hkv, L, d, n, _dtype_code(q.dtype),
                                                              _dtype_code(grad_dtype)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _need_workspace(workspace, need, q.device)
    _check(library().ring_attn_ulysses_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                                           _ptr(dk), _ptr(dv), _dtype_code(grad_dtype), _ptr(workspace),
                                           workspace.numel(), B, H, Hkv, L, d, n, int(causal), _layout(layout),
                                           _dtype_code(q.dtype), _stream(stream, q.device)))
    return dq, dk, dv


def selftest_bounded_wait(limit_ns=2_000_000, stream=None, device=None):
    """ring_attn_selftest_bounded_wait: a GPU wait that nothing completes runs out after limit_ns.
    Returns the kernel's report (1: gave up, 2: completed); the status word then has the timeout bit."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    flag = torch.zeros(4, dtype=torch.int32, device=dev)
    _check(library().ring_attn_selftest_bounded_wait(int(limit_ns), _ptr(flag), _stream(stream, dev)))
    return int(flag[0].item())


def device_status(stream=None, device=None):
    """Reads and clears the device status word (bit RA_DEVICE_TIMEOUT: a bounded wait ran out)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    st = ctypes.c_uint(0)
    _check(library().ring_attn_device_status(ctypes.byref(st), _stream(stream, dev)))
    return int(st.value)


def device_check(stream=None, device=None):
    """ring_attn_device_check: synchronises the stream, reads and clears the device status word and
    raises RingAttnError (status RA_ERR_TIMEOUT) if a bounded wait inside a kernel ran out."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _check(library().ring_attn_device_check(_stream(stream, dev)))


# ------------------------------------------------------------------------------------------------
# One device of the multi-device ring: local shard buffers of S = L / n_shards rows per head
# ------------------------------------------------------------------------------------------------
def _need_block(q, k, v, n_shards, shard_q, shard_kv):
    """q [B,H,S,d] (shard shard_q's rows), k and v [B,Hkv,S,d] (shard shard_kv's rows), same dtype and
    device; returns (B, H, Hkv, S, d, L = n_shards * S)."""
    B, H, Hkv, S, d = _need_qkv(q, k, v)
    n = int(n_shards)
    if n < 1 or not (0 <= int(shard_q) < n and 0 <= int(shard_kv) < n):
        raise ValueError("shard indices must lie in [0, n_shards)")
    return B, H, Hkv, S, d, n * S


def block_fwd(q, k, v, o_acc, lse_acc, n_shards, shard_q, shard_kv, accumulate, causal=True, layout="zigzag",
              stream=None):
    """ring_attn_block_fwd: block attention of the local query shard shard_q against the K/V block of
    shard shard_kv, written to (accumulate=False) or folded into (accumulate=True) the running state
    o_acc [B,H,S,d] float32 (normalised output) and lse_acc [B,H,S] float32.  Returns (o_acc, lse_acc)."""
    B, H, Hkv, S, d, L = _need_block(q, k, v, n_shards, shard_q, shard_kv)
    _need(o_acc, "o_acc", q.device, (B, H, S, d), torch.float32)
    _need(lse_acc, "lse_acc", q.device, (B, H, S), torch.float32)
    _check(library().ring_attn_block_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o_acc), _ptr(lse_acc), B, H, Hkv, L, d,
                                         int(n_shards), int(shard_q), int(shard_kv), int(bool(accumulate)),
                                         int(causal), _layout(layout), _dtype_code(q.dtype),
                                         _stream(stream, q.device)))
    return o_acc, lse_acc


def block_bwd(q, k, v, dout, lse, D, dq_acc, dk, dv, n_shards, shard_q, shard_kv, accumulate_kv, causal=True,
              layout="zigzag", stream=None):
    """ring_attn_block_bwd: the gradient contributions of the pairs (query of shard shard_q, key of shard
    shard_kv): added into dq_acc [B,H,S,d] float32; added into (accumulate_kv=True) or stored to dk, dv
    [B,Hkv,S,d] float32.  lse and D [B,H,S] float32 are the query rows' full log-sum-exp and
    rowsum(dout * out).  Returns (dq_acc, dk, dv)."""
    B, H, Hkv, S, d, L = _need_block(q, k, v, n_shards, shard_q, shard_kv)
    _need(dout, "dout", q.device, q.shape, q.dtype)
    _need(lse, "lse", q.device, (B, H, S), torch.float32)
    _need(D, "D", q.device, (B, H, S), torch.float32)
    _need(dq_acc, "dq_acc", q.device, (B, H, S, d), torch.float32)
    _need(dk, "dk", q.device, (B, Hkv, S, d), torch.float32)
    _need(dv, "dv", q.device, (B, Hkv, S, d), torch.float32)
    _check(library().ring_attn_block_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse), _ptr(D), _ptr(dq_acc),
                                         _ptr(dk), _ptr(dv), B, H, Hkv, L, d, int(n_shards), int(shard_q),
                                         int(shard_kv), int(bool(accumulate_kv)), int(causal), _layout(layout),
                                         _dtype_code(q.dtype), _stream(stream, q.device)))
    return dq_acc, dk, dv


def bwd_preprocess(out, dout, D=None, stream=None):
    """ring_attn_bwd_preprocess: D = rowsum(out * dout) over the last dimension, float32.  out may be
    float32 while dout is bf16 (ring_attn_bwd_preprocess_f32out: the unrounded output)."""
    _need(out, "out", out.device)
    _dtype_code(dout.dtype)
    f32out = out.dtype == torch.float32 and dout.dtype != torch.float32
    _need(dout, "dout", out.device, out.shape, dout.dtype if f32out else out.dtype)
    if D is None:
        D = torch.empty(out.shape[:-1], dtype=torch.float32, device=out.device)
    _need(D, "D", out.device, out.shape[:-1], torch.float32)
    d = int(out.shape[-1])
    call = library().ring_attn_bwd_preprocess_f32out if f32out else library().ring_attn_bwd_preprocess
    _check(call(_ptr(out), _ptr(dout), _ptr(D), int(D.numel()), d, _dtype_code(dout.dtype),
                _stream(stream, out.device)))
    return D


def f32_zero(x, stream=None):
    """ring_attn_f32_zero: x (float32) = 0.  Returns x."""
    _need(x, "x", x.device, None, torch.float32)
    _check(library().ring_attn_f32_zero(_ptr(x), int(x.numel()), _stream(stream, x.device)))
    return x


def f32_add(acc, part, stream=None):
    """ring_attn_f32_add: acc += part (float32, same shape).  Returns acc."""
    _need(acc, "acc", acc.device, None, torch.float32)
    _need(part, "part", acc.device, acc.shape, torch.float32)
    _check(library().ring_attn_f32_add(_ptr(acc), _ptr(part), int(acc.numel()), _stream(stream, acc.device)))
    return acc


def f32_convert(src, dtype, dst=None, stream=None):
    """ring_attn_f32_convert: src (float32) converted to dtype (float32 or bfloat16).  Returns dst."""
    _need(src, "src", src.device, None, torch.float32)
    if dst is None:
        dst = torch.empty(src.shape, dtype=dtype, device=src.device)
    _need(dst, "dst", src.device, src.shape, dtype)
    _check(library().ring_attn_f32_convert(_ptr(src), _ptr(dst), int(src.numel()), _dtype_code(dtype),
                                           _stream(stream, src.device)))
    return dst


def block_rope(x, n_shards, shard, layout="zigzag", base=10000.0, inverse=False, stream=None):
    """ring_attn_block_rope: rotary position embedding, in place, of one device's shard x [B, H, S, d]
    (shard `shard` of n_shards; bf16 or float32), each row by its natural position in the whole
    sequence.  Returns x."""
    if x.dim() != 4:
        raise ValueError("x must be [B, H, S, d]")
    _need(x, "x", x.device)
    B, H, S, d = (int(t) for t in x.shape)
    n = int(n_shards)
    if not 0 <= int(shard) < n:
        raise ValueError("shard must lie in [0, n_shards)")
    _check(library().ring_attn_block_rope(_ptr(x), B, H, n * S, d, n, int(shard), _layout(layout),
                                          _dtype_code(x.dtype), float(base), int(bool(inverse)),
                                          _stream(stream, x.device)))
    return x


# ------------------------------------------------------------------------------------------------
# Norms and rotation of queries and keys, the key/value cache and the attention over it
# ------------------------------------------------------------------------------------------------
# The calls of a serving step take a few microseconds on the GPU, so on the current stream they go through their compiled
# form (csrc/calls.cpp: 24 -> 10 us for the attention over a short cache), which answers None to whatever it does not take:
# then, and where it was not built, the Python form runs, which says what is wrong.  Its checks are kept cheap too: one
# expression per tensor on the way that passes, and the checks that name what is wrong only where it fails.
_Strides = ctypes.c_longlong * 3
_E4M3 = torch.float8_e4m3fn
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream, index):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _hand_over(stream, index, *tensors):
    """Memory that a call allocates (given: None, new: a tensor) comes from the current stream.  The caller's other stream waits
    for what that one still has to do with it, and has to be done with it before it is given out again."""
    new = [t for given, t in tensors if given is None]
    if stream is None or not new:
        return
    current = torch.cuda.current_stream(index)
    if stream != current:
        if _capturing(stream) == _capturing(current):  # (what a capture records waits for nothing outside it)
            stream.wait_stream(current)
        for t in new:
            t.record_stream(stream)


def _capturing(stream):
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _run(index, call, *args):
    """Calls the library with device `index` current: a kernel is launched on the device of its tensors."""
    if torch.cuda.current_device() == index:
        st = call(*args)
    else:
        with torch.cuda.device(index):
            st = call(*args)
    if st != RA_OK:
        _check(st)


def _fits(t, name, device, shape, dtype):
    """A contiguous tensor of this device, shape and dtype; returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda
            and t.is_contiguous()):
        _need(t, name, device, shape, dtype)
    return t.data_ptr()


def _output(t, name, device, shape, dtype):
    """The caller's output, checked, or a new one; and its address."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _fits(t, name, device, shape, dtype)


def _rows(t, name, device, shape, dtype):
    """A tensor read by strides: any [B, heads, rows, d] whose rows are contiguous and lie on 16-byte boundaries.
    Returns its address and its (batch, head, row) element strides, None if it is contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda or t.device != device:
            raise ValueError(f"{name} must be a CUDA tensor on {device}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.is_contiguous():
        return t.data_ptr(), None
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 or (s0 | s1 | s2) % (16 // t.element_size()):
        per = 16 // t.element_size()
        if s3 != 1 or any(n > 1 and s % per for n, s in zip(shape, (s0, s1, s2))):
            raise ValueError(f"{name} must have contiguous rows on 16-byte boundaries")
    return t.data_ptr(), _Strides(s0, s1, s2)


def as_rows(t):
    """t, or a contiguous copy if its rows cannot be read where they lie."""
    per = 16 // t.element_size()
    if t.dim() == 4 and t.stride(3) == 1 and not any(n > 1 and s % per for n, s in zip(t.shape, t.stride()[:3])) \
            and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _dims4(q, k, name):
    """The shapes [B, heads, rows, d] of two tensors and q's dtype code."""
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor):
        raise TypeError("the inputs must be torch tensors")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"{name} must be [B, heads, rows, d]")
    code = _DTYPES.get(q.dtype)
    return q.shape, k.shape, _dtype_code(q.dtype) if code is None else code


def _norm_rope_args(q, k, wq, wk, n_shards, layout, base, eps, shard, positions):
    (B, H, rows, d), (_, Hkv, _, _), code = _dims4(q, k, "q and k")
    dev, dt = q.device, q.dtype
    qp, qs = _rows(q, "q", dev, (B, H, rows, d), dt)
    kp, ks = _rows(k, "k", dev, (B, Hkv, rows, d), dt)
    head = (qp, qs, kp, ks, _fits(wq, "wq", dev, (d,), torch.float32), _fits(wk, "wk", dev, (d,), torch.float32))
    n = int(n_shards)
    L, which, pos = rows, -1, None
    if positions is not None:
        pos = _fits(positions, "positions", dev, (B, rows), torch.int32)
        if shard is not None or n != 1:
            raise ValueError("positions stand in place of a layout: n_shards must be 1 and shard None")
        layout = 0
    elif shard is not None:
        which = int(shard)
        if not 0 <= which < n:
            raise ValueError("shard must lie in [0, n_shards)")
        L = n * rows
    return head, (B, H, Hkv, L, d, n, which, _layout(layout), code, float(base), float(eps), pos)


def qk_norm_rope(q, k, wq, wk, n_shards=1, layout="contiguous", base=10000.0, eps=1e-6, shard=None, positions=None,
                 q_out=None, k_out=None, stream=None):
    """ring_attn_qk_norm_rope: every head of q [B,H,rows,d] and k [B,Hkv,rows,d] divided by its root mean square
    (eps added to the mean square), times wq or wk [d] float32, then rotated by its natural position -- the
    layout's over n_shards shards, shard `shard`'s of them, or positions [B, rows] int32.  q and k may be
    slices of a fused projection (rows contiguous, on 16-byte boundaries).  Returns (q_out, k_out), contiguous,
    in q's dtype; q_out may be q and k_out may be k, where those are contiguous."""
    if _calls is not None and stream is None:
        done = _calls.qk_norm_rope(q, k, wq, wk, n_shards, layout, base, eps, shard, positions, q_out, k_out)
        if done is not None:
            return done
    head, tail = _norm_rope_args(q, k, wq, wk, n_shards, layout, base, eps, shard, positions)
    dev, dt = q.device, q.dtype
    given = q_out, k_out
    q_out, qo = _output(q_out, "q_out", dev, q.shape, dt)
    k_out, ko = _output(k_out, "k_out", dev, k.shape, dt)
    _hand_over(stream, dev.index, (given[0], q_out), (given[1], k_out))
    _run(dev.index, library().ring_attn_qk_norm_rope, *head, qo, ko, *tail, _stream_ptr(stream, dev.index))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, wq, wk, dq_out, dk_out, n_shards=1, layout="contiguous", base=10000.0, eps=1e-6, shard=None,
                     positions=None, dq=None, dk=None, workspace=None, stream=None):
    """ring_attn_qk_norm_rope_bwd: the gradients of qk_norm_rope's inputs from those of its outputs (contiguous).
    Returns (dq, dk) in q's dtype, contiguous (dq may be dq_out, dk may be dk_out), and (dwq, dwk) [d] float32."""
    if _calls is not None and stream is None:
        done = _calls.qk_norm_rope_bwd(q, k, wq, wk, dq_out, dk_out, n_shards, layout, base, eps, shard, positions, dq, dk,
                                       workspace)
        if done is not None:
            return done
    head, tail = _norm_rope_args(q, k, wq, wk, n_shards, layout, base, eps, shard, positions)
    dev, dt, d = q.device, q.dtype, q.shape[3]
    gq, gk = _fits(dq_out, "dq_out", dev, q.shape, dt), _fits(dk_out, "dk_out", dev, k.shape, dt)
    given = dq, dk, workspace
    dq, dqp = _output(dq, "dq", dev, q.shape, dt)
    dk, dkp = _output(dk, "dk", dev, k.shape, dt)
    dwq, dwk = torch.empty(d, dtype=torch.float32, device=dev), torch.empty(d, dtype=torch.float32, device=dev)
    lib = library()
    need = lib.ring_attn_qk_norm_rope_bwd_workspace_size(d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    _hand_over(stream, dev.index, (given[0], dq), (given[1], dk), (None, dwq), (None, dwk), (given[2], workspace))
    _run(dev.index, lib.ring_attn_qk_norm_rope_bwd, *head, gq, gk, dqp, dkp, dwq.data_ptr(), dwk.data_ptr(),
         workspace.data_ptr(), workspace.numel(), *tail, _stream_ptr(stream, dev.index))
    return dq, dk, dwq, dwk


def _axes_args(dev, B, rows, d, positions, sections, spectrum, wq, wk):
    """(address of the positions, number of axes, the sections as a C array, the spectrum's code, addresses of the weights)"""
    sections = [_whole(x, "a section") for x in sections]
    if not 1 <= len(sections) <= 4:
        raise ValueError("sections must name 1 to 4 axes")
    if spectrum not in SPECTRA:
        raise ValueError(f"spectrum must be one of {tuple(SPECTRA)}")
    pos = _fits(positions, "positions", dev, (len(sections), B, rows), torch.int32)
    if (wq is None) != (wk is None):
        raise ValueError("wq and wk must both be given, or neither")
    w = (None, None) if wq is None else (_fits(wq, "wq", dev, (d,), torch.float32), _fits(wk, "wk", dev, (d,), torch.float32))
    return pos, len(sections), (ctypes.c_int * len(sections))(*sections), SPECTRA[spectrum], w


def qk_rope_axes(q, k, positions, sections, wq=None, wk=None, base=10000.0, eps=1e-6, spectrum="whole", q_out=None, k_out=None,
                 stream=None):
    """ring_attn_qk_rope_axes: every head of q [B,H,rows,d] and k [B,Hkv,rows,d] rotated by positions with several axes,
    positions [axes, B, rows] int32: the first sections[0] pairs of a head by its token's position along axis 0, the next
    sections[1] by axis 1 and so on (d/2 pairs in all).  spectrum "whole": pair i of the head has the frequency
    base^(-2i/d); "axis": pair u of an axis's m has base^(-u/m).  With weights wq, wk [d] float32 the heads are normed
    first, as in qk_norm_rope.  q and k may be slices of a fused projection.  Returns (q_out, k_out), contiguous, in q's
    dtype."""
    if _calls is not None and stream is None:
        done = _calls.qk_rope_axes(q, k, positions, sections, wq, wk, base, eps, spectrum, q_out, k_out)
        if done is not None:
            return done
    (B, H, rows, d), (_, Hkv, _, _), code = _dims4(q, k, "q and k")
    dev, dt = q.device, q.dtype
    qp, qs = _rows(q, "q", dev, (B, H, rows, d), dt)
    kp, ks = _rows(k, "k", dev, (B, Hkv, rows, d), dt)
    pos, axes, sec, spec, w = _axes_args(dev, B, rows, d, positions, sections, spectrum, wq, wk)
    given = q_out, k_out
    q_out, qo = _output(q_out, "q_out", dev, q.shape, dt)
    k_out, ko = _output(k_out, "k_out", dev, k.shape, dt)
    _hand_over(stream, dev.index, (given[0], q_out), (given[1], k_out))
    _run(dev.index, library().ring_attn_qk_rope_axes, qp, qs, kp, ks, *w, qo, ko, B, H, Hkv, rows, d, axes, sec, spec, code,
         float(base), float(eps), pos, _stream_ptr(stream, dev.index))
    return q_out, k_out


def qk_rope_axes_bwd(dq_out, dk_out, positions, sections, q=None, k=None, wq=None, wk=None, base=10000.0, eps=1e-6,
                     spectrum="whole", dq=None, dk=None, workspace=None, stream=None):
    """ring_attn_qk_rope_axes_bwd: the gradients of qk_rope_axes' inputs from those of its outputs, dq_out [B,H,rows,d] and
    dk_out [B,Hkv,rows,d] (contiguous).  With the norm's weights q and k are needed too.  Returns (dq, dk, dwq, dwk), the
    last two None without weights; dq may be dq_out, dk may be dk_out."""
    (B, H, rows, d), (_, Hkv, _, _), code = _dims4(dq_out, dk_out, "dq_out and dk_out")
    dev, dt = dq_out.device, dq_out.dtype
    gq, gk = _fits(dq_out, "dq_out", dev, (B, H, rows, d), dt), _fits(dk_out, "dk_out", dev, (B, Hkv, rows, d), dt)
    pos, axes, sec, spec, w = _axes_args(dev, B, rows, d, positions, sections, spectrum, wq, wk)
    lib, given = library(), (dq, dk, workspace)
    qp = qs = kp = ks = dwq = dwk = None
    new = []
    if wq is None:
        if q is not None or k is not None:
            raise ValueError("q and k are the norm's inputs: they need its weights")
        ws, ws_bytes = None, 0
    else:
        qp, qs = _rows(q, "q", dev, (B, H, rows, d), dt)
        kp, ks = _rows(k, "k", dev, (B, Hkv, rows, d), dt)
        dwq, dwk = torch.empty(d, dtype=torch.float32, device=dev), torch.empty(d, dtype=torch.float32, device=dev)
        need = lib.ring_attn_qk_norm_rope_bwd_workspace_size(d)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            _need_workspace(workspace, need, dev)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
        new = [(None, dwq), (None, dwk), (given[2], workspace)]
    dq, dqp = _output(dq, "dq", dev, (B, H, rows, d), dt)
    dk, dkp = _output(dk, "dk", dev, (B, Hkv, rows, d), dt)
    _hand_over(stream, dev.index, (given[0], dq), (given[1], dk), *new)
    _run(dev.index, lib.ring_attn_qk_rope_axes_bwd, qp, qs, kp, ks, *w, gq, gk, dqp, dkp,
         None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(), ws, ws_bytes, B, H, Hkv, rows, d, axes,
         sec, spec, code, float(base), float(eps), pos, _stream_ptr(stream, dev.index))
    return dq, dk, dwq, dwk


def _whole(x, name):
    """An integer argument that the library takes as a C int."""
    x = operator.index(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} does not fit 32 bits")
    return x


def window_fwd(q, k, v, n_shards, window, sinks=0, causal=True, layout="zigzag", out_dtype=None, out=None, lse=None,
               workspace=None, stream=None):
    """ring_attn_window_fwd: attention of whole sequences, q [B,H,L,d], k and v [B,Hkv,L,d] in the layout's order, where
    the token at natural position p sees the tokens j <= p with p - j < window, and the first `sinks` ones (causal=False:
    |p - j| < window, and the first ones).  Returns (out [B,H,L,d] in out_dtype -- q's, or float32 -- and lse [B,H,L]
    float32)."""
    if _calls is not None and stream is None:
        done = _calls.window_fwd(q, k, v, n_shards, window, sinks, causal, layout, out_dtype, out, lse, workspace)
        if done is not None:
            return done
    B, H, Hkv, L, d = _need_qkv(q, k, v)
    dev, lib = q.device, library()
    if out_dtype is None:
        out_dtype = q.dtype
    elif out_dtype not in (q.dtype, torch.float32):
        raise ValueError("out_dtype must be q's dtype or float32")
    n, window, sinks = _whole(n_shards, "n_shards"), _whole(window, "window"), _whole(sinks, "sinks")
    code, lay = _dtype_code(q.dtype), _layout(layout)
    given = out, lse, workspace
    out, op = _output(out, "out", dev, q.shape, out_dtype)
    lse, lp = _output(lse, "lse", dev, (B, H, L), torch.float32)
    need = int(lib.ring_attn_window_fwd_workspace_size(B, H, Hkv, L, d, n, lay, code))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    _hand_over(stream, dev.index, (given[0], out), (given[1], lse), (given[2], workspace))
    _run(dev.index, lib.ring_attn_window_fwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), op, lp, workspace.data_ptr(),
         workspace.numel(), B, H, Hkv, L, d, n, window, sinks, int(bool(causal)), lay, code, _DTYPES[out_dtype],
         _stream_ptr(stream, dev.index))
    return out, lse


def window_bwd(q, k, v, out, lse, dout, n_shards, window, sinks=0, causal=True, layout="zigzag", grad_dtype=torch.float32,
               dq=None, dk=None, dv=None, workspace=None, stream=None):
    """ring_attn_window_bwd: the gradients of window_fwd's inputs from that of its output, dout (q's dtype), with the
    forward's out (q's dtype or float32) and lse.  Returns (dq, dk, dv) in grad_dtype."""
    if _calls is not None and stream is None:
        done = _calls.window_bwd(q, k, v, out, lse, dout, n_shards, window, sinks, causal, layout, grad_dtype, dq, dk, dv, workspace)
        if done is not None:
            return done
    B, H, Hkv, L, d = _need_qkv(q, k, v)
    dev, lib = q.device, library()
    _need(out, "out", dev, q.shape)
    if out.dtype not in (q.dtype, torch.float32):
        raise ValueError("out must be in q's dtype or float32")
    _need(lse, "lse", dev, (B, H, L), torch.float32)
    _need(dout, "dout", dev, q.shape, q.dtype)
    n, window, sinks = _whole(n_shards, "n_shards"), _whole(window, "window"), _whole(sinks, "sinks")
    code, gcode, lay, causal = _dtype_code(q.dtype), _dtype_code(grad_dtype), _layout(layout), int(bool(causal))
    given = dq, dk, dv, workspace
    dq, dqp = _output(dq, "dq", dev, q.shape, grad_dtype)
    dk, dkp = _output(dk, "dk", dev, k.shape, grad_dtype)
    dv, dvp = _output(dv, "dv", dev, k.shape, grad_dtype)
    need = int(lib.ring_attn_window_bwd_workspace_size(B, H, Hkv, L, d, n, window, sinks, causal, lay, code))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    _hand_over(stream, dev.index, (given[0], dq), (given[1], dk), (given[2], dv), (given[3], workspace))
    _run(dev.index, lib.ring_attn_window_bwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
         dout.data_ptr(), dqp, dkp, dvp, workspace.data_ptr(), workspace.numel(), B, H, Hkv, L, d, n, window, sinks, causal,
         lay, code, _DTYPES[out.dtype], gcode, _stream_ptr(stream, dev.index))
    return dq, dk, dv


class KVCache(NamedTuple):
    """A key/value cache: k, v [B, Hkv, cap, d], bfloat16 or float32 like the tensors written to it, or
    float8_e4m3fn with the rows' exponents + 127 in k_exp, v_exp [B, Hkv, cap] uint8 (an element stands for
    its e4m3 value times 2^(byte - 127), byte 1 to 247).  The caller keeps the lengths."""
    k: torch.Tensor
    v: torch.Tensor
    k_exp: Optional[torch.Tensor] = None
    v_exp: Optional[torch.Tensor] = None


def cache_alloc(B, Hkv, cap, d, dtype=_E4M3, device=None):
    """A KVCache of zeros: dtype float8_e4m3fn (quantised as it is written), bfloat16 or float32."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    _cache_code(dtype)
    k, v = (torch.zeros((B, Hkv, cap, d), dtype=dtype, device=dev) for _ in range(2))
    if dtype != _E4M3:
        return KVCache(k, v)
    return KVCache(k, v, *(torch.zeros((B, Hkv, cap), dtype=torch.uint8, device=dev) for _ in range(2)))


def _cache_code(dtype):
    return RA_E4M3 if dtype == _E4M3 else _dtype_code(dtype)


def _cache_args(cache, device, B, Hkv, d, dtype):
    """Checks a cache against the tensors it is used with; returns its addresses, its rows and its dtype's code."""
    k, v, ke, ve = cache
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("the cache's k must be a [B, Hkv, cap, d] tensor")
    cap, kind = k.shape[2], k.dtype
    shape = (B, Hkv, cap, d)
    if kind is not _E4M3:
        if kind is not dtype:
            raise ValueError(f"the cache must hold {dtype} or float8_e4m3fn, not {kind}")
        return (_fits(k, "the cache's k", device, shape, kind), _fits(v, "the cache's v", device, shape, kind), None, None), cap, \
            _DTYPES[kind]
    rows = shape[:3]
    return (_fits(k, "the cache's k", device, shape, kind), _fits(v, "the cache's v", device, shape, kind),
            _fits(ke, "the cache's k_exp", device, rows, torch.uint8), _fits(ve, "the cache's v_exp", device, rows, torch.uint8)), \
        cap, RA_E4M3


def cache_write(cache, k, v, lens=None, ntok=None, stream=None):
    """ring_attn_cache_write: tokens t < ntok[b] (all T without ntok) of k and v [B, Hkv, T, d] to the rows
    lens[b] + t (t without lens) of the cache, quantised there if it is float8_e4m3fn.  lens, ntok: int32 [B] on
    the device.  k and v may be slices of a fused projection.  Rows outside the cache are not written (the
    device status word then has the range bit).  Returns the cache."""
    if _calls is not None and stream is None:
        done = _calls.cache_write(cache, k, v, lens, ntok)
        if done is not None:
            return cache
    shape, _, code = _dims4(k, v, "k and v")
    B, Hkv, T, d = shape
    dev, dt = k.device, k.dtype
    kp, ks = _rows(k, "k", dev, shape, dt)
    vp, vs = _rows(v, "v", dev, shape, dt)
    ptrs, cap, kind = _cache_args(cache, dev, B, Hkv, d, dt)
    _run(dev.index, library().ring_attn_cache_write, kp, ks, vp, vs, *ptrs,
         None if lens is None else _fits(lens, "lens", dev, (B,), torch.int32),
         None if ntok is None else _fits(ntok, "ntok", dev, (B,), torch.int32), B, Hkv, T, d, cap, code, kind,
         _stream_ptr(stream, dev.index))
    return cache


def cache_read(cache, rows, row0=0, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """ring_attn_cache_read: rows [row0, row0 + rows) of every sequence and kv head as (k, v) [B, Hkv, rows, d] in
    dtype: the values the cache stands for."""
    if _calls is not None and stream is None:
        done = _calls.cache_read(cache, rows, row0, dtype, k, v)
        if done is not None:
            return done
    if not isinstance(cache.k, torch.Tensor) or cache.k.dim() != 4:
        raise ValueError("the cache's k must be a [B, Hkv, cap, d] tensor")
    B, Hkv, _, d = cache.k.shape
    dev = cache.k.device
    code = _dtype_code(dtype)
    ptrs, cap, kind = _cache_args(cache, dev, B, Hkv, d, dtype)
    rows, row0 = int(rows), int(row0)
    if rows < 0 or row0 < 0 or row0 + rows > cap:
        raise ValueError(f"rows [{row0}, {row0 + rows}) lie outside the cache ({cap} rows)")
    shape = (B, Hkv, rows, d)
    given = k, v
    k, kp = _output(k, "k", dev, shape, dtype)
    v, vp = _output(v, "v", dev, shape, dtype)
    _hand_over(stream, dev.index, (given[0], k), (given[1], v))
    _run(dev.index, library().ring_attn_cache_read, *ptrs, kp, vp, B, Hkv, row0, rows, d, cap, code, kind,
         _stream_ptr(stream, dev.index))
    return k, v


def tree_workspace_size(B, H, Hkv, T, d, cap, dtype, cache_dtype):
    return _tree_workspace(B, H, Hkv, T, d, cap, _dtype_code(dtype), _cache_code(cache_dtype))


@functools.lru_cache(maxsize=256)
def _tree_workspace(*sizes):
    return int(library().ring_attn_tree_fwd_workspace_size(*sizes))


def tree_fwd(q, cache, lens, mask=None, ntok=None, out_dtype=None, out=None, lse=None, workspace=None, stream=None, window=None,
             sinks=0, positions=None):
    """ring_attn_tree_fwd: attention of T new tokens per sequence, q [B, H, T, d], over a cache that already holds
    their keys and values in the rows lens[b] + t (cache_write): token t of sequence b sees the prefix, rows
    [0, lens[b]), and the step's tokens j < ntok[b] with mask[b, t, j] ([B, T, T] or [T, T] bool; without a mask
    j <= t).  lens, ntok: int32 [B] on the device.  Returns (out [B, H, T, d] in out_dtype -- q's, or float32 --
    and lse [B, H, T] float32); a row that sees nothing, and tokens t >= ntok[b], have 0 and -infinity.
    window, sinks (ring_attn_tree_window_fwd): of the prefix a token at position p sees the rows j > p - window and the
    first `sinks` ones alone.  positions [B, T] int32: the tokens' positions where a mask says which of the step's tokens
    they see (lens[b] + depth in a tree); without them, and without a mask, token t is at lens[b] + t, and without a mask
    it sees the step's tokens j <= t with t - j < window and those among the first `sinks` of the sequence."""
    if _calls is not None and stream is None:
        if window is None and not sinks and positions is None:
            done = _calls.tree_fwd(q, cache, lens, mask, ntok, out_dtype, out, lse, workspace)
        else:
            done = _calls.tree_window_fwd(q, cache, lens, mask, ntok, out_dtype, out, lse, workspace, window, sinks, positions)
        if done is not None:
            return done
    (B, H, T, d), kshape, code = _dims4(q, cache.k, "q and the cache's k")
    Hkv, dev, dt = kshape[1], q.device, q.dtype
    qp = _fits(q, "q", dev, q.shape, dt)
    ptrs, cap, kind = _cache_args(cache, dev, B, Hkv, d, dt)
    if out_dtype is None:
        out_dtype = dt
    elif out_dtype not in (dt, torch.float32):
        raise ValueError("out_dtype must be q's dtype or float32")
    if lens is None:
        raise ValueError("lens is required")
    if window is None and (sinks or positions is not None):
        raise ValueError("sinks and positions need a window")
    mp, batched = None, 0
    if mask is not None:
        batched = int(isinstance(mask, torch.Tensor) and mask.dim() == 3)
        mp = _fits(mask, "mask", dev, (B, T, T) if batched else (T, T), torch.bool)
    given = out, lse, workspace
    out, op = _output(out, "out", dev, q.shape, out_dtype)
    lse, lp = _output(lse, "lse", dev, (B, H, T), torch.float32)
    lib = library()
    need = _tree_workspace(B, H, Hkv, T, d, cap, code, kind)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    _hand_over(stream, dev.index, (given[0], out), (given[1], lse), (given[2], workspace))
    head = (qp, *ptrs, _fits(lens, "lens", dev, (B,), torch.int32),
            None if ntok is None else _fits(ntok, "ntok", dev, (B,), torch.int32), mp, batched)
    tail = (op, lp, workspace.data_ptr(), workspace.numel(), B, H, Hkv, T, d, cap)
    types = (code, kind, _DTYPES[out_dtype], _stream_ptr(stream, dev.index))
    if window is None:
        _run(dev.index, lib.ring_attn_tree_fwd, *head, *tail, *types)
    else:
        pos = None if positions is None else _fits(positions, "positions", dev, (B, T), torch.int32)
        _run(dev.index, lib.ring_attn_tree_window_fwd, *head, pos, *tail, _whole(window, "window"), _whole(sinks, "sinks"), *types)
    return out, lse
