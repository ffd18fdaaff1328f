"""Thin ctypes binding of liblf_attn.so (include/lf_attn.h, lf_proj.h,
lf_paged.h).

Argument marshalling only: torch tensors supply device memory and the CUDA
stream; every step of the attention runs in the library's kernels.  The
functions carry the C names.  There is no fallback of any kind: if the
library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblf_attn.so")

LF_OK, LF_ERR_INVALID, LF_ERR_UNSUPPORTED, LF_ERR_CUDA, LF_ERR_DEVICE_TIMEOUT, LF_ERR_DEVICE_INPUT = range(6)
LF_F32, LF_BF16, LF_F16 = 0, 1, 2
LF_KERNEL_AUTO, LF_KERNEL_SIMT, LF_KERNEL_TC = 0, 1, 2
ERROR_NAMES = {1: "LF_ERR_INVALID", 2: "LF_ERR_UNSUPPORTED", 3: "LF_ERR_CUDA",
               4: "LF_ERR_DEVICE_TIMEOUT", 5: "LF_ERR_DEVICE_INPUT"}

# every symbol include/lf_attn.h declares
EXPORTS = ["lf_attn_version", "lf_attn_workspace_size", "lf_attn_fwd", "lf_attn_bwd",
           "lf_attn_count_pairs", "lf_attn_mask_dump", "lf_attn_status",
           "lf_attn_set_timing_events", "lf_attn_launch_count", "lf_attn_last_error",
           "lf_attn_fwd_noalloc", "lf_attn_status_noalloc", "lf_attn_decode",
           "lf_attn_set_test_hooks", "lf_attn_cross_workspace_size", "lf_attn_cross_fwd"]
# every symbol include/lf_proj.h declares
PROJ_EXPORTS = ["lf_proj_workspace_size", "lf_proj_in", "lf_proj_out", "lf_proj_set_timing_events"]
# every symbol include/lf_paged.h declares
PAGED_EXPORTS = ["lf_rope_fwd", "lf_rope_bwd", "lf_paged_workspace_size", "lf_cache_append", "lf_paged_decode"]
LF_STATIC_WORKSPACE_BYTES = 16 << 20


class LfError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("%s: %s" % (ERROR_NAMES.get(code, str(code)), msg))
        self.code = code


class lf_attn_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("n", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("window", ctypes.c_int),
                ("dilation", ctypes.POINTER(ctypes.c_int32)), ("causal", ctypes.c_int),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int), ("max_global", ctypes.c_int),
                ("kernel", ctypes.c_int)]


class lf_cross_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("Lq", ctypes.c_int), ("Lk", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class lf_proj_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("n", ctypes.c_int), ("H", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int)]


class lf_rope_params(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("n_axes", ctypes.c_int),
                ("pair_axis", ctypes.POINTER(ctypes.c_int32)), ("freqs", ctypes.POINTER(ctypes.c_double)),
                ("base", ctypes.c_double)]


class lf_rope_tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("x_stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3)]


class lf_paged_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("Hkv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("window", ctypes.c_int), ("dilation", ctypes.POINTER(ctypes.c_int32)), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int), ("prefix_len", ctypes.c_int)]


_lib = None


def load(path: str = LIB_PATH):
    """Load the library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError("liblf_attn.so is not built (python -m sparse_sliding_window_b200.build)")
        lib = ctypes.CDLL(path)
        P, sz, i32, vp = ctypes.POINTER(lf_attn_params), ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p
        lib.lf_attn_version.restype = i32
        lib.lf_attn_workspace_size.argtypes = [P, i32]
        lib.lf_attn_workspace_size.restype = sz
        lib.lf_attn_fwd.argtypes = [P] + [vp] * 6 + [vp, vp, vp, vp, sz, vp]
        lib.lf_attn_bwd.argtypes = [P] + [vp] * 6 + [vp, vp, vp, vp] + [vp] * 6 + [vp, sz, vp]
        lib.lf_attn_count_pairs.argtypes = [P, vp, vp, vp, sz, vp]
        lib.lf_attn_mask_dump.argtypes = [P, vp, vp, vp, sz, vp]
        lib.lf_attn_status.argtypes = [vp, vp]
        lib.lf_attn_set_timing_events.argtypes = [vp, vp]
        lib.lf_attn_last_error.restype = ctypes.c_char_p
        lib.lf_attn_launch_count.restype = ctypes.c_uint64
        lib.lf_attn_fwd_noalloc.argtypes = [P] + [vp] * 6 + [vp, vp, vp, vp]
        lib.lf_attn_decode.argtypes = [P, vp, vp, vp, vp, vp, vp, vp]
        lib.lf_attn_decode.restype = i32
        lib.lf_attn_fwd_noalloc.restype = i32
        lib.lf_attn_set_test_hooks.argtypes = [ctypes.c_uint32, i32]
        lib.lf_attn_set_test_hooks.restype = i32
        lib.lf_attn_status_noalloc.argtypes = [vp]
        lib.lf_attn_status_noalloc.restype = i32
        for f in ("fwd", "bwd", "count_pairs", "mask_dump", "status", "set_timing_events"):
            getattr(lib, "lf_attn_" + f).restype = i32
        CP = ctypes.POINTER(lf_cross_params)
        lib.lf_attn_cross_workspace_size.argtypes = [CP]
        lib.lf_attn_cross_workspace_size.restype = sz
        lib.lf_attn_cross_fwd.argtypes = [CP, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.lf_attn_cross_fwd.restype = i32
        PP = ctypes.POINTER(lf_proj_params)
        lib.lf_proj_workspace_size.argtypes = [PP, i32]
        lib.lf_proj_workspace_size.restype = sz
        lib.lf_proj_in.argtypes = [PP, i32, vp, vp, vp, ctypes.POINTER(vp), vp, i32, i32, vp, sz, vp]
        lib.lf_proj_in.restype = i32
        lib.lf_proj_out.argtypes = [PP, vp, vp, vp, vp, vp, sz, vp]
        lib.lf_proj_out.restype = i32
        lib.lf_proj_set_timing_events.argtypes = [vp, vp]
        lib.lf_proj_set_timing_events.restype = i32
        RP, GP = ctypes.POINTER(lf_rope_params), ctypes.POINTER(lf_paged_params)
        for f in (lib.lf_rope_fwd, lib.lf_rope_bwd):
            f.argtypes = [RP, i32, i32, i32, i32, ctypes.POINTER(lf_rope_tensor), vp, vp]
            f.restype = i32
        lib.lf_paged_workspace_size.argtypes = [GP]
        lib.lf_paged_workspace_size.restype = sz
        lib.lf_cache_append.argtypes = [GP, RP, i32] + [vp] * 3 + [ctypes.POINTER(ctypes.c_int64)] + [vp] * 8 + [sz, vp]
        lib.lf_cache_append.restype = i32
        lib.lf_paged_decode.argtypes = [GP, vp, ctypes.POINTER(ctypes.c_int64)] + [vp] * 8 + [sz, vp]
        lib.lf_paged_decode.restype = i32
        _lib = lib
    return _lib


def _check(code: int):
    if code != LF_OK:
        raise LfError(code, load().lf_attn_last_error().decode())


_DT = {"f32": LF_F32, "bf16": LF_BF16, "f16": LF_F16}


def dtype_code(t) -> int:
    import torch
    return {torch.float32: LF_F32, torch.bfloat16: LF_BF16, torch.float16: LF_F16}[t.dtype]


def make_params(B: int, H: int, n: int, window: int, dilation: Optional[Sequence[int]] = None,
                causal: bool = False, scale: float = 0.0, dtype: int = LF_BF16,
                max_global: int = -1, kernel: int = LF_KERNEL_AUTO, head_dim: int = 64):
    """Build an lf_attn_params (the dilation array is kept alive on it)."""
    p = lf_attn_params()
    p.B, p.H, p.n, p.head_dim, p.window = B, H, n, head_dim, window
    if dilation is not None:
        arr = (ctypes.c_int32 * H)(*[int(x) for x in dilation])
        p._dil_keep = arr  # type: ignore[attr-defined]
        p.dilation = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
    p.causal, p.scale, p.dtype, p.max_global, p.kernel = int(causal), float(scale), dtype, max_global, kernel
    return p


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def lf_attn_workspace_size(p, for_bwd: bool = False) -> int:
    return int(load().lf_attn_workspace_size(ctypes.byref(p), int(for_bwd)))


def workspace(p, for_bwd: bool = False, device="cuda"):
    """Allocate a workspace for params p (a uint8 torch tensor, 256-B aligned)."""
    import torch
    nbytes = lf_attn_workspace_size(p, for_bwd)
    if nbytes == 0:
        _check(LF_ERR_INVALID)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)  # status words start at zero


def lf_attn_fwd(p, q_s, k_s, v_s, q_g, k_g, v_g, mask, o, lse, ws, stream=None):
    _check(load().lf_attn_fwd(ctypes.byref(p), _ptr(q_s), _ptr(k_s), _ptr(v_s), _ptr(q_g),
                              _ptr(k_g), _ptr(v_g), _ptr(mask), _ptr(o), _ptr(lse), _ptr(ws),
                              ws.numel(), _stream(stream)))


def lf_attn_fwd_noalloc(p, q_s, k_s, v_s, q_g, k_g, v_g, mask, o, lse, stream=None):
    """Forward without a workspace argument (library-internal static scratch);
    for callers that cannot allocate device memory."""
    _check(load().lf_attn_fwd_noalloc(ctypes.byref(p), _ptr(q_s), _ptr(k_s), _ptr(v_s), _ptr(q_g),
                                      _ptr(k_g), _ptr(v_g), _ptr(mask), _ptr(o), _ptr(lse),
                                      _stream(stream)))


def lf_attn_set_test_hooks(wait_limit_us: int = 0, skip_kv_tile: int = 0):
    """Test hook of the device-side failure detection (see lf_attn.h)."""
    _check(load().lf_attn_set_test_hooks(int(wait_limit_us), int(skip_kv_tile)))


def lf_attn_status_noalloc(stream=None):
    """Read and clear the device status word of lf_attn_fwd_noalloc's static
    scratch on the current device (raises LfError on a device-side error)."""
    _check(load().lf_attn_status_noalloc(_stream(stream)))


def lf_attn_decode(p, q, k_cache, v_cache, lengths, o, lse=None, stream=None):
    """Causal-window decode step: q [B,H,64] against the caches [B,H,n,64]
    whose row lengths[b]-1 holds the new token; writes o [B,H,64] (+ lse)."""
    _check(load().lf_attn_decode(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(lengths), _ptr(o), _ptr(lse), _stream(stream)))


def lf_attn_bwd(p, q_s, k_s, v_s, q_g, k_g, v_g, mask, o, lse, d_o, dq_s, dk_s, dv_s, dq_g, dk_g,
                dv_g, ws, stream=None):
    _check(load().lf_attn_bwd(ctypes.byref(p), _ptr(q_s), _ptr(k_s), _ptr(v_s), _ptr(q_g),
                              _ptr(k_g), _ptr(v_g), _ptr(mask), _ptr(o), _ptr(lse), _ptr(d_o),
                              _ptr(dq_s), _ptr(dk_s), _ptr(dv_s), _ptr(dq_g), _ptr(dk_g),
                              _ptr(dv_g), _ptr(ws), ws.numel(), _stream(stream)))


def lf_attn_count_pairs(p, mask, counts, ws, stream=None):
    _check(load().lf_attn_count_pairs(ctypes.byref(p), _ptr(mask), _ptr(counts), _ptr(ws),
                                      ws.numel(), _stream(stream)))


def lf_attn_mask_dump(p, mask, out, ws, stream=None):
    _check(load().lf_attn_mask_dump(ctypes.byref(p), _ptr(mask), _ptr(out), _ptr(ws), ws.numel(),
                                    _stream(stream)))


def lf_attn_status(ws, stream=None):
    _check(load().lf_attn_status(_ptr(ws), _stream(stream)))


def lf_attn_set_timing_events(ev_start, ev_stop):
    a = None if ev_start is None else ev_start.cuda_event
    b = None if ev_stop is None else ev_stop.cuda_event
    _check(load().lf_attn_set_timing_events(a, b))


def lf_attn_launch_count() -> int:
    return int(load().lf_attn_launch_count())


def make_cross_params(B: int, H: int, Lq: int, Lk: int, dtype: int = LF_BF16, scale: float = 0.0,
                      head_dim: int = 64):
    p = lf_cross_params()
    p.B, p.H, p.Lq, p.Lk, p.head_dim, p.scale, p.dtype = B, H, Lq, Lk, head_dim, float(scale), dtype
    return p


def lf_attn_cross_workspace_size(p) -> int:
    return int(load().lf_attn_cross_workspace_size(ctypes.byref(p)))


def cross_workspace(p, device="cuda"):
    import torch
    nbytes = lf_attn_cross_workspace_size(p)
    if nbytes == 0:
        _check(LF_ERR_INVALID)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)  # status words start at zero


def lf_attn_cross_fwd(p, q, k, v, key_mask, o, lse, ws, stream=None):
    """LED decoder cross-attention: q [B,H,Lq,64] against k, v [B,H,Lk,64]
    (keys with key_mask != 0; key_mask None: all) -> o [B,H,Lq,64], lse."""
    _check(load().lf_attn_cross_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(key_mask), _ptr(o),
                                    _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def make_proj_params(B: int, n: int, H: int, dtype: int = LF_BF16, head_dim: int = 64):
    p = lf_proj_params()
    p.B, p.n, p.H, p.head_dim, p.dtype = B, n, H, head_dim, dtype
    return p


def lf_proj_workspace_size(p, max_rows: int = 0) -> int:
    return int(load().lf_proj_workspace_size(ctypes.byref(p), int(max_rows)))


def proj_workspace(p, max_rows: int = 0, device="cuda"):
    """Allocate a projection workspace (a uint8 torch tensor, 256-B aligned)."""
    import torch
    nbytes = lf_proj_workspace_size(p, max_rows)
    if nbytes == 0:
        _check(LF_ERR_INVALID)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)  # status words start at zero


def lf_proj_in(p, x, w_in, b_in, outs, ws, rows_mask=None, rows_code: int = 2, max_rows: int = 0,
               stream=None):
    """Input projections: outs[k][b,h,t,:] = x[b,t,:] . w_in[k*D + h*64 + :, :] + b_in[...]
    (only rows with rows_mask == rows_code when a mask is given)."""
    arr = (ctypes.c_void_p * len(outs))(*[o.data_ptr() for o in outs])
    _check(load().lf_proj_in(ctypes.byref(p), len(outs), _ptr(x), _ptr(w_in), _ptr(b_in), arr,
                             _ptr(rows_mask), int(rows_code), int(max_rows), _ptr(ws), ws.numel(),
                             _stream(stream)))


def lf_proj_out(p, o, w_out, b_out, y, ws, stream=None):
    """Output projection: y[b,t,:] = concat_h o[b,h,t,:] . w_out^T + b_out."""
    _check(load().lf_proj_out(ctypes.byref(p), _ptr(o), _ptr(w_out), _ptr(b_out), _ptr(y), _ptr(ws),
                              ws.numel(), _stream(stream)))


def lf_proj_set_timing_events(ev_start, ev_stop):
    a = None if ev_start is None else ev_start.cuda_event
    b = None if ev_stop is None else ev_stop.cuda_event
    _check(load().lf_proj_set_timing_events(a, b))


# ------------------------------------- rotation, paged cache, paged decode --
#
# These calls check shapes, dtypes and devices: the library sees bare
# pointers, and a wrong shape would send a kernel out of its buffers.  The
# checks are native (csrc/lf_bind.cpp): from Python they would take longer than
# a decode step.

BIND_PATH = os.path.join(HERE, "_lf_bind.so")
_bind = None


def _load_bind():
    global _bind
    if _bind is None:
        load()
        if not os.path.exists(BIND_PATH):
            raise RuntimeError("_lf_bind.so is not built (python -m sparse_sliding_window_b200.build)")
        import importlib.util
        import torch  # noqa: F401  the module uses its libraries
        spec = importlib.util.spec_from_file_location("_lf_bind", BIND_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _bind = module
    return _bind


def _bad(msg: str):
    raise LfError(LF_ERR_INVALID, msg)


def _done(result):
    """None, an LF_* code of the library, or the text of a refused argument."""
    if result is not None:
        _bad(result) if isinstance(result, str) else _check(result)


def _on(stream):
    return None if stream is None else (stream.device_index, stream.cuda_stream)


def make_rope_params(rot_dim: int = 64, interleaved: bool = False, n_axes: int = 1,
                     pair_axis: Optional[Sequence[int]] = None, freqs: Optional[Sequence[float]] = None,
                     base: float = 10000.0):
    """Build an lf_rope_params (the arrays are kept alive on it)."""
    r = lf_rope_params()
    r.rot_dim, r.interleaved, r.n_axes, r.base = rot_dim, int(interleaved), n_axes, float(base)
    if freqs is None and 2 <= rot_dim <= 64 and rot_dim % 2 == 0 and 0 < base < math.inf:
        # what the library would compute at every call (or refuse, naming the base)
        logs = [-2.0 * p / rot_dim * math.log10(base) for p in range(rot_dim // 2)]
        if max(logs) <= 6:
            freqs = [math.pow(base, -2.0 * p / rot_dim) for p in range(rot_dim // 2)]
    for field, values, kind in (("pair_axis", pair_axis, ctypes.c_int32), ("freqs", freqs, ctypes.c_double)):
        if values is not None:
            if len(values) != (rot_dim or 64) // 2:
                _bad("%s has %d entries for %d pairs" % (field, len(values), (rot_dim or 64) // 2))
            arr = (kind * len(values))(*values)
            setattr(r, "_%s_keep" % field, arr)
            setattr(r, field, ctypes.cast(arr, ctypes.POINTER(kind)))
    return r


def lf_rope_fwd(r, xs, outs, positions=None, stream=None):
    """Rotate every x [B, heads, n, 64] of the list xs into its out (which may
    be x) by positions int32 [n_axes, B, n] (None: the token index)."""
    _done((_bind or _load_bind()).rope(False, r, xs, outs, positions, _on(stream)))


def lf_rope_bwd(r, grads, outs, positions=None, stream=None):
    """The backward of lf_rope_fwd: gradients of its outputs -> of its inputs."""
    _done((_bind or _load_bind()).rope(True, r, grads, outs, positions, _on(stream)))


def make_paged_params(B: int, H: int, Hkv: int, page_size: int, num_pages: int, max_pages: int, window: int = -1,
                      dilation: Optional[Sequence[int]] = None, scale: float = 0.0, dtype: int = LF_BF16,
                      prefix_len: int = 0, head_dim: int = 64):
    """Build an lf_paged_params (the dilation array is kept alive on it)."""
    p = lf_paged_params()
    p.B, p.H, p.Hkv, p.head_dim, p.page_size = B, H, Hkv, head_dim, page_size
    p.num_pages, p.max_pages, p.window, p.scale, p.dtype, p.prefix_len = (num_pages, max_pages, window, float(scale),
                                                                          dtype, prefix_len)
    if dilation is not None:
        if len(dilation) != Hkv:
            _bad("dilation has %d entries for %d key/value heads" % (len(dilation), Hkv))
        arr = (ctypes.c_int32 * Hkv)(*[int(x) for x in dilation])
        p._dil_keep = arr  # type: ignore[attr-defined]
        p.dilation = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
    return p


def lf_paged_workspace_size(p) -> int:
    return int(load().lf_paged_workspace_size(ctypes.byref(p)))


def paged_workspace(p, device="cuda"):
    """Allocate a workspace for lf_cache_append and lf_paged_decode."""
    import torch
    nbytes = lf_paged_workspace_size(p)
    if nbytes == 0:
        _check(LF_ERR_INVALID)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)  # status words start at zero


def lf_cache_append(p, rope, q, k, v, lengths, block_table, q_out, k_pages, v_pages, ws, cu_new=None,
                    positions=None, stream=None):
    """Append new tokens to the paged cache: q [T,H,64] (or None), k, v
    [T,Hkv,64], any strides (a projection's [1,H,T,64] is x[0].transpose(0, 1));
    K rotated by rope (None: not) and V go to the pages, rotated Q to q_out."""
    _done((_bind or _load_bind()).append(p, rope, q, k, v, lengths, block_table, q_out, k_pages, v_pages, ws, cu_new,
                                         positions, _on(stream)))


def lf_paged_decode(p, q, k_pages, v_pages, block_table, lengths, o, lse, ws, prefix_table=None, stream=None):
    """Decode step over the paged cache: q [B,H,64] (any strides) against the
    window of each sequence's own rows and the shared prefix; writes o
    [B,H,64] and lse [B,H] (or None)."""
    _done((_bind or _load_bind()).decode(p, q, k_pages, v_pages, block_table, lengths, o, lse, ws, prefix_table,
                                         _on(stream)))


# ------------------------------------------------------------ convenience --

class LongformerAttention:
    """Holds params + workspace for one problem shape; call fwd / bwd with
    torch tensors [B, H, n, 64] on the GPU and an int32 mask [B, n]."""

    def __init__(self, B, H, n, window, dilation=None, causal=False, scale=0.0, dtype="bf16",
                 max_global=-1, kernel=LF_KERNEL_AUTO, device="cuda"):
        self.p = make_params(B, H, n, window, dilation, causal, scale, _DT[dtype], max_global, kernel)
        self.ws_f = workspace(self.p, False, device)
        self.ws_b = None
        self.device = device

    def fwd(self, q_s, k_s, v_s, q_g, k_g, v_g, mask, o=None, lse=None, stream=None, need_lse=True):
        import torch
        if o is None:
            o = torch.empty_like(q_s)
        if lse is None and need_lse:
            lse = torch.empty(q_s.shape[:3], dtype=torch.float32, device=q_s.device)
        lf_attn_fwd(self.p, q_s, k_s, v_s, q_g, k_g, v_g, mask, o, lse, self.ws_f, stream)
        return o, lse

    def bwd(self, q_s, k_s, v_s, q_g, k_g, v_g, mask, o, lse, d_o, stream=None):
        import torch
        if self.ws_b is None:
            self.ws_b = workspace(self.p, True, self.device)
        grads = [torch.empty_like(q_s) for _ in range(6)]
        lf_attn_bwd(self.p, q_s, k_s, v_s, q_g, k_g, v_g, mask, o, lse, d_o, *grads, self.ws_b, stream)
        return tuple(grads)

    def count_pairs(self, mask, stream=None):
        import torch
        c = torch.empty((self.p.B, self.p.H), dtype=torch.int64, device=mask.device)
        lf_attn_count_pairs(self.p, mask, c, self.ws_f, stream)
        return c

    def mask_dump(self, mask, stream=None):
        import torch
        out = torch.empty((self.p.B, self.p.H, self.p.n, self.p.n), dtype=torch.uint8, device=mask.device)
        lf_attn_mask_dump(self.p, mask, out, self.ws_f, stream)
        return out

    def status(self, bwd=False, stream=None):
        lf_attn_status(self.ws_b if bwd else self.ws_f, stream)
