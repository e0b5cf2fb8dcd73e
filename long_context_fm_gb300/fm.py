"""Python binding of ``libfm.so`` (include/fm.h): the same entry points, with
torch tensors and numpy arrays marshalled to pointers.  Every step of the
computation runs inside the library; this module only checks types,
allocates caller-owned buffers with torch where a helper says so, and
forwards.  Importing it fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import numpy as np
import torch

from . import build as _build

# FM_LIBRARY selects another build of the same library (the FM_DEBUG build of
# build.build(debug=True)); by default the in-tree release build.
_LIB_PATH = os.environ.get("FM_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libfm.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with "
                      "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
_lib = ctypes.CDLL(_LIB_PATH)

FM_OK, FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED, FM_ERR_UNREPRESENTABLE = 0, 1, 2, 3
FM_ERR_BAD_BOUNDS, FM_ERR_PLAN_MISMATCH, FM_ERR_WORKSPACE, FM_ERR_CUDA, FM_ERR_TIMEOUT = 4, 5, 6, 7, 8
FM_ERR_DEBUG_CHECK, FM_ERR_LENGTHS, FM_ERR_PAGES = 9, 10, 11
FM_TILE_SKIP, FM_TILE_FULL, FM_TILE_PARTIAL = 0, 1, 2
FM_DT_BF16, FM_DT_F32, FM_DT_E4M3 = 0, 1, 2
FM_FLAG_PRECISE = 1
KERNEL_NAMES = ["classify_minmax", "classify_lists", "fwd", "bwd_pre", "bwd", "bwd_post",
                "classify_order", "fp8_amax", "fp8_convert", "paged_plan", "paged_append", "paged_decode",
                "paged_chunk"]

EXPORTED = ["fm_status_string", "fm_abi_version", "fm_mask_from_rows", "fm_mask_from_row_intervals",
            "fm_plan_bytes", "fm_tile_classify", "fm_fwd_workspace_bytes", "fm_attn_fwd", "fm_bwd_workspace_bytes",
            "fm_attn_bwd", "fm_profile_begin", "fm_profile_end", "fm_selftest_wait_timeout",
            "fm_attn_bwd_noalloc", "fm_step_graph_create", "fm_step_graph_launch", "fm_step_graph_destroy",
            "fm_plan_bytes_rows", "fm_tile_classify_rows", "fm_attn_fwd_rows", "fm_attn_bwd_rows",
            "fm_quantize_fp8", "fm_attn_fwd_fp8", "fm_debug_wait_test", "fm_bounds_compressed_bytes",
            "fm_bounds_compress", "fm_bounds_decompress", "fm_paged_plan_bytes", "fm_paged_plan", "fm_paged_append",
            "fm_attn_paged"]
# Size of the library's built-in backward workspace (FM_NOALLOC_SCRATCH_BYTES in fm.h).
NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


class FmError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = int(code)
        super().__init__(f"{where}: {fm_status_string(code)} ({code})")


class Bounds(ctypes.Structure):
    _fields_ = [("lts", ctypes.c_void_p), ("lte", ctypes.c_void_p), ("uts", ctypes.c_void_p),
                ("ute", ctypes.c_void_p), ("B", ctypes.c_int32), ("Hm", ctypes.c_int32),
                ("N", ctypes.c_int32)]


class StepArgs(ctypes.Structure):
    """fm_step_args of include/fm.h (field order and C layout)."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("dO", ctypes.c_void_p), ("mask", Bounds), ("plan", ctypes.c_void_p),
                ("plan_bytes", ctypes.c_size_t), ("o", ctypes.c_void_p), ("o_dtype", ctypes.c_int),
                ("lse", ctypes.c_void_p), ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p),
                ("dv", ctypes.c_void_p), ("grad_dtype", ctypes.c_int), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t), ("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int),
                ("d", ctypes.c_int), ("scale", ctypes.c_float), ("flags", ctypes.c_int),
                ("dev_status", ctypes.c_void_p)]


class PagedStep(ctypes.Structure):
    """fm_paged_step of include/fm.h: the sizes that a step's plan is built for."""
    _fields_ = [(n, ctypes.c_int32) for n in ("requests", "max_tokens", "max_q", "max_pages", "num_pages", "page_size",
                                              "Hq", "Hkv", "d", "window", "sink")]

    def __init__(self, *sizes, **named):
        for name, x in [*((n, x) for (n, _), x in zip(self._fields_, sizes)), *named.items()]:
            # (ctypes would keep the low 32 bits)
            if not -1 << 31 <= x < 1 << 31:
                raise ValueError(f"{name} = {x} does not fit 32 bits")
        super().__init__(*sizes, **named)


class PagedCache(ctypes.Structure):
    """fm_paged_cache of include/fm.h."""
    _fields_ = ([("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] +
                [(n, ctypes.c_int64) for n in ("k_page", "k_head", "k_tok", "v_page", "v_head", "v_tok")] +
                [("k_descale", ctypes.c_void_p), ("v_descale", ctypes.c_void_p)] +
                [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "Hkv", "d", "dtype")])


class KernelTime(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("ms", ctypes.c_float)]


_P, _I, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_lib.fm_status_string.restype = ctypes.c_char_p
_lib.fm_status_string.argtypes = [_I]
_lib.fm_abi_version.restype = _I
_lib.fm_mask_from_rows.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P, _P]
_lib.fm_mask_from_row_intervals.argtypes = [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P]
_lib.fm_plan_bytes.restype = _SZ
_lib.fm_plan_bytes.argtypes = [_I, _I, _I, _I, _I]
_lib.fm_tile_classify.argtypes = [Bounds, _I, _I, _P, _SZ, _P, _P, _P]
_lib.fm_fwd_workspace_bytes.restype = _SZ
_lib.fm_fwd_workspace_bytes.argtypes = [_I, _I, _I, _I]
_lib.fm_attn_fwd.argtypes = [_P, _P, _P, Bounds, _P, _I, _I, _I, _I, _F, _P, _I, _P, _P, _SZ, _I, _P, _P]
_lib.fm_bwd_workspace_bytes.restype = _SZ
_lib.fm_bwd_workspace_bytes.argtypes = [_I, _I, _I, _I]
_lib.fm_attn_bwd.argtypes = [_P, _P, _P, _P, _I, _P, _P, Bounds, _P, _I, _I, _I, _I, _F, _P, _P, _P,
                             _I, _I, _P, _SZ, _P, _P]
_lib.fm_attn_bwd_noalloc.argtypes = [_P, _P, _P, _P, _I, _P, _P, Bounds, _P, _I, _I, _I, _I, _F, _P,
                                     _P, _P, _I, _I, _P, _P]
_lib.fm_profile_begin.argtypes = []
_lib.fm_profile_end.restype = _I
_lib.fm_profile_end.argtypes = [_P, _I]
_lib.fm_selftest_wait_timeout.argtypes = [ctypes.c_longlong, _P, _P]
_lib.fm_debug_wait_test.argtypes = [ctypes.c_int, ctypes.c_longlong]
_lib.fm_bounds_compressed_bytes.argtypes = [_P, _P, _P, _P, _I, _I, _I]
_lib.fm_bounds_compressed_bytes.restype = _SZ
_lib.fm_bounds_compress.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P, _SZ]
_lib.fm_bounds_decompress.argtypes = [_P, _SZ, Bounds, _P, _P]
_lib.fm_plan_bytes_rows.restype = _SZ
_lib.fm_plan_bytes_rows.argtypes = [_I, _I, _I, _I, _I, _I, _I]
_lib.fm_tile_classify_rows.argtypes = [Bounds, _I, _I, _I, _I, _P, _SZ, _P, _P, _P]
_lib.fm_attn_fwd_rows.argtypes = [_P, _P, _P, Bounds, _P, _I, _I, _I, _I, _I, _I, _F, _P, _I, _P, _P, _SZ, _I,
                                  _P, _P]
_lib.fm_attn_bwd_rows.argtypes = [_P, _P, _P, _P, _I, _P, _P, Bounds, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P,
                                  _P, _I, _I, _P, _SZ, _P, _P]
_lib.fm_quantize_fp8.argtypes = [_P, _I, _I, _I, _I, _I, _P, _P, _P]
_lib.fm_attn_fwd_fp8.argtypes = [_P, _P, _P, _P, Bounds, _P, _I, _I, _I, _I, _F, _P, _I, _P, _P, _P]
_lib.fm_paged_plan_bytes.restype = _SZ
_lib.fm_paged_plan_bytes.argtypes = [ctypes.POINTER(PagedStep)]
_lib.fm_paged_plan.argtypes = [ctypes.POINTER(PagedStep), _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]
_lib.fm_paged_append.argtypes = [_P, ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_int64, ctypes.c_int64, _P, _I,
                                 ctypes.POINTER(PagedCache), _P, _P]
_lib.fm_attn_paged.argtypes = [ctypes.POINTER(PagedStep), _P, ctypes.c_int64, ctypes.c_int64, _I,
                               ctypes.POINTER(PagedCache), _P, _P, _SZ, _F, _P, _I, _P, _P, _P]
_lib.fm_step_graph_create.argtypes = [ctypes.POINTER(StepArgs), ctypes.POINTER(ctypes.c_void_p)]
_lib.fm_step_graph_launch.argtypes = [_P, _P]
_lib.fm_step_graph_destroy.argtypes = [_P]


def _check(code, where):
    if code != FM_OK:
        raise FmError(code, where)


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if hasattr(stream, "cuda_stream"):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _dt(t):
    if t.dtype == torch.bfloat16:
        return FM_DT_BF16
    if t.dtype == torch.float32:
        return FM_DT_F32
    raise TypeError(f"unsupported output dtype {t.dtype}")


def fm_status_string(code: int) -> str:
    return _lib.fm_status_string(int(code)).decode()


def fm_abi_version() -> int:
    return _lib.fm_abi_version()


def make_bounds(lts, lte, uts, ute) -> Bounds:
    """fm_bounds from four device int32 tensors [B, Hm, N]."""
    for n, t in zip(("lts", "lte", "uts", "ute"), (lts, lte, uts, ute)):
        _dev(t, torch.int32, n)
        if t.dim() != 3 or t.shape != lts.shape:
            raise ValueError(f"{n} must be [B, Hm, N] like lts")
    B, Hm, N = lts.shape
    return Bounds(lts.data_ptr(), lte.data_ptr(), uts.data_ptr(), ute.data_ptr(), B, Hm, N)


def fm_mask_from_rows(cs, ce):
    """Host conversion of row intervals (int32 [B, Hm, N]) to column bounds."""
    cs = np.ascontiguousarray(cs, dtype=np.int32)
    ce = np.ascontiguousarray(ce, dtype=np.int32)
    if cs.ndim != 3 or cs.shape != ce.shape:
        raise ValueError("cs and ce must be int32 [B, Hm, N]")
    B, Hm, N = cs.shape
    out = [np.empty_like(cs) for _ in range(4)]
    code = _lib.fm_mask_from_rows(cs.ctypes.data, ce.ctypes.data, B, Hm, N,
                                  *[o.ctypes.data for o in out])
    _check(code, "fm_mask_from_rows")
    return tuple(out)


def fm_mask_from_row_intervals(starts, ends):
    """Host conversion of K inclusive intervals per row (int32 [B, Hm, N, K];
    start > end marks an unused slot) to column bounds [B, Hm, N]."""
    starts = np.ascontiguousarray(starts, dtype=np.int32)
    ends = np.ascontiguousarray(ends, dtype=np.int32)
    if starts.ndim != 4 or starts.shape != ends.shape:
        raise ValueError("starts and ends must be int32 [B, Hm, N, K]")
    B, Hm, N, K = starts.shape
    out = [np.empty((B, Hm, N), np.int32) for _ in range(4)]
    code = _lib.fm_mask_from_row_intervals(starts.ctypes.data, ends.ctypes.data, K, B, Hm, N,
                                           *[o.ctypes.data for o in out])
    _check(code, "fm_mask_from_row_intervals")
    return tuple(out)


def fm_plan_bytes(B, Hm, N, bq=128, bk=128) -> int:
    return int(_lib.fm_plan_bytes(B, Hm, N, bq, bk))


def fm_tile_classify(bounds: Bounds, plan, dev_status, bq=128, bk=128, labels=None, stream=None):
    _dev(plan, torch.uint8, "plan")
    _dev(dev_status, torch.int32, "dev_status")
    if labels is not None:
        _dev(labels, torch.uint8, "labels")
    code = _lib.fm_tile_classify(bounds, bq, bk, _ptr(plan), plan.numel(), _ptr(labels),
                                 _ptr(dev_status), _stream(stream))
    _check(code, "fm_tile_classify")


def fm_fwd_workspace_bytes(B, H, N, d) -> int:
    return int(_lib.fm_fwd_workspace_bytes(B, H, N, d))


def fm_attn_fwd(q, k, v, bounds: Bounds, plan, scale, o, lse, dev_status, ws=None, stream=None,
                flags=0):
    for n, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, torch.bfloat16, n)
    B, H, N, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or o.shape != q.shape:
        raise ValueError("q, k, v, o must share the shape [B, H, N, d]")
    _dev(o, o.dtype, "o")
    _dev(lse, torch.float32, "lse")
    _dev(plan, torch.uint8, "plan")
    _dev(dev_status, torch.int32, "dev_status")
    code = _lib.fm_attn_fwd(_ptr(q), _ptr(k), _ptr(v), bounds, _ptr(plan), B, H, N, d, float(scale),
                            _ptr(o), _dt(o), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(),
                            int(flags), _ptr(dev_status), _stream(stream))
    _check(code, "fm_attn_fwd")


def fm_bwd_workspace_bytes(B, H, N, d) -> int:
    return int(_lib.fm_bwd_workspace_bytes(B, H, N, d))


def fm_attn_bwd(q, k, v, o, lse, dO, bounds: Bounds, plan, scale, dq, dk, dv, ws, dev_status,
                stream=None, flags=0):
    for n, t in (("q", q), ("k", k), ("v", v), ("dO", dO)):
        _dev(t, torch.bfloat16, n)
    B, H, N, d = q.shape
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        _dev(t, t.dtype, n)
        if t.shape != q.shape:
            raise ValueError(f"{n} must have the shape of q")
    if not (dq.dtype == dk.dtype == dv.dtype):
        raise TypeError("dq, dk, dv must share one dtype")
    _dev(lse, torch.float32, "lse")
    _dev(ws, torch.uint8, "ws")
    code = _lib.fm_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _dt(o), _ptr(lse), _ptr(dO), bounds,
                            _ptr(plan), B, H, N, d, float(scale), _ptr(dq), _ptr(dk), _ptr(dv),
                            _dt(dq), int(flags), _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream))
    _check(code, "fm_attn_bwd")


def fm_attn_bwd_noalloc(q, k, v, o, lse, dO, bounds: Bounds, plan, scale, dq, dk, dv, dev_status,
                        stream=None, flags=0):
    """fm_attn_bwd without a caller workspace: for callers that cannot
    allocate device memory; the library's fixed built-in array is used
    instead (see fm.h for the size limit and the rules on overlapping calls)."""
    for n, t in (("q", q), ("k", k), ("v", v), ("dO", dO)):
        _dev(t, torch.bfloat16, n)
    B, H, N, d = q.shape
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        _dev(t, t.dtype, n)
        if t.shape != q.shape:
            raise ValueError(f"{n} must have the shape of q")
    if not (dq.dtype == dk.dtype == dv.dtype):
        raise TypeError("dq, dk, dv must share one dtype")
    _dev(lse, torch.float32, "lse")
    code = _lib.fm_attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _dt(o), _ptr(lse), _ptr(dO),
                                    bounds, _ptr(plan), B, H, N, d, float(scale), _ptr(dq), _ptr(dk),
                                    _ptr(dv), _dt(dq), int(flags), _ptr(dev_status), _stream(stream))
    _check(code, "fm_attn_bwd_noalloc")


def fm_profile_begin():
    _check(_lib.fm_profile_begin(), "fm_profile_begin")


def fm_profile_end(max_entries=4096):
    """[(kernel name, ms)] of every launch since fm_profile_begin."""
    buf = (KernelTime * max_entries)()
    n = _lib.fm_profile_end(buf, max_entries)
    if n < 0:
        raise FmError(FM_ERR_CUDA, "fm_profile_end")
    return [(KERNEL_NAMES[buf[i].kernel], float(buf[i].ms)) for i in range(n)]


def fm_bounds_compress(lts, lte, uts, ute):
    """Host int32 [B, Hm, N] bounds -> the compressed form (numpy uint8)."""
    arr = [np.ascontiguousarray(x, dtype=np.int32) for x in (lts, lte, uts, ute)]
    if not all(a.shape == arr[0].shape and a.ndim == 3 for a in arr):
        raise ValueError("bounds must be int32 [B, Hm, N], all of one shape")
    B, Hm, N = arr[0].shape
    p = [a.ctypes.data_as(ctypes.c_void_p) for a in arr]
    n = _lib.fm_bounds_compressed_bytes(*p, B, Hm, N)
    if n == 0:
        raise FmError(FM_ERR_INVALID_ARG, "fm_bounds_compressed_bytes")
    out = np.zeros(n, np.uint8)
    _check(_lib.fm_bounds_compress(*p, B, Hm, N, out.ctypes.data_as(ctypes.c_void_p), n), "fm_bounds_compress")
    return out


def fm_bounds_decompress(cbounds, bounds: Bounds, dev_status, stream=None):
    """Device uint8 compressed buffer -> the device int32 arrays of `bounds`."""
    _dev(cbounds, torch.uint8, "cbounds")
    _dev(dev_status, torch.int32, "dev_status")
    _check(_lib.fm_bounds_decompress(_ptr(cbounds), cbounds.numel(), bounds, _ptr(dev_status), _stream(stream)),
           "fm_bounds_decompress")


def fm_debug_wait_test(kernel, limit_cycles):
    """Test hook: the next forward (kernel=0), backward (kernel=1) or paged
    attention launch (KERNEL_NAMES' index of "paged_decode" or "paged_chunk") runs
    with every device-side wait bounded by limit_cycles and its first CTA
    withholds one tile load, so it must end with FM_ERR_TIMEOUT in dev_status."""
    _check(_lib.fm_debug_wait_test(int(kernel), int(limit_cycles)), "fm_debug_wait_test")


def fm_selftest_wait_timeout(limit_cycles, dev_status, stream=None):
    _dev(dev_status, torch.int32, "dev_status")
    _check(_lib.fm_selftest_wait_timeout(int(limit_cycles), _ptr(dev_status), _stream(stream)),
           "fm_selftest_wait_timeout")


# ---------------------------------------------------------------------------
# Convenience layer: allocates the caller-owned buffers with torch and calls
# the entry points above.
# ---------------------------------------------------------------------------
def fm_plan_bytes_rows(B, Hm, N, q_row0, Nq, bq=128, bk=128) -> int:
    return int(_lib.fm_plan_bytes_rows(B, Hm, N, q_row0, Nq, bq, bk))


def fm_tile_classify_rows(bounds: Bounds, q_row0, Nq, plan, dev_status, bq=128, bk=128, labels=None, stream=None):
    _dev(plan, torch.uint8, "plan")
    _dev(dev_status, torch.int32, "dev_status")
    if labels is not None:
        _dev(labels, torch.uint8, "labels")
    code = _lib.fm_tile_classify_rows(bounds, int(q_row0), int(Nq), bq, bk, _ptr(plan), plan.numel(),
                                      _ptr(labels), _ptr(dev_status), _stream(stream))
    _check(code, "fm_tile_classify_rows")


def fm_attn_fwd_rows(q, k, v, bounds: Bounds, plan, q_row0, scale, o, lse, dev_status, stream=None, flags=0):
    """Q rows [q_row0, q_row0 + Nq) (q: [B, H, Nq, d]) against all N keys (k, v: [B, H, N, d])."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, torch.bfloat16, n)
    B, H, Nq, d = q.shape
    N = k.shape[2]
    if k.shape != (B, H, N, d) or v.shape != k.shape or o.shape != q.shape:
        raise ValueError("q, o: [B, H, Nq, d]; k, v: [B, H, N, d]")
    _dev(o, o.dtype, "o")
    _dev(lse, torch.float32, "lse")
    _dev(plan, torch.uint8, "plan")
    _dev(dev_status, torch.int32, "dev_status")
    code = _lib.fm_attn_fwd_rows(_ptr(q), _ptr(k), _ptr(v), bounds, _ptr(plan), B, H, N, int(q_row0), Nq, d,
                                 float(scale), _ptr(o), _dt(o), _ptr(lse), None, 0, int(flags), _ptr(dev_status),
                                 _stream(stream))
    _check(code, "fm_attn_fwd_rows")


def fm_attn_bwd_rows(q, k, v, o, lse, dO, bounds: Bounds, plan, q_row0, scale, dq, dk, dv, ws, dev_status,
                     stream=None, flags=0):
    """dQ of the window's rows; dK, dV receive the window's contribution (all N rows)."""
    for n, t in (("q", q), ("k", k), ("v", v), ("dO", dO)):
        _dev(t, torch.bfloat16, n)
    B, H, Nq, d = q.shape
    N = k.shape[2]
    for n, t, shp in (("o", o, q.shape), ("dq", dq, q.shape), ("dO", dO, q.shape), ("dk", dk, k.shape),
                      ("dv", dv, k.shape)):
        _dev(t, t.dtype, n)
        if t.shape != shp:
            raise ValueError(f"{n} has the wrong shape")
    if not (dq.dtype == dk.dtype == dv.dtype):
        raise TypeError("dq, dk, dv must share one dtype")
    _dev(lse, torch.float32, "lse")
    _dev(ws, torch.uint8, "ws")
    code = _lib.fm_attn_bwd_rows(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _dt(o), _ptr(lse), _ptr(dO), bounds,
                                 _ptr(plan), B, H, N, int(q_row0), Nq, d, float(scale), _ptr(dq), _ptr(dk),
                                 _ptr(dv), _dt(dq), int(flags), _ptr(ws), ws.numel(), _ptr(dev_status),
                                 _stream(stream))
    _check(code, "fm_attn_bwd_rows")


def fm_quantize_fp8(x, transpose=False, out=None, descale=None, stream=None):
    """Per-tensor e4m3 codes (uint8) of a bf16 [B, H, N, d] tensor and its
    descale (device float32 [1]); transpose=True gives the [B, H, d, N] layout."""
    _dev(x, torch.bfloat16, "x")
    B, H, N, d = x.shape
    shape = (B, H, d, N) if transpose else (B, H, N, d)
    out = torch.empty(shape, dtype=torch.uint8, device=x.device) if out is None else _dev(out, torch.uint8, "out")
    descale = torch.empty(1, dtype=torch.float32, device=x.device) if descale is None else descale
    _dev(descale, torch.float32, "descale")
    _check(_lib.fm_quantize_fp8(_ptr(x), B, H, N, d, int(bool(transpose)), _ptr(out), _ptr(descale),
                                _stream(stream)), "fm_quantize_fp8")
    return out, descale


def fm_attn_fwd_fp8(q8, k8, vt8, descale, bounds: Bounds, plan, scale, o, lse, dev_status, stream=None):
    """Forward on e4m3 q8, k8 [B, H, N, d] and vt8 [B, H, d, N]; descale: device
    float32 [3] (Q, K, V)."""
    for n, t in (("q8", q8), ("k8", k8), ("vt8", vt8)):
        _dev(t, torch.uint8, n)
    B, H, N, d = q8.shape
    if k8.shape != q8.shape or vt8.shape != (B, H, d, N) or o.shape != q8.shape:
        raise ValueError("q8, k8, o: [B, H, N, d]; vt8: [B, H, d, N]")
    _dev(descale, torch.float32, "descale")
    if descale.numel() != 3:
        raise ValueError("descale holds the Q, K and V descales")
    _dev(o, o.dtype, "o")
    _dev(lse, torch.float32, "lse")
    _dev(plan, torch.uint8, "plan")
    _dev(dev_status, torch.int32, "dev_status")
    code = _lib.fm_attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(descale), bounds, _ptr(plan), B, H, N, d,
                                float(scale), _ptr(o), _dt(o), _ptr(lse), _ptr(dev_status), _stream(stream))
    _check(code, "fm_attn_fwd_fp8")


# The paged calls are made once per layer and decoding step, where the host's time
# counts.  What a program normally calls them with goes through _call; it answers
# None to anything else, which these functions then check in full, and raise or run.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)      # (a torch without CUDA has neither)
_current_device = getattr(torch._C, "_cuda_getDevice", lambda: -1)


class _NoCall:
    """In _call's place where the extension was not built, or against another torch: the functions here then do it all."""
    plan = append = attend = staticmethod(lambda *args: None)


def _load_call():
    """The marshalling in C++ (csrc/fm_call.cpp), bound to the library loaded above."""
    if not _build.call_fits():
        return _NoCall
    try:
        spec = importlib.util.spec_from_loader("_fm_call", importlib.machinery.ExtensionFileLoader("_fm_call", _build.CALL))
        call = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(call)
    except ImportError:
        return _NoCall
    call.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (_lib.fm_paged_plan, _lib.fm_paged_append, _lib.fm_attn_paged)])
    return call


_call = _load_call()


def _on(t, name):
    """Index of the CUDA device of t, which has to be the current one (kernels launch there)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is cuda:{_current_device()}")
    return dev


def _flat(t, dtype, dev, name, shape=None):
    """Address of a contiguous tensor of that type (and shape) on device dev."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError(f"{name} must be a CUDA tensor on cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _rows(t, dev, name, d):
    """bf16 [T, H, d] rows with any token and head strides: (T, H, token stride, head stride)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError(f"{name} must be a CUDA tensor on cuda:{dev}")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"{name} must be [T, H, {d}], got {list(shape)}")
    st, sh, se = t.stride()
    if se != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    T, H, _ = shape
    if T >= 1 << 31:
        raise ValueError(f"{name} has 2^31 - 1 rows at most")
    return T, H, st if T > 1 else d, sh if H > 1 else d     # the stride of a dimension of size one is never used


def paged_cache(k_cache, v_cache, k_descale=None, v_descale=None) -> PagedCache:
    """fm_paged_cache of two page pools [num_pages, Hkv, page_size, d]: bf16, or
    e4m3 (uint8 codes or torch.float8_e4m3fn) with device float32 [1] descales.
    Views with other strides (tokens before heads, K and V interleaved) serve
    as they are, so long as the last dimension is contiguous."""
    dev = _on(k_cache, "k_cache")
    if not isinstance(v_cache, torch.Tensor) or v_cache.get_device() != dev:
        raise TypeError(f"v_cache must be a CUDA tensor on cuda:{dev}")
    dtype, shape = k_cache.dtype, k_cache.shape
    kd = vd = None
    if v_cache.dtype is not dtype or dtype not in (torch.bfloat16, torch.uint8, torch.float8_e4m3fn):
        raise TypeError("caches must both be bfloat16, or both hold e4m3 codes (uint8 or float8_e4m3fn)")
    code = FM_DT_BF16
    if dtype is not torch.bfloat16:
        code = FM_DT_E4M3
        if k_descale is None or v_descale is None:
            raise ValueError("an e4m3 cache needs k_descale and v_descale")
        kd = _flat(k_descale, torch.float32, dev, "k_descale")
        vd = _flat(v_descale, torch.float32, dev, "v_descale")
        if k_descale.numel() != 1 or v_descale.numel() != 1:
            raise ValueError("k_descale and v_descale hold one value each")
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("caches must be [num_pages, Hkv, page_size, d], of one shape")
    kp, kh, kt, ke = k_cache.stride()
    vp, vh, vt, ve = v_cache.stride()
    if ke != 1 or ve != 1:
        raise ValueError("the last dimension of the caches must be contiguous")
    P, Hkv, page, d = shape
    if P == 1 or Hkv == 1 or page == 1:                     # the stride of a dimension of size one is never used
        kp, vp = (kp, vp) if P > 1 else (d, d)
        kh, vh = (kh, vh) if Hkv > 1 else (d, d)
        kt, vt = (kt, vt) if page > 1 else (d, d)
    return PagedCache(k_cache.data_ptr(), v_cache.data_ptr(), kp, kh, kt, vp, vh, vt, kd, vd, P, page, Hkv, d, code)


def fm_paged_plan_bytes(step: PagedStep) -> int:
    return int(_lib.fm_paged_plan_bytes(step))


def fm_paged_plan(step: PagedStep, ctx_lens, q_lens, block_table, seq_lens, cu_q, slots, positions, plan, dev_status,
                  free_pages=None, free_head=None, free_next=None, stream=None):
    """Block tables, slot map, positions and attention plan of a step (see fm.h).
    ctx_lens, q_lens, seq_lens: int32 [requests]; block_table: int32 [requests,
    max_pages]; cu_q: int32 [requests + 1]; slots: int64, positions: int32 or
    None [max_tokens]; free_pages: int32 [n] with free_head and free_next int32 [1]."""
    if stream is None:
        code = _call.plan(ctypes.addressof(step), ctx_lens, q_lens, block_table, seq_lens, cu_q, slots, positions, plan,
                          dev_status, free_pages, free_head, free_next)
        if code == 0:
            return
        if code is not None:
            raise FmError(code, "fm_paged_plan")
    dev, i32 = _on(ctx_lens, "ctx_lens"), torch.int32
    R, T = step.requests, step.max_tokens
    free = head = after = None
    n_free = 0
    if free_pages is not None:
        if free_head is None or free_next is None:
            raise ValueError("free_pages comes with free_head and free_next")
        n_free = free_pages.numel()
        if n_free >= 1 << 31:
            raise ValueError("free_pages has 2^31 - 1 entries at most")
        free = _flat(free_pages, i32, dev, "free_pages", (n_free,))
        head = _flat(free_head, i32, dev, "free_head", (1,))
        after = _flat(free_next, i32, dev, "free_next", (1,))
        free = free or head         # an empty tensor has no address, but an empty list is not "no list"
    code = _lib.fm_paged_plan(
        step, _flat(ctx_lens, i32, dev, "ctx_lens", (R,)), _flat(q_lens, i32, dev, "q_lens", (R,)),
        _flat(block_table, i32, dev, "block_table", (R, step.max_pages)), free, n_free, head, after,
        _flat(seq_lens, i32, dev, "seq_lens", (R,)), _flat(cu_q, i32, dev, "cu_q", (R + 1,)),
        _flat(slots, torch.int64, dev, "slots", (T,)),
        None if positions is None else _flat(positions, i32, dev, "positions", (T,)),
        _flat(plan, torch.uint8, dev, "plan"), plan.numel(), _flat(dev_status, i32, dev, "dev_status", (1,)),
        _raw_stream(dev) if stream is None else _stream(stream))
    if code:
        raise FmError(code, "fm_paged_plan")


def fm_paged_append(k, v, slots, k_cache, v_cache, dev_status, k_descale=None, v_descale=None, stream=None):
    """Rows of k and v (bf16 [T, Hkv, d], any token and head strides) to the cache's
    slots (int64, T of them at least; negative ones are skipped)."""
    if stream is None:
        code = _call.append(k, v, slots, k_cache, v_cache, dev_status, k_descale, v_descale)
        if code == 0:
            return
        if code is not None:
            raise FmError(code, "fm_paged_append")
    cache = paged_cache(k_cache, v_cache, k_descale, v_descale)
    dev = k_cache.get_device()
    T, H, kt, kh = _rows(k, dev, "k", cache.d)
    Tv, Hv, vt, vh = _rows(v, dev, "v", cache.d)
    if T != Tv or H != Hv or H != cache.Hkv:
        raise ValueError("k and v must be [T, Hkv, d] of the cache")
    if slots.dim() != 1 or slots.shape[0] < T:
        raise ValueError("slots must be int64 with an entry for every row of k")
    at, status = _flat(slots, torch.int64, dev, "slots"), _flat(dev_status, torch.int32, dev, "dev_status", (1,))
    if T == 0:
        return
    code = _lib.fm_paged_append(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, at, T, cache, status,
                                _raw_stream(dev) if stream is None else _stream(stream))
    if code:
        raise FmError(code, "fm_paged_append")


def fm_attn_paged(step: PagedStep, q, k_cache, v_cache, block_table, plan, scale, o, lse, dev_status, k_descale=None,
                  v_descale=None, stream=None):
    """Attention of a step's new tokens (q: bf16 [rows, Hq, d]) over the paged cache;
    o: bf16 or fp32 [rows, Hq, d], lse: fp32 [rows, Hq] (see fm.h)."""
    dev = _on(q, "q")
    _flat(o, o.dtype, dev, "o", q.shape)
    _flat(lse, torch.float32, dev, "lse", q.shape[:2])
    _attn_paged(step, q, k_cache, v_cache, block_table, plan, scale, o, lse, dev_status, k_descale, v_descale, stream)


def _attn_paged(step, q, k_cache, v_cache, block_table, plan, scale, o, lse, dev_status, k_descale, v_descale, stream):
    """fm_attn_paged with o and lse known to fit q."""
    cache = paged_cache(k_cache, v_cache, k_descale, v_descale)
    dev = k_cache.get_device()
    T, H, qt, qh = _rows(q, dev, "q", step.d)
    if H != step.Hq:
        raise ValueError("q must be [rows, Hq, d] of the step")
    table = _flat(block_table, torch.int32, dev, "block_table", (step.requests, step.max_pages))
    buf, status = _flat(plan, torch.uint8, dev, "plan"), _flat(dev_status, torch.int32, dev, "dev_status", (1,))
    if T == 0:
        return
    code = _lib.fm_attn_paged(step, q.data_ptr(), qt, qh, T, cache, table, buf, plan.numel(), scale, o.data_ptr(), _dt(o),
                              lse.data_ptr(), status, _raw_stream(dev) if stream is None else _stream(stream))
    if code:
        raise FmError(code, "fm_attn_paged")


def fm_step_graph_create(q, k, v, dO, bounds: Bounds, plan, scale, o, lse, dev_status, dq=None, dk=None,
                         dv=None, ws=None, flags=0):
    """Capture classify + forward (+ backward when dO is given) for these
    buffers; returns the opaque handle (an int)."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, torch.bfloat16, n)
    B, H, N, d = q.shape
    a = StepArgs()
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    a.dO = None if dO is None else _dev(dO, torch.bfloat16, "dO").data_ptr()
    a.mask = bounds
    a.plan, a.plan_bytes = _dev(plan, torch.uint8, "plan").data_ptr(), plan.numel()
    a.o, a.o_dtype = _dev(o, o.dtype, "o").data_ptr(), _dt(o)
    a.lse = _dev(lse, torch.float32, "lse").data_ptr()
    if dO is not None:
        if not (dq.dtype == dk.dtype == dv.dtype):
            raise TypeError("dq, dk, dv must share one dtype")
        a.dq, a.dk, a.dv = (_dev(t, t.dtype, n).data_ptr() for n, t in (("dq", dq), ("dk", dk), ("dv", dv)))
        a.grad_dtype = _dt(dq)
        a.ws, a.ws_bytes = _dev(ws, torch.uint8, "ws").data_ptr(), ws.numel()
    a.B, a.H, a.N, a.d = B, H, N, d
    a.scale, a.flags = float(scale), int(flags)
    a.dev_status = _dev(dev_status, torch.int32, "dev_status").data_ptr()
    h = ctypes.c_void_p()
    _check(_lib.fm_step_graph_create(ctypes.byref(a), ctypes.byref(h)), "fm_step_graph_create")
    return h.value


def fm_step_graph_launch(graph, stream=None):
    _check(_lib.fm_step_graph_launch(ctypes.c_void_p(graph), _stream(stream)), "fm_step_graph_launch")


def fm_step_graph_destroy(graph):
    _check(_lib.fm_step_graph_destroy(ctypes.c_void_p(graph)), "fm_step_graph_destroy")


class StepGraph:
    """One captured step over fixed buffers (keeps them referenced while the
    graph lives); refill the inputs in place and call launch()."""

    def __init__(self, q, k, v, dO, att: "MaskedAttention", scale, o, lse, dq=None, dk=None, dv=None, ws=None,
                 flags=0):
        self._keep = (q, k, v, dO, att, o, lse, dq, dk, dv, ws)
        self.handle = fm_step_graph_create(q, k, v, dO, att.bounds, att.plan, scale, o, lse, att.status,
                                           dq, dk, dv, ws, flags)

    def launch(self, stream=None):
        fm_step_graph_launch(self.handle, stream)

    def close(self):
        if self.handle is not None:
            fm_step_graph_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MaskedAttention:
    """Holds the device bounds, plan and status word of one mask."""

    def __init__(self, lts, lte, uts, ute, device="cuda", stream=None):
        t = [torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(device) for x in
             (lts, lte, uts, ute)]
        self.lts, self.lte, self.uts, self.ute = t
        self.bounds = make_bounds(*t)
        self.B, self.Hm, self.N = self.lts.shape
        self.plan = torch.empty(fm_plan_bytes(self.B, self.Hm, self.N), dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.stream = stream
        fm_tile_classify(self.bounds, self.plan, self.status, stream=stream)

    def labels(self, bq=128, bk=128):
        """Labels uint8 [B, Hm, n_q, n_k] (a separate plan of tile size bq x bk)."""
        n_q, n_k = -(-self.N // bq), -(-self.N // bk)
        out = torch.empty((self.B, self.Hm, n_q, n_k), dtype=torch.uint8, device=self.plan.device)
        plan = torch.empty(fm_plan_bytes(self.B, self.Hm, self.N, bq, bk), dtype=torch.uint8,
                           device=self.plan.device)
        fm_tile_classify(self.bounds, plan, self.status, bq, bk, labels=out, stream=self.stream)
        return out

    def forward(self, q, k, v, scale=None, o_dtype=torch.bfloat16, flags=0):
        B, H, N, d = q.shape
        scale = 1.0 / d ** 0.5 if scale is None else scale
        o = torch.empty(q.shape, dtype=o_dtype, device=q.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        fm_attn_fwd(q, k, v, self.bounds, self.plan, scale, o, lse, self.status, stream=self.stream,
                    flags=flags)
        return o, lse

    def backward(self, q, k, v, o, lse, dO, scale=None, grad_dtype=torch.float32, ws=None, flags=0):
        B, H, N, d = q.shape
        scale = 1.0 / d ** 0.5 if scale is None else scale
        if ws is None:
            ws = torch.empty(fm_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)
        dq, dk, dv = (torch.empty(q.shape, dtype=grad_dtype, device=q.device) for _ in range(3))
        fm_attn_bwd(q, k, v, o, lse, dO, self.bounds, self.plan, scale, dq, dk, dv, ws, self.status,
                    stream=self.stream, flags=flags)
        return dq, dk, dv

    def check_status(self):
        code = int(self.status.item())
        if code != 0:
            raise FmError(code, "device")


class PagedAttention:
    """A batch of requests over a paged cache: the step's sizes, plan, slot map and
    status word.  Per step one plan() (lengths and block table on the device), then
    per layer an append() and an attend() with that layer's cache.  The plan's buffer
    takes 45 MB at d = 128 (23 at 64), 5 and 3 if no request can have more than
    32 rows (max_q * Hq / Hkv)."""

    def __init__(self, requests, Hq, Hkv, d, page_size, num_pages, max_pages, max_tokens, max_q, window=0, sink=0,
                 device="cuda"):
        self.step = PagedStep(requests, max_tokens, max_q, max_pages, num_pages, page_size, Hq, Hkv, d, window, sink)
        n = fm_paged_plan_bytes(self.step)
        if n == 0:
            raise ValueError("sizes of the step outside what fm.h allows")
        if _call is _NoCall:
            warnings.warn("the paged calls go through ctypes, about 10 us more each: _lib/_fm_call.so is missing or does not fit this torch "
                          "(build it with `python -c 'import __graft_entry__ as g; g.build()'`)", RuntimeWarning, stacklevel=2)
        i32 = dict(dtype=torch.int32, device=device)
        self.plan_buffer = torch.empty(n, dtype=torch.uint8, device=device)
        self.cu_q = torch.empty(requests + 1, **i32)
        self.seq_lens = torch.empty(requests, **i32)
        self.slots = torch.empty(max_tokens, dtype=torch.int64, device=device)
        self.positions = torch.empty(max_tokens, **i32)
        self.free_next = torch.empty(1, **i32)
        self.status = torch.zeros(1, **i32)

    def plan(self, ctx_lens, q_lens, block_table, free_pages=None, free_head=None, in_place=False):
        """Plans a step; with in_place, ctx_lens and free_head are advanced too
        (a captured step can then be replayed)."""
        fm_paged_plan(self.step, ctx_lens, q_lens, block_table, ctx_lens if in_place else self.seq_lens, self.cu_q,
                      self.slots, self.positions, self.plan_buffer, self.status, free_pages, free_head,
                      None if free_pages is None else free_head if in_place else self.free_next)

    def append(self, k, v, k_cache, v_cache, k_descale=None, v_descale=None):
        fm_paged_append(k, v, self.slots, k_cache, v_cache, self.status, k_descale, v_descale)

    def attend(self, q, k_cache, v_cache, block_table, scale=None, o_dtype=torch.bfloat16, k_descale=None,
               v_descale=None):
        """(o, lse) of q's rows, newly allocated.  Rows at or behind cu_q[requests] (a padded
        batch), and all of them after a plan that failed, hold what that memory held before."""
        scale = 1.0 / self.step.d ** 0.5 if scale is None else scale
        if o_dtype is torch.bfloat16 or o_dtype is torch.float32:
            r = _call.attend(ctypes.addressof(self.step), q, k_cache, v_cache, block_table, self.plan_buffer, scale,
                             o_dtype is torch.float32, self.status, k_descale, v_descale)
            if type(r) is tuple:
                return r
            if r is not None:
                raise FmError(r, "fm_attn_paged")
        shape = q.shape
        o = torch.empty(shape, dtype=o_dtype, device=q.device)
        lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device)
        _attn_paged(self.step, q, k_cache, v_cache, block_table, self.plan_buffer, scale, o, lse, self.status, k_descale,
                    v_descale, None)
        return o, lse

    def check_status(self):
        code = int(self.status.item())
        if code != 0:
            raise FmError(code, "device")
