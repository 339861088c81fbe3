"""Thin Python binding of ``libawq_mi355x.so`` (ctypes).

Argument marshalling only: every step of the path runs in the HIP library.
Torch supplies device memory and the current stream.  Importing this module
loads the library and fails loudly if it has not been built; there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import NamedTuple

import numpy as np
import torch

__all__ = [
    "AwqError",
    "AwqNonFinite",
    "lib_path",
    "load",
    "version",
    "act_stats",
    "weight_stats",
    "search_workspace_size",
    "search_workspace_min_size",
    "search_layer",
    "SearchResult",
    "clip_workspace_size",
    "clip_search",
    "ClipResult",
    "pack",
    "w4a16_gemm",
    "w4a16_workspace_size",
    "w4a16_gemm_noalloc",
    "KvCache",
    "kv_page_size",
    "kv_cache",
    "KvStep",
    "kv_tables",
    "kv_append",
    "kv_rotation_table",
    "kv_append_rotated",
    "kv_read",
    "kv_attention_workspace_size",
    "kv_attention",
    "AWQ_F32",
    "AWQ_BF16",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIBNAME = "libawq_mi355x.so"

AWQ_F32 = 0
AWQ_BF16 = 1
AWQ_F16 = 2                     # stored steps, and the key/value cache
AWQ_SEARCH_ZERO_POINT = 1       # awq_search_layer_flags
AWQ_SEARCH_FP16_STEPS = 2
AWQ_SEARCH_MATRIX_BF16 = 4      # loss contraction on bf16 matrix cores (with correction rows)
AWQ_SEARCH_MATRIX_FP16 = 8      # loss contraction on fp16 matrix cores

_STATUS = {
    0: "AWQ_OK",
    -1: "AWQ_ERR_ARG",
    -2: "AWQ_ERR_SHAPE",
    -3: "AWQ_ERR_DTYPE",
    -4: "AWQ_ERR_WORKSPACE",
    -5: "AWQ_ERR_NONFINITE",
    -6: "AWQ_ERR_HIP",
}


class AwqError(RuntimeError):
    """A C-ABI call returned a negative awq_status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class AwqNonFinite(AwqError):
    """The search met a NaN or Inf (best == -1)."""


def lib_path() -> str:
    return os.path.join(_PKG, _LIBNAME)


_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_uint = ctypes.c_uint
_sz = ctypes.c_size_t


class _KvCacheC(ctypes.Structure):
    """awq_kv_cache"""
    _fields_ = [("pages", _vp), ("n_pages", _i64), ("page_stride", _i64), ("heads", _i64), ("dim", _int),
                ("group", _int), ("page", _int)]


class _KvBatchC(ctypes.Structure):
    """awq_kv_batch"""
    _fields_ = [("rows", _i64), ("batch", _i64), ("max_pages", _i64), ("row_start", _vp), ("kv_len", _vp),
                ("block_table", _vp)]


class _KvRotationC(ctypes.Structure):
    """awq_kv_rotation"""
    _fields_ = [("cos_sin", _vp), ("positions", _i64), ("rot", _int), ("interleaved", _int), ("q_weight", _vp),
                ("k_weight", _vp), ("eps", ctypes.c_double)]


class _KvStepC(ctypes.Structure):
    """awq_kv_step"""
    _fields_ = [("kv_len", _vp), ("row_start", _vp), ("taken", _vp), ("position", _vp), ("slot", _vp)]


class _KvViewC(ctypes.Structure):
    """awq_kv_view"""
    _fields_ = [("window", _i64), ("sinks", _i64), ("prefix_table", _vp), ("prefix_len", _vp), ("prefix_pages", _i64)]


_kvc = ctypes.POINTER(_KvCacheC)
_kvb = ctypes.POINTER(_KvBatchC)

SIGNATURES = {
    "awq_last_error": (ctypes.c_char_p, []),
    "awq_version": (ctypes.c_char_p, []),
    "awq_act_stats": (_int, [_vp, _int, _i64, _i64, _vp, _vp]),
    "awq_act_stats_ex": (_int, [_vp, _int, _i64, _i64, _int, _vp, _vp]),
    "awq_weight_stats": (_int, [_vp, _int, _i64, _i64, _vp, _vp]),
    "awq_search_workspace_size": (_sz, [_i64, _i64, _i64, _int, _int, _int, _int]),
    "awq_search_workspace_min_size": (_sz, [_i64, _i64, _i64, _int, _int, _int, _int]),
    "awq_search_status": (_int, [_vp, _vp, _vp]),
    "awq_search_layer": (_int, [_vp, _int, _i64, _i64, _vp, _int, _i64, _vp, _vp, _int, _int, _int,
                                _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "awq_search_layer_ex": (_int, [_vp, _int, _i64, _i64, _vp, _int, _i64, _vp, _vp, _int, _int, _int,
                                   _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp, _int]),
    "awq_search_layer_wscale": (_int, [_vp, _int, _i64, _i64, _vp, _int, _i64, _vp, _vp, _vp, _int, _int, _int,
                                       _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "awq_clip_workspace_size": (_sz, [_i64, _i64, _int]),
    "awq_clip_search": (_int, [_vp, _int, _i64, _i64, _vp, _int, _i64, _vp, _vp, _int, _int, _int,
                               _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "awq_search_layer_zp": (_int, [_vp, _int, _i64, _i64, _vp, _int, _i64, _vp, _vp, _vp, _int, _int, _int,
                                   _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "awq_search_layer_flags": (_int, [_vp, _int, _i64, _i64, _vp, _int, _i64, _vp, _vp, _vp, _int, _int, _int,
                                      _uint, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "awq_pack": (_int, [_vp, _i64, _i64, _int, _vp, _vp]),
    "awq_pack_ex": (_int, [_vp, _i64, _i64, _int, _int, _vp, _vp]),
    "awq_w4a16_gemm_zp": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _int, _vp, _vp, _int, _vp, _sz, _vp]),
    "awq_w4a16_workspace_size": (_sz, [_i64, _i64, _i64, _int]),
    "awq_w4a16_gemm": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _int, _vp, _vp, _int, _vp, _sz, _vp]),
    "awq_w4a16_workspace_size_ex": (_sz, [_i64, _i64, _i64, _int, _int]),
    "awq_w4a16_noalloc_scratch_bytes": (_sz, []),
    "awq_w4a16_gemm_noalloc": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _int, _vp, _vp, _int, _vp]),
    "awq_w4a16_gemm_ex": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _int, _vp, _int, _vp, _vp, _int, _vp, _sz,
                                 _vp]),
    "awq_kv_page_size": (_sz, [_int, _i64, _int, _int]),
    "awq_kv_append": (_int, [_kvc, _kvb, _vp, _vp, _int, _i64, _i64, _vp]),
    "awq_kv_append_rotated": (_int, [_kvc, _kvb, ctypes.POINTER(_KvRotationC), _vp, _vp, _vp, _int, _i64, _i64, _i64, _i64,
                                     _vp, _i64, _vp]),
    "awq_kv_tables": (_int, [_int, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _i64, ctypes.POINTER(_KvStepC), _vp]),
    "awq_kv_tables_ex": (_int, [_int, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _i64, ctypes.POINTER(_KvStepC), _vp]),
    "awq_kv_read": (_int, [_kvc, _kvb, _vp, _vp, _int, _i64, _i64, _vp]),
    "awq_kv_attention_workspace_size": (_sz, [_kvc, _kvb, _i64, _i64]),
    "awq_kv_attention": (_int, [_kvc, _kvb, _vp, _int, _i64, _i64, _i64, ctypes.c_float, _int, _i64, _vp, _i64, _vp,
                                _vp, _sz, _vp]),
    "awq_kv_attention_workspace_size_ex": (_sz, [_kvc, _kvb, ctypes.POINTER(_KvViewC), _i64, _i64]),
    "awq_kv_attention_ex": (_int, [_kvc, _kvb, ctypes.POINTER(_KvViewC), _vp, _int, _i64, _i64, _i64, ctypes.c_float, _int, _vp,
                                   _i64, _vp, _vp, _sz, _vp]),
}


def load() -> ctypes.CDLL:
    """Load the HIP library (raises if it is missing: no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it first with "
            "`python -c 'import __graft_entry__ as g; g.build()'` "
            "or `python -m weight_only_quantization_awq_amd.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def version() -> str:
    return load().awq_version().decode()


def _check(status: int):
    if status != 0:
        msg = load().awq_last_error().decode(errors="replace")
        raise AwqError(status, msg)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return AWQ_F32
    if t == torch.bfloat16:
        return AWQ_BF16
    raise TypeError(f"unsupported dtype {t} (float32 or bfloat16)")


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# ---------------------------------------------------------------------------

_STATS = {"mean": 0, "max": 1}


def act_stats(X: torch.Tensor, statistic: str = "mean") -> torch.Tensor:
    """a_j = mean_n |X[n, j]| (or max_n with statistic="max") as float32 [D_in]."""
    lib = load()
    if statistic not in _STATS:
        raise ValueError("statistic must be 'mean' or 'max'")
    N, D_in = X.shape
    a = torch.empty(D_in, dtype=torch.float32, device=X.device)
    _check(lib.awq_act_stats_ex(_dev(X, "X"), _dtype_code(X.dtype), N, D_in, _STATS[statistic], _dev(a, "a"),
                                _stream(X.device)))
    return a


def weight_stats(W: torch.Tensor) -> torch.Tensor:
    """b_j = mean_o |W[j, o]| as float32 [D_in] (W is [D_in, D_out])."""
    lib = load()
    D_in, D_out = W.shape
    b = torch.empty(D_in, dtype=torch.float32, device=W.device)
    _check(lib.awq_weight_stats(_dev(W, "W"), _dtype_code(W.dtype), D_in, D_out, _dev(b, "b"), _stream(W.device)))
    return b


def search_workspace_size(N: int, D_in: int, D_out: int, x_dtype: torch.dtype, bits: int = 4,
                          group: int = 128, n_alpha: int = 21) -> int:
    lib = load()
    n = lib.awq_search_workspace_size(N, D_in, D_out, _dtype_code(x_dtype), bits, group, n_alpha)
    if n == 0:
        raise AwqError(-2, lib.awq_last_error().decode(errors="replace"))
    return int(n)


def search_workspace_min_size(N: int, D_in: int, D_out: int, x_dtype: torch.dtype, bits: int = 4,
                              group: int = 128, n_alpha: int = 21) -> int:
    """The smallest workspace the search accepts (it then runs in column chunks)."""
    lib = load()
    n = lib.awq_search_workspace_min_size(N, D_in, D_out, _dtype_code(x_dtype), bits, group, n_alpha)
    if n == 0:
        raise AwqError(-2, lib.awq_last_error().decode(errors="replace"))
    return int(n)


@dataclass
class SearchResult:
    losses: torch.Tensor   # float64 [n_alpha]
    best: torch.Tensor     # int32 [1] (device)
    s_best: torch.Tensor   # float32 [D_in]
    scales: torch.Tensor   # float32 [D_in/group, D_out]
    codes: torch.Tensor | None  # int8 [D_in, D_out] (uint8 zero-point codes with zero_point=True)
    zeros: torch.Tensor | None = None  # uint8 [D_in/group, D_out] (zero_point=True)

    def best_index(self) -> int:
        """alpha* index, through awq_search_status (waits for the current stream)."""
        lib = load()
        out = ctypes.c_int32(-1)
        st = lib.awq_search_status(_dev(self.best, "best"), _stream(self.best.device), ctypes.byref(out))
        if st == -5:
            raise AwqNonFinite(st, lib.awq_last_error().decode(errors="replace"))
        _check(st)
        return int(out.value)


def default_alphas(n: int = 21) -> np.ndarray:
    return (np.arange(n, dtype=np.float64) / max(n - 1, 1)).astype(np.float32)


SEARCH_EVENTS = 5


def search_layer(X: torch.Tensor, W: torch.Tensor, alphas=None, bits: int = 4, group: int = 128,
                 a: torch.Tensor | None = None, want_codes: bool = True,
                 workspace: torch.Tensor | None = None, events=None,
                 b: torch.Tensor | None = None, zero_point: bool = False,
                 f16_steps: bool = False, matrix: str | None = None) -> SearchResult:
    """Run the alpha grid search for one layer (asynchronous on the current stream).

    ``workspace``: a caller buffer of at least :func:`search_workspace_min_size`
    bytes (below :func:`search_workspace_size` the search runs in column
    chunks, with identical results); None allocates the one-pass size.

    ``events``: optional list of 5 ``torch.cuda.Event(enable_timing=True)``
    recorded at the phase boundaries (see awq_search_layer_ex).
    ``b``: a weight statistic (e.g. :func:`weight_stats`) selects the
    candidates s = a^alpha / b^(1-alpha) (awq_search_layer_wscale; no events).
    ``zero_point``: asymmetric codes in [0, 2^bits - 1] with zero points
    (awq_search_layer_zp; no events).
    ``f16_steps``: steps rounded to and returned in FP16 (``scales`` is
    float16), with either code kind (awq_search_layer_flags; no events).
    ``matrix``: "bf16" or "fp16" picks the loss contraction's matrix cores on
    layers that may take the bf16 path, instead of the size rule
    (awq_search_layer_flags; no events).
    """
    lib = load()
    N, D_in = X.shape
    D_in2, D_out = W.shape
    if D_in2 != D_in:
        raise ValueError("X and W disagree on D_in")
    dev = X.device
    if alphas is None:
        alphas = default_alphas(21)
    al = np.ascontiguousarray(np.asarray(alphas, dtype=np.float32))
    if a is None:
        a = act_stats(X)
    if workspace is None:
        workspace = torch.empty(search_workspace_size(N, D_in, D_out, X.dtype, bits, group, al.size),
                                dtype=torch.uint8, device=dev)
    losses = torch.empty(al.size, dtype=torch.float64, device=dev)
    best = torch.empty(1, dtype=torch.int32, device=dev)
    s_best = torch.empty(D_in, dtype=torch.float32, device=dev)
    scales = torch.empty(D_in // group, D_out, dtype=torch.float32, device=dev)
    codes = torch.empty(D_in, D_out, dtype=torch.int8, device=dev) if want_codes else None
    ev_arr, n_ev = None, 0
    if events is not None:
        if len(events) != SEARCH_EVENTS:
            raise ValueError(f"events must hold {SEARCH_EVENTS} torch.cuda.Event objects")
        st = torch.cuda.current_stream(dev)
        for e in events:            # materialise the underlying hipEvent_t handles
            if not e.cuda_event:
                e.record(st)
        ev_arr = (ctypes.c_void_p * SEARCH_EVENTS)(*[e.cuda_event for e in events])
        n_ev = SEARCH_EVENTS
    if matrix not in (None, "bf16", "fp16"):
        raise ValueError(f"matrix must be None, 'bf16' or 'fp16' (got {matrix!r})")
    if f16_steps or matrix is not None:
        if events is not None:
            raise ValueError("phase events are not available with FP16 steps or a chosen matrix format")
        flags = ((AWQ_SEARCH_FP16_STEPS if f16_steps else 0) | (AWQ_SEARCH_ZERO_POINT if zero_point else 0)
                 | {None: 0, "bf16": AWQ_SEARCH_MATRIX_BF16, "fp16": AWQ_SEARCH_MATRIX_FP16}[matrix])
        if f16_steps:
            scales = torch.empty(D_in // group, D_out, dtype=torch.float16, device=dev)
        zeros = torch.empty(D_in // group, D_out, dtype=torch.uint8, device=dev) if zero_point else None
        if zero_point and codes is not None:
            codes = codes.view(torch.uint8)
        _check(lib.awq_search_layer_flags(
            _dev(X, "X"), _dtype_code(X.dtype), N, D_in, _dev(W, "W"), _dtype_code(W.dtype), D_out,
            _dev(a, "a"), _dev(b, "b") if b is not None else None, al.ctypes.data, al.size, bits, group, flags,
            _dev(losses, "losses"), _dev(best, "best"), _dev(s_best, "s_best"), _dev(scales, "scales"),
            _dev(zeros, "zeros") if zeros is not None else None, _dev(codes, "codes") if codes is not None else None,
            _dev(workspace, "workspace"), workspace.numel(), _stream(dev)))
        return SearchResult(losses, best, s_best, scales, codes, zeros)
    if zero_point:
        if events is not None:
            raise ValueError("phase events are not available with zero-point codes")
        zeros = torch.empty(D_in // group, D_out, dtype=torch.uint8, device=dev)
        codes = codes.view(torch.uint8) if codes is not None else None
        _check(lib.awq_search_layer_zp(
            _dev(X, "X"), _dtype_code(X.dtype), N, D_in, _dev(W, "W"), _dtype_code(W.dtype), D_out,
            _dev(a, "a"), _dev(b, "b") if b is not None else None, al.ctypes.data, al.size, bits, group,
            _dev(losses, "losses"), _dev(best, "best"), _dev(s_best, "s_best"), _dev(scales, "scales"),
            _dev(zeros, "zeros"), _dev(codes, "codes") if codes is not None else None,
            _dev(workspace, "workspace"), workspace.numel(), _stream(dev)))
        return SearchResult(losses, best, s_best, scales, codes, zeros)
    if b is not None:
        if events is not None:
            raise ValueError("phase events are not available with a weight statistic")
        _check(lib.awq_search_layer_wscale(
            _dev(X, "X"), _dtype_code(X.dtype), N, D_in, _dev(W, "W"), _dtype_code(W.dtype), D_out,
            _dev(a, "a"), _dev(b, "b"), al.ctypes.data, al.size, bits, group,
            _dev(losses, "losses"), _dev(best, "best"), _dev(s_best, "s_best"), _dev(scales, "scales"),
            _dev(codes, "codes") if codes is not None else None,
            _dev(workspace, "workspace"), workspace.numel(), _stream(dev)))
        return SearchResult(losses, best, s_best, scales, codes)
    _check(lib.awq_search_layer_ex(
        _dev(X, "X"), _dtype_code(X.dtype), N, D_in, _dev(W, "W"), _dtype_code(W.dtype), D_out,
        _dev(a, "a"), al.ctypes.data, al.size, bits, group,
        _dev(losses, "losses"), _dev(best, "best"), _dev(s_best, "s_best"), _dev(scales, "scales"),
        _dev(codes, "codes") if codes is not None else None,
        _dev(workspace, "workspace"), workspace.numel(), _stream(dev),
        ctypes.cast(ev_arr, ctypes.c_void_p) if ev_arr is not None else None, n_ev))
    return SearchResult(losses, best, s_best, scales, codes)


def clip_workspace_size(N: int, D_in: int, group: int = 128) -> int:
    lib = load()
    n = lib.awq_clip_workspace_size(N, D_in, group)
    if n == 0:
        raise AwqError(-1, lib.awq_last_error().decode(errors="replace"))
    return int(n)


@dataclass
class ClipResult:
    ratio_idx: torch.Tensor          # int32 [D_in/group, D_out]
    scales: torch.Tensor             # float32 [D_in/group, D_out]
    codes: torch.Tensor | None       # int8 [D_in, D_out]
    errors: torch.Tensor | None      # float32 [n_ratio, D_in/group, D_out]


def default_clip_ratios(n: int = 11, lowest: float = 0.5) -> np.ndarray:
    """1, ..., lowest in n equal steps (1 = no clipping)."""
    return np.linspace(1.0, lowest, n).astype(np.float32)


def clip_search(X: torch.Tensor, W: torch.Tensor, s: torch.Tensor, ratios=None, bits: int = 4,
                group: int = 128, want_codes: bool = True, want_errors: bool = False,
                workspace: torch.Tensor | None = None) -> ClipResult:
    """Per-group weight-clipping search with fixed scales s (asynchronous on the current stream)."""
    lib = load()
    N, D_in = X.shape
    D_in2, D_out = W.shape
    if D_in2 != D_in:
        raise ValueError("X and W disagree on D_in")
    dev = X.device
    r = np.ascontiguousarray(np.asarray(default_clip_ratios() if ratios is None else ratios, dtype=np.float32))
    need = clip_workspace_size(N, D_in, group)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    G = D_in // group
    ratio_idx = torch.empty(G, D_out, dtype=torch.int32, device=dev)
    scales = torch.empty(G, D_out, dtype=torch.float32, device=dev)
    codes = torch.empty(D_in, D_out, dtype=torch.int8, device=dev) if want_codes else None
    errors = torch.empty(r.size, G, D_out, dtype=torch.float32, device=dev) if want_errors else None
    _check(lib.awq_clip_search(
        _dev(X, "X"), _dtype_code(X.dtype), N, D_in, _dev(W, "W"), _dtype_code(W.dtype), D_out,
        _dev(s, "s"), r.ctypes.data, r.size, bits, group,
        _dev(ratio_idx, "ratio_idx"), _dev(scales, "scales"),
        _dev(codes, "codes") if codes is not None else None,
        _dev(errors, "errors") if errors is not None else None,
        _dev(workspace, "workspace"), workspace.numel(), _stream(dev)))
    return ClipResult(ratio_idx, scales, codes, errors)


def pack(codes: torch.Tensor, bits: int = 4) -> torch.Tensor:
    """Codes [D_in, D_out] -> uint32 words [D_in/8, D_out] (stored as int32).

    int8 codes are signed (nibble = q + 8); uint8 codes are the zero-point
    codes of ``search_layer(..., zero_point=True)`` (nibble = q).
    """
    lib = load()
    if codes.dtype not in (torch.int8, torch.uint8):
        raise TypeError("codes must be int8 (signed) or uint8 (zero-point codes)")
    D_in, D_out = codes.shape
    packed = torch.empty(D_in // 8, D_out, dtype=torch.int32, device=codes.device)
    _check(lib.awq_pack_ex(_dev(codes, "codes"), D_in, D_out, bits, 1 if codes.dtype == torch.uint8 else 0,
                           _dev(packed, "packed"), _stream(codes.device)))
    return packed


def w4a16_workspace_size(M: int, D_in: int, D_out: int, has_inv_s: bool) -> int:
    return int(load().awq_w4a16_workspace_size(M, D_in, D_out, 1 if has_inv_s else 0))


def w4a16_gemm(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, group: int = 128,
               inv_s: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               zeros: torch.Tensor | None = None) -> torch.Tensor:
    """Y = (X·diag(inv_s))·Dequant(packed, scales[, zeros]); X bf16 [M, D_in].

    ``scales`` float32, or float16 (FP16 steps: awq_w4a16_gemm_ex).
    """
    lib = load()
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    M, D_in = X.shape
    D_out = packed.shape[1]
    if packed.shape[0] * 8 != D_in:
        raise ValueError("packed rows must be D_in/8")
    if out is None:
        out = torch.empty(M, D_out, dtype=out_dtype, device=X.device)
    if scales.dtype == torch.float16:
        need = int(lib.awq_w4a16_workspace_size_ex(M, D_in, D_out, group, AWQ_F16))
        if need == 0:
            raise AwqError(-1, lib.awq_last_error().decode(errors="replace"))
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
        _check(lib.awq_w4a16_gemm_ex(
            _dev(X, "X"), M, D_in, D_out, _dev(packed, "packed"), _dev(scales, "scales"), AWQ_F16,
            _dev(zeros, "zeros") if zeros is not None else None, group,
            _dev(inv_s, "inv_s") if inv_s is not None else None, _dev(out, "Y"), _dtype_code(out.dtype),
            _dev(workspace, "workspace"), workspace.numel(), _stream(X.device)))
        return out
    need = w4a16_workspace_size(M, D_in, D_out, inv_s is not None)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    if zeros is not None:
        _check(lib.awq_w4a16_gemm_zp(
            _dev(X, "X"), M, D_in, D_out, _dev(packed, "packed"), _dev(scales, "scales"), _dev(zeros, "zeros"),
            group, _dev(inv_s, "inv_s") if inv_s is not None else None,
            _dev(out, "Y"), _dtype_code(out.dtype),
            _dev(workspace, "workspace") if need else None, workspace.numel() if need else 0,
            _stream(X.device)))
        return out
    _check(lib.awq_w4a16_gemm(
        _dev(X, "X"), M, D_in, D_out, _dev(packed, "packed"), _dev(scales, "scales"), group,
        _dev(inv_s, "inv_s") if inv_s is not None else None,
        _dev(out, "Y"), _dtype_code(out.dtype),
        _dev(workspace, "workspace") if need else None, workspace.numel() if need else 0,
        _stream(X.device)))
    return out


def w4a16_gemm_noalloc(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, group: int = 128,
                       inv_s: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """awq_w4a16_gemm_noalloc: the W4A16 product on the library's static scratch
    (no workspace; float32 steps, signed codes).  Pass ``out`` to allocate
    nothing at all; calls that overlap on one GPU race on the scratch."""
    lib = load()
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    M, D_in = X.shape
    D_out = packed.shape[1]
    if out is None:
        out = torch.empty(M, D_out, dtype=out_dtype, device=X.device)
    _check(lib.awq_w4a16_gemm_noalloc(
        _dev(X, "X"), M, D_in, D_out, _dev(packed, "packed"), _dev(scales, "scales"), group,
        _dev(inv_s, "inv_s") if inv_s is not None else None, _dev(out, "Y"), _dtype_code(out.dtype),
        _stream(X.device)))
    return out


# ---------------------------------------------------------------------------
# The 4-bit key/value cache

_KV_TYPES = {torch.float32: AWQ_F32, torch.bfloat16: AWQ_BF16, torch.float16: AWQ_F16}


@dataclass(frozen=True, eq=False)   # a cache equals itself alone
class KvCache:
    """A pool of pages of 4-bit keys and values (include/awq.h: awq_kv_cache).

    ``pages`` is uint8 [n_pages, heads, block]; the pages may lie apart (a slice
    of a larger pool), each one contiguous.  :func:`kv_cache` makes one.  Calls use the
    memory that ``pages`` has at the time: it may be given other storage (``set_``).
    """
    pages: torch.Tensor
    dim: int           # channels of a head: 64, 128 or 256
    group: int = 128   # channels that share a step: 32, 64 or 128
    page: int = 16     # tokens of a page: 16, 32, 64, 128 or 256

    def __post_init__(self):
        p = self.pages
        if p.dtype != torch.uint8 or p.dim() != 3:
            raise TypeError("pages must be uint8 [n_pages, heads, block]")
        n, heads, block = p.shape
        size = kv_page_size(self.page, heads, self.dim, self.group)
        if heads * block != size:
            raise ValueError(f"a page must hold {size} bytes (got {heads} x {block})")
        if p.stride(2) != 1 or p.stride(1) != block:
            raise ValueError("each page must be contiguous")
        stride = p.stride(0) if n > 1 else size    # torch gives a single page any stride
        end = p.storage_offset() + (n - 1) * stride + size if n else 0
        if p.untyped_storage().nbytes() < end:
            raise ValueError("the memory of the pages has been given up, or is smaller than they are")
        object.__setattr__(self, "_c", _KvCacheC(p.data_ptr(), n, stride, heads, self.dim, self.group, self.page))
        object.__setattr__(self, "_at", p.data_ptr())
        object.__setattr__(self, "_ptr", p.data_ptr)
        object.__setattr__(self, "_device", p.device)
        object.__setattr__(self, "heads", heads)


def kv_page_size(page: int, heads: int, dim: int, group: int = 128) -> int:
    """Bytes of one page: heads * (page*dim + 8*page*(dim/group))."""
    lib = load()
    n = lib.awq_kv_page_size(page, heads, dim, group)
    if n == 0:
        raise AwqError(-1, lib.awq_last_error().decode(errors="replace"))
    return int(n)


def kv_cache(n_pages: int, heads: int, dim: int, group: int = 128, page: int = 16, device="cuda") -> KvCache:
    """A pool of ``n_pages`` pages (all zero, which reads back as zero)."""
    block = kv_page_size(page, heads, dim, group) // heads
    return KvCache(torch.zeros(n_pages, heads, block, dtype=torch.uint8, device=device), dim, group, page)


def _kv_pool(cache: KvCache):
    """The cache's C struct and its device, anew where the pages' memory is no longer where it was
    (0.15 us; resizing storage, smaller or larger, moves it)."""
    if cache._ptr() != cache._at:
        cache.__post_init__()
    return cache._c, cache._device


def _kv_rows(x: torch.Tensor, name: str, device, shape) -> tuple[int, int]:
    """Pointer and row stride of a [rows, heads, dim] tensor whose rows may lie apart."""
    if x.device != device:
        raise ValueError(f"{name} must be on the cache's GPU")
    if x.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(x.shape)})")
    if x.is_contiguous():
        return x.data_ptr(), shape[1] * shape[2]
    if x.stride(2) != 1 or (shape[1] > 1 and x.stride(1) != shape[2]):
        raise ValueError(f"each row of {name} must be contiguous")
    # torch gives a single row any stride
    return x.data_ptr(), x.stride(0) if shape[0] > 1 else shape[1] * shape[2]


def _kv_ints(x: torch.Tensor, name: str, device, shape) -> int:
    """Pointer of an int32 tensor on the cache's GPU."""
    if x.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32 (got {x.dtype})")
    if x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on the cache's GPU")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(x.shape)})")
    return x.data_ptr()


def _kv_batch(device, block_table, kv_len, row_start, rows: int) -> _KvBatchC:
    if device.type != "cuda":
        raise ValueError("pages must be a GPU tensor")
    table = _kv_ints(block_table, "block_table", device, None)
    batch, max_pages = block_table.shape
    return _KvBatchC(rows, batch, max_pages,
                     None if row_start is None else _kv_ints(row_start, "row_start", device, (batch + 1,)),
                     _kv_ints(kv_len, "kv_len", device, (batch,)), table)


def _kv_type(t: torch.dtype) -> int:
    if t not in _KV_TYPES:
        raise TypeError(f"unsupported dtype {t} (float32, bfloat16 or float16)")
    return _KV_TYPES[t]


# torch's own handle of the current stream where it offers it (0.1 us); the Stream
# object costs 1.9 us, a fifth of a call on a few tokens.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _kv_call(device: torch.device, fn, *args):
    """fn(*args, current stream of `device`), with that device current."""
    index = device.index
    if torch.cuda.current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        _check(status)


def kv_append(cache: KvCache, K: torch.Tensor, V: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor,
              row_start: torch.Tensor | None = None) -> None:
    """Quantise the rows' keys and values [rows, heads, dim] into the cache.

    Sequence b's rows are ``row_start[b] .. row_start[b+1] - 1`` (the same number
    for each sequence without ``row_start``) and become the last of its ``kv_len[b]``
    positions; position p lies in page ``block_table[b, p // page]``.
    """
    c, dev = _kv_pool(cache)
    rows = K.shape[0]
    shape = (rows, cache.heads, cache.dim)
    if V.dtype != K.dtype:
        raise TypeError("K and V must have one dtype")
    b = _kv_batch(dev, block_table, kv_len, row_start, rows)
    k, k_stride = _kv_rows(K, "K", dev, shape)
    v, v_stride = _kv_rows(V, "V", dev, shape)
    _kv_call(dev, _lib.awq_kv_append, c, b, k, v, _kv_type(K.dtype), k_stride, v_stride)


class KvStep(NamedTuple):
    """What :func:`kv_tables` gives: a step's ``kv_len`` and ``row_start`` for the other calls, the
    free pages ``taken`` so far, and each row's ``position`` and ``slot`` (None without ``rows``)."""
    kv_len: torch.Tensor              # int32 [batch]
    row_start: torch.Tensor           # int32 [batch + 1]
    taken: torch.Tensor               # int32 [1]
    position: torch.Tensor | None     # int32 [rows]
    slot: torch.Tensor | None         # int64 [rows]


def kv_tables(block_table: torch.Tensor, kv_len: torch.Tensor, count: torch.Tensor, free_pages: torch.Tensor,
              taken: torch.Tensor | None = None, page: int = 16, rows: int = 0, out: KvStep | None = None,
              n_pages: int = 0) -> KvStep:
    """The tables of a step in which sequence b, ``kv_len[b]`` tokens long, adds ``count[b]`` rows.

    The pages that new rows begin come from ``free_pages`` behind the first ``taken`` of them
    and are written into ``block_table`` (-1 where none are left; ``taken`` of the result then
    exceeds their number).  ``rows``: with positions and slots of so many rows, -1 for those
    that belong to no sequence.  A slot on a page of a negative number is -1, too, and with
    ``n_pages`` (of the pool) one on a page from there on.  ``out``: a :class:`KvStep` to write to; none of its tensors may
    share memory with an input.  Everything stays on the GPU: a captured step can grow its sequences.
    """
    dev = block_table.device
    if dev.type != "cuda":
        raise ValueError("block_table must be a GPU tensor")
    table = _kv_ints(block_table, "block_table", dev, None)
    batch, max_pages = block_table.shape
    if out is None:
        ints = torch.empty(2 * batch + 2 + rows, dtype=torch.int32, device=dev).split_with_sizes((batch, batch + 1, 1, rows))
        out = KvStep(ints[0], ints[1], ints[2], ints[3] if rows else None,
                     torch.empty(rows, dtype=torch.int64, device=dev) if rows else None)
        s = _KvStepC(*[x.data_ptr() for x in ints], out.slot.data_ptr() if rows else None)
    else:
        if out.slot is not None and (out.slot.dtype is not torch.int64 or out.slot.device != dev
                                     or out.slot.shape != (rows,) or not out.slot.is_contiguous()):
            raise ValueError(f"slot must be contiguous int64 [{rows}] on the table's GPU")
        s = _KvStepC(_kv_ints(out.kv_len, "out.kv_len", dev, (batch,)), _kv_ints(out.row_start, "out.row_start", dev, (batch + 1,)),
                     _kv_ints(out.taken, "out.taken", dev, (1,)),
                     None if out.position is None else _kv_ints(out.position, "out.position", dev, (rows,)),
                     None if out.slot is None else out.slot.data_ptr())
    if free_pages.dim() != 1:
        raise ValueError("free_pages must have one dimension")
    _kv_call(dev, _lib.awq_kv_tables_ex, page, batch, max_pages, _kv_ints(kv_len, "kv_len", dev, (batch,)),
             _kv_ints(count, "count", dev, (batch,)), _kv_ints(free_pages, "free_pages", dev, None), free_pages.shape[0],
             None if taken is None else _kv_ints(taken, "taken", dev, (1,)), table, rows, n_pages, s)
    return out


def kv_rotation_table(positions: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines [positions, 2, rot/2] of the angles p * base^(-2i/rot), taken in 64 bits and
    rounded once to float32 (for :func:`kv_append_rotated`; scaled frequencies are a table of one's own)."""
    if rot < 0 or rot % 2:
        raise ValueError(f"rot must be even (got {rot})")
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), 1).float()


def _kv_floats(x: torch.Tensor, name: str, device, shape) -> int:
    """Pointer of a float32 tensor on the cache's GPU."""
    if x.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32 (got {x.dtype})")
    if x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on the cache's GPU")
    if x.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(x.shape)})")
    return x.data_ptr()


def kv_append_rotated(cache: KvCache, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, block_table: torch.Tensor,
                      kv_len: torch.Tensor, cos_sin: torch.Tensor | None, row_start: torch.Tensor | None = None,
                      q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                      interleaved: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Normalise and rotate queries [rows, q_heads, dim] and keys, and append keys and values.

    Rows and positions as in :func:`kv_append`.  ``q_weight`` / ``k_weight`` (float32 [dim]):
    each head's row is divided by the root of its mean square plus ``eps`` and multiplied by
    the weight; None leaves it.  ``cos_sin`` (float32 [positions, 2, rot/2], see
    :func:`kv_rotation_table`): the first rot channels are rotated by the row's position, in
    halves or (``interleaved``) in neighbouring pairs; None rotates nothing.  A position that
    it does not hold gives NaN.  Returns the queries for :func:`kv_attention`.  ``out`` may be Q,
    but no other tensor that shares memory with Q; K and V are read before it is written.
    """
    c, dev = _kv_pool(cache)
    rows, q_heads = Q.shape[0], Q.shape[1]
    shape, kv_shape, dtype = (rows, q_heads, cache.dim), (rows, cache.heads, cache.dim), Q.dtype
    if K.dtype != dtype or V.dtype != dtype:
        raise TypeError("Q, K and V must have one dtype")
    b = _kv_batch(dev, block_table, kv_len, row_start, rows)
    q, q_stride = _kv_rows(Q, "Q", dev, shape)
    k, k_stride = _kv_rows(K, "K", dev, kv_shape)
    v, v_stride = _kv_rows(V, "V", dev, kv_shape)
    if out is None:
        out = torch.empty_like(Q) if Q.is_contiguous() else torch.empty(shape, dtype=dtype, device=dev)
        o, o_stride = out.data_ptr(), q_heads * cache.dim
    elif out.dtype != dtype:
        raise TypeError("out must have the dtype of Q")
    else:
        o, o_stride = _kv_rows(out, "out", dev, shape)
    positions = rot = table = 0
    if cos_sin is not None:
        if cos_sin.dim() != 3:
            raise ValueError("cos_sin must be [positions, 2, rot/2]")
        positions, rot = cos_sin.shape[0], 2 * cos_sin.shape[2]
        table = _kv_floats(cos_sin, "cos_sin", dev, (positions, 2, rot // 2))
    weights = (cache.dim,)
    r = _KvRotationC(table, positions, rot, 1 if interleaved else 0,
                     None if q_weight is None else _kv_floats(q_weight, "q_weight", dev, weights),
                     None if k_weight is None else _kv_floats(k_weight, "k_weight", dev, weights), eps)
    _kv_call(dev, _lib.awq_kv_append_rotated, c, b, r, q, k, v, _kv_type(dtype), q_heads, q_stride, k_stride, v_stride, o, o_stride)
    return out


def kv_read(cache: KvCache, block_table: torch.Tensor, kv_len: torch.Tensor, rows: int,
            row_start: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
            out: tuple[torch.Tensor, torch.Tensor] | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """The rows' keys and values [rows, heads, dim] as the cache stands for them.

    Rows and positions as in :func:`kv_append`: the last positions of each
    sequence, all of them where its rows are ``kv_len[b]``.  Rows that belong to
    no sequence are left as they were in ``out`` (unspecified in new tensors).
    """
    c, dev = _kv_pool(cache)
    shape = (rows, cache.heads, cache.dim)
    b = _kv_batch(dev, block_table, kv_len, row_start, rows)
    if out is None:
        out = torch.empty((2,) + shape, dtype=dtype, device=dev).unbind(0)
    K, V = out
    if V.dtype != K.dtype:
        raise TypeError("both outputs must have one dtype")
    k, k_stride = _kv_rows(K, "K", dev, shape)
    v, v_stride = _kv_rows(V, "V", dev, shape)
    _kv_call(dev, _lib.awq_kv_read, c, b, k, v, _kv_type(K.dtype), k_stride, v_stride)
    return K, V


def _kv_workspace(cache_c, batch_c, view_c, q_heads: int, max_rows: int) -> int:
    if view_c is None:
        n = _lib.awq_kv_attention_workspace_size(cache_c, batch_c, q_heads, max_rows)
    else:
        n = _lib.awq_kv_attention_workspace_size_ex(cache_c, batch_c, view_c, q_heads, max_rows)
    if n == 0:
        msg = _lib.awq_last_error()
        if msg:
            raise AwqError(-2, msg.decode(errors="replace"))
    return n


def kv_attention_workspace_size(cache: KvCache, q_heads: int, rows: int, batch: int, max_pages: int,
                                ragged: bool = False, max_rows: int | None = None, prefix_pages: int = 0) -> int:
    """Bytes of workspace of a :func:`kv_attention` call (``ragged``: with row_start; ``prefix_pages``: of its prefix)."""
    b = _KvBatchC(rows, batch, max_pages, 4 if ragged else None, None, None)   # only whether it is NULL counts
    return _kv_workspace(cache._c, b, _KvViewC(0, 0, None, 4, prefix_pages) if prefix_pages else None, q_heads, max_rows or 0)


def kv_attention(Q: torch.Tensor, cache: KvCache, block_table: torch.Tensor, kv_len: torch.Tensor,
                 row_start: torch.Tensor | None = None, max_rows: int | None = None, scale: float | None = None,
                 causal: bool = True, window: int = 0, want_lse: bool = False, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, sinks: int = 0,
                 prefix: tuple[torch.Tensor, torch.Tensor] | None = None):
    """Attention of the queries [rows, q_heads, dim] (bf16 or fp16) over the cache.

    Rows and positions as in :func:`kv_append` (append the rows' keys first:
    a row sees its own position).  ``max_rows``: an upper bound on any
    sequence's rows, known on the host; give it with ``row_start``.  ``scale``
    defaults to dim ** -0.5.  ``window`` > 0: only the last ``window`` positions,
    and with ``sinks`` > 0 the first ``sinks`` ones too.
    Without ``causal`` every row sees all ``kv_len[b]`` positions, whatever its own.
    ``prefix`` = (table int32 [pages], length int32 [1]): the first length positions of every
    sequence (counted by ``kv_len``) lie in the table's pages instead of ``block_table``'s and are
    read once for the whole batch; not with a window.  It pays from about 8 sequences behind 32768
    positions, 32 behind 8192 or 128 behind 2048 on (8 heads of 128; with fewer or smaller ones
    from more on); below, shared pages in each row of ``block_table`` are up to three times as fast.
    ``out`` may be Q, but no other tensor that shares memory with it.
    ``workspace``: uint8 of :func:`kv_attention_workspace_size` bytes (None
    allocates it).  Returns the output like Q, and with ``want_lse`` also the
    float32 log-sum-exp [rows, q_heads] (-inf, and output 0, where a row sees
    nothing).
    """
    c, dev = _kv_pool(cache)
    rows, q_heads = Q.shape[0], Q.shape[1]
    shape = (rows, q_heads, cache.dim)
    dtype = Q.dtype
    if dtype != torch.bfloat16 and dtype != torch.float16:
        raise TypeError(f"Q must be bfloat16 or float16 (got {dtype})")
    q, q_stride = _kv_rows(Q, "Q", dev, shape)
    b = _kv_batch(dev, block_table, kv_len, row_start, rows)
    if out is None:   # (empty_like costs 0.5 us less)
        out = torch.empty_like(Q) if Q.is_contiguous() else torch.empty(shape, dtype=dtype, device=dev)
        o, o_stride = out.data_ptr(), q_heads * cache.dim
    elif out.dtype != dtype:
        raise TypeError("out must have the dtype of Q")
    else:
        o, o_stride = _kv_rows(out, "out", dev, shape)
    lse = torch.empty((rows, q_heads), dtype=torch.float32, device=dev) if want_lse else None
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.device != dev
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous uint8 on the cache's GPU")
    view = None
    if prefix is not None:
        table, length = prefix
        if table.dim() != 1:
            raise ValueError("the prefix's table must have one dimension")
        view = _KvViewC(window, sinks, _kv_ints(table, "the prefix's table", dev, None),
                        _kv_ints(length, "the prefix's length", dev, (1,)), table.shape[0])
    elif sinks != 0:
        view = _KvViewC(window, sinks, None, None, 0)
    need = _kv_workspace(c, b, view, q_heads, max_rows or 0)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if view is None:
        _kv_call(dev, _lib.awq_kv_attention, c, b, q, _KV_TYPES[dtype], q_heads, q_stride, max_rows or 0,
                 cache.dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, o, o_stride,
                 lse.data_ptr() if want_lse else None, workspace.data_ptr() if need else None,
                 workspace.numel() if need else 0)
    else:
        _kv_call(dev, _lib.awq_kv_attention_ex, c, b, view, q, _KV_TYPES[dtype], q_heads, q_stride, max_rows or 0,
                 cache.dim ** -0.5 if scale is None else scale, 1 if causal else 0, o, o_stride,
                 lse.data_ptr() if want_lse else None, workspace.data_ptr() if need else None,
                 workspace.numel() if need else 0)
    return (out, lse) if want_lse else out


# Load at import time: a missing library is an error, never a silent fallback.
load()
