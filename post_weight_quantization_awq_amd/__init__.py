"""AWQ per-layer hot path on MI355X (gfx950): Python binding of libawq.so.

This module only marshals arguments: torch tensors are checked for device,
dtype and layout, their device pointers and the current HIP stream are handed
to the C ABI declared in ``include/awq.h``, and errors come back as
``AwqError``.  Every step of the computation runs in the library's HIP
kernels; there is no CPU fallback.  The library must have been built
(``python -m post_weight_quantization_awq_amd.build``); the first call without
it raises ImportError.

Entry points (same names as the C ABI):

* ``act_stats``           per-input-channel mean |x|        ("AWQ scaling", konic.io)
* ``candidate_scales``    s_k = clamp(x^(k/n), s_min) / sqrt(max*min)   ("The scale search as code", aicassindra.com)
* ``search_scales``       alpha grid search, weight or output score, optional clip search
* ``quantize_pack``       INT4 codes + fp16 scales in the AutoAWQ GEMM layout
* ``unpack_dequant``      inverse of quantize_pack
* ``mx_quantize``         microscaled 8-bit or 4-bit codes (blocks of 32, power-of-two scales)
* ``mx_dequant``          inverse of mx_quantize
* ``rms_norm_mx``         RMS norm with the residual's addition, microscaled result
* ``silu_mul_mx``         SiLU gating, microscaled result
* ``mx_matmul``           product of microscaled activations with 4-bit microscaled weights
* ``mx_linear``           the same with bias, activation and residual in its epilogue, also with a microscaled result
* ``moe_route``           each token's experts and shares, and the (token, expert) pairs in expert order
* ``mx_matmul_grouped``   products grouped by expert with ragged sizes
* ``block_norm_mx``       the experts' sum, the norm after a block, gate, residual, and the norm before the next one
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import os
from typing import List, NamedTuple, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libawq.so")

AWQ_OK, AWQ_EINVAL, AWQ_ESHAPE, AWQ_EDTYPE, AWQ_EWORKSPACE, AWQ_EALIGN, AWQ_EHIP = range(7)
AWQ_F16, AWQ_BF16, AWQ_F32 = 0, 1, 2
AWQ_SCORE_WEIGHT, AWQ_SCORE_OUTPUT = 0, 1
AWQ_MX_FP8, AWQ_MX_FP4 = 0, 1
AWQ_FLAG_DUO = 1
AWQ_FLAG_ASYM = 2
AWQ_FLAG_OUT_DIRECT = 4
AWQ_FLAG_OUT_GRAM = 8
_OUT_FORM = {"auto": 0, "direct": AWQ_FLAG_OUT_DIRECT, "gram": AWQ_FLAG_OUT_GRAM}
STATUS_NAMES = {0: "AWQ_OK", 1: "AWQ_EINVAL", 2: "AWQ_ESHAPE", 3: "AWQ_EDTYPE",
                4: "AWQ_EWORKSPACE", 5: "AWQ_EALIGN", 6: "AWQ_EHIP"}

EXPORTED = ("awq_act_stats_workspace", "awq_act_stats", "awq_candidate_scales_workspace", "awq_candidate_scales",
            "awq_search_workspace", "awq_search_output_form", "awq_search_scales", "awq_quantize_pack", "awq_quantize_pack_asym",
            "awq_unpack_dequant", "awq_norm_group_fold", "awq_weight_channel_mean_workspace",
            "awq_weight_channel_mean", "awq_candidate_scales_duo_workspace", "awq_candidate_scales_duo",
            "awq_w4a16_workspace", "awq_w4a16_matmul", "awq_search_scales_noalloc",
            "awq_mx_quantize", "awq_mx_dequant", "awq_rms_norm_mx", "awq_silu_mul_mx", "awq_mx_matmul_workspace",
            "awq_mx_matmul", "awq_mx_linear_workspace", "awq_mx_linear", "awq_moe_route_workspace", "awq_moe_route",
            "awq_mx_matmul_grouped_workspace", "awq_mx_matmul_grouped", "awq_block_norm_mx",
            "awq_last_error", "awq_abi_version", "awq_set_timing_events")


class AwqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class SearchCfg(ctypes.Structure):
    _fields_ = [("group_size", ctypes.c_int32), ("n_grid", ctypes.c_int32),
                ("score", ctypes.c_int32), ("n_clip", ctypes.c_int32),
                ("s_min", ctypes.c_double), ("clip_lo", ctypes.c_float),
                ("flags", ctypes.c_int32)]


class WGroup(ctypes.Structure):
    _fields_ = [("n_parts", ctypes.c_int32), ("w", ctypes.POINTER(ctypes.c_void_p)),
                ("rows", ctypes.POINTER(ctypes.c_int64))]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m post_weight_quantization_awq_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F32, F64, SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_double, ctypes.c_size_t)
    PSZ = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "awq_act_stats_workspace": [I64, I64, PSZ],
        "awq_act_stats": [P, I32, I64, I64, I64, F32, I32, P, P, SZ, P],
        "awq_candidate_scales_workspace": [I64, I32, PSZ],
        "awq_candidate_scales": [P, I64, I32, F64, P, P, SZ, P],
        "awq_search_workspace": [ctypes.POINTER(SearchCfg), I64, I64, I64, PSZ],
        "awq_search_output_form": [ctypes.POINTER(SearchCfg), I64, I64, I64, ctypes.POINTER(I32)],
        "awq_search_scales": [ctypes.POINTER(SearchCfg), ctypes.POINTER(WGroup), I64, P, P, I32, I64, I64,
                              P, P, P, P, P, P, SZ, P],
        "awq_quantize_pack": [P, I64, I64, I32, P, P, P, P, P, P],
        "awq_quantize_pack_asym": [P, I64, I64, I32, P, P, P, P, P, P],
        "awq_unpack_dequant": [P, P, P, I64, I64, I32, P, P, I32, P],
        "awq_norm_group_fold": [ctypes.POINTER(ctypes.c_void_p), I32, I64, P, I32, P, P, P],
        "awq_weight_channel_mean_workspace": [I64, I64, PSZ],
        "awq_weight_channel_mean": [ctypes.POINTER(WGroup), I64, P, P, SZ, P],
        "awq_candidate_scales_duo_workspace": [I64, I32, PSZ],
        "awq_candidate_scales_duo": [P, P, I64, I32, F64, P, P, SZ, P],
        "awq_w4a16_workspace": [I64, I64, I64, PSZ],
        "awq_w4a16_matmul": [P, I64, I64, P, P, P, I64, I64, I32, P, I64, I32, P, SZ, P],
        "awq_mx_quantize": [P, I32, I64, I64, I64, P, I32, P, P, P],
        "awq_mx_dequant": [P, P, I32, I64, I64, P, P, I32, I64, P],
        "awq_rms_norm_mx": [P, I32, I64, I64, I64, P, I64, P, I32, F32, P, I64, I32, P, P, P],
        "awq_silu_mul_mx": [P, I64, P, I64, I32, I64, I64, I32, P, P, P],
        "awq_mx_matmul_workspace": [I32, I64, I64, I64, PSZ],
        "awq_mx_matmul": [P, P, I32, I64, P, P, I64, I64, P, I64, I32, P, SZ, P],
        "awq_mx_linear_workspace": [I32, I64, I64, I64, PSZ],
        "awq_mx_linear": [P, P, I32, I64, P, P, I64, I64, P, I32, I32, P, I32, I64, P, I64, I32, I32, P, P, P, SZ, P],
        "awq_moe_route_workspace": [I64, I32, PSZ],
        "awq_moe_route": [P, I32, I64, I32, I64, I32, I32, F32, P, P, P, P, P, P, SZ, P],
        "awq_mx_matmul_grouped_workspace": [I32, I64, I64, I64, I32, PSZ],
        "awq_mx_matmul_grouped": [P, P, I32, I64, P, I64, P, P, I32, I64, I64, P, P, I64, I32, P, SZ, P],
        "awq_block_norm_mx": [P, I32, I64, I64, P, P, I32, I64, I64, P, I32, P, I32, I64, P, I64, F32, P, I32, F32,
                              P, I64, I32, P, P, P],
        "awq_set_timing_events": [P, P],
        "awq_search_scales_noalloc": [ctypes.POINTER(SearchCfg), ctypes.POINTER(WGroup), I64, P, P, P, P, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int32
    lib.awq_last_error.argtypes = []
    lib.awq_last_error.restype = ctypes.c_char_p
    lib.awq_abi_version.argtypes = []
    lib.awq_abi_version.restype = ctypes.c_int32
    return lib


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded libawq.so (loaded on first use; ImportError if it is not built)."""
    global _lib
    if _lib is None:
        _lib = _load()
    return _lib


def _check(st: int) -> None:
    if st != AWQ_OK:
        raise AwqError(st, lib().awq_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def _tensor(t: Optional[torch.Tensor], name: str, dtype, shape=None, *, contiguous: bool = True,
            unit_col_stride: bool = False, min_numel: Optional[int] = None, like: Optional[torch.Tensor] = None,
            optional: bool = False) -> None:
    """Checks a tensor the library will read or write before anything is launched:
    dtype, shape (a tuple, entries None = any), layout (contiguous, or 2-D with
    unit column stride), size, and that it lives where `like` does.  That the
    tensors are on the device is checked once all of them passed (_dev).
    Raises ValueError."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if shape is not None:
        if t.dim() != len(shape) or any(w is not None and g != w for g, w in zip(t.shape, shape)):
            want = "[" + ", ".join("*" if w is None else str(w) for w in shape) + "]"
            raise ValueError(f"{name} must have shape {want}, got {list(t.shape)}")
    if unit_col_stride:
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
            raise ValueError(f"{name} must be 2-D with unit column stride and rows at least a row apart")
    elif contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {min_numel}")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")


def _x_dtype(X: torch.Tensor) -> int:
    if X.dtype == torch.bfloat16:
        return AWQ_BF16
    if X.dtype == torch.float16:
        return AWQ_F16
    raise ValueError(f"activations must be bf16 or fp16, got {X.dtype}")


def _rows_view(X: torch.Tensor, name: str):
    if X.dim() != 2 or (X.shape[1] > 1 and X.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    # a tensor of at most one row may report any row stride; its rows are never stepped over
    ld = X.stride(0) if X.shape[0] > 1 else max(X.stride(0), X.shape[1])
    return X.shape[0], X.shape[1], ld


def workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# Prepared calls: the ctypes argument tuple is built once; run() is one call
# into the library (no allocation, no size queries), so repeated use costs a
# few microseconds of host time.
# ---------------------------------------------------------------------------
class _Prepared:
    _fn = ""

    def _bind(self, *args) -> None:
        self._f = getattr(lib(), self._fn)
        self._args = args

    def launch(self) -> None:
        _check(self._f(*self._args))


def act_stats_workspace_bytes(T: int, d_in: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().awq_act_stats_workspace(T, d_in, ctypes.byref(n)))
    return n.value


class ActStatsPlan(_Prepared):
    """x_mean[i] (+)= inv_count * sum_t |X[t, i]| (inv_count defaults to 1/T)."""
    _fn = "awq_act_stats"

    def __init__(self, X: torch.Tensor, x_mean: Optional[torch.Tensor] = None, inv_count: Optional[float] = None,
                 accumulate: bool = False, ws: Optional[torch.Tensor] = None, stream=None):
        _tensor(X, "X", (torch.bfloat16, torch.float16), (None, None), unit_col_stride=True)
        T, d_in, ld = _rows_view(X, "X")
        _tensor(x_mean, "x_mean", torch.float32, (d_in,), like=X, optional=True)
        _tensor(ws, "ws", torch.uint8, (None,), like=X, optional=True)
        _dev(X, "X")
        self.x_mean = torch.empty(d_in, dtype=torch.float32, device=X.device) if x_mean is None else x_mean
        if inv_count is None:
            inv_count = 1.0 / T if T > 0 else 0.0
        need = act_stats_workspace_bytes(T, d_in)
        self.ws = workspace(need, X.device) if (ws is None or ws.numel() < need) else ws
        self._keep = (X,)
        self._bind(_ptr(X), _x_dtype(X), T, d_in, ld, inv_count, int(accumulate), _ptr(self.x_mean),
                   _ptr(self.ws), self.ws.numel(), _stream(stream))

    def run(self) -> torch.Tensor:
        self.launch()
        return self.x_mean


def act_stats(X: torch.Tensor, x_mean: Optional[torch.Tensor] = None, inv_count: Optional[float] = None,
              accumulate: bool = False, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x_mean[i] (+)= inv_count * sum_t |X[t, i]| (inv_count defaults to 1/T)."""
    return ActStatsPlan(X, x_mean, inv_count, accumulate, ws, stream).run()


def candidate_scales(x_mean: torch.Tensor, n_grid: int = 20, s_min: float = 1e-4, stream=None) -> torch.Tensor:
    _tensor(x_mean, "x_mean", torch.float32, (None,))
    _dev(x_mean, "x_mean")
    d_in = x_mean.numel()
    S = torch.empty((n_grid, d_in), dtype=torch.float32, device=x_mean.device)
    n = ctypes.c_size_t()
    _check(lib().awq_candidate_scales_workspace(d_in, n_grid, ctypes.byref(n)))
    ws = workspace(n.value, x_mean.device)
    _check(lib().awq_candidate_scales(_ptr(x_mean), d_in, n_grid, s_min, _ptr(S), _ptr(ws), ws.numel(),
                                      _stream(stream)))
    return S


def _wgroup(parts):
    ptrs = (ctypes.c_void_p * len(parts))(*[p.data_ptr() for p in parts])
    rows = (ctypes.c_int64 * len(parts))(*[p.shape[0] for p in parts])
    return WGroup(len(parts), ctypes.cast(ptrs, ctypes.POINTER(ctypes.c_void_p)),
                  ctypes.cast(rows, ctypes.POINTER(ctypes.c_int64))), (ptrs, rows)


def weight_channel_mean(W_parts: Sequence[torch.Tensor], stream=None) -> torch.Tensor:
    """Duo scaling's w_mean: row-normalised mean |w| per input channel of the
    group's concatenated rows (fp32 [d_in])."""
    parts = list(W_parts)
    for p in parts:
        _dev(p, "W")
        if p.dtype != torch.float16 or p.dim() != 2 or not p.is_contiguous() or p.shape[1] != parts[0].shape[1]:
            raise ValueError("weights must be contiguous fp16 [rows, d_in] with one d_in")
    d_in, dev = parts[0].shape[1], parts[0].device
    d_out = sum(p.shape[0] for p in parts)
    n = ctypes.c_size_t()
    _check(lib().awq_weight_channel_mean_workspace(d_out, d_in, ctypes.byref(n)))
    ws = workspace(n.value, dev)
    out = torch.empty(d_in, dtype=torch.float32, device=dev)
    grp, keep = _wgroup(parts)
    _check(lib().awq_weight_channel_mean(ctypes.byref(grp), d_in, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def candidate_scales_duo(x_mean: torch.Tensor, w_mean: torch.Tensor, n_grid: int = 20, s_min: float = 1e-4,
                         stream=None) -> torch.Tensor:
    """Duo-scaling candidate table S [n_grid, d_in]."""
    _tensor(x_mean, "x_mean", torch.float32, (None,))
    _tensor(w_mean, "w_mean", torch.float32, (x_mean.numel(),), like=x_mean)
    _dev(x_mean, "x_mean")
    d_in = x_mean.numel()
    S = torch.empty((n_grid, d_in), dtype=torch.float32, device=x_mean.device)
    n = ctypes.c_size_t()
    _check(lib().awq_candidate_scales_duo_workspace(d_in, n_grid, ctypes.byref(n)))
    ws = workspace(n.value, x_mean.device)
    _check(lib().awq_candidate_scales_duo(_ptr(x_mean), _ptr(w_mean), d_in, n_grid, s_min, _ptr(S), _ptr(ws),
                                          ws.numel(), _stream(stream)))
    return S


@dataclasses.dataclass
class SearchResult:
    err: torch.Tensor                 # fp32 [n_grid]
    best_idx: torch.Tensor            # int32 [1]
    best_s: torch.Tensor              # fp32 [d_in]
    clip: Optional[torch.Tensor]      # fp32 [d_out] or None
    clip_err: Optional[torch.Tensor]  # fp32 [d_out, n_clip] or None


def _cfg(group_size, n_grid, score, n_clip, clip_lo, s_min, duo=False, asym=False, out_form="auto") -> SearchCfg:
    sc = {"weight": AWQ_SCORE_WEIGHT, "output": AWQ_SCORE_OUTPUT}[score] if isinstance(score, str) else score
    if out_form not in _OUT_FORM:
        raise ValueError(f"out_form {out_form!r} not in {sorted(_OUT_FORM)}")
    flags = (AWQ_FLAG_DUO if duo else 0) | (AWQ_FLAG_ASYM if asym else 0) | _OUT_FORM[out_form]
    return SearchCfg(group_size, n_grid, sc, n_clip, s_min, clip_lo, flags)


def search_workspace_bytes(d_out: int, d_in: int, T: int = 0, *, group_size: int = 128, n_grid: int = 20,
                           score="weight", n_clip: int = 0, clip_lo: float = 0.5, s_min: float = 1e-4,
                           duo: bool = False, asym: bool = False, out_form: str = "auto") -> int:
    cfg = _cfg(group_size, n_grid, score, n_clip, clip_lo, s_min, duo, asym, out_form)
    n = ctypes.c_size_t()
    _check(lib().awq_search_workspace(ctypes.byref(cfg), d_out, d_in, T, ctypes.byref(n)))
    return n.value


def search_output_form(d_out: int, d_in: int, T: int, *, group_size: int = 128, n_grid: int = 20, n_clip: int = 0,
                       clip_lo: float = 0.5, s_min: float = 1e-4, duo: bool = False, asym: bool = False,
                       out_form: str = "auto") -> str:
    """The form the output-score alpha search takes for these arguments: "direct" or "gram"."""
    return search_output_forms(d_out, d_in, T, group_size=group_size, n_grid=n_grid, n_clip=n_clip,
                               clip_lo=clip_lo, s_min=s_min, duo=duo, asym=asym, out_form=out_form)[0]


def search_output_forms(d_out: int, d_in: int, T: int, *, group_size: int = 128, n_grid: int = 20, n_clip: int = 0,
                        clip_lo: float = 0.5, s_min: float = 1e-4, duo: bool = False, asym: bool = False,
                        out_form: str = "auto"):
    """(alpha search form, clip search form or None): "direct" or "gram" each."""
    cfg = _cfg(group_size, n_grid, "output", n_clip, clip_lo, s_min, duo, asym, out_form)
    f = ctypes.c_int32()
    _check(lib().awq_search_output_form(ctypes.byref(cfg), d_out, d_in, T, ctypes.byref(f)))
    return ("gram" if f.value & 1 else "direct",
            ("gram" if f.value & 2 else "direct") if n_clip >= 2 else None)


class SearchPlan(_Prepared):
    """Grid search of alpha for one group of linears sharing an input (rows concatenated).
    out_form (output score): "auto" (the library picks), "direct" (X times each candidate's
    dW) or "gram" (the second-moment form dW H dW^T with H = X^T X)."""
    _fn = "awq_search_scales"

    def __init__(self, W_parts: Sequence[torch.Tensor], x_mean: torch.Tensor, *, group_size: int = 128,
                 n_grid: int = 20, score="weight", X: Optional[torch.Tensor] = None, n_clip: int = 0,
                 clip_lo: float = 0.5, s_min: float = 1e-4, want_clip_err: bool = False,
                 ws: Optional[torch.Tensor] = None, out: Optional[SearchResult] = None, stream=None,
                 duo: bool = False, asym: bool = False, out_form: str = "auto"):
        parts: List[torch.Tensor] = list(W_parts)
        if not parts:
            raise ValueError("empty weight group")
        d_in = parts[0].shape[1]
        for p in parts:
            if p.dtype != torch.float16 or p.dim() != 2 or not p.is_contiguous() or p.shape[1] != d_in:
                raise ValueError("weights must be contiguous fp16 [rows, d_in] with one d_in")
        dev = parts[0].device
        for p in parts[1:]:
            if p.device != dev:
                raise ValueError("the parts of a group must live on one device")
        d_out = sum(p.shape[0] for p in parts)
        _tensor(x_mean, "x_mean", torch.float32, (d_in,), like=parts[0])
        self.cfg = _cfg(group_size, n_grid, score, n_clip, clip_lo, s_min, duo, asym, out_form)
        T, ld, xdt = 0, 0, AWQ_BF16
        if X is not None:
            _tensor(X, "X", (torch.bfloat16, torch.float16), (None, d_in), unit_col_stride=True, like=parts[0])
            T, dx, ld = _rows_view(X, "X")
            xdt = _x_dtype(X)
        if out is not None:
            _tensor(out.err, "out.err", torch.float32, (n_grid,), like=parts[0])
            _tensor(out.best_idx, "out.best_idx", torch.int32, (1,), like=parts[0])
            _tensor(out.best_s, "out.best_s", torch.float32, (d_in,), like=parts[0])
            _tensor(out.clip, "out.clip", torch.float32, (d_out,), like=parts[0], optional=not n_clip)
            _tensor(out.clip_err, "out.clip_err", torch.float32, (d_out, n_clip), like=parts[0], optional=True)
        _tensor(ws, "ws", torch.uint8, (None,), like=parts[0], optional=True)
        _dev(parts[0], "W")
        n = ctypes.c_size_t()
        _check(lib().awq_search_workspace(ctypes.byref(self.cfg), d_out, d_in, max(T, 1), ctypes.byref(n)))
        self.ws = workspace(n.value, dev) if (ws is None or ws.numel() < n.value) else ws
        if out is None:
            out = SearchResult(
                err=torch.empty(n_grid, dtype=torch.float32, device=dev),
                best_idx=torch.empty(1, dtype=torch.int32, device=dev),
                best_s=torch.empty(d_in, dtype=torch.float32, device=dev),
                clip=torch.empty(d_out, dtype=torch.float32, device=dev) if n_clip else None,
                clip_err=torch.empty((d_out, n_clip), dtype=torch.float32, device=dev)
                if (n_clip and want_clip_err) else None)
        self.out = out
        self._wptrs = (ctypes.c_void_p * len(parts))(*[p.data_ptr() for p in parts])
        self._rows = (ctypes.c_int64 * len(parts))(*[p.shape[0] for p in parts])
        self.grp = WGroup(len(parts), ctypes.cast(self._wptrs, ctypes.POINTER(ctypes.c_void_p)),
                          ctypes.cast(self._rows, ctypes.POINTER(ctypes.c_int64)))
        self._keep = (parts, x_mean, X)
        self._bind(ctypes.byref(self.cfg), ctypes.byref(self.grp), d_in, _ptr(x_mean), _ptr(X), xdt, T, ld,
                   _ptr(out.err), _ptr(out.best_idx), _ptr(out.best_s), _ptr(out.clip), _ptr(out.clip_err),
                   _ptr(self.ws), self.ws.numel(), _stream(stream))

    def run(self) -> SearchResult:
        self.launch()
        return self.out


def search_scales_noalloc(W_parts: Sequence[torch.Tensor], x_mean: torch.Tensor, out: SearchResult, *,
                          group_size: int = 128, n_grid: int = 20, s_min: float = 1e-4, duo: bool = False,
                          asym: bool = False, stream=None) -> SearchResult:
    """Weight-score search through awq_search_scales_noalloc: the library's own
    per-GPU scratch, no workspace, nothing allocated (the caller passes `out`).
    Calls that overlap on one GPU share that scratch and must not run concurrently."""
    parts: List[torch.Tensor] = list(W_parts)
    if not parts:
        raise ValueError("empty weight group")
    d_in = parts[0].shape[1]
    for p in parts:
        if p.dtype != torch.float16 or p.dim() != 2 or not p.is_contiguous() or p.shape[1] != d_in:
            raise ValueError("weights must be contiguous fp16 [rows, d_in] with one d_in")
        if p.device != parts[0].device:
            raise ValueError("the parts of a group must live on one device")
    _tensor(x_mean, "x_mean", torch.float32, (d_in,), like=parts[0])
    _tensor(out.err, "out.err", torch.float32, (n_grid,), like=parts[0])
    _tensor(out.best_idx, "out.best_idx", torch.int32, (1,), like=parts[0])
    _tensor(out.best_s, "out.best_s", torch.float32, (d_in,), like=parts[0])
    _dev(parts[0], "W")
    cfg = _cfg(group_size, n_grid, "weight", 0, 0.5, s_min, duo, asym)
    grp, keep = _wgroup(parts)
    _check(lib().awq_search_scales_noalloc(ctypes.byref(cfg), ctypes.byref(grp), d_in, _ptr(x_mean), _ptr(out.err),
                                           _ptr(out.best_idx), _ptr(out.best_s), _stream(stream)))
    return out


def search_scales(W_parts: Sequence[torch.Tensor], x_mean: torch.Tensor, **kw) -> SearchResult:
    """Grid search of alpha for one group of linears sharing an input (rows concatenated)."""
    return SearchPlan(W_parts, x_mean, **kw).run()


class PackPlan(_Prepared):
    """INT4 quantize + pack of W*s: qweight int32 [d_in, d_out/8], scales fp16 [d_in/G, d_out],
    qzeros int32 [d_in/G, d_out/8] (or None; always written for the asymmetric grid)."""
    _fn = "awq_quantize_pack"

    def __init__(self, W: torch.Tensor, group_size: int = 128, s: Optional[torch.Tensor] = None,
                 clip: Optional[torch.Tensor] = None, with_zeros: bool = True, out=None, stream=None,
                 asym: bool = False):
        if asym:
            self._fn = "awq_quantize_pack_asym"
            with_zeros = True
        _tensor(W, "W", torch.float16, (None, None))
        d_out, d_in = W.shape
        if group_size not in (32, 64, 128) or d_in % group_size or d_out % 8:
            raise ValueError(f"W [{d_out}, {d_in}]: need d_out % 8 == 0 and d_in a multiple of "
                             f"group_size in {{32, 64, 128}}, got {group_size}")
        _tensor(s, "s", torch.float32, (d_in,), like=W, optional=True)
        _tensor(clip, "clip", torch.float32, (d_out,), like=W, optional=True)
        if out is not None:
            qweight, scales, qzeros = out
            _tensor(qweight, "qweight", torch.int32, (d_in, d_out // 8), like=W)
            _tensor(scales, "scales", torch.float16, (d_in // group_size, d_out), like=W)
            _tensor(qzeros, "qzeros", torch.int32, (d_in // group_size, d_out // 8), like=W, optional=not asym)
        _dev(W, "W")
        if out is None:
            qweight = torch.empty((d_in, d_out // 8), dtype=torch.int32, device=W.device)
            scales = torch.empty((d_in // group_size, d_out), dtype=torch.float16, device=W.device)
            qzeros = torch.empty((d_in // group_size, d_out // 8), dtype=torch.int32, device=W.device) \
                if with_zeros else None
            out = (qweight, scales, qzeros)
        self.out = out
        self._keep = (W, s, clip)
        qweight, scales, qzeros = out
        self._bind(_ptr(W), d_out, d_in, group_size, _ptr(s), _ptr(clip), _ptr(qweight), _ptr(scales),
                   _ptr(qzeros), _stream(stream))

    def run(self):
        self.launch()
        return self.out


def quantize_pack(W: torch.Tensor, group_size: int = 128, s: Optional[torch.Tensor] = None,
                  clip: Optional[torch.Tensor] = None, with_zeros: bool = True, out=None, stream=None,
                  asym: bool = False):
    """Returns (qweight int32 [d_in, d_out/8], scales fp16 [d_in/G, d_out], qzeros int32 [d_in/G, d_out/8]);
    asym = True: the asymmetric grid with data zero points."""
    return PackPlan(W, group_size, s, clip, with_zeros, out, stream, asym).run()


class W4A16Plan(_Prepared):
    """Y [M, d_out] = X [M, d_in] (fp16, carrying the folded 1/s) times the
    dequantized packed weights, transposed (the decode GEMV)."""
    _fn = "awq_w4a16_matmul"

    def __init__(self, X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                 qzeros: Optional[torch.Tensor], d_out: int, group_size: int = 128, out_dtype=torch.float16,
                 out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
        _tensor(X, "X", torch.float16, (None, None), unit_col_stride=True)
        M, d_in, ld = _rows_view(X, "X")
        if group_size not in (32, 64, 128) or d_in % group_size or d_out % 8:
            raise ValueError(f"need d_out % 8 == 0 and d_in ({d_in}) a multiple of group_size in "
                             f"{{32, 64, 128}}, got d_out {d_out}, group_size {group_size}")
        _tensor(qweight, "qweight", torch.int32, (d_in, d_out // 8), like=X)
        _tensor(scales, "scales", torch.float16, (d_in // group_size, d_out), like=X)
        _tensor(qzeros, "qzeros", torch.int32, (d_in // group_size, d_out // 8), like=X, optional=True)
        if out is not None:
            _tensor(out, "out", (torch.float16, torch.float32), (M, d_out), unit_col_stride=True, like=X)
        _tensor(ws, "ws", torch.uint8, (None,), like=X, optional=True)
        _dev(X, "X")
        n = ctypes.c_size_t()
        _check(lib().awq_w4a16_workspace(M, d_out, d_in, ctypes.byref(n)))
        self.ws = workspace(n.value, X.device) if (ws is None or ws.numel() < n.value) else ws
        self.out = torch.empty((M, d_out), dtype=out_dtype, device=X.device) if out is None else out
        ydt = {torch.float32: AWQ_F32, torch.float16: AWQ_F16}[self.out.dtype]
        self._keep = (X, qweight, scales, qzeros)
        self._bind(_ptr(X), M, ld, _ptr(qweight), _ptr(scales), _ptr(qzeros), d_out, d_in, group_size,
                   _ptr(self.out), self.out.stride(0), ydt, _ptr(self.ws), self.ws.numel(), _stream(stream))

    def run(self) -> torch.Tensor:
        self.launch()
        return self.out


def w4a16_matmul(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, qzeros: Optional[torch.Tensor],
                 d_out: int, group_size: int = 128, out_dtype=torch.float16, stream=None) -> torch.Tensor:
    """Y = X W_hat^T on the packed layout (W_hat = (u - z) * scale in the stored domain)."""
    return W4A16Plan(X, qweight, scales, qzeros, d_out, group_size, out_dtype, stream=stream).run()


def unpack_dequant(qweight: torch.Tensor, scales: torch.Tensor, qzeros: Optional[torch.Tensor], d_out: int,
                   group_size: int = 128, s: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                   stream=None) -> torch.Tensor:
    _tensor(qweight, "qweight", torch.int32, (None, d_out // 8))
    d_in = qweight.shape[0]
    if group_size not in (32, 64, 128) or d_in % group_size or d_out % 8:
        raise ValueError(f"need d_out % 8 == 0 and d_in ({d_in}) a multiple of group_size in "
                         f"{{32, 64, 128}}, got d_out {d_out}, group_size {group_size}")
    _tensor(scales, "scales", torch.float16, (d_in // group_size, d_out), like=qweight)
    _tensor(qzeros, "qzeros", torch.int32, (d_in // group_size, d_out // 8), like=qweight, optional=True)
    _tensor(s, "s", torch.float32, (d_in,), like=qweight, optional=True)
    _dev(qweight, "qweight")
    out = torch.empty((d_out, d_in), dtype=out_dtype, device=qweight.device)
    odt = {torch.float32: AWQ_F32, torch.float16: AWQ_F16}[out_dtype]
    _check(lib().awq_unpack_dequant(_ptr(qweight), _ptr(scales), _ptr(qzeros), d_out, d_in, group_size, _ptr(s),
                                    _ptr(out), odt, _stream(stream)))
    return out


class FoldPlan(_Prepared):
    """Shared scale of a norm group (per-channel geometric mean of the members'
    scales) and the norm folded with it (norm / s_shared in the norm's dtype)."""
    _fn = "awq_norm_group_fold"

    def __init__(self, s_members: Sequence[torch.Tensor], norm: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, s_shared: Optional[torch.Tensor] = None, stream=None):
        members = list(s_members)
        if not members:
            raise ValueError("no member scales")
        d_in = members[0].numel()
        for t in members:
            _dev(t, "s")
            if t.dtype != torch.float32 or t.numel() != d_in or not t.is_contiguous():
                raise ValueError("member scales must be contiguous fp32 [d_in] with one d_in")
        dev = members[0].device
        ndt = 0
        if norm is not None:
            _dev(norm, "norm")
            if norm.numel() != d_in or not norm.is_contiguous():
                raise ValueError("norm must be contiguous [d_in]")
            ndt = {torch.float16: AWQ_F16, torch.bfloat16: AWQ_BF16, torch.float32: AWQ_F32}[norm.dtype]
            if out is None:
                out = torch.empty_like(norm)
        self.s_shared = torch.empty(d_in, dtype=torch.float32, device=dev) if s_shared is None else s_shared
        self.norm_out = out
        self._sptrs = (ctypes.c_void_p * len(members))(*[t.data_ptr() for t in members])
        self._keep = (members, norm)
        self._bind(ctypes.cast(self._sptrs, ctypes.POINTER(ctypes.c_void_p)), len(members), d_in, _ptr(norm), ndt,
                   _ptr(out), _ptr(self.s_shared), _stream(stream))

    def run(self):
        self.launch()
        return self.s_shared, self.norm_out


def norm_group_fold(s_members: Sequence[torch.Tensor], norm: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, s_shared: Optional[torch.Tensor] = None, stream=None):
    """Returns (s_shared fp32 [d_in], norm_out or None): the geometric mean of the
    member scales and norm / s_shared (out may be norm itself, in place)."""
    return FoldPlan(s_members, norm, out, s_shared, stream).run()


# ---------------------------------------------------------------------------
# Microscaled (MX) operators.  codes: float8_e4m3fn [rows, cols] ("fp8") or uint8
# [rows, cols / 2] with two 4-bit codes a byte ("fp4"); scales: float8_e8m0fnu
# [rows, cols / 32].  The plans run on the device that holds their tensors, and
# on the stream that is current in each run unless one is given.  A captured graph
# works on its plan's buffers: the plan stays as long as the graph.
# ---------------------------------------------------------------------------
_MX_FMT = {"fp8": AWQ_MX_FP8, "fp4": AWQ_MX_FP4}
_X16 = (torch.float16, torch.bfloat16)
_FLOATS = {torch.float16: AWQ_F16, torch.bfloat16: AWQ_BF16, torch.float32: AWQ_F32}


_raw_stream = torch._C._cuda_getCurrentRawStream   # handle of a device's current stream, without a Stream object


class _MxPrepared(_Prepared):
    """A prepared call on the device of `like`, made current around the launch when it is not: on the stream
    given, or else on the one that is current in every run, so that a plan built anywhere can be run under
    another stream or captured.  The arguments are kept as C values for a function without argument types,
    which spares their conversion in every run."""

    def _place(self, like: torch.Tensor, stream) -> int:
        self._device, self._index = like.device, like.device.index
        self._alone = torch.cuda.device_count() == 1
        self._follow = stream is None
        if stream is None:
            return torch.cuda.current_stream(like.device).cuda_stream
        if stream.device != like.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {like.device}")
        return stream.cuda_stream

    def _bind(self, *args) -> None:
        types = getattr(lib(), self._fn).argtypes
        if len(types) != len(args):
            raise TypeError(f"{self._fn} takes {len(types)} arguments, got {len(args)}")
        self._f = lib()[self._fn]
        self._f.restype = ctypes.c_int32
        self._bound = args[-1], tuple(t(a) for t, a in zip(types, args))     # the stream, which comes last, and all
        self._used = {args[-1]}

    def _follow_to(self, stream: int):
        """The current stream is another one than in the last run.  Memory that the plan allocated goes back to
        its pool only when that stream is done with it, too."""
        if stream not in self._used:
            self._used.add(stream)
            s = torch.cuda.current_stream(self._device)
            for t in self._mine:
                t.record_stream(s)
        self._bound = stream, (*self._bound[1][:-1], ctypes.c_void_p(stream))
        return self._bound

    def launch(self) -> None:
        at, args = self._bound
        if self._follow:
            stream = _raw_stream(self._index)
            if stream != at:
                at, args = self._follow_to(stream)
        if self._alone or torch.cuda.current_device() == self._index:
            st = self._f(*args)
        else:
            with torch.cuda.device(self._device):
                st = self._f(*args)
        if st != AWQ_OK:
            _check(st)


def _mx_alloc(stream):
    """Results and workspaces come from the memory pool of the stream that uses them: freed, they are
    handed out again in that stream's order."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _mx_fmt(fmt: str) -> int:
    if fmt not in _MX_FMT:
        raise ValueError(f"fmt {fmt!r} not in {sorted(_MX_FMT)}")
    return _MX_FMT[fmt]


def _mx_rows(t: torch.Tensor, name: str, dtype=_X16, shape=(None, None), like=None, optional=False) -> int:
    """Checks a 2-D operand with unit column stride; returns its row stride (at least a row)."""
    _tensor(t, name, dtype, shape, unit_col_stride=True, like=like, optional=optional)
    if t is None:
        return 0
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _mx_out(out, rows: int, cols: int, fmt: str, like: torch.Tensor):
    """Checks the shape of a quantized result, and `out` if given."""
    _mx_fmt(fmt)
    if cols % 32:
        raise ValueError(f"need columns in whole blocks of 32, got {cols}")
    if out is not None:
        codes, scales = out
        if fmt == "fp8":
            _tensor(codes, "codes", torch.float8_e4m3fn, (rows, cols), like=like)
        else:
            _tensor(codes, "codes", torch.uint8, (rows, cols // 2), like=like)
        _tensor(scales, "scales", torch.float8_e8m0fnu, (rows, cols // 32), like=like)


def _mx_empty(out, rows: int, cols: int, fmt: str, device, stream):
    if out is not None:
        return tuple(out)
    with _mx_alloc(stream):
        codes = (torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=device) if fmt == "fp8" else
                 torch.empty((rows, cols // 2), dtype=torch.uint8, device=device))
        return codes, torch.empty((rows, cols // 32), dtype=torch.float8_e8m0fnu, device=device)


def _mx_operand(codes: torch.Tensor, scales: torch.Tensor, name: str, like=None):
    """(fmt, rows, cols) of a quantized operand."""
    _tensor(codes, f"{name}codes", (torch.float8_e4m3fn, torch.uint8), (None, None), like=like)
    fmt = "fp8" if codes.dtype == torch.float8_e4m3fn else "fp4"
    rows, cols = codes.shape[0], codes.shape[1] * (1 if fmt == "fp8" else 2)
    if cols % 32:
        raise ValueError(f"{name}codes: need columns in whole blocks of 32, got {cols}")
    _tensor(scales, f"{name}scales", torch.float8_e8m0fnu, (rows, cols // 32), like=codes)
    return fmt, rows, cols


class MxQuantPlan(_MxPrepared):
    """codes, scales of X [rows, cols] (fp16 or bf16, rows any stride apart), or of X * s."""
    _fn = "awq_mx_quantize"

    def __init__(self, X: torch.Tensor, fmt: str = "fp8", s: Optional[torch.Tensor] = None, out=None, stream=None):
        ld = _mx_rows(X, "X")
        rows, cols = X.shape
        _tensor(s, "s", torch.float32, (cols,), like=X, optional=True)
        _mx_out(out, rows, cols, fmt, X)
        _dev(X, "X")
        self.out = _mx_empty(out, rows, cols, fmt, X.device, stream)
        self._mine = self.out if out is None else ()
        self._keep = (X, s)
        self._bind(_ptr(X), _FLOATS[X.dtype], rows, cols, ld, _ptr(s), _mx_fmt(fmt), _ptr(self.out[0]),
                   _ptr(self.out[1]), self._place(X, stream))

    def run(self):
        self.launch()
        return self.out


def mx_quantize(X: torch.Tensor, fmt: str = "fp8", s: Optional[torch.Tensor] = None, out=None, stream=None):
    """Returns (codes, scales) of X, or of X * s (s fp32 [cols], the AWQ scale of the input channels):
    blocks of 32 values sharing a power of two, elements e4m3 ("fp8") or e2m1 ("fp4")."""
    return MxQuantPlan(X, fmt, s, out, stream).run()


class MxDequantPlan(_MxPrepared):
    """The values of codes and scales [rows, cols], divided by s if given."""
    _fn = "awq_mx_dequant"

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, s: Optional[torch.Tensor] = None,
                 out_dtype=torch.float32, out: Optional[torch.Tensor] = None, stream=None):
        fmt, rows, cols = _mx_operand(codes, scales, "")
        _tensor(s, "s", torch.float32, (cols,), like=codes, optional=True)
        if out_dtype not in _FLOATS:
            raise ValueError(f"out_dtype must be one of {list(_FLOATS)}, got {out_dtype}")
        if out is not None:
            _mx_rows(out, "out", tuple(_FLOATS), (rows, cols), like=codes)
        _dev(codes, "codes")
        with _mx_alloc(stream):
            self.out = torch.empty((rows, cols), dtype=out_dtype, device=codes.device) if out is None else out
        ld = self.out.stride(0) if rows > 1 else max(self.out.stride(0), cols)
        self._mine = (self.out,) if out is None else ()
        self._keep = (codes, scales, s)
        self._bind(_ptr(codes), _ptr(scales), _MX_FMT[fmt], rows, cols, _ptr(s), _ptr(self.out),
                   _FLOATS[self.out.dtype], ld, self._place(codes, stream))

    def run(self) -> torch.Tensor:
        self.launch()
        return self.out


def mx_dequant(codes: torch.Tensor, scales: torch.Tensor, s: Optional[torch.Tensor] = None, out_dtype=torch.float32,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values that codes and scales stand for (divided by s if given): inverse of mx_quantize."""
    return MxDequantPlan(codes, scales, s, out_dtype, out, stream).run()


class RmsNormMxPlan(_MxPrepared):
    """h = X + residual; codes, scales of h / sqrt(mean h^2 + eps) * weight; residual_out = h in X's dtype.
    residual_out may be residual or X itself."""
    _fn = "awq_rms_norm_mx"

    def __init__(self, X: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None, fmt: str = "fp8",
                 residual_out: Optional[torch.Tensor] = None, out=None, stream=None):
        ld_x = _mx_rows(X, "X")
        rows, cols = X.shape
        _tensor(weight, "weight", tuple(_FLOATS), (cols,), like=X)
        ld_r = _mx_rows(residual, "residual", X.dtype, (rows, cols), like=X, optional=True)
        if residual is None and residual_out is not None:
            raise ValueError("residual_out without residual")
        ld_ro = _mx_rows(residual_out, "residual_out", X.dtype, (rows, cols), like=X, optional=True)
        _mx_out(out, rows, cols, fmt, X)
        _dev(X, "X")
        self._mine = ()
        if residual is not None and residual_out is None:
            with _mx_alloc(stream):
                residual_out = torch.empty((rows, cols), dtype=X.dtype, device=X.device)
            ld_ro = cols
            self._mine = (residual_out,)
        self.out = (*_mx_empty(out, rows, cols, fmt, X.device, stream), residual_out)
        if out is None:
            self._mine += self.out[:2]
        self._keep = (X, weight, residual)
        self._bind(_ptr(X), _FLOATS[X.dtype], rows, cols, ld_x, _ptr(residual), ld_r, _ptr(weight),
                   _FLOATS[weight.dtype], eps, _ptr(residual_out), ld_ro, _mx_fmt(fmt), _ptr(self.out[0]),
                   _ptr(self.out[1]), self._place(X, stream))

    def run(self):
        self.launch()
        return self.out


def rms_norm_mx(X: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                fmt: str = "fp8", residual_out: Optional[torch.Tensor] = None, out=None, stream=None):
    """Returns (codes, scales, residual_out): the RMS norm of h = X + residual, quantized, and h in X's
    dtype (None without a residual)."""
    return RmsNormMxPlan(X, weight, eps, residual, fmt, residual_out, out, stream).run()


class SiluMulMxPlan(_MxPrepared):
    """codes, scales of silu(gate) * up (fp16 or bf16 [rows, cols] each, rows any stride apart)."""
    _fn = "awq_silu_mul_mx"

    def __init__(self, gate: torch.Tensor, up: torch.Tensor, fmt: str = "fp8", out=None, stream=None):
        ld_g = _mx_rows(gate, "gate")
        rows, cols = gate.shape
        ld_u = _mx_rows(up, "up", gate.dtype, (rows, cols), like=gate)
        _mx_out(out, rows, cols, fmt, gate)
        _dev(gate, "gate")
        self.out = _mx_empty(out, rows, cols, fmt, gate.device, stream)
        self._mine = self.out if out is None else ()
        self._keep = (gate, up)
        self._bind(_ptr(gate), ld_g, _ptr(up), ld_u, _FLOATS[gate.dtype], rows, cols, _mx_fmt(fmt),
                   _ptr(self.out[0]), _ptr(self.out[1]), self._place(gate, stream))

    def run(self):
        self.launch()
        return self.out


def silu_mul_mx(gate: torch.Tensor, up: torch.Tensor, fmt: str = "fp8", out=None, stream=None):
    """Returns (codes, scales) of silu(gate) * up; gate and up may be the halves of one tensor's columns."""
    return SiluMulMxPlan(gate, up, fmt, out, stream).run()


def mx_matmul_workspace_bytes(fmt: str, M: int, N: int, K: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().awq_mx_matmul_workspace(_mx_fmt(fmt), M, N, K, ctypes.byref(n)))
    return n.value


class MxMatmulPlan(_MxPrepared):
    """Y [M, N] = A [M, K] W [N, K]^T from quantized operands: A "fp8" or "fp4", W "fp4"."""
    _fn = "awq_mx_matmul"

    def __init__(self, a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                 out_dtype=torch.float16, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None):
        fmt, M, K = _mx_operand(a_codes, a_scales, "a_")
        w_fmt, N, Kw = _mx_operand(w_codes, w_scales, "w_", like=a_codes)
        if w_fmt != "fp4":
            raise ValueError("w_codes must hold 4-bit codes (uint8)")
        if Kw != K:
            raise ValueError(f"a_codes have {K} columns, w_codes {Kw}")
        if out is not None:
            _mx_rows(out, "out", tuple(_FLOATS), (M, N), like=a_codes)
            out_dtype = out.dtype
        if out_dtype not in _FLOATS:
            raise ValueError(f"out_dtype must be one of {list(_FLOATS)}, got {out_dtype}")
        _tensor(ws, "ws", torch.uint8, (None,), like=a_codes, optional=True)
        _dev(a_codes, "a_codes")
        need = mx_matmul_workspace_bytes(fmt, M, N, K)
        with _mx_alloc(stream):
            self.ws = workspace(need, a_codes.device) if (ws is None or ws.numel() < need) else ws
            self.out = torch.empty((M, N), dtype=out_dtype, device=a_codes.device) if out is None else out
        self._mine = (() if self.ws is ws else (self.ws,)) + (() if out is not None else (self.out,))
        ld = self.out.stride(0) if M > 1 else max(self.out.stride(0), N)
        self._keep = (a_codes, a_scales, w_codes, w_scales)
        self._bind(_ptr(a_codes), _ptr(a_scales), _MX_FMT[fmt], M, _ptr(w_codes), _ptr(w_scales), N, K,
                   _ptr(self.out), ld, _FLOATS[self.out.dtype], _ptr(self.ws), self.ws.numel(),
                   self._place(a_codes, stream))

    def run(self) -> torch.Tensor:
        self.launch()
        return self.out


def mx_matmul(a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
              out_dtype=torch.float16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = A W^T of quantized A ("fp8" or "fp4" codes) and W ("fp4" codes), rounded once to out_dtype
    (float16, bfloat16, or float32 for 4-bit A)."""
    return MxMatmulPlan(a_codes, a_scales, w_codes, w_scales, out_dtype, out, stream=stream).run()


# ---------------------------------------------------------------------------
# A block with experts, and the linears and norms around it
# ---------------------------------------------------------------------------
_ACT = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def mx_linear_workspace_bytes(fmt: str, M: int, N: int, K: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().awq_mx_linear_workspace(_mx_fmt(fmt), M, N, K, ctypes.byref(n)))
    return n.value


class MxLinearPlan(_MxPrepared):
    """act(A W^T + bias) + residual from quantized operands (as MxMatmulPlan takes them), rounded once to out_dtype,
    or with fmt quantized to (codes, scales)."""
    _fn = "awq_mx_linear"

    def __init__(self, a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                 bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                 residual: Optional[torch.Tensor] = None, out_dtype=torch.float16, fmt: Optional[str] = None, out=None,
                 ws: Optional[torch.Tensor] = None, stream=None):
        a_fmt, M, K = _mx_operand(a_codes, a_scales, "a_")
        w_fmt, N, Kw = _mx_operand(w_codes, w_scales, "w_", like=a_codes)
        if w_fmt != "fp4":
            raise ValueError("w_codes must hold 4-bit codes (uint8)")
        if Kw != K:
            raise ValueError(f"a_codes have {K} columns, w_codes {Kw}")
        if activation not in _ACT:
            raise ValueError(f"activation {activation!r} not in {list(_ACT)}")
        _tensor(bias, "bias", tuple(_FLOATS), (N,), like=a_codes, optional=True)
        ld_r = _mx_rows(residual, "residual", tuple(_FLOATS), (M, N), like=a_codes, optional=True)
        if fmt is not None:
            _mx_out(out, M, N, fmt, a_codes)
        elif out is not None:
            _mx_rows(out, "out", tuple(_FLOATS), (M, N), like=a_codes)
            out_dtype = out.dtype
        if out_dtype not in _FLOATS:
            raise ValueError(f"out_dtype must be one of {list(_FLOATS)}, got {out_dtype}")
        _tensor(ws, "ws", torch.uint8, (None,), like=a_codes, optional=True)
        _dev(a_codes, "a_codes")
        need = mx_linear_workspace_bytes(a_fmt, M, N, K)
        y = codes = scales = None
        ld = N
        with _mx_alloc(stream):
            self.ws = workspace(need, a_codes.device) if (ws is None or ws.numel() < need) else ws
            if fmt is not None:
                self.out = codes, scales = _mx_empty(out, M, N, fmt, a_codes.device, stream)
            else:
                self.out = y = torch.empty((M, N), dtype=out_dtype, device=a_codes.device) if out is None else out
                ld = y.stride(0) if M > 1 else max(y.stride(0), N)
        self._mine = (() if self.ws is ws else (self.ws,))
        if out is None:
            self._mine += (y,) if fmt is None else (codes, scales)
        self._keep = (a_codes, a_scales, w_codes, w_scales, bias, residual)
        self._bind(_ptr(a_codes), _ptr(a_scales), _MX_FMT[a_fmt], M, _ptr(w_codes), _ptr(w_scales), N, K, _ptr(bias),
                   0 if bias is None else _FLOATS[bias.dtype], _ACT[activation], _ptr(residual),
                   0 if residual is None else _FLOATS[residual.dtype], ld_r, _ptr(y), ld, _FLOATS[out_dtype],
                   -1 if fmt is None else _mx_fmt(fmt), _ptr(codes), _ptr(scales), _ptr(self.ws), self.ws.numel(),
                   self._place(a_codes, stream))

    def run(self):
        self.launch()
        return self.out


def mx_linear(a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
              bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
              residual: Optional[torch.Tensor] = None, out_dtype=torch.float16, fmt: Optional[str] = None, out=None,
              stream=None):
    """act(A W^T + bias) + residual of quantized A and W: activation None, "relu", "silu", "gelu" or "gelu_tanh"; bias
    [N]; residual [M, N] (which may be `out`).  Rounded once to out_dtype, or with fmt "fp8" / "fp4" returned
    as (codes, scales), the operand of the next product."""
    return MxLinearPlan(a_codes, a_scales, w_codes, w_scales, bias, activation, residual, out_dtype, fmt, out,
                        stream=stream).run()


class MoeRouting(NamedTuple):
    experts: torch.Tensor   # int32 [T, top]: descending by logit, -1 where none is left
    weights: torch.Tensor   # fp32 [T, top]
    rows: torch.Tensor      # int32 [T * top]: the token of each place, -1 behind the last
    places: torch.Tensor    # int32 [T, top]: the place of each pair, -1 where experts is -1
    offsets: torch.Tensor   # int32 [n_experts + 1]: each expert's first place


class MoeRoutePlan(_MxPrepared):
    """The `top` experts of each token by its logits [T, n_experts] and their shares, and the (token, expert) pairs
    in expert order."""
    _fn = "awq_moe_route"

    def __init__(self, logits: torch.Tensor, top: int, renormalize: bool = True, scale: float = 1.0,
                 out: Optional[MoeRouting] = None, ws: Optional[torch.Tensor] = None, stream=None):
        ld = _mx_rows(logits, "logits", tuple(_FLOATS))
        T, n = logits.shape
        shapes = {"experts": (T, top), "weights": (T, top), "rows": (T * top,), "places": (T, top), "offsets": (n + 1,)}
        types = {k: torch.float32 if k == "weights" else torch.int32 for k in shapes}
        if not 1 <= top <= min(n, 32):
            raise ValueError(f"top must be in [1, min({n}, 32)], got {top}")
        if out is not None:
            for k, shape in shapes.items():
                _tensor(getattr(out, k), k, types[k], shape, like=logits)
        _tensor(ws, "ws", torch.uint8, (None,), like=logits, optional=True)
        _dev(logits, "logits")
        need = ctypes.c_size_t()
        _check(lib().awq_moe_route_workspace(T, n, ctypes.byref(need)))
        need = need.value
        with _mx_alloc(stream):
            self.ws = workspace(need, logits.device) if (ws is None or ws.numel() < need) else ws
            self.out = MoeRouting(**{k: torch.empty(shape, dtype=types[k], device=logits.device)
                                     for k, shape in shapes.items()}) if out is None else MoeRouting(*out)
        self._mine = (() if self.ws is ws else (self.ws,)) + (() if out is not None else tuple(self.out))
        self._keep = (logits,)
        self._bind(_ptr(logits), _FLOATS[logits.dtype], T, n, ld, top, int(renormalize), scale,
                   *(_ptr(t) for t in self.out), _ptr(self.ws), self.ws.numel(), self._place(logits, stream))

    def run(self) -> MoeRouting:
        self.launch()
        return self.out


def moe_route(logits: torch.Tensor, top: int, renormalize: bool = True, scale: float = 1.0,
              out: Optional[MoeRouting] = None, stream=None) -> MoeRouting:
    """(experts, weights, rows, places, offsets) of logits [T, n_experts]: each token's `top` largest (ties to the
    lower index, -inf never), the shares exp(l - max) / sum (over the chosen, or over all without renormalize)
    times scale, and the pairs in expert order for mx_matmul_grouped and block_norm_mx."""
    return MoeRoutePlan(logits, top, renormalize, scale, out, stream=stream).run()


def mx_matmul_grouped_workspace_bytes(fmt: str, M: int, N: int, K: int, n_groups: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().awq_mx_matmul_grouped_workspace(_mx_fmt(fmt), M, N, K, n_groups, ctypes.byref(n)))
    return n.value


class MxMatmulGroupedPlan(_MxPrepared):
    """Y [M, N]: rows [offsets[e], offsets[e + 1]) are A's rows (or those that `rows` names) times W[e]^T.  offsets
    and rows are read in each run."""
    _fn = "awq_mx_matmul_grouped"

    def __init__(self, a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                 offsets: torch.Tensor, rows: Optional[torch.Tensor] = None, out_dtype=torch.float16,
                 out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
        fmt, a_rows, K = _mx_operand(a_codes, a_scales, "a_")
        _tensor(w_codes, "w_codes", torch.uint8, (None, None, K // 2), like=a_codes)
        n_groups, N = w_codes.shape[:2]
        _tensor(w_scales, "w_scales", torch.float8_e8m0fnu, (n_groups, N, K // 32), like=a_codes)
        _tensor(offsets, "offsets", torch.int32, (n_groups + 1,), like=a_codes)
        _tensor(rows, "rows", torch.int32, (None,), like=a_codes, optional=True)
        M = a_rows if rows is None else rows.shape[0]
        if out is not None:
            _mx_rows(out, "out", tuple(_FLOATS), (M, N), like=a_codes)
            out_dtype = out.dtype
        if out_dtype not in _FLOATS:
            raise ValueError(f"out_dtype must be one of {list(_FLOATS)}, got {out_dtype}")
        _tensor(ws, "ws", torch.uint8, (None,), like=a_codes, optional=True)
        _dev(a_codes, "a_codes")
        need = mx_matmul_grouped_workspace_bytes(fmt, M, N, K, n_groups)
        with _mx_alloc(stream):
            self.ws = workspace(need, a_codes.device) if (ws is None or ws.numel() < need) else ws
            self.out = torch.empty((M, N), dtype=out_dtype, device=a_codes.device) if out is None else out
        self._mine = (() if self.ws is ws else (self.ws,)) + (() if out is not None else (self.out,))
        ld = self.out.stride(0) if M > 1 else max(self.out.stride(0), N)
        self._keep = (a_codes, a_scales, w_codes, w_scales, offsets, rows)
        self._bind(_ptr(a_codes), _ptr(a_scales), _MX_FMT[fmt], a_rows, _ptr(rows), M, _ptr(w_codes), _ptr(w_scales),
                   n_groups, N, K, _ptr(offsets), _ptr(self.out), ld, _FLOATS[self.out.dtype], _ptr(self.ws),
                   self.ws.numel(), self._place(a_codes, stream))

    def run(self) -> torch.Tensor:
        self.launch()
        return self.out


def mx_matmul_grouped(a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                      offsets: torch.Tensor, rows: Optional[torch.Tensor] = None, out_dtype=torch.float16,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y[m] = A[rows[m]] W[e]^T (A[m] without rows) for offsets[e] <= m < offsets[e + 1]: quantized A [*, K], W
    [n_groups, N, K] (mx_quantize of each matrix, stacked), offsets and rows as of moe_route.  Rows of `out` outside
    the groups are left as they were."""
    return MxMatmulGroupedPlan(a_codes, a_scales, w_codes, w_scales, offsets, rows, out_dtype, out,
                               stream=stream).run()


class BlockNormMxPlan(_MxPrepared):
    """y = X, or the sum of its rows places[t] weighted by shares[t]; h = residual_scale residual + gate norm(y) (the
    norm with post_weight, if given); codes, scales of h / sqrt(mean h^2 + eps) * weight; residual_out = h in X's
    dtype, which may be residual, or X itself without places."""
    _fn = "awq_block_norm_mx"

    def __init__(self, X: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                 residual_scale: float = 1.0, places: Optional[torch.Tensor] = None,
                 shares: Optional[torch.Tensor] = None, fmt: str = "fp8",
                 residual_out: Optional[torch.Tensor] = None, out=None, stream=None):
        ld_x = _mx_rows(X, "X")
        ld_r = _mx_rows(residual, "residual", X.dtype, (None, X.shape[1]), like=X)
        rows, cols = residual.shape
        if (places is None) != (shares is None):
            raise ValueError("places and shares go together")
        if places is None:
            _mx_rows(X, "X", X.dtype, (rows, cols))
        else:
            _tensor(places, "places", torch.int32, (rows, None), like=X)
            _tensor(shares, "shares", torch.float32, tuple(places.shape), like=X)
        _tensor(weight, "weight", tuple(_FLOATS), (cols,), like=X)
        _tensor(post_weight, "post_weight", tuple(_FLOATS), (cols,), like=X, optional=True)
        ld_g = 0
        if gate is not None and gate.dim() == 2 and not (rows > 0 and gate.stride(0) == 0 and gate.shape[0] == rows):
            ld_g = _mx_rows(gate, "gate", tuple(_FLOATS), (rows, cols), like=X)
        elif gate is not None and gate.dim() == 2:
            _tensor(gate[0], "gate", tuple(_FLOATS), (cols,), like=X)
        else:
            _tensor(gate, "gate", tuple(_FLOATS), (cols,), like=X, optional=True)
        ld_ro = _mx_rows(residual_out, "residual_out", X.dtype, (rows, cols), like=X, optional=True)
        _mx_out(out, rows, cols, fmt, X)
        _dev(X, "X")
        self._mine = ()
        if residual_out is None:
            with _mx_alloc(stream):
                residual_out = torch.empty((rows, cols), dtype=X.dtype, device=X.device)
            ld_ro = cols
            self._mine = (residual_out,)
        self.out = (*_mx_empty(out, rows, cols, fmt, X.device, stream), residual_out)
        if out is None:
            self._mine += self.out[:2]
        self._keep = (X, residual, weight, post_weight, gate, places, shares)
        dt = lambda t: 0 if t is None else _FLOATS[t.dtype]  # noqa: E731
        self._bind(_ptr(X), _FLOATS[X.dtype], X.shape[0], ld_x, _ptr(places), _ptr(shares),
                   0 if places is None else places.shape[1], rows, cols, _ptr(post_weight), dt(post_weight), _ptr(gate),
                   dt(gate), ld_g, _ptr(residual), ld_r, residual_scale, _ptr(weight), dt(weight), eps,
                   _ptr(residual_out), ld_ro, _mx_fmt(fmt), _ptr(self.out[0]), _ptr(self.out[1]),
                   self._place(X, stream))

    def run(self):
        self.launch()
        return self.out


def block_norm_mx(X: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                  post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  residual_scale: float = 1.0, places: Optional[torch.Tensor] = None,
                  shares: Optional[torch.Tensor] = None, fmt: str = "fp8", residual_out: Optional[torch.Tensor] = None,
                  out=None, stream=None):
    """Returns (codes, scales, residual_out): h = residual_scale * residual + gate * norm(y), with y = X or the sum of
    its rows places[t] weighted by shares[t] (places and weights of moe_route), the norm by post_weight (none
    without), gate [cols] or [rows, cols]; the RMS norm of h by weight, quantized; and h in X's dtype."""
    return BlockNormMxPlan(X, residual, weight, eps, post_weight, gate, residual_scale, places, shares, fmt,
                           residual_out, out, stream).run()


def set_timing_events(before: Optional[int], after: Optional[int]) -> None:
    """Record raw hipEvent_t handles around the main kernel of every later call (None clears)."""
    _check(lib().awq_set_timing_events(before, after))


__all__ = ["set_timing_events", "ActStatsPlan", "SearchPlan", "search_scales_noalloc", "PackPlan", "FoldPlan", "norm_group_fold",
           "weight_channel_mean", "candidate_scales_duo", "W4A16Plan", "w4a16_matmul", "AwqError", "act_stats", "candidate_scales", "search_scales", "quantize_pack", "unpack_dequant",
           "search_workspace_bytes", "act_stats_workspace_bytes", "SearchResult", "lib", "LIB_PATH",
           "MxQuantPlan", "mx_quantize", "MxDequantPlan", "mx_dequant", "RmsNormMxPlan", "rms_norm_mx",
           "SiluMulMxPlan", "silu_mul_mx", "MxMatmulPlan", "mx_matmul", "mx_matmul_workspace_bytes",
           "MxLinearPlan", "mx_linear", "mx_linear_workspace_bytes", "MoeRouting", "MoeRoutePlan", "moe_route",
           "MxMatmulGroupedPlan", "mx_matmul_grouped", "mx_matmul_grouped_workspace_bytes", "BlockNormMxPlan",
           "block_norm_mx"]
