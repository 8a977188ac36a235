"""Python binding of libqlin (include/qlin.h): argument marshalling only.

Every step of the computation runs in the HIP kernels behind the C ABI.
PyTorch supplies device memory and the current stream.  There is no fallback:
if libqlin.so is missing or the GPU is not gfx950, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import List, Optional, Sequence, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqlin.so")

FMT_PACKED = 0
FMT_FP16_MASTER = 1

STATUS_NAMES = {
    0: "QLIN_OK", 1: "QLIN_ERR_NULL", 2: "QLIN_ERR_SHAPE", 3: "QLIN_ERR_BITS",
    4: "QLIN_ERR_GROUP", 5: "QLIN_ERR_ALIGN", 6: "QLIN_ERR_FORMAT", 7: "QLIN_ERR_ALIAS",
    8: "QLIN_ERR_WORKSPACE", 9: "QLIN_ERR_NO_DEVICE", 10: "QLIN_ERR_HIP",
}

# Every symbol include/qlin.h declares.
EXPORTS = (
    "qlin_status_string", "qlin_last_hip_error", "qlin_abi_version", "qlin_packed_bytes",
    "qlin_meta_entries", "qlin_quantize", "qlin_gemv_workspace_bytes",
    "qlin_gemm_workspace_bytes", "qlin_gemv", "qlin_gemm",
    "qlin_gemv_multi_workspace_bytes", "qlin_gemv_multi",
    "qlin_gemv_swiglu_workspace_bytes", "qlin_gemv_swiglu", "qlin_embed_rows",
    "qlin_quantize_batch", "qlin_gemm_multi_workspace_bytes", "qlin_gemm_multi",
    "qlin_gemm_swiglu_workspace_bytes", "qlin_gemm_swiglu", "qlin_gemv_noalloc",
)
# include/qlin_tune.h (launch-shape sweeps and tests only)
TUNE_EXPORTS = ("qlin_set_launch_override",)
TUNE_FAMILIES = {"gemv": 0, "gemm": 1}
# include/qlin_rows.h (products whose weights differ from row to row)
ROWS_EXPORTS = (
    "qlin_route", "qlin_moe_mlp_workspace_bytes", "qlin_moe_mlp",
    "qlin_gemm_lora_workspace_bytes", "qlin_gemm_lora",
)
# include/qlin_kv.h (the cache of keys and values)
KV_EXPORTS = (
    "qlin_kv_page_bytes", "qlin_kv_write", "qlin_kv_read", "qlin_kv_attention_workspace_bytes",
    "qlin_kv_attention",
)
# include/qlin_sample.h (drawing tokens)
SAMPLE_EXPORTS = ("qlin_sample_workspace_bytes", "qlin_sample")


class QlinError(RuntimeError):
    def __init__(self, status: int, where: str, hip_error: int = 0):
        self.status = status
        self.hip_error = hip_error
        msg = f"{where}: {_lib().qlin_status_string(status).decode()}"
        if hip_error:
            msg += f" (hip error {hip_error})"
        super().__init__(msg)


class QlinWeightC(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("bits", ctypes.c_int32),
        ("group", ctypes.c_int32), ("format", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("data", ctypes.c_void_p), ("ld", ctypes.c_int64),
        ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p),
    ]


class QlinQuantJobC(ctypes.Structure):
    _fields_ = [
        ("w16", ctypes.c_void_p), ("ld_w", ctypes.c_int64), ("n", ctypes.c_int32),
        ("k", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("zero", ctypes.c_void_p),
    ]


class QlinRouterC(ctypes.Structure):
    _fields_ = [
        ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("score", ctypes.c_int32),
        ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
        ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("bias", ctypes.c_void_p),
    ]


class QlinAdaptersC(ctypes.Structure):
    _fields_ = [
        ("slots", ctypes.c_int32), ("rank", ctypes.c_int32), ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p),
    ]


class QlinKvCacheC(ctypes.Structure):
    _fields_ = [
        ("pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page", ctypes.c_int32), ("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32),
        ("data", ctypes.c_void_p),
    ]


class QlinKvSeqsC(ctypes.Structure):
    _fields_ = [
        ("seqs", ctypes.c_int32), ("width", ctypes.c_int32), ("table", ctypes.c_void_p),
        ("ld", ctypes.c_int64), ("lengths", ctypes.c_void_p),
    ]


class QlinSamplingC(ctypes.Structure):
    _fields_ = [
        ("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
        ("min_p", ctypes.c_void_p),
    ]


_LIB: Optional[ctypes.CDLL] = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libqlin.so not built at {LIB_PATH}; run "
                              "`python -m group_wise_bit_amd.build` (no CPU fallback exists)")
        lib = ctypes.CDLL(LIB_PATH)
        i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        wp = ctypes.POINTER(QlinWeightC)
        lib.qlin_status_string.argtypes = [ctypes.c_int]
        lib.qlin_status_string.restype = ctypes.c_char_p
        lib.qlin_last_hip_error.argtypes = []
        lib.qlin_last_hip_error.restype = ctypes.c_int
        lib.qlin_abi_version.argtypes = []
        lib.qlin_abi_version.restype = ctypes.c_int
        lib.qlin_packed_bytes.argtypes = [i32, i32, i32]
        lib.qlin_packed_bytes.restype = i64
        lib.qlin_meta_entries.argtypes = [i32, i32, i32]
        lib.qlin_meta_entries.restype = i64
        lib.qlin_quantize.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp]
        lib.qlin_quantize.restype = ctypes.c_int
        lib.qlin_gemv_workspace_bytes.argtypes = [wp]
        lib.qlin_gemv_workspace_bytes.restype = i64
        lib.qlin_gemm_workspace_bytes.argtypes = [wp, i32]
        lib.qlin_gemm_workspace_bytes.restype = i64
        lib.qlin_gemv.argtypes = [wp, vp, vp, vp, i64, vp]
        lib.qlin_gemv.restype = ctypes.c_int
        lib.qlin_gemm.argtypes = [wp, vp, i32, i64, vp, i64, vp, i64, vp]
        lib.qlin_gemm.restype = ctypes.c_int
        lib.qlin_gemv_multi_workspace_bytes.argtypes = [wp, i32]
        lib.qlin_gemv_multi_workspace_bytes.restype = i64
        lib.qlin_gemv_multi.argtypes = [wp, i32, vp, ctypes.POINTER(vp), vp, i64, vp]
        lib.qlin_gemv_multi.restype = ctypes.c_int
        lib.qlin_gemv_swiglu_workspace_bytes.argtypes = [wp]
        lib.qlin_gemv_swiglu_workspace_bytes.restype = i64
        lib.qlin_gemv_swiglu.argtypes = [wp, wp, vp, vp, vp, vp, i64, vp]
        lib.qlin_gemv_swiglu.restype = ctypes.c_int
        lib.qlin_embed_rows.argtypes = [wp, vp, i32, vp, vp, i64, vp]
        lib.qlin_embed_rows.restype = ctypes.c_int
        lib.qlin_quantize_batch.argtypes = [ctypes.POINTER(QlinQuantJobC), i32, i32, i32, vp]
        lib.qlin_quantize_batch.restype = ctypes.c_int
        lib.qlin_gemm_multi_workspace_bytes.argtypes = [wp, i32, i32]
        lib.qlin_gemm_multi_workspace_bytes.restype = i64
        lib.qlin_gemm_multi.argtypes = [wp, i32, vp, i32, i64, ctypes.POINTER(vp),
                                        ctypes.POINTER(i64), vp, i64, vp]
        lib.qlin_gemm_multi.restype = ctypes.c_int
        lib.qlin_gemm_swiglu_workspace_bytes.argtypes = [wp, i32]
        lib.qlin_gemm_swiglu_workspace_bytes.restype = i64
        lib.qlin_gemm_swiglu.argtypes = [wp, wp, vp, i32, i64, vp, vp, i64, vp, i64, vp]
        lib.qlin_gemm_swiglu.restype = ctypes.c_int
        lib.qlin_gemv_noalloc.argtypes = [wp, vp, vp, vp]
        lib.qlin_gemv_noalloc.restype = ctypes.c_int
        lib.qlin_set_launch_override.argtypes = [i32, ctypes.POINTER(i32)]
        lib.qlin_set_launch_override.restype = ctypes.c_int
        rp, ap = ctypes.POINTER(QlinRouterC), ctypes.POINTER(QlinAdaptersC)
        lib.qlin_route.argtypes = [rp, vp, i32, i64, vp, vp, vp]
        lib.qlin_route.restype = ctypes.c_int
        lib.qlin_moe_mlp_workspace_bytes.argtypes = [wp, wp, i32, i32, i32]
        lib.qlin_moe_mlp_workspace_bytes.restype = i64
        lib.qlin_moe_mlp.argtypes = [wp, wp, wp, i32, vp, i32, i64, vp, vp, i32, vp, vp, i64, vp,
                                     i64, vp]
        lib.qlin_moe_mlp.restype = ctypes.c_int
        lib.qlin_gemm_lora_workspace_bytes.argtypes = [wp, ap, i32]
        lib.qlin_gemm_lora_workspace_bytes.restype = i64
        lib.qlin_gemm_lora.argtypes = [wp, ap, vp, i32, i64, vp, vp, vp, i64, vp, i64, vp]
        lib.qlin_gemm_lora.restype = ctypes.c_int
        kp, sp = ctypes.POINTER(QlinKvCacheC), ctypes.POINTER(QlinKvSeqsC)
        lib.qlin_kv_page_bytes.argtypes = [i32, i32, i32, i32]
        lib.qlin_kv_page_bytes.restype = i64
        lib.qlin_kv_write.argtypes = [kp, vp, i64, vp, i64, i32, sp, vp, vp]
        lib.qlin_kv_write.restype = ctypes.c_int
        lib.qlin_kv_read.argtypes = [kp, sp, vp, i32, vp, i64, vp, i64, i32, vp]
        lib.qlin_kv_read.restype = ctypes.c_int
        lib.qlin_kv_attention_workspace_bytes.argtypes = [kp, sp, i32]
        lib.qlin_kv_attention_workspace_bytes.restype = i64
        lib.qlin_kv_attention.argtypes = [kp, sp, vp, i64, i32, ctypes.c_float, i32, vp, vp, i64, vp,
                                          vp, i64, vp]
        lib.qlin_kv_attention.restype = ctypes.c_int
        lib.qlin_sample_workspace_bytes.argtypes = [i32, i32]
        lib.qlin_sample_workspace_bytes.restype = i64
        lib.qlin_sample.argtypes = [ctypes.POINTER(QlinSamplingC), vp, i32, i32, i64, vp, vp, vp, vp,
                                    i64, vp]
        lib.qlin_sample.restype = ctypes.c_int
        _LIB = lib
    return _LIB


def library() -> ctypes.CDLL:
    """The loaded libqlin (raises ImportError when it is not built)."""
    return _lib()


def _check(status: int, where: str) -> None:
    if status != 0:
        raise QlinError(status, where, _lib().qlin_last_hip_error() if status == 10 else 0)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need_out(t: torch.Tensor, dtype: torch.dtype, device: torch.device, rows: int, cols: int,
              name: str) -> None:
    """An output the library writes (it cannot see buffer sizes): the right
    dtype, on the inputs' device, unit-stride rows, room for rows x cols
    (rows = 0: a vector of cols elements)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the inputs on {device}")
    if rows == 0:
        if not t.is_contiguous() or t.numel() < cols:
            raise ValueError(f"{name} must be contiguous with at least {cols} elements")
        return
    if t.dim() != 2 or t.stride(1) != 1 or t.shape[0] < rows or t.shape[1] < cols:
        raise ValueError(f"{name} must be 2-D [>= {rows}, >= {cols}] with contiguous rows, "
                         f"got shape {tuple(t.shape)} strides {t.stride()}")


def _need_x(w: "QWeight", x: torch.Tensor) -> None:
    if x.dtype != torch.float16 or x.numel() != w.k or not x.is_contiguous():
        raise TypeError(f"x must be a contiguous float16 tensor of k = {w.k} elements")


def set_launch_override(family: str, cfg=None) -> None:
    """qlin_set_launch_override (include/qlin_tune.h): force the launch shape of
    every later GEMV ("gemv": waves, splits[, rows]) or GEMM ("gemm": form,
    splits) call, or restore the library's own choice (cfg None).  cfg is a
    tuple or a "a,b[,c]" string.  For launch-shape sweeps and tests."""
    fam = TUNE_FAMILIES[family]
    if cfg is None:
        _check(_lib().qlin_set_launch_override(fam, None), "qlin_set_launch_override")
        return
    vals = [int(v) for v in cfg.split(",")] if isinstance(cfg, str) else [int(v) for v in cfg]
    if family == "gemv" and len(vals) == 2:
        vals.append(64)
    arr = (ctypes.c_int32 * 3)(*(vals + [0] * (3 - len(vals))))
    _check(_lib().qlin_set_launch_override(fam, arr), "qlin_set_launch_override")


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def packed_bytes(n: int, k: int, bits: int) -> int:
    return int(_lib().qlin_packed_bytes(n, k, bits))


def meta_entries(n: int, k: int, group: int) -> int:
    return int(_lib().qlin_meta_entries(n, k, group))


@dataclass
class QWeight:
    """A weight matrix for qlin_gemv / qlin_gemm (tensors stay owned here)."""
    n: int
    k: int
    bits: int
    group: int
    format: int
    data: torch.Tensor
    scale: Optional[torch.Tensor] = None
    zero: Optional[torch.Tensor] = None
    ld: int = 0

    def c_struct(self) -> QlinWeightC:
        return QlinWeightC(self.n, self.k, self.bits, self.group, self.format, 0,
                           _ptr(self.data), self.ld, _ptr(self.scale), _ptr(self.zero))

    @property
    def weight_bytes(self) -> int:
        """Bytes a matmul must read for this weight (codes or fp16 + metadata)."""
        b = self.data.numel() * self.data.element_size() if self.format == FMT_PACKED \
            else self.n * self.k * 2
        if self.bits != 16:
            b += self.scale.numel() * 2 + self.zero.numel()
        return b


def _check_room(cbuf, code_bytes, scale, zero, entries) -> None:
    """The output buffers must hold what the library writes (it cannot check)."""
    if cbuf is not None and cbuf.numel() * cbuf.element_size() < code_bytes:
        raise ValueError(f"codes buffer holds {cbuf.numel() * cbuf.element_size()} bytes, "
                         f"{code_bytes} needed")
    if scale.numel() < entries or zero.numel() < entries:
        raise ValueError(f"scale/zero buffers hold fewer than {entries} entries")


def quantize(w16: torch.Tensor, bits: int, group: int, codes: bool = True,
             out: Optional[QWeight] = None) -> QWeight:
    """qlin_quantize on a cuda fp16 [n, k] tensor -> packed QWeight (codes=False:
    scale/zero only, returned with the masters as an FP16_MASTER weight)."""
    if w16.dtype != torch.float16 or w16.dim() != 2 or not w16.is_cuda:
        raise TypeError("w16 must be a 2-D cuda float16 tensor")
    if w16.stride(1) != 1:
        raise ValueError("w16 rows must be contiguous")
    n, k = w16.shape
    g = k if group in ("k", "K") else int(group)
    me = meta_entries(n, k, g)
    pb = packed_bytes(n, k, bits)
    if out is None:
        scale = torch.empty(max(me, 1), dtype=torch.float16, device=w16.device)
        zero = torch.empty(max(me, 1), dtype=torch.uint8, device=w16.device)
        cbuf = torch.empty(max(pb // 4, 1), dtype=torch.int32, device=w16.device) if codes else None
    else:
        scale, zero, cbuf = out.scale, out.zero, (out.data if codes else None)
    _check_room(cbuf, pb, scale, zero, me)
    st = _lib().qlin_quantize(w16.data_ptr(), w16.stride(0), n, k, bits, g, _ptr(cbuf),
                              scale.data_ptr(), zero.data_ptr(), _stream())
    _check(st, "qlin_quantize")
    if codes:
        return QWeight(n, k, bits, g, FMT_PACKED, cbuf, scale, zero)
    return QWeight(n, k, bits, g, FMT_FP16_MASTER, w16, scale, zero, ld=w16.stride(0))


def master_weight(w16: torch.Tensor, bits: int, group: int, scale=None, zero=None) -> QWeight:
    """FP16_MASTER weight over existing masters (bits=16: the plain fp16 control)."""
    n, k = w16.shape
    g = k if group in ("k", "K") else int(group)
    return QWeight(n, k, bits, g, FMT_FP16_MASTER, w16, scale, zero, ld=w16.stride(0))


_WS: dict = {}
_WS_RECORDED: list = []       # buffers whose addresses a graph may hold: never freed


def workspace(nbytes: int, device: torch.device) -> Optional[torch.Tensor]:
    """Zero-filled workspace, cached per (device, stream); the kernels leave it
    zero-filled again after every call.  A buffer handed out under stream capture
    stays allocated when a larger one takes its place in the cache: the graph
    goes on writing to it."""
    if nbytes <= 0:
        return None
    key = (device.index, _stream())
    buf = _WS.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _WS[key] = buf
    if _capturing() and not any(b is buf for b in _WS_RECORDED):
        _WS_RECORDED.append(buf)
    return buf


def gemv(w: QWeight, x: torch.Tensor, y: Optional[torch.Tensor] = None,
         ws: Optional[torch.Tensor] = "auto") -> torch.Tensor:
    _need_x(w, x)
    if y is None:
        y = torch.empty(w.n, dtype=torch.float32, device=x.device)
    _need_out(y, torch.float32, x.device, 0, w.n, "y")
    ws_struct = w.c_struct()
    if isinstance(ws, str):
        need = int(_lib().qlin_gemv_workspace_bytes(ctypes.byref(ws_struct)))
        ws = workspace(need, x.device)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib().qlin_gemv(ctypes.byref(ws_struct), x.data_ptr(), y.data_ptr(), _ptr(ws), wsb,
                          _stream())
    _check(st, "qlin_gemv")
    return y


def gemv_noalloc(w: QWeight, x: torch.Tensor, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_gemv_noalloc: qlin_gemv with the library's static split-K scratch
    (no workspace, no allocation inside the library; y is allocated here only
    when not given)."""
    _need_x(w, x)
    if y is None:
        y = torch.empty(w.n, dtype=torch.float32, device=x.device)
    _need_out(y, torch.float32, x.device, 0, w.n, "y")
    ws_struct = w.c_struct()
    st = _lib().qlin_gemv_noalloc(ctypes.byref(ws_struct), x.data_ptr(), y.data_ptr(), _stream())
    _check(st, "qlin_gemv_noalloc")
    return y


def gemm(w: QWeight, X: torch.Tensor, Y: Optional[torch.Tensor] = None,
         ws: Optional[torch.Tensor] = "auto") -> torch.Tensor:
    if X.dtype != torch.float16 or X.dim() != 2 or X.shape[1] != w.k or X.stride(1) != 1:
        raise TypeError("X must be a float16 [m, k] tensor with contiguous rows")
    m = X.shape[0]
    if Y is None:
        Y = torch.empty(m, w.n, dtype=torch.float32, device=X.device)
    _need_out(Y, torch.float32, X.device, m, w.n, "Y")
    ws_struct = w.c_struct()
    if isinstance(ws, str):
        need = int(_lib().qlin_gemm_workspace_bytes(ctypes.byref(ws_struct), m))
        ws = workspace(need, X.device)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib().qlin_gemm(ctypes.byref(ws_struct), X.data_ptr(), m, X.stride(0), Y.data_ptr(),
                          Y.stride(0), _ptr(ws), wsb, _stream())
    _check(st, "qlin_gemm")
    return Y


def gemv_multi(ws_list: Sequence[QWeight], x: torch.Tensor,
               ys: Optional[Sequence[torch.Tensor]] = None,
               ws: Optional[torch.Tensor] = "auto") -> List[torch.Tensor]:
    """qlin_gemv_multi: y_i = W_i . x for up to 4 packed weights sharing x, one launch."""
    count = len(ws_list)
    for w in ws_list:
        _need_x(w, x)
    arr = (QlinWeightC * max(count, 1))(*[w.c_struct() for w in ws_list])
    if ys is None:
        ys = [torch.empty(w.n, dtype=torch.float32, device=x.device) for w in ws_list]
    if len(ys) != count:
        raise ValueError("one output per weight")
    for i, (w, y) in enumerate(zip(ws_list, ys)):
        _need_out(y, torch.float32, x.device, 0, w.n, f"ys[{i}]")
    yp = (ctypes.c_void_p * max(count, 1))(*[y.data_ptr() for y in ys])
    if isinstance(ws, str):
        need = int(_lib().qlin_gemv_multi_workspace_bytes(arr, count))
        ws = workspace(need, x.device)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib().qlin_gemv_multi(arr, count, x.data_ptr(), yp, _ptr(ws), wsb, _stream())
    _check(st, "qlin_gemv_multi")
    return list(ys)


def gemv_swiglu(gate: QWeight, up: QWeight, x: torch.Tensor,
                h: Optional[torch.Tensor] = None, h16: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = "auto", want_h: bool = True,
                want_h16: bool = True) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """qlin_gemv_swiglu: h = silu(gate . x) * (up . x), fp32 and/or fp16, one launch."""
    _need_x(gate, x)
    _need_x(up, x)
    if h is None and want_h:
        h = torch.empty(gate.n, dtype=torch.float32, device=x.device)
    if h16 is None and want_h16:
        h16 = torch.empty(gate.n, dtype=torch.float16, device=x.device)
    if h is not None:
        _need_out(h, torch.float32, x.device, 0, gate.n, "h")
    if h16 is not None:
        _need_out(h16, torch.float16, x.device, 0, gate.n, "h16")
    g, u = gate.c_struct(), up.c_struct()
    if isinstance(ws, str):
        need = int(_lib().qlin_gemv_swiglu_workspace_bytes(ctypes.byref(g)))
        ws = workspace(need, x.device)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib().qlin_gemv_swiglu(ctypes.byref(g), ctypes.byref(u), x.data_ptr(), _ptr(h),
                                 _ptr(h16), _ptr(ws), wsb, _stream())
    _check(st, "qlin_gemv_swiglu")
    return h, h16


def embed_rows(w: QWeight, ids: torch.Tensor, want16: bool = True, want32: bool = False
               ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """qlin_embed_rows: dequantized rows ids of a packed weight, fp16 and/or fp32 [len(ids), k]."""
    if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous():
        raise TypeError("ids must be a contiguous 1-D int32 tensor")
    count = ids.numel()
    out16 = torch.empty(count, w.k, dtype=torch.float16, device=ids.device) if want16 else None
    out32 = torch.empty(count, w.k, dtype=torch.float32, device=ids.device) if want32 else None
    ws_struct = w.c_struct()
    st = _lib().qlin_embed_rows(ctypes.byref(ws_struct), ids.data_ptr(), count, _ptr(out16),
                                _ptr(out32), w.k, _stream())
    _check(st, "qlin_embed_rows")
    return out16, out32


def quantize_batch(masters: Sequence[torch.Tensor], bits: int, group, codes: bool = True,
                   outs: Optional[Sequence[QWeight]] = None) -> List[QWeight]:
    """qlin_quantize_batch: every cuda fp16 [n, k] master quantized at one bit
    width, group 64 or "K" (per row), one launch per 64 matrices.  outs: the
    QWeights of an earlier call to overwrite (scale/zero, and codes)."""
    row = group in ("k", "K")
    if not row and int(group) != 64:
        raise ValueError("group must be 64 or 'K'")
    res, jobs = [], []
    for i, w16 in enumerate(masters):
        if w16.dtype != torch.float16 or w16.dim() != 2 or not w16.is_cuda or w16.stride(1) != 1:
            raise TypeError("masters must be 2-D cuda float16 tensors with contiguous rows")
        n, k = w16.shape
        g = k if row else 64
        me = meta_entries(n, k, g)
        if outs is not None:
            o = outs[i]
            scale, zero, cbuf = o.scale, o.zero, (o.data if codes else None)
            _check_room(cbuf, packed_bytes(n, k, bits), scale, zero, me)
        else:
            scale = torch.empty(max(me, 1), dtype=torch.float16, device=w16.device)
            zero = torch.empty(max(me, 1), dtype=torch.uint8, device=w16.device)
            cbuf = (torch.empty(max(packed_bytes(n, k, bits) // 4, 1), dtype=torch.int32,
                                device=w16.device) if codes else None)
        jobs.append(QlinQuantJobC(w16.data_ptr(), w16.stride(0), n, k, _ptr(cbuf),
                                  scale.data_ptr(), zero.data_ptr()))
        res.append(QWeight(n, k, bits, g, FMT_PACKED, cbuf, scale, zero) if codes else
                   QWeight(n, k, bits, g, FMT_FP16_MASTER, w16, scale, zero, ld=w16.stride(0)))
    arr = (QlinQuantJobC * max(len(jobs), 1))(*jobs)
    st = _lib().qlin_quantize_batch(arr, len(jobs), bits, 0 if row else 64, _stream())
    _check(st, "qlin_quantize_batch")
    return res


def gemm_multi(ws_list: Sequence[QWeight], X: torch.Tensor,
               Ys: Optional[Sequence[torch.Tensor]] = None,
               ws: Optional[torch.Tensor] = "auto") -> List[torch.Tensor]:
    """qlin_gemm_multi: Y_i = X . W_i^T for up to 4 packed weights sharing X, one launch."""
    if X.dtype != torch.float16 or X.dim() != 2 or X.stride(1) != 1:
        raise TypeError("X must be a float16 [m, k] tensor with contiguous rows")
    m, count = X.shape[0], len(ws_list)
    if Ys is None:
        Ys = [torch.empty(m, w.n, dtype=torch.float32, device=X.device) for w in ws_list]
    if len(Ys) != count:
        raise ValueError("one output per weight")
    for i, (w, Y) in enumerate(zip(ws_list, Ys)):
        if X.shape[1] != w.k:
            raise TypeError(f"X has {X.shape[1]} columns, weight {i} k = {w.k}")
        _need_out(Y, torch.float32, X.device, m, w.n, f"Ys[{i}]")
    arr = (QlinWeightC * max(count, 1))(*[w.c_struct() for w in ws_list])
    yp = (ctypes.c_void_p * max(count, 1))(*[y.data_ptr() for y in Ys])
    ld = (ctypes.c_int64 * max(count, 1))(*[y.stride(0) for y in Ys])
    if isinstance(ws, str):
        need = int(_lib().qlin_gemm_multi_workspace_bytes(arr, count, m))
        ws = workspace(need, X.device)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib().qlin_gemm_multi(arr, count, X.data_ptr(), m, X.stride(0), yp, ld, _ptr(ws), wsb,
                                _stream())
    _check(st, "qlin_gemm_multi")
    return list(Ys)


def gemm_swiglu(gate: QWeight, up: QWeight, X: torch.Tensor,
                H: Optional[torch.Tensor] = None, H16: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = "auto", want_h: bool = True,
                want_h16: bool = True) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """qlin_gemm_swiglu: H = silu(X . gate^T) * (X . up^T), fp32 and/or fp16 [m, n], one launch.
    H and H16, when both given, must share one row stride."""
    if X.dtype != torch.float16 or X.dim() != 2 or X.stride(1) != 1:
        raise TypeError("X must be a float16 [m, k] tensor with contiguous rows")
    m = X.shape[0]
    if H is None and want_h:
        H = torch.empty(m, gate.n, dtype=torch.float32, device=X.device)
    if H16 is None and want_h16:
        H16 = torch.empty(m, gate.n, dtype=torch.float16, device=X.device)
    if X.shape[1] != gate.k or X.shape[1] != up.k:
        raise TypeError("X must have k columns")
    if H is not None:
        _need_out(H, torch.float32, X.device, m, gate.n, "H")
    if H16 is not None:
        _need_out(H16, torch.float16, X.device, m, gate.n, "H16")
    outs = [t for t in (H, H16) if t is not None]
    ld = outs[0].stride(0) if outs else gate.n
    if any(t.stride(0) != ld for t in outs):
        raise ValueError("H and H16 must share one row stride")
    g, u = gate.c_struct(), up.c_struct()
    if isinstance(ws, str):
        need = int(_lib().qlin_gemm_swiglu_workspace_bytes(ctypes.byref(g), m))
        ws = workspace(need, X.device)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib().qlin_gemm_swiglu(ctypes.byref(g), ctypes.byref(u), X.data_ptr(), m, X.stride(0),
                                 _ptr(H), _ptr(H16), ld, _ptr(ws), wsb, _stream())
    _check(st, "qlin_gemm_swiglu")
    return H, H16


# ---------------------------------------- products whose weights differ by row
# (include/qlin_rows.h).  Every tensor of a call is on one device, and the
# kernels run on that device's current stream, whichever device is current.

def _same_device(dev: torch.device, named) -> None:
    for name, t in named:
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the inputs on {dev}")


# The current stream's handle, device and capture state without the wrappers (the
# object torch.cuda.current_stream() builds takes about 3 us of a call's 12, the
# initialization checks 1), where torch offers them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing",
                     torch.cuda.is_current_stream_capturing)


def _launch(dev: torch.device, call):
    """call(raw stream) with the tensors' device current and its current stream."""
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be on a GPU, not on {dev}")
    index = dev.index
    if index == _current_device():
        return call(_raw_stream(index))
    with torch.cuda.device(dev):
        return call(_raw_stream(index))


# Workspaces of the row-wise calls, by device and stream: apart from workspace()'s,
# whose users do not grow with a batch's rows and are recorded by graphs.
_ROWS_WS: dict = {}
# Held while a call is enqueued on such a buffer: its launches hand their results on in
# it, and another thread's call on the same stream must not come between them.
_ROWS_LOCK = threading.Lock()


def _with_workspace(ws, dev: torch.device, need, call, where: str) -> None:
    """call(workspace pointer, bytes, raw stream) with the caller's workspace or
    the device and stream's own (grown to need() bytes when the library finds
    it too small, before any launch).  Under stream capture a buffer of the
    graph's own memory: one that a later, larger call may replace must not be
    recorded."""
    def run(stream):
        if not isinstance(ws, str):
            if ws is None:
                return call(None, 0, stream)
            if ws.device != dev:
                raise ValueError(f"ws is on {ws.device}, the inputs on {dev}")
            if not ws.is_contiguous():
                raise ValueError("ws must be contiguous")
            return call(ws.data_ptr(), ws.numel() * ws.element_size(), stream)
        if _capturing():
            size = need()
            own = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
            return call(_ptr(own), size, stream)
        with _ROWS_LOCK:
            buf = _ROWS_WS.get((dev.index, stream))
            st = call(None, 0, stream) if buf is None else call(buf.data_ptr(), buf.numel(), stream)
            if st == 8:                       # QLIN_ERR_WORKSPACE
                buf = torch.empty(need(), dtype=torch.uint8, device=dev)
                _ROWS_WS[dev.index, stream] = buf
                st = call(buf.data_ptr(), buf.numel(), stream)
            return st
    _check(_launch(dev, run), where)


class _CStruct:
    """The ctypes form of an object of tensors, built and checked again whenever
    one of its tensors is at another address or of another shape, stride or type."""

    def _cached(self, tensors, extra, build):
        key = (*[None if t is None else (t.data_ptr(), t.shape, t.stride(), t.dtype)
                 for t in tensors], *extra)
        got = self.__dict__.get("_c")
        if got is None or got[0] != key:
            got = self.__dict__["_c"] = (key, build())
        return got[1]


def _need_rows_x(X: torch.Tensor, k: int) -> None:
    if not isinstance(X, torch.Tensor) or X.dtype != torch.float16 or X.dim() != 2 or \
            X.shape[1] != k or (X.shape[0] > 0 and X.stride(1) != 1):
        raise TypeError(f"X must be a float16 [m, {k}] tensor with contiguous rows")


def _row_pitch(t: torch.Tensor) -> int:
    """Elements from one row to the next (one row has no next: its own length)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _need_flat(t: torch.Tensor, dtype: torch.dtype, shape: Tuple[int, ...], name: str) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or \
            not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")


def _row_outputs(m: int, n: int, dev, Y, Y16, want_y: bool, want_y16: bool):
    """fp32 and fp16 [m, n] outputs of a row-wise product and their common row stride."""
    ld = n
    if Y is not None or Y16 is not None:
        given = [(t, dtype, name) for t, dtype, name in ((Y, torch.float32, "Y"),
                                                         (Y16, torch.float16, "Y16"))
                 if t is not None]
        for t, dtype, name in given:
            if m:
                _need_out(t, dtype, dev, m, n, name)
        if m > 1:
            ld = given[0][0].stride(0)
            if given[-1][0].stride(0) != ld or (len(given) < 2 and want_y and want_y16 and ld != n):
                raise ValueError("Y and Y16 must share one row stride")
    elif not want_y and not want_y16:
        raise ValueError("one of Y and Y16 must be wanted")
    if Y is None and want_y:
        Y = torch.empty(m, n, dtype=torch.float32, device=dev)
    if Y16 is None and want_y16:
        Y16 = torch.empty(m, n, dtype=torch.float16, device=dev)
    return Y, Y16, ld


@dataclass(eq=False)
class Router(_CStruct):
    """How route() turns logits into experts (qlin_router in qlin_rows.h)."""
    experts: int
    top_k: int
    score: str = "softmax"                # or "sigmoid"
    bias: Optional[torch.Tensor] = None   # fp32 [experts]: added for the choice only
    groups: int = 1
    top_groups: Optional[int] = None      # None: all groups
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0

    def c_struct(self) -> QlinRouterC:
        return self._cached((self.bias,), (self.experts, self.top_k, self.score, self.groups,
                                           self.top_groups, self.group_top, self.renormalize,
                                           self.scale), self._build)

    def _build(self) -> QlinRouterC:
        if self.score not in ("softmax", "sigmoid"):
            raise ValueError("score must be 'softmax' or 'sigmoid'")
        if self.bias is not None:
            _need_flat(self.bias, torch.float32, (self.experts,), "bias")
        return QlinRouterC(self.experts, self.top_k, int(self.score == "sigmoid"), self.groups,
                           self.groups if self.top_groups is None else self.top_groups,
                           self.group_top, int(bool(self.renormalize)), self.scale,
                           _ptr(self.bias))


def route(router: Router, logits: torch.Tensor, ids: Optional[torch.Tensor] = None,
          weights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """qlin_route: (ids int32, weights fp32), both [m, top_k], of fp32 logits [m, experts]."""
    experts = router.experts
    if not isinstance(logits, torch.Tensor) or logits.dtype != torch.float32 or \
            logits.dim() != 2 or logits.shape[1] != experts or \
            (experts > 1 and logits.shape[0] > 0 and logits.stride(1) != 1):
        raise TypeError(f"logits must be a float32 [m, {experts}] tensor with contiguous rows")
    m, dev = logits.shape[0], logits.device
    c = router.c_struct()
    if router.top_k < 1:
        raise ValueError("top_k must be at least 1")
    shape = (m, router.top_k)
    _same_device(dev, (("bias", router.bias), ("ids", ids), ("weights", weights)))
    if ids is None:
        ids = torch.empty(shape, dtype=torch.int32, device=dev)
    else:
        _need_flat(ids, torch.int32, shape, "ids")
    if weights is None:
        weights = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _need_flat(weights, torch.float32, shape, "weights")
    _check(_launch(dev, lambda stream: _lib().qlin_route(
        ctypes.byref(c), logits.data_ptr(), m, _row_pitch(logits), ids.data_ptr(),
        weights.data_ptr(), stream)), "qlin_route")
    return ids, weights


@dataclass(eq=False)
class QExperts(_CStruct):
    """A stack of packed weights of one shape, expert after expert (the layout
    qlin_moe_mlp takes): each tensor holds `count` times one QWeight's."""
    count: int
    n: int
    k: int
    bits: int
    group: int
    data: torch.Tensor
    scale: torch.Tensor
    zero: torch.Tensor

    def c_struct(self) -> QlinWeightC:
        return self._cached((self.data, self.scale, self.zero),
                            (self.count, self.n, self.k, self.bits, self.group), self._build)

    def _build(self) -> QlinWeightC:
        words = self.count * (packed_bytes(self.n, self.k, self.bits) // 4)
        entries = self.count * meta_entries(self.n, self.k, self.group)
        for t, dtype, size, name in ((self.data, torch.int32, words, "data"),
                                     (self.scale, torch.float16, entries, "scale"),
                                     (self.zero, torch.uint8, entries, "zero")):
            if t.dtype != dtype or not t.is_contiguous() or t.numel() < size or \
                    t.device != self.data.device:
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {size} "
                                 "elements on the codes' device")
        return QlinWeightC(self.n, self.k, self.bits, self.group, FMT_PACKED, 0,
                           self.data.data_ptr(), 0, self.scale.data_ptr(), self.zero.data_ptr())

    def expert(self, e: int) -> QWeight:
        """Expert e as a QWeight over the same memory."""
        if not 0 <= e < self.count:
            raise IndexError(f"expert {e} of {self.count}")
        w, s = packed_bytes(self.n, self.k, self.bits) // 4, meta_entries(self.n, self.k, self.group)
        return QWeight(self.n, self.k, self.bits, self.group, FMT_PACKED,
                       self.data.reshape(-1)[e * w:(e + 1) * w],
                       self.scale.reshape(-1)[e * s:(e + 1) * s],
                       self.zero.reshape(-1)[e * s:(e + 1) * s])


def quantize_experts(w16: torch.Tensor, bits: int, group) -> QExperts:
    """qlin_quantize_batch of fp16 masters [count, n, k] into one stack."""
    if w16.dim() != 3 or w16.shape[0] < 1:
        raise TypeError("w16 must be a float16 [count, n, k] tensor")
    count, n, k = w16.shape
    g = k if group in ("k", "K") else int(group)
    words, entries = packed_bytes(n, k, bits) // 4, meta_entries(n, k, g)
    if not words or not entries:
        raise ValueError(f"no packed layout for n = {n}, k = {k}, bits = {bits}, group = {group}")
    dev = w16.device
    q = QExperts(count, n, k, bits, g, torch.empty(count * words, dtype=torch.int32, device=dev),
                 torch.empty(count * entries, dtype=torch.float16, device=dev),
                 torch.empty(count * entries, dtype=torch.uint8, device=dev))
    _launch(dev, lambda stream: quantize_batch(
        [w16[e] for e in range(count)], bits, "K" if g != 64 else 64,
        outs=[q.expert(e) for e in range(count)]))
    return q


def moe_mlp(gate: QExperts, up: QExperts, down: QExperts, X: torch.Tensor, ids: torch.Tensor,
            weights: torch.Tensor, Y: Optional[torch.Tensor] = None,
            Y16: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = "auto",
            want_y: bool = True, want_y16: bool = True
            ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """qlin_moe_mlp: Y[i] = sum_j weights[i, j] * down_e(silu(gate_e x_i) * up_e x_i), e =
    ids[i, j]; fp32 and / or fp16 [m, n].  ids and weights [m, top_k] as route() gives them."""
    _need_rows_x(X, gate.k)
    m, dev = X.shape[0], X.device
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise TypeError("ids must be a contiguous torch.int32 [m, top_k] tensor")
    top_k = ids.shape[1]
    _need_flat(ids, torch.int32, (m, top_k), "ids")
    _need_flat(weights, torch.float32, (m, top_k), "weights")
    if not gate.count == up.count == down.count:
        raise ValueError("gate, up and down must hold the same number of experts")
    _same_device(dev, (("gate", gate.data), ("up", up.data), ("down", down.data), ("ids", ids),
                       ("weights", weights)))
    Y, Y16, ld = _row_outputs(m, down.n, dev, Y, Y16, want_y, want_y16)
    g, u, d = (ctypes.byref(w.c_struct()) for w in (gate, up, down))
    lib = _lib()
    _with_workspace(
        ws, dev, lambda: lib.qlin_moe_mlp_workspace_bytes(g, d, gate.count, m, top_k),
        lambda wp, wb, stream: lib.qlin_moe_mlp(
            g, u, d, gate.count, X.data_ptr(), m, _row_pitch(X), ids.data_ptr(),
            weights.data_ptr(), top_k, _ptr(Y), _ptr(Y16), ld, wp, wb, stream), "qlin_moe_mlp")
    return Y, Y16


@dataclass(eq=False)
class Adapters(_CStruct):
    """A pool of low-rank adapters of one projection: a fp16 [slots, rank, k],
    b fp16 [slots, n, rank], scale fp32 [slots] or None (all 1)."""
    a: torch.Tensor
    b: torch.Tensor
    scale: Optional[torch.Tensor] = None

    def c_struct(self, w: "QWeight") -> QlinAdaptersC:
        return self._cached((self.a, self.b, self.scale), (w.n, w.k), lambda: self._build(w))

    def _build(self, w: "QWeight") -> QlinAdaptersC:
        if self.a.dim() != 3:
            raise TypeError("a must be a contiguous torch.float16 [slots, rank, k] tensor")
        slots, rank = self.a.shape[0], self.a.shape[1]
        _need_flat(self.a, torch.float16, (slots, rank, w.k), "a")
        _need_flat(self.b, torch.float16, (slots, w.n, rank), "b")
        if self.scale is not None:
            _need_flat(self.scale, torch.float32, (slots,), "scale")
        return QlinAdaptersC(slots, rank, self.a.data_ptr(), self.b.data_ptr(), _ptr(self.scale))


def gemm_lora(w: QWeight, X: torch.Tensor, adapters: Adapters, ids: torch.Tensor,
              Y: Optional[torch.Tensor] = None, Y16: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = "auto", want_y: bool = True, want_y16: bool = True
              ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """qlin_gemm_lora: Y[i] = W x_i + scale[a] * B_a (A_a x_i), a = ids[i] (W x_i alone where
    ids[i] is no slot); fp32 and / or fp16 [m, n]."""
    _need_rows_x(X, w.k)
    m, dev = X.shape[0], X.device
    _need_flat(ids, torch.int32, (m,), "ids")
    ad = adapters.c_struct(w)
    _same_device(dev, (("w", w.data), ("a", adapters.a), ("b", adapters.b),
                       ("scale", adapters.scale), ("ids", ids)))
    Y, Y16, ld = _row_outputs(m, w.n, dev, Y, Y16, want_y, want_y16)
    c, a = ctypes.byref(w.c_struct()), ctypes.byref(ad)
    lib = _lib()
    _with_workspace(
        ws, dev, lambda: lib.qlin_gemm_lora_workspace_bytes(c, a, m),
        lambda wp, wb, stream: lib.qlin_gemm_lora(
            c, a, X.data_ptr(), m, _row_pitch(X), ids.data_ptr(), _ptr(Y), _ptr(Y16), ld, wp, wb,
            stream), "qlin_gemm_lora")
    return Y, Y16


# ------------------------------------------------ the cache of keys and values
# (include/qlin_kv.h).  Devices and streams as for the row-wise calls.

def kv_page_bytes(head_dim: int, page_size: int, k_bits: int, v_bits: int) -> int:
    """Bytes of one page of one head."""
    return int(_lib().qlin_kv_page_bytes(head_dim, page_size, k_bits, v_bits))


@dataclass(eq=False)
class KVCache(_CStruct):
    """A layer's cache: pages of `page_size` tokens of keys and values in groups of 64 with
    k_bits and v_bits (4, 8, or 16: not quantized), each on its own.  data uint8 [pages, kv_heads,
    kv_page_bytes(...)], contiguous; copying a page copies its tokens."""
    data: torch.Tensor
    kv_heads: int
    head_dim: int
    page_size: int = 64
    k_bits: int = 8
    v_bits: int = 8

    def c_struct(self) -> QlinKvCacheC:
        return self._cached((self.data,), (self.kv_heads, self.head_dim, self.page_size,
                                           self.k_bits, self.v_bits), self._build)

    def _build(self) -> QlinKvCacheC:
        size = kv_page_bytes(self.head_dim, self.page_size, self.k_bits, self.v_bits)
        if not size:
            raise ValueError(f"no cache layout for head_dim = {self.head_dim}, page_size = "
                             f"{self.page_size}, k_bits = {self.k_bits}, v_bits = {self.v_bits}")
        if self.data.dim() != 3:
            raise TypeError("data must be a contiguous torch.uint8 [pages, kv_heads, bytes] tensor")
        _need_flat(self.data, torch.uint8, (self.data.shape[0], self.kv_heads, size), "data")
        return QlinKvCacheC(self.data.shape[0], self.kv_heads, self.head_dim, self.page_size,
                            self.k_bits, self.v_bits, self.data.data_ptr())


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, k_bits: int = 8,
             v_bits: int = 8, device="cuda") -> KVCache:
    """An empty cache (no page needs initialization: what is not written is not read)."""
    size = kv_page_bytes(head_dim, page_size, k_bits, v_bits)
    if not size:
        raise ValueError(f"no cache layout for head_dim = {head_dim}, page_size = {page_size}, "
                         f"k_bits = {k_bits}, v_bits = {v_bits}")
    return KVCache(torch.empty(pages, kv_heads, size, dtype=torch.uint8, device=device), kv_heads,
                   head_dim, page_size, k_bits, v_bits)


def _kv_seqs(cache: KVCache, table: torch.Tensor, lengths: torch.Tensor,
             starts: Optional[torch.Tensor]) -> QlinKvSeqsC:
    shape = table.shape if isinstance(table, torch.Tensor) and table.dtype is torch.int32 else ()
    if len(shape) != 2:
        raise TypeError("table must be an int32 [seqs, pages per sequence] tensor with contiguous "
                        "rows")
    seqs, width = shape
    ld, step = table.stride()
    if seqs > 0 and width > 1 and step != 1:
        raise TypeError("table's rows must be contiguous")
    _need_flat(lengths, torch.int32, (seqs,), "lengths")
    dev = cache.data.device
    if starts is not None:
        _need_flat(starts, torch.int32, (seqs + 1,), "starts")
    if table.device != dev or lengths.device != dev or \
            (starts is not None and starts.device != dev):
        _same_device(dev, (("table", table), ("lengths", lengths), ("starts", starts)))
    return QlinKvSeqsC(seqs, width, table.data_ptr(), ld if seqs > 1 else width, lengths.data_ptr())


def _kv_rows(t: torch.Tensor, dtype: torch.dtype, heads: int, head_dim: int, name: str) -> int:
    """The pitch of [m, heads, head_dim] rows, whose heads follow one another."""
    shape = t.shape if isinstance(t, torch.Tensor) and t.dtype is dtype else ()
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim:
        raise TypeError(f"{name} must be a {dtype} [rows, {heads}, {head_dim}] tensor")
    if shape[0] == 0:
        return heads * head_dim
    pitch, head, one = t.stride()
    if one != 1 or (head != head_dim and heads > 1):
        raise ValueError(f"{name}'s rows must be contiguous, got strides {t.stride()}")
    return pitch if shape[0] > 1 else heads * head_dim


def kv_write(cache: KVCache, K: torch.Tensor, V: torch.Tensor, table: torch.Tensor,
             lengths: torch.Tensor, starts: Optional[torch.Tensor] = None) -> None:
    """qlin_kv_write: rows starts[b] .. starts[b + 1] - 1 of K and V (fp16 [m, kv_heads, head_dim])
    become the last tokens of sequence b; without starts row b is the last token of sequence b.
    lengths counts them already."""
    c = cache.c_struct()
    s = _kv_seqs(cache, table, lengths, starts)
    ldk = _kv_rows(K, torch.float16, cache.kv_heads, cache.head_dim, "K")
    ldv = _kv_rows(V, torch.float16, cache.kv_heads, cache.head_dim, "V")
    m, dev = K.shape[0], cache.data.device
    if V.shape[0] != m:
        raise ValueError(f"K has {m} rows, V {V.shape[0]}")
    if K.device != dev or V.device != dev:
        _same_device(dev, (("K", K), ("V", V)))
    _check(_launch(dev, lambda stream: _lib().qlin_kv_write(
        c, K.data_ptr(), ldk, V.data_ptr(), ldv, m, s, _ptr(starts), stream)), "qlin_kv_write")


def kv_read(cache: KVCache, table: torch.Tensor, lengths: torch.Tensor,
            starts: Optional[torch.Tensor] = None, rows: Optional[int] = None,
            K: Optional[torch.Tensor] = None, V: Optional[torch.Tensor] = None,
            dtype: torch.dtype = torch.float16) -> Tuple[torch.Tensor, torch.Tensor]:
    """qlin_kv_read: the last starts[b + 1] - starts[b] tokens of every sequence b as rows
    starts[b] on of K and V ([rows, kv_heads, head_dim], fp16 or fp32); without starts row b is the
    last token of sequence b.  rows: how many K and V have where they are not given (default: one
    per sequence); rows from starts[-1] on are not written."""
    c = cache.c_struct()
    s = _kv_seqs(cache, table, lengths, starts)
    h, d, dev = cache.kv_heads, cache.head_dim, cache.data.device
    if dtype not in (torch.float16, torch.float32):
        raise TypeError("dtype must be torch.float16 or torch.float32")
    if rows is None:
        given = next((t for t in (K, V) if t is not None), None)
        if given is None and starts is not None:
            raise ValueError("rows must be given along with starts, unless K or V is")
        rows = s.seqs if given is None else given.shape[0]
    if K is None:
        K = torch.empty(rows, h, d, dtype=dtype, device=dev)
    if V is None:
        V = torch.empty(rows, h, d, dtype=dtype, device=dev)
    ldk, ldv = _kv_rows(K, dtype, h, d, "K"), _kv_rows(V, dtype, h, d, "V")
    if K.shape[0] < rows or V.shape[0] < rows:
        raise ValueError(f"K and V must have {rows} rows")
    if K.device != dev or V.device != dev:
        _same_device(dev, (("K", K), ("V", V)))
    _check(_launch(dev, lambda stream: _lib().qlin_kv_read(
        c, s, _ptr(starts), rows, K.data_ptr(), ldk, V.data_ptr(), ldv, int(dtype is torch.float32),
        stream)), "qlin_kv_read")
    return K, V


def kv_attention(cache: KVCache, Q: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                 scale: Optional[float] = None, window: int = 0,
                 O: Optional[torch.Tensor] = None, O16: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = "auto",
                 want_o: bool = True, want_o16: bool = True, want_lse: bool = False
                 ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """qlin_kv_attention: (O fp32, O16 fp16, lse fp32) of one query row per sequence (Q fp16 [seqs,
    heads, head_dim]) over its cached tokens, the last `window` of them if that is not 0; scale is
    1 / sqrt(head_dim) by default."""
    c = cache.c_struct()
    s = _kv_seqs(cache, table, lengths, None)
    d, dev, seqs = cache.head_dim, cache.data.device, s.seqs
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3:
        raise TypeError(f"Q must be a {torch.float16} [seqs, heads, {d}] tensor")
    heads = Q.shape[1]
    ldq = _kv_rows(Q, torch.float16, heads, d, "Q")
    if Q.shape[0] != seqs:
        raise ValueError(f"Q has {Q.shape[0]} rows for {seqs} sequences")
    if O is None and want_o:
        O = torch.empty(seqs, heads, d, dtype=torch.float32, device=dev)
    if O16 is None and want_o16:
        O16 = torch.empty(seqs, heads, d, dtype=torch.float16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty(seqs, heads, dtype=torch.float32, device=dev)
    ldo = ldo16 = None
    if O is not None:
        ldo = _kv_rows(O, torch.float32, heads, d, "O")
    if O16 is not None:
        ldo16 = _kv_rows(O16, torch.float16, heads, d, "O16")
    for t, name in ((O, "O"), (O16, "O16")):
        if t is not None and (t.shape[0] != seqs or t.device != dev):
            _same_device(dev, ((name, t),))
            raise ValueError(f"{name} has {t.shape[0]} rows for {seqs} sequences")
    if ldo is None:
        ldo = heads * d if ldo16 is None else ldo16
    elif ldo16 is not None and ldo16 != ldo:
        raise ValueError("O and O16 must share one row stride")
    if lse is not None:
        _need_flat(lse, torch.float32, (seqs, heads), "lse")
        _same_device(dev, (("lse", lse),))
    if Q.device != dev:
        _same_device(dev, (("Q", Q),))
    if scale is None:
        scale = d ** -0.5
    if not 0 <= window < 1 << 31:            # (ctypes would cut it to 32 bits)
        raise ValueError(f"window must be from 0 to 2^31 - 1, got {window}")
    lib = _lib()
    _with_workspace(
        ws, dev, lambda: lib.qlin_kv_attention_workspace_bytes(c, s, heads),
        lambda wp, wb, stream: lib.qlin_kv_attention(
            c, s, Q.data_ptr(), ldq, heads, scale, window, _ptr(O), _ptr(O16), ldo, _ptr(lse), wp,
            wb, stream), "qlin_kv_attention")
    return O, O16, lse


# ------------------------------------------------------------- drawing a token
# (include/qlin_sample.h).  Devices and streams as for the row-wise calls.

@dataclass(eq=False)
class Sampling(_CStruct):
    """How sample() draws, one setting per row (None: off for all): temperature fp32 [m] (not above
    0: the first of the largest), top_k int32 [m] (below 1: off), top_p fp32 [m] (not below 1: off)
    and min_p fp32 [m] (not above 0: off; above 1: one token)."""
    temperature: Optional[torch.Tensor] = None
    top_k: Optional[torch.Tensor] = None
    top_p: Optional[torch.Tensor] = None
    min_p: Optional[torch.Tensor] = None

    def c_struct(self, m: int) -> QlinSamplingC:
        return self._cached((self.temperature, self.top_k, self.top_p, self.min_p), (m,),
                            lambda: self._build(m))

    def _build(self, m: int) -> QlinSamplingC:
        for t, dtype, name in ((self.temperature, torch.float32, "temperature"),
                               (self.top_k, torch.int32, "top_k"),
                               (self.top_p, torch.float32, "top_p"),
                               (self.min_p, torch.float32, "min_p")):
            if t is not None:
                _need_flat(t, dtype, (m,), name)
        return QlinSamplingC(_ptr(self.temperature), _ptr(self.top_k), _ptr(self.top_p),
                             _ptr(self.min_p))


def sample(sampling: Sampling, logits: torch.Tensor, u: torch.Tensor,
           ids: Optional[torch.Tensor] = None, probs: Optional[torch.Tensor] = None,
           ws: Optional[torch.Tensor] = "auto") -> Tuple[torch.Tensor, torch.Tensor]:
    """qlin_sample: (ids int32 [m], probs fp32 [m]) of fp32 logits [m, vocab] and u fp32 [m] in
    [0, 1): the token that u falls on among the kept ones, and its probability among them."""
    if not isinstance(logits, torch.Tensor) or logits.dtype != torch.float32 or \
            logits.dim() != 2 or \
            (logits.shape[1] > 1 and logits.shape[0] > 0 and logits.stride(1) != 1):
        raise TypeError("logits must be a float32 [m, vocab] tensor with contiguous rows")
    m, vocab = logits.shape
    dev = logits.device
    c = ctypes.byref(sampling.c_struct(m))
    _need_flat(u, torch.float32, (m,), "u")
    if ids is None:
        ids = torch.empty(m, dtype=torch.int32, device=dev)
    else:
        _need_flat(ids, torch.int32, (m,), "ids")
    if probs is None:
        probs = torch.empty(m, dtype=torch.float32, device=dev)
    else:
        _need_flat(probs, torch.float32, (m,), "probs")
    _same_device(dev, (("temperature", sampling.temperature), ("top_k", sampling.top_k),
                       ("top_p", sampling.top_p), ("min_p", sampling.min_p), ("u", u),
                       ("ids", ids), ("probs", probs)))
    lib = _lib()
    _with_workspace(
        ws, dev, lambda: lib.qlin_sample_workspace_bytes(m, vocab),
        lambda wp, wb, stream: lib.qlin_sample(
            c, logits.data_ptr(), m, vocab, _row_pitch(logits), u.data_ptr(), ids.data_ptr(),
            probs.data_ptr(), wp, wb, stream), "qlin_sample")
    return ids, probs
