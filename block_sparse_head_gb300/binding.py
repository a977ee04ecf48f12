"""ctypes binding of libbsa (include/bsa.h): argument marshalling only.

Every step of the forward runs inside the library's CUDA kernel; torch supplies device
memory and streams.  Calls fail loudly (``BsaError``) when the library is missing or
a call returns an error; there is no fallback path.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))

BSA_ORDER_GLOBAL = 0
BSA_ORDER_GROUPED = 1
_ORDERS = {"global": BSA_ORDER_GLOBAL, "grouped": BSA_ORDER_GROUPED,
           BSA_ORDER_GLOBAL: BSA_ORDER_GLOBAL, BSA_ORDER_GROUPED: BSA_ORDER_GROUPED}

BSA_ERR_DEVICE_TIMEOUT = -8

# Every symbol declared in include/bsa.h.
EXPORTED = (
    "bsa_build_lut", "bsa_lut_info", "bsa_lut_export", "bsa_lut_schedule", "bsa_lut_upload",
    "bsa_lut_free",
    "bsa_forward", "bsa_device_status", "bsa_set_schedule", "bsa_set_wait_limit",
    "bsa_wait_selftest",
    "bsa_status_string", "bsa_version", "bsa_forward_noalloc", "bsa_debug_expire_wait",
    "bsa_build_lut_rect", "bsa_lut_kv_blocks", "bsa_forward_ext", "bsa_lut_export_csc",
    "bsa_backward", "bsa_topk_forward", "bsa_cache_resize", "bsa_cache_append",
    "bsa_cache_forward", "bsa_cache_workspace", "bsa_diff_forward", "bsa_diff_backward",
    "bsa_diff_workspace", "bsa_cache_diff_forward", "bsa_rotary_table", "bsa_rotary",
)

_ACTIVATIONS = {torch.bfloat16: 0, torch.float16: 1}          # BSA_BF16, BSA_FP16
_CACHE_TYPES = {torch.float8_e4m3fn: 2, torch.int8: 3}        # BSA_E4M3, BSA_INT8


class ExtArgs(ctypes.Structure):
    """bsa_ext_args of include/bsa.h."""
    _fields_ = [("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
                ("softcap", ctypes.c_float), ("sinks", ctypes.c_void_p),
                ("q_segment_ids", ctypes.c_void_p), ("kv_segment_ids", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()


class BsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        text = _lib.bsa_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{what}: {text} ({status})")


def library_path() -> str:
    return os.path.join(_HERE, "libbsa.so")


def load_library():
    """Load libbsa.so (built by ``block_sparse_head_gb300.build``) and declare its ABI."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m block_sparse_head_gb300.build` "
                "(the CUDA path has no fallback)")
        lib = ctypes.CDLL(path)
        i32p = ctypes.POINTER(ctypes.c_int32)
        ip = ctypes.POINTER(ctypes.c_int)
        vp = ctypes.c_void_p
        lib.bsa_build_lut.argtypes = [vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.POINTER(vp)]
        lib.bsa_build_lut_rect.argtypes = [vp, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
        lib.bsa_lut_kv_blocks.argtypes = [vp, ip]
        lib.bsa_forward_ext.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.POINTER(ExtArgs), vp]
        lib.bsa_topk_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_float, vp]
        ci, i64 = ctypes.c_int, ctypes.c_int64
        lib.bsa_cache_resize.argtypes = [vp] * 10 + [ci] * 5 + [vp]
        lib.bsa_cache_append.argtypes = [vp, vp, vp, vp, ci, ci, i64, i64, i64,
                                         i64, vp]
        lib.bsa_cache_forward.argtypes = [vp] + [vp] * 8 + [i64] + [ci] * 6 + \
            [i64, i64, ctypes.c_float, vp, vp]
        lib.bsa_cache_diff_forward.argtypes = [vp] * 10 + [i64] + [ci] * 8 + \
            [i64, i64, ctypes.c_float, vp, vp]
        lib.bsa_cache_workspace.argtypes = [ci, ci, ci, ci, ctypes.POINTER(i64)]
        lib.bsa_diff_forward.argtypes = [vp] * 8 + [ci] * 7 + [ctypes.c_float, ci, ci, vp]
        lib.bsa_diff_backward.argtypes = [vp] * 14 + [i64] + [ci] * 7 + [ctypes.c_float, ci, ci, vp]
        lib.bsa_diff_workspace.argtypes = [ci] * 5 + [ctypes.POINTER(i64)]
        lib.bsa_rotary_table.argtypes = [vp, vp, ci, vp]
        lib.bsa_rotary.argtypes = [vp, vp]
        lib.bsa_lut_export_csc.argtypes = [vp, vp, vp, vp]
        lib.bsa_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                                     ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                     ctypes.c_int, ctypes.c_int, vp]
        lib.bsa_lut_info.argtypes = [vp, ip, ip, ip, ip, ip]
        lib.bsa_lut_export.argtypes = [vp, vp, vp, vp]
        lib.bsa_lut_schedule.argtypes = [vp, ctypes.c_int, ctypes.c_int, vp, vp]
        lib.bsa_lut_upload.argtypes = [vp, vp]
        lib.bsa_lut_free.argtypes = [vp]
        lib.bsa_lut_free.restype = None
        lib.bsa_forward.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_int,
                                    ctypes.c_int, vp]
        lib.bsa_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                            ctypes.c_int, ctypes.c_int, vp, ctypes.c_int]
        lib.bsa_forward_noalloc.restype = ctypes.c_int
        lib.bsa_device_status.argtypes = [vp, vp, i32p]
        lib.bsa_set_wait_limit.argtypes = [vp, ctypes.c_uint64]
        lib.bsa_set_schedule.argtypes = [vp, ctypes.c_int]
        lib.bsa_debug_expire_wait.argtypes = [vp, ctypes.c_int]
        lib.bsa_wait_selftest.argtypes = [ctypes.c_uint64, vp]
        lib.bsa_status_string.argtypes = [ctypes.c_int]
        lib.bsa_status_string.restype = ctypes.c_char_p
        lib.bsa_version.argtypes = []
        lib.bsa_version.restype = ctypes.c_char_p
        for name in ("bsa_build_lut", "bsa_lut_info", "bsa_lut_export", "bsa_lut_schedule",
                     "bsa_lut_upload",
                     "bsa_forward", "bsa_device_status", "bsa_set_schedule", "bsa_set_wait_limit",
                     "bsa_wait_selftest", "bsa_debug_expire_wait", "bsa_build_lut_rect",
                     "bsa_lut_kv_blocks", "bsa_forward_ext", "bsa_lut_export_csc",
                     "bsa_backward", "bsa_topk_forward", "bsa_cache_resize", "bsa_cache_append",
                     "bsa_cache_forward", "bsa_cache_workspace", "bsa_diff_forward",
                     "bsa_diff_backward", "bsa_diff_workspace", "bsa_cache_diff_forward",
                     "bsa_rotary_table", "bsa_rotary"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _check(status: int, what: str) -> None:
    if status != 0:
        raise BsaError(status, what)


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


class Lut:
    """A built look-up table (CSR of active column blocks + work list)."""

    def __init__(self, layout, batch: int, order="global"):
        lib = load_library()
        lay = layout.detach().cpu().numpy() if isinstance(layout, torch.Tensor) else np.asarray(layout)
        if lay.ndim != 3:
            raise ValueError(f"layout must be [H, nb, nbk], got {lay.shape}")
        lay = np.ascontiguousarray(lay.astype(np.int32, copy=False))
        self._lib = lib
        self.handle = ctypes.c_void_p()
        if lay.shape[1] == lay.shape[2]:
            _check(lib.bsa_build_lut(lay.ctypes.data, lay.shape[0], lay.shape[1], int(batch),
                                     _ORDERS[order], ctypes.byref(self.handle)), "bsa_build_lut")
        else:
            _check(lib.bsa_build_lut_rect(lay.ctypes.data, lay.shape[0], lay.shape[1],
                                          lay.shape[2], int(batch), _ORDERS[order],
                                          ctypes.byref(self.handle)), "bsa_build_lut_rect")
        H, nb, b, nnz, n, nbk = (ctypes.c_int() for _ in range(6))
        _check(lib.bsa_lut_info(self.handle, *(ctypes.byref(x) for x in (H, nb, b, nnz, n))),
               "bsa_lut_info")
        _check(lib.bsa_lut_kv_blocks(self.handle, ctypes.byref(nbk)), "bsa_lut_kv_blocks")
        self.H, self.nb, self.batch, self.nbk = H.value, nb.value, b.value, nbk.value
        self.nnz_total, self.n_items = nnz.value, n.value
        self.device = None

    def export(self):
        """(row_ptr [H*nb+1], col_idx [nnz], items [n_items, 4]) as int32 numpy arrays."""
        rp = np.empty(self.H * self.nb + 1, np.int32)
        ci = np.empty(max(self.nnz_total, 1), np.int32)
        it = np.empty((self.n_items, 4), np.int32)
        _check(self._lib.bsa_lut_export(self.handle, rp.ctypes.data, ci.ctypes.data, it.ctypes.data),
               "bsa_lut_export")
        return rp, ci[:self.nnz_total], it

    def export_csc(self):
        """(col_ptr [H*nb+1], row_idx [nnz], items [n_items, 4]) of the column view."""
        cp = np.empty(self.H * self.nb + 1, np.int32)
        ri = np.empty(max(self.nnz_total, 1), np.int32)
        it = np.empty((self.n_items, 4), np.int32)
        _check(self._lib.bsa_lut_export_csc(self.handle, cp.ctypes.data, ri.ctypes.data,
                                            it.ctypes.data), "bsa_lut_export_csc")
        return cp, ri[:self.nnz_total], it

    def schedule(self, grid: int, by_head: bool = False):
        """(items [n_items, 4], cta_start [grid + 1]) of the per-CTA schedule for ``grid``
        CTAs: CTA c runs items[cta_start[c]:cta_start[c + 1]].  ``by_head`` hands the items
        out (batch, head) by (batch, head) instead of in work-list order."""
        it = np.empty((max(self.n_items, 1), 4), np.int32)
        cs = np.empty(int(grid) + 1, np.int32)
        _check(self._lib.bsa_lut_schedule(self.handle, int(grid), int(bool(by_head)),
                                          it.ctypes.data, cs.ctypes.data), "bsa_lut_schedule")
        return it[:self.n_items], cs

    def upload(self, stream=None):
        _check(self._lib.bsa_lut_upload(self.handle, _stream_handle(stream)), "bsa_lut_upload")
        self.device = torch.cuda.current_device()
        return self

    _SCHEDULES = {"auto": 0, "list": 1, "by_head": 2}

    def set_schedule(self, policy: str = "auto"):
        """Device schedule of later forwards: "auto", "list" or "by_head"."""
        _check(self._lib.bsa_set_schedule(self.handle, self._SCHEDULES[policy]), "bsa_set_schedule")

    def set_wait_limit(self, ns: int):
        _check(self._lib.bsa_set_wait_limit(self.handle, int(ns)), "bsa_set_wait_limit")

    def debug_expire_wait(self, site: int):
        """Test knob: later forwards (cache_forward with this layout too) treat every wait at
        ``site`` as run out (0: off)."""
        _check(self._lib.bsa_debug_expire_wait(self.handle, int(site)), "bsa_debug_expire_wait")

    def device_status(self, stream=None) -> tuple[int, int]:
        """(status, raw word) of the device status word; synchronizes the stream."""
        word = ctypes.c_int32(0)
        st = self._lib.bsa_device_status(self.handle, _stream_handle(stream), ctypes.byref(word))
        return st, word.value

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self._lib.bsa_lut_free(h)
            self.handle = None


def build_lut(layout, batch: int, order="global", upload: bool | None = None, stream=None) -> Lut:
    """Build the LUT on the host; upload it to the current CUDA device when one exists
    (or when ``upload`` is True)."""
    lut = Lut(layout, batch, order)
    if upload is None:
        upload = torch.cuda.is_available()
    if upload:
        lut.upload(stream)
    return lut


def _check_qkv(t: torch.Tensor, name: str, shape) -> None:
    if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lut: Lut, scale: float,
            block: int, causal_diag: bool, out: torch.Tensor | None = None,
            lse: torch.Tensor | None = None, stream=None):
    """Block-sparse attention forward.  q, k, v: bf16 [B, H, L, d] on the LUT's device.
    Returns (out bf16 [B, H, L, d], lse fp32 [B, H, L])."""
    lib = load_library()
    B, H, L, d = q.shape
    _check_qkv(q, "q", (B, H, L, d))
    _check_qkv(k, "k", (B, H, L, d))
    _check_qkv(v, "v", (B, H, L, d))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, H, L, device=q.device, dtype=torch.float32)
    _check_qkv(out, "out", (B, H, L, d))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, L) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, L] tensor")
    _check(lib.bsa_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), lut.handle, out.data_ptr(),
                           lse.data_ptr(), B, H, L, d, float(scale), int(block), int(bool(causal_diag)),
                           _stream_handle(stream)), "bsa_forward")
    return out, lse


def forward_ext(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lut: Lut, scale: float,
                q_block: int, kv_block: int, causal_diag: bool, window=None, softcap: float = 0.0,
                sinks: torch.Tensor | None = None, q_segment_ids: torch.Tensor | None = None,
                kv_segment_ids: torch.Tensor | None = None, out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, stream=None):
    """Extended forward (bsa_forward_ext): q [B,H,Lq,d], k/v [B,H,Lk,d] bf16; ``window``
    an int (both sides) or a (left, right) pair (None or negative: no bound); ``sinks``
    fp32 [H]; segment ids int32 [B,Lq] / [B,Lk].  Returns (out [B,H,Lq,d], lse [B,H,Lq])."""
    lib = load_library()
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    _check_qkv(q, "q", (B, H, Lq, d))
    _check_qkv(k, "k", (B, H, Lk, d))
    _check_qkv(v, "v", (B, H, Lk, d))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, H, Lq, device=q.device, dtype=torch.float32)
    _check_qkv(out, "out", (B, H, Lq, d))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Lq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, Lq] tensor")
    if window is None:
        wl = wr = -1
    elif isinstance(window, int):
        wl = wr = window
    else:
        wl, wr = (-1 if w is None else int(w) for w in window)

    def dev_arr(t, dtype, shape, name):
        if t is None:
            return None
        if not t.is_cuda or t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != shape:
            raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {shape}")
        return t.data_ptr()

    x = ExtArgs(wl, wr, float(softcap), dev_arr(sinks, torch.float32, (H,), "sinks"),
                dev_arr(q_segment_ids, torch.int32, (B, Lq), "q_segment_ids"),
                dev_arr(kv_segment_ids, torch.int32, (B, Lk), "kv_segment_ids"))
    _check(lib.bsa_forward_ext(q.data_ptr(), k.data_ptr(), v.data_ptr(), lut.handle,
                               out.data_ptr(), lse.data_ptr(), B, H, Lq, Lk, d, float(scale),
                               int(q_block), int(kv_block), int(bool(causal_diag)),
                               ctypes.byref(x), _stream_handle(stream)), "bsa_forward_ext")
    return out, lse


def backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
             lse: torch.Tensor, dout: torch.Tensor, lut: Lut, scale: float, block: int,
             causal_diag: bool, dq=None, dk=None, dv=None, delta=None, stream=None):
    """Gradients (dq, dk, dv) of the forward (bsa_backward).  q, k, v, out, dout: bf16
    [B, H, L, d] on the LUT's device; lse fp32 [B, H, L] from the forward.  ``delta`` is
    an fp32 [B, H, L] workspace (allocated when None)."""
    lib = load_library()
    B, H, L, d = q.shape
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _check_qkv(t, name, (B, H, L, d))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, L) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, L] tensor")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for t, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check_qkv(t, name, (B, H, L, d))
    if delta is None:
        delta = torch.empty(B, H, L, device=q.device, dtype=torch.float32)
    _check(lib.bsa_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            lse.data_ptr(), dout.data_ptr(), lut.handle, dq.data_ptr(),
                            dk.data_ptr(), dv.data_ptr(), delta.data_ptr(), B, H, L, d,
                            float(scale), int(block), int(bool(causal_diag)),
                            _stream_handle(stream)), "bsa_backward")
    return dq, dk, dv


def topk_forward(q: torch.Tensor, kv: torch.Tensor, sink: torch.Tensor, idx: torch.Tensor,
                 scale: float, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 status: torch.Tensor | None = None, stream=None):
    """Top-k token-gather attention with a sink (bsa_topk_forward).  q bf16 [B, M, H, D],
    kv bf16 [B, N, D], sink fp32 [H], idx int32 [B, M, K] (-1: unused).  Returns
    (out bf16 [B, M, H, D], lse fp32 [B, M, H], status int32 [1]); a nonzero status
    (read after the stream is synchronized) means a bounded wait gave up."""
    lib = load_library()
    B, M, H, D = q.shape
    N, K = kv.shape[1], idx.shape[2]
    _check_qkv(q, "q", (B, M, H, D))
    _check_qkv(kv, "kv", (B, N, D))
    if not sink.is_cuda or sink.dtype != torch.float32 or tuple(sink.shape) != (H,):
        raise ValueError("sink must be a CUDA fp32 tensor of shape [H]")
    if not idx.is_cuda or idx.dtype != torch.int32 or not idx.is_contiguous() or idx.shape[:2] != (B, M):
        raise ValueError("idx must be a contiguous CUDA int32 tensor [B, M, K]")
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, M, H, device=q.device, dtype=torch.float32) if lse is None else lse
    status = torch.zeros(4, device=q.device, dtype=torch.int32) if status is None else status
    _check_qkv(out, "out", (B, M, H, D))
    _check(lib.bsa_topk_forward(q.data_ptr(), kv.data_ptr(), sink.contiguous().data_ptr(),
                                idx.data_ptr(), out.data_ptr(), lse.data_ptr(), status.data_ptr(),
                                B, M, N, H, D, K, float(scale), _stream_handle(stream)),
           "bsa_topk_forward")
    return out, lse, status


# Raw handle of the current stream of a device: torch.cuda.current_stream() builds an object
# for it, which takes longer than all the other checks of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

_CACHE = struct.Struct("@4P5i4x")        # bsa_cache
_CACHE_ARGS = struct.Struct("@ifPPi4x")  # bsa_cache_args


def _this_device(t, name: str) -> int:
    """Index of the current device, which the cache calls launch on; t has to be there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = torch.cuda.current_device()
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    return dev


# torch.cuda.current_device() without its look whether CUDA has been initialised: the callers have
# a tensor there.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_of(t, name: str) -> int:
    """_this_device for the calls whose host time counts most."""
    if isinstance(t, torch.Tensor):
        dev = t.get_device()
        if dev >= 0 and dev == _current_device():
            return dev
    return _this_device(t, name)


def _dev_ptr(t, name: str, dtype, shape, dev: int) -> int:
    """Pointer of a contiguous tensor of this type and shape on device dev."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor
        pass
    if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}")


def _rows_ptr(t, name: str, heads: int | None, d: int, dev: int):
    """Pointer and (token, head) strides of a [T, heads, d] activation tensor whose numbers
    of one head are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _ACTIVATIONS or t.dim() != 3 or \
            t.shape[2] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be a bf16 or fp16 CUDA tensor [T, heads, {d}]")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    token, head, one = t.stride()
    if one != 1 and t.numel() > 0:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # The stride of a dimension of one is never used, whatever the tensor says.
    return t.data_ptr(), token if t.shape[0] > 1 else 0, head if t.shape[1] > 1 else 0


_HERE_AND_NOW = contextlib.nullcontext()


def _on(stream):
    """Context in which a call allocates what the caller did not give it: memory of the
    stream that the call runs on, so that neither earlier nor later work of the current
    stream touches it meanwhile."""
    if stream is None:
        return _HERE_AND_NOW
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _cache_view(k_cache, v_cache, k_scale, v_scale):
    """(device, bsa_cache as bytes, kv_heads, d)."""
    dev = _device_of(k_cache, "k_cache")
    kind = _CACHE_TYPES.get(k_cache.dtype)
    if kind is None or k_cache.dim() != 4:
        raise ValueError("k_cache must be float8_e4m3fn or int8 [pages, kv_heads, page, d]")
    shape = k_cache.shape
    pages, heads, page, d = shape
    return dev, _CACHE.pack(
        _dev_ptr(k_cache, "k_cache", k_cache.dtype, shape, dev),
        _dev_ptr(v_cache, "v_cache", k_cache.dtype, shape, dev),
        _dev_ptr(k_scale, "k_scale", torch.float32, (pages, heads), dev),
        _dev_ptr(v_scale, "v_scale", torch.float32, (pages, heads), dev),
        pages, heads, page, d, kind), heads, d


def _cache_stream(stream, dev: int):
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream_handle(stream)


def cache_resize(block_table: torch.Tensor, kv_len: torch.Tensor, new_len: torch.Tensor,
                 free_pages: torch.Tensor, free_count: torch.Tensor, page: int, tokens: int,
                 kv_len_out: torch.Tensor | None = None, free_count_out: torch.Tensor | None = None,
                 cu_new: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                 status: torch.Tensor | None = None, stream=None):
    """Block tables and slots from request lengths (bsa_cache_resize).  int32 on the current
    device: block_table [B, max_pages], kv_len and new_len [B], free_pages [pages], free_count
    [1]; ``tokens`` is the capacity of the packed new tokens.  kv_len and free_count are
    updated in place unless other outputs are given.  Returns (cu_new [B + 1], slots
    [tokens], status [1]); a nonzero status means that nothing was changed."""
    lib = _lib or load_library()
    dev = _this_device(block_table, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, max_pages]")
    B, max_pages = block_table.shape
    i32 = torch.int32
    tokens = int(tokens)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    if cu_new is None or slots is None or status is None:
        with _on(stream):
            where = block_table.device
            cu_new = torch.empty(B + 1, dtype=i32, device=where) if cu_new is None else cu_new
            slots = torch.empty(tokens, dtype=i32, device=where) if slots is None else slots
            status = torch.empty(1, dtype=i32, device=where) if status is None else status
    n_pages = free_pages.numel()
    len_ptr = _dev_ptr(kv_len, "kv_len", i32, (B,), dev)
    count_ptr = _dev_ptr(free_count, "free_count", i32, (1,), dev)
    _check(lib.bsa_cache_resize(
        _dev_ptr(block_table, "block_table", i32, (B, max_pages), dev), len_ptr,
        _dev_ptr(new_len, "new_len", i32, (B,), dev),
        _dev_ptr(free_pages, "free_pages", i32, (n_pages,), dev), count_ptr,
        len_ptr if kv_len_out is None else _dev_ptr(kv_len_out, "kv_len_out", i32, (B,), dev),
        count_ptr if free_count_out is None else
        _dev_ptr(free_count_out, "free_count_out", i32, (1,), dev),
        _dev_ptr(cu_new, "cu_new", i32, (B + 1,), dev), _dev_ptr(slots, "slots", i32, (tokens,), dev),
        _dev_ptr(status, "status", i32, (1,), dev), B, max_pages, n_pages, int(page), tokens,
        _cache_stream(stream, dev)), "bsa_cache_resize")
    return cu_new, slots, status


def cache_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 stream=None) -> None:
    """Quantise new keys and values into the cache (bsa_cache_append).  k, v: bf16 or fp16
    [T, kv_heads, d], 16-byte aligned, token and head strides any multiples of 8 elements; slots
    int32 [T] (cache_resize; -1: skip); caches float8_e4m3fn or int8 [pages, kv_heads, page, d],
    scales fp32 [pages, kv_heads], all on the current device and updated in place."""
    lib = _lib or load_library()
    dev, cache, heads, d = _cache_view(k_cache, v_cache, k_scale, v_scale)
    kp, kt, kh = _rows_ptr(k, "k", heads, d, dev)
    vp, vt, vh = _rows_ptr(v, "v", heads, d, dev)
    if v.dtype is not k.dtype or v.shape != k.shape:
        raise ValueError("k and v must have one type and shape")
    T = k.shape[0]
    _check(lib.bsa_cache_append(cache, kp, vp, _dev_ptr(slots, "slots", torch.int32, (T,), dev), T,
                                _ACTIVATIONS[k.dtype], kt, kh, vt, vh, _cache_stream(stream, dev)),
           "bsa_cache_append")


def cache_workspace(heads: int, kv_heads: int, d: int, max_q: int) -> torch.Tensor:
    """A workspace for cache_forward on the current device, zeroed as its first call wants
    it; calls that may overlap on the GPU need one each."""
    lib = _lib or load_library()
    n = ctypes.c_int64()
    _check(lib.bsa_cache_workspace(int(heads), int(kv_heads), int(d), int(max_q), ctypes.byref(n)),
           "bsa_cache_workspace")
    return torch.zeros(n.value, dtype=torch.uint8, device=torch.device("cuda", torch.cuda.current_device()))


def cache_status(workspace: torch.Tensor) -> int:
    """Waits for the device and returns the status that calls with this workspace and no
    ``status`` of their own have left: 0, or nonzero when a bounded wait gave up in one of them
    (its outputs are undefined and the workspace has to be zeroed)."""
    torch.cuda.synchronize(workspace.device)
    return int(workspace[:4].view(torch.int32).item())


def _cache_args(window, softcap, sinks, heads: int, lut, block, dev: int):
    """bsa_cache_args as bytes (None: none of them)."""
    if not ((window is not None and window >= 0) or softcap or sinks is not None or lut is not None):
        return None
    return _CACHE_ARGS.pack(-1 if window is None else min(max(-1, int(window)), 2 ** 31 - 1), float(softcap),
                            0 if sinks is None else _dev_ptr(sinks, "sinks", torch.float32, (heads,), dev),
                            0 if lut is None else lut.handle.value, 0 if block is None else int(block))


def cache_forward(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor,
                  kv_len: torch.Tensor, cu_q: torch.Tensor, scale: float, max_q: int | None = None,
                  window: int | None = None, softcap: float = 0.0,
                  sinks: torch.Tensor | None = None, lut: Lut | None = None,
                  block: int | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, status: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None):
    """Attention of the newest tokens of every request over its cache (bsa_cache_forward).
    q: bf16 or fp16 [T, heads, d], strides as in cache_append, packed by cu_q int32 [B + 1];
    caches and scales as in cache_append; block_table int32 [B, max_pages], kv_len int32 [B]
    with the new tokens counted.  ``max_q``: the most queries of a request (T when None, which is
    right but takes a batch of decoding requests through the kernel for many rows: give 1 there);
    ``window``: keys further back than that are masked (None or negative: no bound); ``lut``
    with ``block``: only the layout's active blocks, one layout head per kv head;
    ``workspace``: from cache_workspace (a zeroed one is made for the call when None).
    Returns (out [T, heads, d], lse fp32 [T, heads], status); a nonzero status int32 [1] (read
    after the stream is synchronized) means a bounded wait gave up.  With a workspace and no
    ``status`` the workspace keeps it (cache_status) and None is returned."""
    lib = _lib or load_library()
    dev, cache, kv_heads, d = _cache_view(k_cache, v_cache, k_scale, v_scale)
    qp, qt, qh = _rows_ptr(q, "q", None, d, dev)
    T, heads, _ = q.shape
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, max_pages]")
    B, max_pages = block_table.shape
    if lut is not None and block is None:
        raise ValueError("a lut needs its block")
    max_q = max(T, 1) if max_q is None else int(max_q)
    i32, f32 = torch.int32, torch.float32
    if out is None or lse is None or workspace is None:
        with _on(stream):
            where = q.device
            out = torch.empty(T, heads, d, dtype=q.dtype, device=where) if out is None else out
            lse = torch.empty(T, heads, dtype=f32, device=where) if lse is None else lse
            if workspace is None:
                workspace = cache_workspace(heads, kv_heads, d, max_q)
                if status is None:
                    status = torch.empty(1, dtype=i32, device=where)
    args = _cache_args(window, softcap, sinks, heads, lut, block, dev)
    ws_bytes = workspace.numel()
    _check(lib.bsa_cache_forward(
        cache, qp, _dev_ptr(block_table, "block_table", i32, (B, max_pages), dev),
        _dev_ptr(kv_len, "kv_len", i32, (B,), dev), _dev_ptr(cu_q, "cu_q", i32, (B + 1,), dev),
        _dev_ptr(out, "out", q.dtype, (T, heads, d), dev),
        _dev_ptr(lse, "lse", f32, (T, heads), dev),
        None if status is None else _dev_ptr(status, "status", i32, (1,), dev),
        _dev_ptr(workspace, "workspace", torch.uint8, (ws_bytes,), dev), ws_bytes, B, max_pages, T,
        heads, max_q, _ACTIVATIONS[q.dtype], qt, qh, float(scale), args, _cache_stream(stream, dev)),
        "bsa_cache_forward")
    return out, lse, status


def cache_diff_forward(q: torch.Tensor, lam: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor,
                       kv_len: torch.Tensor, cu_q: torch.Tensor, scale: float, max_q: int | None = None,
                       window: int | None = None, softcap: float = 0.0,
                       sinks: torch.Tensor | None = None, lut: Lut | None = None,
                       block: int | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, status: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None):
    """Differential attention of the newest tokens of every request over its cache
    (bsa_cache_diff_forward): out = O_0 - lam O_1 with cache_forward's O of query heads 2h and
    2h + 1.  q: bf16 or fp16 [T, 2 * heads, dq], dq = d or (a key half for each map) d / 2 = 64;
    lam: fp32 [heads] or [T, heads]; sinks [2 * heads]; ``workspace`` from cache_workspace(2 *
    heads, ...); the rest as in cache_forward.  Returns (out [T, heads, d], lse fp32 [T, 2 *
    heads], status)."""
    lib = _lib or load_library()
    dev, cache, kv_heads, d = _cache_view(k_cache, v_cache, k_scale, v_scale)
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[1] % 2:
        raise ValueError("q must be bf16 or fp16 [T, 2 * heads, dq]")
    T, heads2, dq = q.shape
    heads = heads2 // 2
    qp, qt, qh = _rows_ptr(q, "q", None, dq, dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, max_pages]")
    if not isinstance(lam, torch.Tensor) or lam.dim() not in (1, 2):
        raise ValueError("lam must be fp32 [heads] or [T, heads]")
    B, max_pages = block_table.shape
    if lut is not None and block is None:
        raise ValueError("a lut needs its block")
    max_q = max(T, 1) if max_q is None else int(max_q)
    i32, f32 = torch.int32, torch.float32
    out_ptr = None if out is None else _dev_ptr(out, "out", q.dtype, (T, heads, d), dev)
    lse_ptr = None if lse is None else _dev_ptr(lse, "lse", f32, (T, heads2), dev)
    if out is None or lse is None or workspace is None:
        with _on(stream):
            where = q.device
            if out is None:
                out = torch.empty((T, heads, d), dtype=q.dtype, device=where)
                out_ptr = out.data_ptr()
            if lse is None:
                lse = torch.empty((T, heads2), dtype=f32, device=where)
                lse_ptr = lse.data_ptr()
            if workspace is None:
                workspace = cache_workspace(heads2, kv_heads, d, max_q)
                if status is None:
                    status = torch.empty(1, dtype=i32, device=where)
    rows = lam.dim() == 2
    ws_bytes = workspace.numel()
    rc = lib.bsa_cache_diff_forward(
        cache, qp, _dev_ptr(lam, "lam", f32, (T, heads) if rows else (heads,), dev),
        _dev_ptr(block_table, "block_table", i32, (B, max_pages), dev),
        _dev_ptr(kv_len, "kv_len", i32, (B,), dev), _dev_ptr(cu_q, "cu_q", i32, (B + 1,), dev), out_ptr, lse_ptr,
        None if status is None else _dev_ptr(status, "status", i32, (1,), dev),
        _dev_ptr(workspace, "workspace", torch.uint8, (ws_bytes,), dev), ws_bytes, B, max_pages, T,
        heads, dq, max_q, rows, _ACTIVATIONS[q.dtype], qt, qh, float(scale),
        _cache_args(window, softcap, sinks, heads2, lut, block, dev), _cache_stream(stream, dev))
    if rc:
        raise BsaError(rc, "bsa_cache_diff_forward")
    return out, lse, status


def _diff_shapes(q, k, lam):
    """(device, B, H, kv_heads, L, d, dq, shape of lam) of a differential attention call."""
    dev = _device_of(q, "q")
    if q.dim() != 4 or q.shape[1] % 2:
        raise ValueError("q must be bf16 [B, 2H, L, dq]")
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be bf16 [B, kv_heads, L, d]")
    B, H2, L, dq = q.shape
    _, kv, _, d = k.shape
    H = H2 // 2
    rows = lam.dim() if isinstance(lam, torch.Tensor) else 0
    if rows != 1 and rows != 3:
        raise ValueError("lam must be fp32 [H] or [B, H, L]")
    return dev, B, H, kv, L, d, dq, (H,) if rows == 1 else (B, H, L)


def diff_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, lut: Lut,
                 scale: float, block: int, causal_diag: bool, training: bool = False,
                 out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 out2: torch.Tensor | None = None, stream=None):
    """Block-sparse differential attention (bsa_diff_forward): out = (P_0 - lam P_1) V with two
    softmax maps a head.  q: bf16 [B, 2H, L, dq], head h's maps at 2h and 2h + 1; k, v: bf16
    [B, kv_heads, L, d], contiguous, on the current device; dq = d (both maps score the whole
    key) or d / 2 = 64 (the key's first half for map 0, its second for map 1).  lam: fp32 [H] or
    [B, H, L].  lut: of a layout [kv_heads, nb, nb], nb = ceil(L / block), for batch B.
    Returns (out bf16 [B, H, L, d], lse fp32 [B, 2H, L], out2); out2, the second map's output
    that diff_backward takes, is made where ``training`` is set (None else)."""
    lib = _lib or load_library()
    dev, B, H, kv, L, d, dq, lam_shape = _diff_shapes(q, k, lam)
    bf16, f32 = torch.bfloat16, torch.float32
    shape, keys = (B, H, L, d), (B, kv, L, d)
    out_ptr = None if out is None else _dev_ptr(out, "out", bf16, shape, dev)
    lse_ptr = None if lse is None else _dev_ptr(lse, "lse", f32, (B, 2 * H, L), dev)
    out2_ptr = None if out2 is None else _dev_ptr(out2, "out2", bf16, shape, dev)
    if out is None or lse is None or (training and out2 is None):
        with _on(stream):
            if out is None:
                out = torch.empty(shape, dtype=bf16, device=q.device)
                out_ptr = out.data_ptr()
            if lse is None:
                lse = torch.empty((B, 2 * H, L), dtype=f32, device=q.device)
                lse_ptr = lse.data_ptr()
            if training and out2 is None:
                out2 = torch.empty_like(out)
                out2_ptr = out2.data_ptr()
    status = lib.bsa_diff_forward(
        _dev_ptr(q, "q", bf16, q.shape, dev), _dev_ptr(k, "k", bf16, keys, dev), _dev_ptr(v, "v", bf16, keys, dev),
        _dev_ptr(lam, "lam", f32, lam_shape, dev), lut.handle, out_ptr, lse_ptr, out2_ptr, B, H, kv, L, d, dq,
        len(lam_shape) == 3, float(scale), int(block), bool(causal_diag), _cache_stream(stream, dev))
    if status:
        raise BsaError(status, "bsa_diff_forward")
    return out, lse, out2


def diff_workspace(B: int, H: int, L: int, d: int, block: int) -> torch.Tensor:
    """A workspace for diff_backward on the current device; calls that may overlap on the GPU
    need one each."""
    lib = _lib or load_library()
    n = ctypes.c_int64()
    _check(lib.bsa_diff_workspace(int(B), int(H), int(L), int(d), int(block), ctypes.byref(n)),
           "bsa_diff_workspace")
    return torch.empty(n.value, dtype=torch.uint8, device=torch.device("cuda", torch.cuda.current_device()))


def diff_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
                  out: torch.Tensor, out2: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor,
                  lut: Lut, scale: float, block: int, causal_diag: bool, dq: torch.Tensor | None = None,
                  dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                  dlam: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients (dq, dk, dv, dlam) of diff_forward (bsa_diff_backward).  out, out2 (of a call
    with ``training``) and lse as it returned them; dout bf16 [B, H, L, d].  dlam is fp32 in
    lam's shape, the others bf16 in those of q, k, v.  ``workspace``: from diff_workspace (one is
    made for the call when None)."""
    lib = _lib or load_library()
    dev, B, H, kv, L, d, n, lam_shape = _diff_shapes(q, k, lam)
    bf16, f32 = torch.bfloat16, torch.float32
    rows, keys = (B, H, L, d), (B, kv, L, d)
    q_ptr, k_ptr = _dev_ptr(q, "q", bf16, q.shape, dev), _dev_ptr(k, "k", bf16, keys, dev)
    v_ptr, lam_ptr = _dev_ptr(v, "v", bf16, keys, dev), _dev_ptr(lam, "lam", f32, lam_shape, dev)
    given = [None if t is None else _dev_ptr(t, name, like.dtype, like.shape, dev)
             for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v), (dlam, "dlam", lam))]
    if workspace is not None:
        ws_bytes = workspace.numel()
        ws_ptr = _dev_ptr(workspace, "workspace", torch.uint8, (ws_bytes,), dev)
    if workspace is None or None in given:
        with _on(stream):
            if dq is None:
                dq = torch.empty_like(q)
                given[0] = dq.data_ptr()
            if dk is None:
                dk = torch.empty_like(k)
                given[1] = dk.data_ptr()
            if dv is None:
                dv = torch.empty_like(v)
                given[2] = dv.data_ptr()
            if dlam is None:
                dlam = torch.empty_like(lam)
                given[3] = dlam.data_ptr()
            if workspace is None:
                workspace = diff_workspace(B, H, L, d, block)
                ws_bytes, ws_ptr = workspace.numel(), workspace.data_ptr()
    status = lib.bsa_diff_backward(
        q_ptr, k_ptr, v_ptr, lam_ptr, _dev_ptr(out, "out", bf16, rows, dev), _dev_ptr(out2, "out2", bf16, rows, dev),
        _dev_ptr(lse, "lse", f32, (B, 2 * H, L), dev), _dev_ptr(dout, "dout", bf16, rows, dev), lut.handle, *given,
        ws_ptr, ws_bytes, B, H, kv, L, d, n, len(lam_shape) == 3, float(scale), int(block), bool(causal_diag),
        _cache_stream(stream, dev))
    if status:
        raise BsaError(status, "bsa_diff_backward")
    return dq, dk, dv, dlam


_ROTARY_ARGS = struct.Struct("@PPi4x6qPPi4x6qP2qP8i")  # bsa_rotary_args
_PAIRINGS = {"half": 0, "adjacent": 1}


class RotaryTable:
    """Frequencies and axes of the pairs of a head (rotary_table), on one device."""

    def __init__(self, data: torch.Tensor, pairs: int, axes: int):
        self.data, self.pairs, self.axes = data, pairs, axes


def rotary_table(inv_freq, axis=None) -> RotaryTable:
    """Table of rotary's pairs on the current device (bsa_rotary_table).  inv_freq: the pairs'
    frequencies in radians per position, as numbers of 64 bits (1 to 128 of them, at most 1e6 in
    magnitude); axis: the axis of each, 0 to 7 (None: all 0).  A ladder over all pairs whose rungs
    are dealt to three axes, or a ladder for each axis: both are lists of these."""
    lib = _lib or load_library()
    f = np.ascontiguousarray(inv_freq, np.float64)
    if f.ndim != 1 or f.size == 0:
        raise ValueError("inv_freq must be a list of frequencies")
    a = np.zeros(f.size, np.int32)
    if axis is not None:
        given = np.asarray(axis)
        if given.shape != f.shape or given.dtype.kind not in "iu":
            raise ValueError("axis must have a whole number for each frequency")
        a[:] = np.clip(given, -1, 8)  # out of range stays so: the library refuses it
    host = np.zeros((f.size, 2), np.uint64)
    _check(lib.bsa_rotary_table(f.ctypes.data, a.ctypes.data, int(f.size), host.ctypes.data), "bsa_rotary_table")
    dev = torch.device("cuda", torch.cuda.current_device())
    return RotaryTable(torch.from_numpy(host.view(np.int64)).to(dev), int(f.size), int(a.max()) + 1)


def _rotary_rows(t, name: str, dtype, shape, dev: int):
    """(pointer, batch, head and token strides) of q, k or an output of rotary's."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor of shape {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    if len(shape) == 3:
        (token, head, one), batch = t.stride(), 0
        tokens, heads, _ = shape
    else:
        batch, head, token, one = t.stride()
        many, heads, tokens, _ = shape
        if many == 1:
            batch = 0
    if one != 1 and t.numel() > 0:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # The stride of a dimension of one is never used, whatever the tensor says.
    return t.data_ptr(), batch, head if heads > 1 else 0, token if tokens > 1 else 0


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, table: RotaryTable,
           pairing: str = "half", inverse: bool = False, q_out: torch.Tensor | None = None,
           k_out: torch.Tensor | None = None, stream=None):
    """Turns the pairs of q's and k's heads by their positions (bsa_rotary), one launch.  q, k:
    bf16 or fp16 [B, H, L, d] as the layout's calls take them, or packed [T, heads, d] as the
    cache's do, any strides that are multiples of 8 with d contiguous; k may be None.  positions:
    int32 [axes, L] (packed: [axes, T]) or [axes, B, L], last dimension contiguous, with the axes
    of ``table``.  ``pairing``: "half" (numbers i and i + pairs) or "adjacent" (2i and 2i + 1);
    ``inverse`` turns back, which is the gradient.  q_out and k_out may be q and k.  Returns (q, k)
    turned (k None without one)."""
    lib = _lib or load_library()
    dev = _device_of(q, "q")
    dtype, shape = q.dtype, q.shape
    kind = _ACTIVATIONS.get(dtype)
    packed = len(shape) == 3
    if kind is None or not (packed or len(shape) == 4):
        raise ValueError("q must be bf16 or fp16 [B, H, L, d] or [T, heads, d]")
    if packed:
        B, (L, heads, d) = 1, shape
    else:
        B, heads, L, d = shape
    if k is not None and (not isinstance(k, torch.Tensor) or k.dim() != len(shape)):
        raise ValueError("k must have as many dimensions as q")
    if not isinstance(table, RotaryTable):
        raise ValueError("table must come from rotary_table")
    pair = _PAIRINGS.get(pairing)
    if pair is None:
        raise ValueError(f"pairing must be one of {tuple(_PAIRINGS)}")
    if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32 or \
            positions.get_device() != dev:
        raise ValueError("positions must be an int32 tensor on the current device")
    axes = table.axes
    if positions.shape == (axes, L):
        pos_axis, one = positions.stride()
        pos_batch = 0
    elif positions.shape == (axes, B, L):
        pos_axis, pos_batch, one = positions.stride()
    else:
        raise ValueError(f"positions has shape {tuple(positions.shape)}, expected "
                         f"{(axes, L)} or {(axes, B, L)}")
    if one != 1 and L > 1:
        raise ValueError("positions: the last dimension must be contiguous")
    if table.data.get_device() != dev:
        raise ValueError(f"table is on {table.data.device}, not on the current device")
    if q_out is None or (k is not None and k_out is None):
        with _on(stream):
            q_out = torch.empty(shape, dtype=dtype, device=q.device) if q_out is None else q_out
            if k is not None and k_out is None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=q.device)
    qi, q0, q1, q2 = _rotary_rows(q, "q", dtype, shape, dev)
    qo, q3, q4, q5 = _rotary_rows(q_out, "q_out", dtype, shape, dev)
    ki = k0 = k1 = k2 = ko = k3 = k4 = k5 = k_heads = 0
    if k is not None:
        k_heads = k.shape[1]
        shape = (L, k_heads, d) if packed else (B, k_heads, L, d)
        ki, k0, k1, k2 = _rotary_rows(k, "k", dtype, shape, dev)
        ko, k3, k4, k5 = _rotary_rows(k_out, "k_out", dtype, shape, dev)
    status = lib.bsa_rotary(_ROTARY_ARGS.pack(
        qi, qo, heads, q0, q1, q2, q3, q4, q5, ki, ko, k_heads, k0, k1, k2, k3, k4, k5, positions.data_ptr(),
        pos_axis, pos_batch, table.data.data_ptr(), table.pairs, axes, pair, bool(inverse), B, L, d, kind),
        _cache_stream(stream, dev))
    if status:
        raise BsaError(status, "bsa_rotary")
    return q_out, None if k is None else k_out


def forward_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lut: Lut, scale: float,
                 block: int, causal_diag: bool, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, dev_bufs=None, stream=None):
    """Forward from host (ideally pinned) tensors: copies q, k, v to the device, runs
    ``forward`` and copies out / lse back into host tensors, all on one stream.

    ``dev_bufs`` may hold preallocated device tensors (q, k, v, out, lse) to reuse."""
    dev = torch.device("cuda", torch.cuda.current_device())
    if dev_bufs is None:
        dev_bufs = (torch.empty_like(q, device=dev), torch.empty_like(k, device=dev),
                    torch.empty_like(v, device=dev), torch.empty_like(q, device=dev),
                    torch.empty(q.shape[:3], device=dev, dtype=torch.float32))
    dq, dk, dv, do, dl = dev_bufs
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.stream(s):
        dq.copy_(q, non_blocking=True)
        dk.copy_(k, non_blocking=True)
        dv.copy_(v, non_blocking=True)
        forward(dq, dk, dv, lut, scale, block, causal_diag, out=do, lse=dl, stream=s)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=torch.float32, pin_memory=True)
        out.copy_(do, non_blocking=True)
        lse.copy_(dl, non_blocking=True)
    return out, lse


def wait_selftest(limit_ns: int = 1_000_000, stream=None) -> int:
    """Run the bounded-wait self-test kernel; returns its status (expected
    BSA_ERR_DEVICE_TIMEOUT = -8)."""
    lib = load_library()
    return lib.bsa_wait_selftest(int(limit_ns), _stream_handle(stream))


def version() -> str:
    return load_library().bsa_version().decode()
