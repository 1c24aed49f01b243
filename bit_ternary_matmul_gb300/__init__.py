"""GB300-native Q2_0 dequantize-fused matmul — Python binding of libq2_0.

Thin ctypes marshalling over the C ABI declared in ``include/q2_0.h``: the
functions here carry the same names as the C entry points, check tensor
dtype/device/contiguity, pass ``data_ptr()`` values and the current CUDA stream
(or ``stream``: outputs and workspaces that a call makes are then that stream's
memory, and a user on another one waits for it and calls record_stream), and
raise on a non-OK status. Every result is computed by the library's CUDA
kernels; there is no CPU path. PyTorch provides device memory and streams only.

Q2_0 (sources: "WebGPU: add Q2_0 support", bisque.today write-up of llama.cpp
PR 30914, format paragraph; "Llama.cpp umí dvoubitový Q2_0 i na kartách
NVIDIA", aisvetem.cz, section "Osmnáct bajtů na čtyřiašedesát vah"): 64 weights
per 18-byte block — fp16 scale d, then four little-endian u32 words of 2-bit
codes q; a weight is (q - 1) * d.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from ._build import LIB as _LIB_PATH
from ._build import build as _build

BLOCK_WEIGHTS = 64
BLOCK_BYTES = 18

Q2_0_OK = 0
Q2_0_EINVAL = 1
Q2_0_ECUDA = 2
Q2_0_EUNSUPPORTED = 3
Q2_0_EDEVICE = 4
Q2_0_ENOSPACE = 5
Q2_0_NOALLOC_SCRATCH_BYTES = 1 << 20

Q2_0_PREC_F16_SPLIT = 0
Q2_0_PREC_F16 = 1

Q2_0_TYPE_F16 = 0
Q2_0_TYPE_BF16 = 1

Q2_0_ROPE_HALVES = 0
Q2_0_ROPE_PAIRS = 1

Q2_0_DEVERR_NONE = 0
Q2_0_DEVERR_BAD_ID = 1
Q2_0_DEVERR_TIMEOUT = 2

_STATUS = {0: "Q2_0_OK", 1: "Q2_0_EINVAL", 2: "Q2_0_ECUDA", 3: "Q2_0_EUNSUPPORTED",
           4: "Q2_0_EDEVICE", 5: "Q2_0_ENOSPACE"}

# Every symbol include/q2_0.h declares.
EXPORTS = (
    "q2_0_version", "q2_0_device_check", "q2_0_mul_mat_vec", "q2_0_mul_mat_vec_workspace_size",
    "q2_0_mul_mat_vec_ws", "q2_0_mul_mat_vec_noalloc", "q2_0_test_inject_stall",
    "q2_0_test_stall_attention",
    "q2_0_mv_plan_create", "q2_0_mv_plan_execute",
    "q2_0_mv_plan_launches", "q2_0_mv_plan_destroy", "q2_0_mul_mat_workspace_size",
    "q2_0_mul_mat", "q2_0_get_rows", "q2_0_quantize_ref", "q2_0_get_error",
    "q2_0_mul_mat_vec_f16", "q2_0_mul_mat_f16",
    "q2_0_g128_to_g64", "q2_0_g128_get_rows", "q2_0_g128_mul_mat_vec",
    "q2_0_mul_mat_id_workspace_size", "q2_0_mul_mat_id",
    "q2_0_split_bytes", "q2_0_split_layout", "q2_0_join_layout", "q2_0_mul_mat_vec_split",
    "q2_0_mm_plan_create", "q2_0_mm_plan_execute", "q2_0_mm_plan_launches",
    "q2_0_mm_plan_destroy",
    "q2_0_kv_append", "q2_0_attn_plan_create", "q2_0_attn_plan_execute",
    "q2_0_attn_plan_launches", "q2_0_attn_plan_destroy",
    "q2_0_beam_select_workspace_size", "q2_0_beam_select", "q2_0_beam_reorder",
)


class Q2Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)}")
        self.status = status


class _MvDesc(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class _MmDesc(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("M", ctypes.c_int64)]


class _KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("n_layers", ctypes.c_int), ("n_kv", ctypes.c_int), ("page", ctypes.c_int),
                ("dim", ctypes.c_int), ("type", ctypes.c_int)]


class _AttnDesc(ctypes.Structure):
    _fields_ = [("cache", _KvCacheStruct), ("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("n_groups", ctypes.c_int64), ("n_seq", ctypes.c_int64), ("n_q", ctypes.c_int),
                ("scale", ctypes.c_float), ("prefix_table", ctypes.c_void_p),
                ("prefix_len", ctypes.c_void_p), ("prefix_width", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("len", ctypes.c_void_p), ("width", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    """Compile libq2_0.so in-tree for sm_103a (no-op when up to date)."""
    return _build(force=force)


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded libq2_0 (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    "libq2_0.so is not built; run bit_ternary_matmul_gb300.build() "
                    "(the CUDA library is required, there is no CPU fallback)")
            L = ctypes.CDLL(_LIB_PATH)
            vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            L.q2_0_version.restype = ctypes.c_char_p
            L.q2_0_device_check.restype = i32
            L.q2_0_mul_mat_vec.argtypes = [vp, vp, vp, i64, i64, i32, vp]
            L.q2_0_mul_mat_vec.restype = i32
            L.q2_0_mul_mat_vec_workspace_size.argtypes = [i64, i32]
            L.q2_0_mul_mat_vec_workspace_size.restype = sz
            L.q2_0_mul_mat_vec_ws.argtypes = [vp, vp, vp, i64, i64, i32, vp, sz, vp]
            L.q2_0_mul_mat_vec_ws.restype = i32
            L.q2_0_mul_mat_vec_noalloc.argtypes = [vp, vp, vp, i64, i64, i32, vp]
            L.q2_0_mul_mat_vec_noalloc.restype = i32
            L.q2_0_test_inject_stall.argtypes = [i32, ctypes.c_uint64]
            L.q2_0_test_inject_stall.restype = i32
            L.q2_0_test_stall_attention.argtypes = [i32]
            L.q2_0_test_stall_attention.restype = i32
            L.q2_0_mv_plan_create.argtypes = [ctypes.POINTER(_MvDesc), i32, i32,
                                              ctypes.POINTER(vp)]
            L.q2_0_mv_plan_create.restype = i32
            L.q2_0_mv_plan_execute.argtypes = [vp, vp]
            L.q2_0_mv_plan_execute.restype = i32
            L.q2_0_mv_plan_launches.argtypes = [vp]
            L.q2_0_mv_plan_launches.restype = i32
            L.q2_0_mv_plan_destroy.argtypes = [vp]
            L.q2_0_mv_plan_destroy.restype = None
            L.q2_0_mul_mat_workspace_size.argtypes = [i64, i64, i64, i32]
            L.q2_0_mul_mat_workspace_size.restype = sz
            L.q2_0_mul_mat.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]
            L.q2_0_mul_mat.restype = i32
            L.q2_0_mm_plan_create.argtypes = [ctypes.POINTER(_MmDesc), i32, i32,
                                              ctypes.POINTER(vp)]
            L.q2_0_mm_plan_create.restype = i32
            L.q2_0_mm_plan_execute.argtypes = [vp, vp]
            L.q2_0_mm_plan_execute.restype = i32
            L.q2_0_mm_plan_launches.argtypes = [vp]
            L.q2_0_mm_plan_launches.restype = i32
            L.q2_0_mm_plan_destroy.argtypes = [vp]
            L.q2_0_mm_plan_destroy.restype = None
            L.q2_0_mul_mat_vec_f16.argtypes = [vp, vp, vp, i64, i64, i32, vp]
            L.q2_0_mul_mat_vec_f16.restype = i32
            L.q2_0_mul_mat_f16.argtypes = [vp, vp, vp, i64, i64, i64, vp, sz, vp]
            L.q2_0_mul_mat_f16.restype = i32
            L.q2_0_g128_to_g64.argtypes = [vp, vp, i64, i64, vp]
            L.q2_0_g128_to_g64.restype = i32
            L.q2_0_g128_get_rows.argtypes = [vp, i64, i64, vp, i64, vp, vp]
            L.q2_0_g128_get_rows.restype = i32
            L.q2_0_g128_mul_mat_vec.argtypes = [vp, vp, vp, i64, i64, i32, vp]
            L.q2_0_g128_mul_mat_vec.restype = i32
            L.q2_0_get_rows.argtypes = [vp, i64, i64, vp, i64, vp, vp]
            L.q2_0_get_rows.restype = i32
            L.q2_0_mul_mat_id_workspace_size.argtypes = [i64, i64, i64]
            L.q2_0_mul_mat_id_workspace_size.restype = sz
            L.q2_0_mul_mat_id.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, i64, vp, vp, sz, vp]
            L.q2_0_mul_mat_id.restype = i32
            L.q2_0_split_bytes.argtypes = [i64, i64]
            L.q2_0_split_bytes.restype = sz
            L.q2_0_split_layout.argtypes = [vp, vp, i64, i64, vp]
            L.q2_0_split_layout.restype = i32
            L.q2_0_join_layout.argtypes = [vp, vp, i64, i64, vp]
            L.q2_0_join_layout.restype = i32
            L.q2_0_mul_mat_vec_split.argtypes = [vp, vp, vp, i64, i64, i32, vp]
            L.q2_0_mul_mat_vec_split.restype = i32
            L.q2_0_quantize_ref.argtypes = [vp, vp, i64, i64, vp]
            L.q2_0_quantize_ref.restype = i32
            L.q2_0_kv_append.argtypes = [vp, i32, vp, i64, vp, i64, vp, i64, i64, i32, vp, vp, vp,
                                         vp, i64, i64, vp, i64, i32, i32, vp, vp]
            L.q2_0_kv_append.restype = i32
            L.q2_0_attn_plan_create.argtypes = [ctypes.POINTER(_AttnDesc), ctypes.POINTER(vp)]
            L.q2_0_attn_plan_create.restype = i32
            L.q2_0_attn_plan_execute.argtypes = [vp, i32, vp]
            L.q2_0_attn_plan_execute.restype = i32
            L.q2_0_attn_plan_launches.argtypes = [vp]
            L.q2_0_attn_plan_launches.restype = i32
            L.q2_0_attn_plan_destroy.argtypes = [vp]
            L.q2_0_attn_plan_destroy.restype = None
            L.q2_0_beam_select_workspace_size.argtypes = [i64, i32, i64, i32]
            L.q2_0_beam_select_workspace_size.restype = sz
            L.q2_0_beam_select.argtypes = [vp, i64, vp, vp, i32, i64, i32, i64, i32, vp, vp, vp, vp,
                                           sz, vp]
            L.q2_0_beam_select.restype = i32
            L.q2_0_beam_reorder.argtypes = [vp, vp, i64, i32, vp, vp, i64, vp, vp, vp, vp, vp]
            L.q2_0_beam_reorder.restype = i32
            L.q2_0_get_error.argtypes = [vp, ctypes.POINTER(i64)]
            L.q2_0_get_error.restype = i32
            _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != Q2_0_OK:
        raise Q2Error(fn, status)


def _stream(stream) -> int:
    if stream is None:  # the current stream's handle, without a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A buffer that a call allocates for itself: memory of the stream it runs on, as a tensor made
    under torch.cuda.stream(...) has. (The current stream's may be in use there until later, and is
    handed out again there as soon as the last reference goes, whatever runs on `stream`.)"""
    if stream is not None and device.type == "cuda":
        handle = _stream(stream)
        if handle != _stream(None):
            if not isinstance(stream, torch.cuda.Stream):
                # (0 and 1 are the legacy default stream's handles)
                stream = (torch.cuda.ExternalStream(handle, device) if handle > 1
                          else torch.cuda.default_stream(device))
            with torch.cuda.stream(stream):
                return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _dev(t: torch.Tensor, name: str, dtype, numel: int = 0):
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() >= numel:
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def packed_bytes(N: int, K: int) -> int:
    return N * (K // BLOCK_WEIGHTS) * BLOCK_BYTES


def q2_0_version() -> str:
    return lib().q2_0_version().decode()


def q2_0_device_check() -> int:
    return lib().q2_0_device_check()


def q2_0_mul_mat_vec(w: torch.Tensor, x: torch.Tensor, N: int, K: int, ncols: int | None = None,
                     y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[c][n] = sum_k W[n][k] x[c][k]; w uint8 packed, x f32 [ncols][K]."""
    ncols = x.shape[0] if (ncols is None and x.dim() == 2) else (ncols or 1)
    if y is None:
        y = _empty((ncols, N), torch.float32, x.device, stream)
    st = lib().q2_0_mul_mat_vec(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                                _dev(x, "x", torch.float32, ncols * K),
                                _dev(y, "y", torch.float32, ncols * N), N, K, ncols, _stream(stream))
    _check("q2_0_mul_mat_vec", st)
    return y


def q2_0_mul_mat_vec_f16(w: torch.Tensor, x: torch.Tensor, N: int, K: int,
                         ncols: int | None = None, y: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """As q2_0_mul_mat_vec with x F16 [ncols][K]."""
    ncols = x.shape[0] if (ncols is None and x.dim() == 2) else (ncols or 1)
    if y is None:
        y = _empty((ncols, N), torch.float32, x.device, stream)
    st = lib().q2_0_mul_mat_vec_f16(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                                    _dev(x, "x", torch.float16, ncols * K),
                                    _dev(y, "y", torch.float32, ncols * N), N, K, ncols,
                                    _stream(stream))
    _check("q2_0_mul_mat_vec_f16", st)
    return y


def q2_0_mul_mat_vec_workspace_size(K: int, ncols: int) -> int:
    return int(lib().q2_0_mul_mat_vec_workspace_size(K, ncols))


def q2_0_mul_mat_vec_ws(w, x, N, K, ncols, workspace: torch.Tensor, y=None, stream=None):
    if y is None:
        y = _empty((ncols, N), torch.float32, x.device, stream)
    need = q2_0_mul_mat_vec_workspace_size(K, ncols)
    st = lib().q2_0_mul_mat_vec_ws(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                                   _dev(x, "x", torch.float32, ncols * K),
                                   _dev(y, "y", torch.float32, ncols * N), N, K, ncols,
                                   _dev(workspace, "workspace", torch.uint8, need),
                                   workspace.numel(), _stream(stream))
    _check("q2_0_mul_mat_vec_ws", st)
    return y


def q2_0_mul_mat_vec_noalloc(w: torch.Tensor, x: torch.Tensor, N: int, K: int,
                             ncols: int | None = None, y: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """q2_0_mul_mat_vec whose scratch is the library's static device array.

    For callers that cannot allocate device memory at call time. The output
    tensor is allocated here only when ``y`` is None; pass ``y`` to keep the call
    allocation-free. Calls that overlap on the GPU share the array and race.
    """
    ncols = x.shape[0] if (ncols is None and x.dim() == 2) else (ncols or 1)
    if y is None:
        y = _empty((ncols, N), torch.float32, x.device, stream)
    st = lib().q2_0_mul_mat_vec_noalloc(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                                        _dev(x, "x", torch.float32, ncols * K),
                                        _dev(y, "y", torch.float32, ncols * N), N, K, ncols,
                                        _stream(stream))
    _check("q2_0_mul_mat_vec_noalloc", st)
    return y


class MvPlan:
    """A batched mat-vec plan (q2_0_mv_plan_*): keeps references to its tensors."""

    def __init__(self, entries, ncols: int):
        """entries: iterable of (w uint8, x f32 [ncols][K], y f32 [ncols][N], N, K)."""
        self._keep = []
        descs = []
        for (w, x, y, N, K) in entries:
            descs.append(_MvDesc(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                                 _dev(x, "x", torch.float32, ncols * K),
                                 _dev(y, "y", torch.float32, ncols * N), N, K))
            self._keep.append((w, x, y))
        arr = (_MvDesc * len(descs))(*descs)
        h = ctypes.c_void_p()
        _check("q2_0_mv_plan_create",
               lib().q2_0_mv_plan_create(arr, len(descs), ncols, ctypes.byref(h)))
        self._h = h
        self.ncols = ncols
        self.n = len(descs)

    @property
    def launches(self) -> int:
        return int(lib().q2_0_mv_plan_launches(self._h))

    def execute(self, stream=None):
        _check("q2_0_mv_plan_execute", lib().q2_0_mv_plan_execute(self._h, _stream(stream)))

    def close(self):
        if getattr(self, "_h", None):
            lib().q2_0_mv_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def q2_0_mul_mat_workspace_size(M: int, N: int, K: int, prec: int = Q2_0_PREC_F16_SPLIT) -> int:
    return int(lib().q2_0_mul_mat_workspace_size(M, N, K, prec))


def q2_0_mul_mat(w: torch.Tensor, x: torch.Tensor, N: int, K: int, M: int | None = None,
                 prec: int = Q2_0_PREC_F16_SPLIT, y: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[m][n] = sum_k W[n][k] X[m][k]; x f32 [M][K] -> y f32 [M][N]."""
    M = x.shape[0] if M is None else M
    if y is None:
        y = _empty((M, N), torch.float32, x.device, stream)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel()
        ws_ptr = _dev(workspace, "workspace", torch.uint8,
                      q2_0_mul_mat_workspace_size(M, N, K, prec))
    st = lib().q2_0_mul_mat(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                            _dev(x, "x", torch.float32, M * K),
                            _dev(y, "y", torch.float32, M * N), N, K, M, prec, ws_ptr, ws_bytes,
                            _stream(stream))
    _check("q2_0_mul_mat", st)
    return y


class MmPlan:
    """A grouped GEMM plan (q2_0_mm_plan_*): keeps references to its tensors."""

    def __init__(self, entries, prec: int = Q2_0_PREC_F16_SPLIT):
        """entries: iterable of (w uint8, x f32 [M][K], y f32 [M][N], N, K, M)."""
        self._keep = []
        descs = []
        for (w, x, y, N, K, M) in entries:
            descs.append(_MmDesc(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                                 _dev(x, "x", torch.float32, M * K),
                                 _dev(y, "y", torch.float32, M * N), N, K, M))
            self._keep.append((w, x, y))
        arr = (_MmDesc * len(descs))(*descs)
        h = ctypes.c_void_p()
        _check("q2_0_mm_plan_create",
               lib().q2_0_mm_plan_create(arr, len(descs), prec, ctypes.byref(h)))
        self._h = h
        self.prec = prec
        self.n = len(descs)

    @property
    def launches(self) -> int:
        return int(lib().q2_0_mm_plan_launches(self._h))

    def execute(self, stream=None):
        _check("q2_0_mm_plan_execute", lib().q2_0_mm_plan_execute(self._h, _stream(stream)))

    def close(self):
        if getattr(self, "_h", None):
            lib().q2_0_mm_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def q2_0_mul_mat_f16(w: torch.Tensor, x: torch.Tensor, N: int, K: int, M: int | None = None,
                     y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """As q2_0_mul_mat with x F16 [M][K] (exact fp16 operands; workspace size of
    Q2_0_PREC_F16)."""
    M = x.shape[0] if M is None else M
    if y is None:
        y = _empty((M, N), torch.float32, x.device, stream)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel()
        ws_ptr = _dev(workspace, "workspace", torch.uint8,
                      q2_0_mul_mat_workspace_size(M, N, K, Q2_0_PREC_F16))
    st = lib().q2_0_mul_mat_f16(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                                _dev(x, "x", torch.float16, M * K),
                                _dev(y, "y", torch.float32, M * N), N, K, M, ws_ptr, ws_bytes,
                                _stream(stream))
    _check("q2_0_mul_mat_f16", st)
    return y


def q2_0_get_rows(table: torch.Tensor, n_rows: int, K: int, ids: torch.Tensor,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[r] = row ids[r] of the Q2_0 table as F32 (bit-exact)."""
    n_ids = ids.numel()
    if out is None:
        out = _empty((n_ids, K), torch.float32, ids.device, stream)
    if n_ids == 0:
        return out
    st = lib().q2_0_get_rows(_dev(table, "table", torch.uint8, packed_bytes(n_rows, K)), n_rows, K,
                             _dev(ids, "ids", torch.int32, n_ids), n_ids,
                             _dev(out, "out", torch.float32, n_ids * K), _stream(stream))
    _check("q2_0_get_rows", st)
    return out


def q2_0_mul_mat_id_workspace_size(K: int, n_tokens: int, n_x: int) -> int:
    return int(lib().q2_0_mul_mat_id_workspace_size(K, n_tokens, n_x))


def q2_0_mul_mat_id(w: torch.Tensor, n_expert: int, N: int, K: int, x: torch.Tensor,
                    ids: torch.Tensor, y: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Expert mat-vec: y[t][i] = W_{ids[t][i]} x[t][i or 0].

    w: n_expert packed N x K matrices, one after another; x: f32 [n_tokens][n_x][K]
    (n_x = 1 or n_used; a 2-D x is n_x = 1); ids: int32 [n_tokens][n_used];
    y: f32 [n_tokens][n_used][N].
    """
    n_tokens, n_used = ids.shape
    n_x = 1 if x.dim() == 2 else x.shape[1]
    if y is None:
        y = _empty((n_tokens, n_used, N), torch.float32, ids.device, stream)
    if n_tokens == 0:
        return y
    need = q2_0_mul_mat_id_workspace_size(K, n_tokens, n_x)
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, ids.device, stream)
    wsp = _dev(workspace, "workspace", torch.uint8, need) if need > 0 else None
    st = lib().q2_0_mul_mat_id(_dev(w, "w", torch.uint8, n_expert * packed_bytes(N, K)), n_expert,
                               N, K, _dev(x, "x", torch.float32, n_tokens * n_x * K), n_x,
                               _dev(ids, "ids", torch.int32, n_tokens * n_used), n_used, n_tokens,
                               _dev(y, "y", torch.float32, n_tokens * n_used * N), wsp,
                               need if need > 0 else 0, _stream(stream))
    _check("q2_0_mul_mat_id", st)
    return y


def q2_0_split_bytes(N: int, K: int) -> int:
    return int(lib().q2_0_split_bytes(N, K))


def q2_0_split_layout(w: torch.Tensor, N: int, K: int, dst: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """18-byte blocks -> split layout (codes, then 256-byte aligned fp16 scales)."""
    nbytes = q2_0_split_bytes(N, K)
    if dst is None:
        dst = _empty(nbytes, torch.uint8, w.device, stream)
    st = lib().q2_0_split_layout(_dev(w, "w", torch.uint8, packed_bytes(N, K)),
                                 _dev(dst, "dst", torch.uint8, nbytes), N, K, _stream(stream))
    _check("q2_0_split_layout", st)
    return dst


def q2_0_join_layout(src: torch.Tensor, N: int, K: int, w: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Split layout -> 18-byte blocks."""
    if w is None:
        w = _empty(packed_bytes(N, K), torch.uint8, src.device, stream)
    st = lib().q2_0_join_layout(_dev(src, "src", torch.uint8, q2_0_split_bytes(N, K)),
                                _dev(w, "w", torch.uint8, packed_bytes(N, K)), N, K, _stream(stream))
    _check("q2_0_join_layout", st)
    return w


def q2_0_mul_mat_vec_split(w: torch.Tensor, x: torch.Tensor, N: int, K: int, ncols: int = 1,
                           y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[c][n] = sum_k W[n][k] x[c][k] with W in the split layout."""
    if y is None:
        y = _empty((ncols, N), torch.float32, x.device, stream)
    st = lib().q2_0_mul_mat_vec_split(_dev(w, "w", torch.uint8, q2_0_split_bytes(N, K)),
                                      _dev(x, "x", torch.float32, ncols * K),
                                      _dev(y, "y", torch.float32, ncols * N), N, K, ncols,
                                      _stream(stream))
    _check("q2_0_mul_mat_vec_split", st)
    return y


def q2_0_quantize_ref(src: torch.Tensor, nrows: int, K: int, dst: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Reference quantizer: f32 [nrows][K] -> packed uint8 blocks."""
    if dst is None:
        dst = _empty(packed_bytes(nrows, K), torch.uint8, src.device, stream)
    st = lib().q2_0_quantize_ref(_dev(src, "src", torch.float32, nrows * K),
                                 _dev(dst, "dst", torch.uint8, packed_bytes(nrows, K)), nrows, K,
                                 _stream(stream))
    _check("q2_0_quantize_ref", st)
    return dst


# ---- decode step on a paged key/value cache --------------------------------------
_CACHE_TYPES = {torch.float16: Q2_0_TYPE_F16, torch.bfloat16: Q2_0_TYPE_BF16}


def _rows(t: torch.Tensor, name: str, n_tokens: int, heads: int, dim: int):
    """(data_ptr, floats from a token to the next) of f32 [n_tokens][heads][dim] (or
    [n_tokens][heads * dim]) whose tokens are contiguous but may lie apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.float32:
        raise ValueError(f"{name} must be {torch.float32}, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        ok = shape[1] == heads and shape[2] == dim and stride[2] == 1 and \
            (stride[1] == dim or heads == 1)
    else:
        ok = len(shape) == 2 and shape[1] == heads * dim and stride[1] == 1
    if not ok or shape[0] != n_tokens:
        raise ValueError(f"{name} must be [{n_tokens}][{heads}][{dim}] with contiguous tokens")
    return t.data_ptr(), stride[0] if n_tokens > 1 else heads * dim


class KvCache:
    """A paged key/value cache (q2_0_kv_cache): keeps references to its tensors."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        """k, v: f16 or bf16 [n_layers][n_pages][n_kv][page][dim], contiguous."""
        if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor):
            raise TypeError("k and v must be torch.Tensors")
        if k.dtype not in _CACHE_TYPES:
            raise ValueError(f"k must be torch.float16 or torch.bfloat16, got {k.dtype}")
        if k.dim() != 5 or v.shape != k.shape:
            raise ValueError("k and v must both be [n_layers][n_pages][n_kv][page][dim]")
        if v.device != k.device:
            raise ValueError("k and v must be on one device")
        self.k, self.v = k, v
        self.n_layers, self.n_pages, self.n_kv, self.page, self.dim = k.shape
        self._c = _KvCacheStruct(_dev(k, "k", k.dtype), _dev(v, "v", k.dtype), self.n_pages,
                                 self.n_layers, self.n_kv, self.page, self.dim,
                                 _CACHE_TYPES[k.dtype])
        self._ref = ctypes.addressof(self._c)


def q2_0_kv_append(cache: KvCache, layer: int, q: torch.Tensor | None, k: torch.Tensor,
                   v: torch.Tensor, pos: torch.Tensor | None, slot: torch.Tensor,
                   table: torch.Tensor, rope: torch.Tensor | None, style: int = Q2_0_ROPE_HALVES,
                   seq: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor | None:
    """Rotates q and k, stores k and v in the cache's pages; returns the rotated q.

    q f32 [n_tokens][n_q][dim] (or None), k and v f32 [n_tokens][n_kv][dim]: tokens may lie
    apart, as slices of one product's rows do; pos, slot, seq int32 [n_tokens] (seq None:
    token t belongs to row t of the table); table int32 [n_seq][width]; rope f32
    [n_pos][rot], cosines then sines (None: no rotation); q_out [n_tokens][n_q][dim] in the
    cache's type.
    """
    T = k.shape[0]
    qp, qs, n_q, qo = None, 0, 0, None
    if q is not None:
        n_q = q.shape[1] if q.dim() == 3 else q.shape[1] // cache.dim
        qp, qs = _rows(q, "q", T, n_q, cache.dim)
        if q_out is None:
            q_out = _empty((T, n_q, cache.dim), cache.k.dtype, q.device, stream)
            qo = q_out.data_ptr()
        else:
            qo = _dev(q_out, "q_out", cache.k.dtype, T * n_q * cache.dim)
    kp, ks = _rows(k, "k", T, cache.n_kv, cache.dim)
    vp, vs = _rows(v, "v", T, cache.n_kv, cache.dim)
    if table.dim() != 2:
        raise ValueError("table must be [n_seq][width]")
    n_pos, rot = (0, 0) if rope is None else rope.shape
    st = lib().q2_0_kv_append(
        cache._ref, layer, qp, qs, kp, ks, vp, vs, T, n_q,
        None if pos is None else _dev(pos, "pos", torch.int32, T),
        _dev(slot, "slot", torch.int32, T),
        None if seq is None else _dev(seq, "seq", torch.int32, T),
        _dev(table, "table", torch.int32), table.shape[0], table.shape[1],
        None if rope is None else _dev(rope, "rope", torch.float32), n_pos, rot, style, qo,
        _stream(stream))
    _check("q2_0_kv_append", st)
    return q_out


class AttnPlan:
    """Decode attention with shared prefixes (q2_0_attn_plan_*): keeps references to its tensors."""

    def __init__(self, cache: KvCache, q: torch.Tensor, out: torch.Tensor, table: torch.Tensor,
                 length: torch.Tensor, prefix_table: torch.Tensor | None = None,
                 prefix_len: torch.Tensor | None = None, scale: float | None = None):
        """q, out [n_groups * n_seq][n_q][dim] in the cache's type; table int32 [n_groups * n_seq]
        [width], length int32 [n_groups * n_seq]; prefix_table int32 [n_groups][prefix_width],
        prefix_len int32 [n_groups] (None: nothing is shared). scale: 1 / sqrt(dim) if None."""
        if q.dim() != 3 or q.shape[2] != cache.dim or out.shape != q.shape:
            raise ValueError("q and out must be [n_groups * n_seq][n_q][dim]")
        n, n_q = q.shape[0], q.shape[1]
        if table.dim() != 2 or table.shape[0] != n:
            raise ValueError("table must be [n_groups * n_seq][width]")
        groups, pw, pt, pl = 1, 0, None, None
        if prefix_table is None and prefix_len is not None:
            raise ValueError("prefix_table is needed with prefix_len")
        if prefix_table is not None:
            if prefix_table.dim() != 2 or prefix_table.shape[0] < 1 or n % prefix_table.shape[0]:
                raise ValueError("prefix_table must be [n_groups][prefix_width]")
            groups, pw = prefix_table.shape
            pt = _dev(prefix_table, "prefix_table", torch.int32)
            if prefix_len is None:
                raise ValueError("prefix_len is needed with prefix_table")
            pl = _dev(prefix_len, "prefix_len", torch.int32, groups)
        d = _AttnDesc(cache._c, _dev(q, "q", cache.k.dtype), _dev(out, "out", cache.k.dtype), groups,
                      n // groups, n_q, cache.dim ** -0.5 if scale is None else scale, pt, pl, pw,
                      _dev(table, "table", torch.int32), _dev(length, "length", torch.int32, n),
                      table.shape[1])
        self._keep = (cache, q, out, table, length, prefix_table, prefix_len)
        h = ctypes.c_void_p()
        _check("q2_0_attn_plan_create", lib().q2_0_attn_plan_create(ctypes.byref(d), ctypes.byref(h)))
        self._h = h
        self.out = out

    @property
    def launches(self) -> int:
        return int(lib().q2_0_attn_plan_launches(self._h))

    def execute(self, layer: int = 0, stream=None) -> torch.Tensor:
        _check("q2_0_attn_plan_execute",
               lib().q2_0_attn_plan_execute(self._h, layer, _stream(stream)))
        return self.out

    def close(self):
        if getattr(self, "_h", None):
            lib().q2_0_attn_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


@functools.lru_cache(maxsize=256)
def q2_0_beam_select_workspace_size(n_groups: int, n_beams: int, n_vocab: int, n_out: int) -> int:
    return int(lib().q2_0_beam_select_workspace_size(n_groups, n_beams, n_vocab, n_out))


def q2_0_beam_select(logits: torch.Tensor, scores: torch.Tensor, n_out: int | None = None,
                     done: torch.Tensor | None = None, done_token: int = 0,
                     out: tuple | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> tuple:
    """(scores, parent, token) [n_groups][n_out] of the best continuations of each group's beams.

    logits f32 [n_groups][n_beams][n_vocab]: rows contiguous, evenly apart; scores f32 and done
    uint8 or bool [n_groups][n_beams]. n_out: n_beams if None. out: three tensors to write to
    (f32, int32, int32).
    """
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dtype != torch.float32:
        raise ValueError(f"logits must be {torch.float32}, got {logits.dtype}")
    if logits.dim() != 3:
        raise ValueError("logits must be [n_groups][n_beams][n_vocab]")
    G, W, V = logits.shape
    gs, stride, one = logits.stride()
    if W == 1:
        stride = gs if G > 1 else V
    if (V > 1 and one != 1) or (G > 1 and gs != W * stride):
        raise ValueError("logits must have contiguous rows, evenly apart")
    n_out = W if n_out is None else n_out
    if out is None:
        token = _empty((G, n_out), torch.int32, logits.device, stream)
        out = (_empty((G, n_out), torch.float32, logits.device, stream),
               _empty((G, n_out), torch.int32, logits.device, stream), token)
        op = [t.data_ptr() for t in out]
    else:
        op = [_dev(t, f"out[{i}]", torch.int32 if i else torch.float32, G * n_out)
              for i, t in enumerate(out)]
    dp = None
    if done is not None:
        dp = _dev(done, "done", torch.bool if done.dtype == torch.bool else torch.uint8, G * W)
    wp, wb = None, q2_0_beam_select_workspace_size(G, W, V, n_out)
    if wb > 0:
        if workspace is None:
            workspace = _empty(wb, torch.uint8, logits.device, stream)
            wp = workspace.data_ptr()
        else:
            wp = _dev(workspace, "workspace", torch.uint8, wb)
    st = lib().q2_0_beam_select(logits.data_ptr(), stride, _dev(scores, "scores", torch.float32, G * W),
                                dp, done_token, G, W, V, n_out, op[0], op[1], op[2], wp, wb,
                                _stream(stream))
    _check("q2_0_beam_select", st)
    return out


def q2_0_beam_reorder(cache: KvCache, parent: torch.Tensor, table: torch.Tensor,
                      length: torch.Tensor, fresh: torch.Tensor, out: tuple | None = None,
                      stream=None) -> tuple:
    """(table, length, used) after the beams went on from their parents.

    parent int32 [n_groups][n_beams]; table int32 [n_groups * n_beams][width]; length, fresh
    int32 [n_groups * n_beams]. out: three int32 tensors to write to.
    """
    if parent.dim() != 2 or table.dim() != 2 or table.shape[0] != parent.numel():
        raise ValueError("parent must be [n_groups][n_beams], table [n_groups * n_beams][width]")
    G, W = parent.shape
    n, width = table.shape
    if out is None:
        out = tuple(_empty(t.shape, t.dtype, t.device, stream) for t in (table, length, length))
        op = [t.data_ptr() for t in out]
    else:
        op = [_dev(t, f"out[{i}]", torch.int32, n if i else n * width) for i, t in enumerate(out)]
    st = lib().q2_0_beam_reorder(cache._ref, _dev(parent, "parent", torch.int32), G, W,
                                 _dev(table, "table", torch.int32),
                                 _dev(length, "length", torch.int32, n), width,
                                 _dev(fresh, "fresh", torch.int32, n), op[0], op[1], op[2],
                                 _stream(stream))
    _check("q2_0_beam_reorder", st)
    return out


def q2_0_test_inject_stall(stage: int, wait_limit_ns: int) -> None:
    """Test only: the next fp4 mat-vec launch on the current device stalls before
    pipeline stage `stage` and its waits give up after wait_limit_ns."""
    _check("q2_0_test_inject_stall", lib().q2_0_test_inject_stall(int(stage), int(wait_limit_ns)))


def q2_0_test_stall_attention(tiles: int) -> None:
    """Test only: the next attention execute on the current device stalls about `tiles` tiles
    into each block's share."""
    _check("q2_0_test_stall_attention", lib().q2_0_test_stall_attention(int(tiles)))


def q2_0_get_error(stream=None):
    """(code, info): synchronises the stream, reads and clears the device error word."""
    info = ctypes.c_int64(0)
    code = lib().q2_0_get_error(_stream(stream), ctypes.byref(info))
    if code < 0:
        raise Q2Error("q2_0_get_error", Q2_0_ECUDA)
    return code, info.value


# ---- group-128 packing (34-byte blocks of 128 weights) ---------------------------
def packed_bytes_g128(N: int, K: int) -> int:
    return N * (K // 128) * 34


def q2_0_g128_to_g64(src: torch.Tensor, nrows: int, K: int, dst: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Exact repack of a group-128 matrix into the 64-weight layout (uint8)."""
    if dst is None:
        dst = _empty(packed_bytes(nrows, K), torch.uint8, src.device, stream)
    st = lib().q2_0_g128_to_g64(_dev(src, "src", torch.uint8, packed_bytes_g128(nrows, K)),
                               _dev(dst, "dst", torch.uint8, packed_bytes(nrows, K)), nrows, K,
                               _stream(stream))
    _check("q2_0_g128_to_g64", st)
    return dst


def q2_0_g128_get_rows(table: torch.Tensor, n_rows: int, K: int, ids: torch.Tensor,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    n_ids = ids.numel()
    if out is None:
        out = _empty((n_ids, K), torch.float32, ids.device, stream)
    if n_ids == 0:
        return out
    st = lib().q2_0_g128_get_rows(_dev(table, "table", torch.uint8, packed_bytes_g128(n_rows, K)),
                                 n_rows, K, _dev(ids, "ids", torch.int32, n_ids), n_ids,
                                 _dev(out, "out", torch.float32, n_ids * K), _stream(stream))
    _check("q2_0_g128_get_rows", st)
    return out


def q2_0_g128_mul_mat_vec(w: torch.Tensor, x: torch.Tensor, N: int, K: int,
                         ncols: int | None = None, y: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    ncols = x.shape[0] if (ncols is None and x.dim() == 2) else (ncols or 1)
    if y is None:
        y = _empty((ncols, N), torch.float32, x.device, stream)
    st = lib().q2_0_g128_mul_mat_vec(_dev(w, "w", torch.uint8, packed_bytes_g128(N, K)),
                                    _dev(x, "x", torch.float32, ncols * K),
                                    _dev(y, "y", torch.float32, ncols * N), N, K, ncols,
                                    _stream(stream))
    _check("q2_0_g128_mul_mat_vec", st)
    return y
