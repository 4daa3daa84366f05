"""Python binding of libninfer_ternary.so (the GB300 Hadamard-rotated ternary
projection). Argument marshalling only: every step of the computation runs in
the library's CUDA kernels or its host C++ code. There is no fallback: if the
shared library is missing, importing this package raises ImportError.

Names match the C entry points of include/ninfer_ternary.h,
include/ninfer_decode.h and include/ninfer_layer.h. Host entry points take and return numpy arrays; device entry points take torch CUDA tensors and
run on the current torch CUDA stream.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from collections import namedtuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libninfer_ternary.so")

if not os.path.exists(LIBRARY_PATH):
    raise ImportError(f"{LIBRARY_PATH} is not built; run `python bit_gemv_gb300/build.py` "
                      "(or __graft_entry__.build()) first")
_lib = C.CDLL(LIBRARY_PATH)

PQ2_0_G128 = 142
PTQ1_0_G128 = 143
FORMATS = {"PQ2_0_G128": PQ2_0_G128, "PTQ1_0_G128": PTQ1_0_G128}
F32, BF16, F16, E4M3 = 0, 1, 2, 3
# bits of the status words of the decode-step operators
KV_OUT_OF_PAGES, KV_ROW_TOO_SHORT, KV_OUT_OF_SLOTS, KV_BAD_LENGTH, KV_BAD_SLOT, LOGITS_BAD_TOKEN = 1, 2, 4, 8, 16, 32
DELTA_BAD_SLOT = 64
ROTARY_SCALINGS = {"none": 0, "linear": 1, "dimensions": 2, "turns": 3}

GEOMETRY_FIELDS = ("n", "k", "k_pad", "groups_per_row", "base_bytes_per_group",
                   "high_bytes_per_group", "base_row_bytes", "high_row_bytes",
                   "scale_row_bytes", "base_offset", "base_bytes", "high_offset",
                   "high_bytes", "scale_offset", "scale_bytes", "payload_bytes")
RowSplitGeometry = namedtuple("RowSplitGeometry", GEOMETRY_FIELDS)


class _Geom(C.Structure):
    _fields_ = [(f, C.c_uint64) for f in GEOMETRY_FIELDS]


class _KvCacheStruct(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("pages", C.c_uint64), ("page_size", C.c_uint64),
                ("kv_heads", C.c_uint64), ("head_dim", C.c_uint64), ("page_stride", C.c_uint64),
                ("token_stride", C.c_uint64), ("head_stride", C.c_uint64), ("k_scale", C.c_float),
                ("v_scale", C.c_float), ("dtype", C.c_int), ("reserved", C.c_int)]


class _LogitsControls(C.Structure):
    _fields_ = [("history", C.c_void_p), ("history_lengths", C.c_void_p), ("prompt_lengths", C.c_void_p),
                ("history_stride", C.c_uint64), ("repetition", C.c_void_p), ("presence", C.c_void_p),
                ("frequency", C.c_void_p), ("bias_offsets", C.c_void_p), ("bias_ids", C.c_void_p),
                ("bias_values", C.c_void_p), ("bias_count", C.c_uint64), ("mask", C.c_void_p),
                ("mask_rows", C.c_void_p), ("mask_row_count", C.c_uint64), ("mask_stride", C.c_uint64)]


class NinferError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.status_name = _lib.ninfer_status_name(status).decode()
        super().__init__(f"{self.status_name}: {message}")


_u64, _int, _vp = C.c_uint64, C.c_int, C.c_void_p
_sig = {
    "ninfer_last_error": (C.c_char_p, []),
    "ninfer_status_name": (C.c_char_p, [_int]),
    "ninfer_abi_version": (_int, []),
    "ninfer_ternary_geometry": (_int, [_int, _u64, _u64, C.POINTER(_Geom)]),
    "ninfer_ternary_pack": (_int, [_int, _u64, _u64, _vp, _vp, _vp, _u64]),
    "ninfer_ternary_unpack": (_int, [_int, _u64, _u64, _vp, _u64, _vp, _vp]),
    "ninfer_blocks_to_planes": (_int, [_int, _u64, _u64, _vp, _u64, _vp, _u64]),
    "ninfer_planes_to_blocks": (_int, [_int, _u64, _u64, _vp, _u64, _vp, _u64]),
    "ninfer_blocks_to_planes_device": (_int, [_int, _u64, _u64, _vp, _u64, _vp, _u64, _vp]),
    "ninfer_planes_to_blocks_device": (_int, [_int, _u64, _u64, _vp, _u64, _vp, _u64, _vp]),
    "ninfer_validate_signs": (_int, [_vp, _u64]),
    "ninfer_hadamard_fwd": (_int, [_vp, _int, _vp, _int, _vp, _u64, _u64, _vp]),
    "ninfer_hadamard_inv": (_int, [_vp, _int, _vp, _int, _vp, _u64, _u64, _vp]),
    "ninfer_ternary_matmul_workspace": (_int, [_int, _u64, _u64, _u64, _int, C.POINTER(_u64)]),
    "ninfer_ternary_matmul": (_int, [_int, _vp, _u64, _u64, _u64, _vp, _int, _vp, _vp, _int, _u64, _vp, _u64, _vp]),
    "ninfer_ternary_embed": (_int, [_int, _vp, _u64, _u64, _u64, _vp, _u64, _vp, _vp, _int, _vp, _vp]),
    "ninfer_device_errors": (_int, [C.POINTER(C.c_uint32), _int]),
    "ninfer_set_prefetch_before_dependency": (_int, [_int]),
    "ninfer_set_wait_limit": (_int, [C.c_longlong]),
    "ninfer_ternary_matmul_noalloc": (_int, [_int, _vp, _u64, _u64, _u64, _vp, _int, _vp, _vp, _int, _u64, _vp]),
    "ninfer_ternary_gate_up_workspace": (_int, [_int, _u64, _u64, _u64, _int, _int, C.POINTER(_u64)]),
    "ninfer_ternary_gate_up": (_int, [_int, _vp, _vp, _u64, _u64, _u64, _vp, _int, _vp, _vp, _vp, _int, _u64, _vp,
                                      _u64, _vp]),
    "ninfer_kv_tables": (_int, [_vp, _vp, _u64, _u64, _vp, _u64, _vp, _u64, _u64, _vp, _vp, _vp, _u64, _vp, _vp, _vp,
                                _vp, _vp]),
    "ninfer_kv_append": (_int, [_vp, _vp, _int, _u64, _u64, _u64, _u64, _u64, _vp, C.POINTER(_KvCacheStruct), _vp, _vp]),
    "ninfer_kv_attention_workspace": (_int, [C.POINTER(_KvCacheStruct), _u64, _u64, C.POINTER(_u64)]),
    "ninfer_kv_attention": (_int, [_vp, _int, _u64, _u64, _u64, _u64, C.POINTER(_KvCacheStruct), _vp, _u64, _u64, _vp,
                                   C.c_float, _u64, _vp, _int, _vp, _vp, _u64, _vp]),
    "ninfer_logits_process": (_int, [_vp, _u64, _vp, _u64, _int, _u64, _u64, _vp, _vp, _vp]),
    "ninfer_norm": (_int, [_vp, _vp]),
    "ninfer_rotary_frequencies": (_int, [_u64, C.c_double, _int, C.c_double, C.c_double, C.c_double, C.c_double, _vp,
                                         C.POINTER(C.c_float)]),
    "ninfer_rotary": (_int, [_vp, _vp]),
    "ninfer_gated_delta_workspace": (_int, [_u64, _u64, _u64, _u64, _u64, _u64, C.POINTER(_u64)]),
    "ninfer_gated_delta": (_int, [_vp, _vp, _u64, _vp]),
    "ninfer_sample": (_int, [_vp, _vp]),
}
NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sig)


def _check(status: int):
    if status != 0:
        raise NinferError(status, _lib.ninfer_last_error().decode(errors="replace"))


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(C.c_void_p)


def ninfer_abi_version() -> int:
    return _lib.ninfer_abi_version()


# ------------------------------------------------------------------ host ---
def ninfer_ternary_geometry(fmt, n: int, k: int) -> RowSplitGeometry:
    g = _Geom()
    _check(_lib.ninfer_ternary_geometry(_fmt(fmt), n, k, C.byref(g)))
    return RowSplitGeometry(*[getattr(g, f) for f in GEOMETRY_FIELDS])


def ninfer_ternary_pack(fmt, values: np.ndarray, scales_f16: np.ndarray) -> np.ndarray:
    values = np.ascontiguousarray(values, dtype=np.int8)
    scales_f16 = np.ascontiguousarray(scales_f16, dtype=np.uint16)
    n, k = values.shape
    g = ninfer_ternary_geometry(fmt, n, k)
    if scales_f16.size != n * g.groups_per_row:
        raise ValueError("scales must hold n * groups_per_row binary16 words")
    out = np.empty(g.payload_bytes, dtype=np.uint8)
    _check(_lib.ninfer_ternary_pack(_fmt(fmt), n, k, _np_ptr(values), _np_ptr(scales_f16), _np_ptr(out), out.size))
    return out


def ninfer_ternary_unpack(fmt, n: int, k: int, payload: np.ndarray):
    payload = np.ascontiguousarray(payload, dtype=np.uint8).reshape(-1)
    g = ninfer_ternary_geometry(fmt, n, k)
    values = np.empty((n, k), dtype=np.int8)
    scales = np.empty((n, g.groups_per_row), dtype=np.uint16)
    _check(_lib.ninfer_ternary_unpack(_fmt(fmt), n, k, _np_ptr(payload), payload.size, _np_ptr(values), _np_ptr(scales)))
    return values, scales


def ninfer_blocks_to_planes(fmt, n: int, k: int, blocks: np.ndarray) -> np.ndarray:
    blocks = np.ascontiguousarray(blocks, dtype=np.uint8).reshape(-1)
    g = ninfer_ternary_geometry(fmt, n, k)
    out = np.empty(g.payload_bytes, dtype=np.uint8)
    _check(_lib.ninfer_blocks_to_planes(_fmt(fmt), n, k, _np_ptr(blocks), blocks.size, _np_ptr(out), out.size))
    return out


def ninfer_planes_to_blocks(fmt, n: int, k: int, payload: np.ndarray) -> np.ndarray:
    payload = np.ascontiguousarray(payload, dtype=np.uint8).reshape(-1)
    g = ninfer_ternary_geometry(fmt, n, k)
    nb = 34 if _fmt(fmt) == PQ2_0_G128 else 28
    out = np.empty(n * g.groups_per_row * nb, dtype=np.uint8)
    _check(_lib.ninfer_planes_to_blocks(_fmt(fmt), n, k, _np_ptr(payload), payload.size, _np_ptr(out), out.size))
    return out


def ninfer_blocks_to_planes_device(fmt, n: int, k: int, blocks, out=None):
    """Device version of ninfer_blocks_to_planes: blocks is a uint8 CUDA tensor;
    returns (or fills) the uint8 CUDA payload tensor, on the current stream."""
    torch = _torch()
    g = ninfer_ternary_geometry(fmt, n, k)
    if out is None:
        out = torch.empty(g.payload_bytes, dtype=torch.uint8, device=blocks.device)
    _check(_lib.ninfer_blocks_to_planes_device(_fmt(fmt), n, k, _dev(blocks, "blocks"), blocks.numel(),
                                               _dev(out, "payload"), out.numel(), _stream(blocks)))
    return out


def ninfer_planes_to_blocks_device(fmt, n: int, k: int, payload, out=None):
    torch = _torch()
    g = ninfer_ternary_geometry(fmt, n, k)
    nb = 34 if _fmt(fmt) == PQ2_0_G128 else 28
    if out is None:
        out = torch.empty(n * g.groups_per_row * nb, dtype=torch.uint8, device=payload.device)
    _check(_lib.ninfer_planes_to_blocks_device(_fmt(fmt), n, k, _dev(payload, "payload"), payload.numel(),
                                               _dev(out, "blocks"), out.numel(), _stream(payload)))
    return out


def ninfer_device_errors(clear: bool = True) -> int:
    v = C.c_uint32()
    _check(_lib.ninfer_device_errors(C.byref(v), int(bool(clear))))
    return v.value


def ninfer_set_prefetch_before_dependency(enable: bool) -> None:
    _check(_lib.ninfer_set_prefetch_before_dependency(int(bool(enable))))


WAIT_LIMIT_DEFAULT = 4_000_000_000


def ninfer_set_wait_limit(cycles: int) -> None:
    _check(_lib.ninfer_set_wait_limit(int(cycles)))


# ---------------------------------------------------------------- device ---
def _torch():
    import torch
    return torch


def _dt(t) -> int:
    torch = _torch()
    return {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}[t]


def _stream(t):
    torch = _torch()
    return C.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dev(t, name):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return C.c_void_p(t.data_ptr())


def ninfer_validate_signs(signs) -> None:
    """Raise NinferError unless signs (host uint16/int16 bfloat16 bits, length K,
    K % 1024 == 0) holds only +1 and -1."""
    a = np.ascontiguousarray(np.asarray(signs).view(np.uint16).reshape(-1))
    _check(_lib.ninfer_validate_signs(a.ctypes.data_as(C.c_void_p), a.size))


def ninfer_hadamard_fwd(x, signs, out=None, out_dtype=None):
    """Forward signed block transform of a (M, K) CUDA tensor; signs is a (K,)
    CUDA tensor of bfloat16 +-1 (dtype bfloat16, int16 or uint16 bit patterns)."""
    return _hadamard(_lib.ninfer_hadamard_fwd, x, signs, out, out_dtype)


def ninfer_hadamard_inv(x, signs, out=None, out_dtype=None):
    return _hadamard(_lib.ninfer_hadamard_inv, x, signs, out, out_dtype)


def _hadamard(fn, x, signs, out, out_dtype):
    torch = _torch()
    x2 = x.reshape(-1, x.shape[-1])
    if out is None:
        out = torch.empty(x2.shape, dtype=out_dtype or torch.float32, device=x.device)
    _check(fn(_dev(x2, "x"), _dt(x2.dtype), _dev(out, "out"), _dt(out.dtype), _dev(signs, "signs"),
              x2.shape[0], x2.shape[1], _stream(x)))
    return out.reshape(x.shape[:-1] + (x.shape[-1],))


def ninfer_ternary_matmul_workspace(fmt, n: int, k: int, M: int, rotate: bool = True) -> int:
    b = C.c_uint64()
    _check(_lib.ninfer_ternary_matmul_workspace(_fmt(fmt), n, k, M, int(bool(rotate)), C.byref(b)))
    return b.value


def ninfer_ternary_matmul(fmt, payload, n: int, k: int, x, signs=None, y=None, y_dtype=None, workspace=None):
    """y (M, n) = ternary W (n, k) applied to the forward-transformed x (M, k)."""
    torch = _torch()
    x2 = x.reshape(-1, k)
    M = x2.shape[0]
    if y is None:
        y = torch.empty((M, n), dtype=y_dtype or torch.float32, device=x.device)
    need = ninfer_ternary_matmul_workspace(fmt, n, k, M, signs is not None)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.ninfer_ternary_matmul(
        _fmt(fmt), _dev(payload, "payload"), payload.numel(), n, k, _dev(x2, "x"), _dt(x2.dtype),
        _dev(signs, "signs") if signs is not None else None, _dev(y, "y"), _dt(y.dtype), M,
        ws_ptr, ws_bytes, _stream(x)))
    return y


def ninfer_ternary_gate_up_workspace(fmt, n: int, k: int, M: int, rotate: bool, distinct_signs: bool) -> int:
    v = _u64()
    _check(_lib.ninfer_ternary_gate_up_workspace(_fmt(fmt), n, k, M, int(bool(rotate)), int(bool(distinct_signs)),
                                                 C.byref(v)))
    return v.value


def ninfer_ternary_gate_up(fmt, payload_gate, payload_up, n: int, k: int, x, signs_gate=None, signs_up=None, y=None,
                           y_dtype=None, workspace=None):
    """y (M, n) = silu(gate projection) * (up projection) of x (M, k); each
    projection rotates x with its own signs (both or neither given)."""
    torch = _torch()
    x2 = x.reshape(-1, k)
    M = x2.shape[0]
    if y is None:
        y = torch.empty((M, n), dtype=y_dtype or torch.float32, device=x.device)
    distinct = signs_gate is not None and signs_up is not None and signs_gate.data_ptr() != signs_up.data_ptr()
    need = ninfer_ternary_gate_up_workspace(fmt, n, k, M, signs_gate is not None, distinct)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_ptr = _dev(workspace, "workspace") if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if need else 0
    _check(_lib.ninfer_ternary_gate_up(
        _fmt(fmt), _dev(payload_gate, "payload_gate"), _dev(payload_up, "payload_up"), payload_gate.numel(), n, k,
        _dev(x2, "x"), _dt(x2.dtype), _dev(signs_gate, "signs_gate") if signs_gate is not None else None,
        _dev(signs_up, "signs_up") if signs_up is not None else None, _dev(y, "y"), _dt(y.dtype), M,
        ws_ptr, ws_bytes, _stream(x)))
    return y


def ninfer_ternary_matmul_noalloc(fmt, payload, n: int, k: int, x, signs=None, y=None, y_dtype=None):
    """As ninfer_ternary_matmul, for callers that cannot allocate device memory:
    the workspace comes from the library's fixed device array."""
    torch = _torch()
    x2 = x.reshape(-1, k)
    M = x2.shape[0]
    if y is None:
        y = torch.empty((M, n), dtype=y_dtype or torch.float32, device=x.device)
    _check(_lib.ninfer_ternary_matmul_noalloc(
        _fmt(fmt), _dev(payload, "payload"), payload.numel(), n, k, _dev(x2, "x"), _dt(x2.dtype),
        _dev(signs, "signs") if signs is not None else None, _dev(y, "y"), _dt(y.dtype), M, _stream(x)))
    return y


def ninfer_ternary_embed(fmt, payload, n: int, k: int, ids, signs=None, out=None, out_dtype=None, status=None):
    """out (count, k) = inverse transform of the dequantised rows ids (int32 CUDA)."""
    torch = _torch()
    count = ids.numel()
    if out is None:
        out = torch.empty((count, k), dtype=out_dtype or torch.float32, device=ids.device)
    _check(_lib.ninfer_ternary_embed(
        _fmt(fmt), _dev(payload, "payload"), payload.numel(), n, k, _dev(ids, "ids"), count,
        _dev(signs, "signs") if signs is not None else None, _dev(out, "out"), _dt(out.dtype),
        _dev(status, "status") if status is not None else None, _stream(ids)))
    return out


# ------------------------------------------------------------ decode step ---
# A decode step's calls are short, so that their checks are written for speed:
# torch's types and the stream query are looked up once, addresses and strides
# go to the library as plain integers, the controls of the logits as packed bytes.
_TYPES: dict = {}       # torch dtype -> library dtype
_I32 = _I64 = _F32 = _raw_stream = None
_several = False        # whether torch sees more than one GPU
_CONTROLS = struct.Struct("=15Q")


def _types():
    global _I32, _I64, _F32, _raw_stream, _several
    if not _TYPES:
        torch = _torch()
        _several = torch.cuda.device_count() > 1
        _I32, _I64, _F32, _raw_stream = torch.int32, torch.int64, torch.float32, torch._C._cuda_getCurrentRawStream
        _TYPES.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16, torch.float8_e4m3fn: E4M3})
    return _TYPES


def _on(t, name):
    """The GPU that a call's first tensor lies on, and with it all others: the current one, where the library launches."""
    device = t.get_device()
    if device < 0 or _several and device != _torch().cuda.current_device():
        raise ValueError(f"{name} must be a CUDA tensor on the current device, not on {t.device}")
    return device


def _arg(t, name, dtype, count, device):
    """Address of a contiguous tensor of one dtype and `count` elements on a GPU; None is 0."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous() or t.numel() != count:
        raise ValueError(f"{name} must be a contiguous tensor of {count} elements of {dtype} on cuda:{device}, "
                         f"not {tuple(t.shape)} of {t.dtype} on {t.device}")
    return t.data_ptr()


def _rows(t, name, dims, dtypes, device):
    """Checks a tensor on a GPU whose last dimension is contiguous and whose other
    strides are free; returns its library dtype and its strides."""
    code = _TYPES.get(t.dtype, -1)
    strides = t.stride()
    if t.get_device() != device or len(strides) != dims or code not in dtypes or (strides[-1] != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be a tensor of {dims} dimensions, the last one contiguous, of a supported dtype on cuda:{device}")
    return code, strides


def _table(t, name, device):
    """Address, width and row stride of an int32 table with contiguous rows."""
    strides = t.stride()
    if t.dtype is not _I32 or t.get_device() != device or len(strides) != 2 or (strides[1] != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be a two-dimensional int32 tensor with contiguous rows on cuda:{device}")
    n, width = t.shape
    return t.data_ptr(), n, width, strides[0] if n > 1 else width


class KvCache:
    """A paged key/value cache over two pools indexed [page][token][head][element]
    (any strides, the last dimension contiguous; bfloat16, float16 or
    float8_e4m3fn). A stored value stands for itself times k_scale (v_scale). The
    pools are read and checked when the cache is made, and again by the next call
    where their memory was replaced (resize_, set_, .data)."""

    def __init__(self, k, v, k_scale: float = 1.0, v_scale: float = 1.0):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._read()

    def _read(self):
        k, v = self.k, self.v
        _TYPES or _types()
        device = _on(k, "k")
        code, strides = _rows(k, "k", 4, (BF16, F16, E4M3), device)
        if _rows(v, "v", 4, (BF16, F16, E4M3), device) != (code, strides) or v.shape != k.shape:
            raise ValueError("k and v must have the same dtype, shape, strides and device")
        pages, page_size, heads, dim = k.shape
        self.pages, self.page_size, self.kv_heads, self.head_dim = pages, page_size, heads, dim
        strides = [s if n > 1 else 0 for s, n in zip(strides, k.shape)]
        self._struct = _KvCacheStruct(k.data_ptr(), v.data_ptr(), pages, page_size, heads, dim, strides[0], strides[1],
                                      strides[2], self.k_scale, self.v_scale, code, 0)
        self._ref = C.byref(self._struct)
        self._device, self._seen = device, (k.data_ptr(), v.data_ptr())
        self._held = k.detach(), v.detach()

    def _current(self, device):
        """The library's description of the pools as they are now, for a call on a GPU."""
        if self._seen != (self.k.data_ptr(), self.v.data_ptr()):
            self._read()
        if self._device != device:
            raise ValueError(f"the cache lies on cuda:{self._device}, not on cuda:{device}")
        return self._ref


class KvTables(namedtuple("KvTables", ("block_table", "slots", "positions", "token_rows", "offsets", "lengths", "counts"))):
    """What ninfer_kv_tables writes; give one back as `out` to reuse its buffers,
    which are checked when it is first used and again where the memory of one was
    replaced (resize_, set_, .data) or the table has another shape."""

    @classmethod
    def empty(cls, block_table, capacity: int):
        """Buffers for the requests of block_table (requests, table_pages) and `capacity` new tokens."""
        torch = _torch()
        new = lambda n, t: torch.empty(n, dtype=t, device=block_table.device)  # noqa: E731
        n, i32 = block_table.shape[0], torch.int32
        return cls(block_table, new(capacity, torch.int64), new(capacity, i32), new(capacity, i32), new(n + 1, i32),
                   new(n, i32), new(2, i32))

    def _addresses(self, capacity: int, device: int):
        # Aliases keep the checked memory alive, so that an address that is still the same is the same memory.
        table, t, p, r, o, n, c = self
        seen = (capacity, device, table.data_ptr(), table.shape, table.stride(), t is None or t.data_ptr(),
                p is None or p.data_ptr(), r is None or r.data_ptr(), o is None or o.data_ptr(),
                n is None or n.data_ptr(), c is None or c.data_ptr())
        known = self.__dict__.get("_known")
        if known is None or known[0] != seen:
            rows = _table(table, "block_table", device)
            requests = rows[1]
            known = self.__dict__["_known"] = (
                seen, rows,
                (_arg(t, "slots", _I64, capacity, device), _arg(p, "positions", _I32, capacity, device),
                 _arg(r, "token_rows", _I32, capacity, device)),
                (_arg(o, "offsets", _I32, requests + 1, device), _arg(n, "lengths", _I32, requests, device),
                 _arg(c, "counts", _I32, 2, device)),
                [x.detach() for x in self if x is not None])
        return known


def ninfer_kv_tables(lengths, new_tokens, page_size: int, free_pages, block_table, capacity: int, out=None, status=None):
    """Block tables and slot maps of a step's new tokens from the requests'
    lengths: fills the fresh entries of block_table in place and returns a
    KvTables. new_tokens None: one a request; free_pages None: no free page.
    out.lengths may not be lengths: copy them once the step has read both."""
    _TYPES or _types()
    device = _on(lengths, "lengths")
    if out is None:
        out = KvTables.empty(block_table, capacity)
    elif out.block_table is not block_table:
        out = out._replace(block_table=block_table)
    _, (table, n, width, stride), tokens, requests, _ = out._addresses(capacity, device)
    free = free_pages.numel() if free_pages is not None else 0
    _check(_lib.ninfer_kv_tables(
        _arg(lengths, "lengths", _I32, n, device), _arg(new_tokens, "new_tokens", _I32, n, device), n, page_size,
        _arg(free_pages, "free_pages", _I32, free, device), free, table, width, stride, *tokens, capacity, *requests,
        _arg(status, "status", _I32, 1, device), _raw_stream(device)))
    return out


def ninfer_kv_append(cache: KvCache, k, v, slots, status=None) -> None:
    """Writes the new keys and values k, v (tokens, kv_heads, head_dim) into the cache's slots."""
    device = _on(k, "k")
    ref = cache._current(device)
    code, ks = _rows(k, "k", 3, (F32, BF16, F16), device)
    code_v, vs = _rows(v, "v", 3, (F32, BF16, F16), device)
    shape = k.shape
    if code != code_v or shape != v.shape or shape[1] != cache.kv_heads or shape[2] != cache.head_dim:
        raise ValueError("k and v must be (tokens, kv_heads, head_dim) of the cache and of one dtype")
    tokens = shape[0]
    _check(_lib.ninfer_kv_append(k.data_ptr(), v.data_ptr(), code, tokens, ks[0], ks[1], vs[0], vs[1],
                                 _arg(slots, "slots", _I64, tokens, device), ref, _arg(status, "status", _I32, 1, device),
                                 _raw_stream(device)))


def ninfer_kv_attention_workspace(cache: KvCache, requests: int, q_heads: int) -> int:
    b = C.c_uint64()
    _check(_lib.ninfer_kv_attention_workspace(cache._current(cache._device), requests, q_heads, C.byref(b)))
    return b.value


def ninfer_kv_attention(q, cache: KvCache, block_table, lengths, scale=None, window: int = 0, out=None, out_dtype=None,
                        lse=None, workspace=None):
    """Attention of one new token per request, q (requests, q_heads, head_dim),
    over the cache's pages in block_table (requests, table_pages); lengths count
    the new token. scale: head_dim ** -0.5 unless given; window 0: every key.
    lse: a float32 (requests, q_heads) tensor to be written, or None."""
    device = _on(q, "q")
    ref = cache._current(device)
    code, strides = _rows(q, "q", 3, (F32, BF16, F16), device)
    requests, heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError(f"q has head_dim {dim}, the cache {cache.head_dim}")
    table, n, width, stride = _table(block_table, "block_table", device)
    if n != requests:
        raise ValueError(f"block_table has {n} rows for {requests} requests")
    if out is None:
        out = _torch().empty((requests, heads, dim), dtype=out_dtype or q.dtype, device=q.device)
    if workspace is None:
        need = ninfer_kv_attention_workspace(cache, requests, heads)
        workspace = _torch().empty(need, dtype=_torch().uint8, device=q.device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    dtype = out.dtype
    _check(_lib.ninfer_kv_attention(
        q.data_ptr(), code, requests, heads, strides[0], strides[1], ref, table, width, stride,
        _arg(lengths, "lengths", _I32, requests, device), dim ** -0.5 if scale is None else scale, window,
        _arg(out, "out", dtype, requests * heads * dim, device), _TYPES.get(dtype, -1), _arg(lse, "lse", _F32, requests * heads, device),
        workspace.data_ptr(), workspace.nbytes, _raw_stream(device)))
    return out


def ninfer_logits_process(logits, out=None, history=None, history_lengths=None, prompt_lengths=None, repetition=None,
                          presence=None, frequency=None, bias_offsets=None, bias_ids=None, bias_values=None, mask=None,
                          mask_rows=None, status=None):
    """Penalties, biases and grammar masks on logits (rows, vocab); out may be
    logits itself. history: int32 (rows, longest); mask: int32 words (mask rows,
    ceil(vocab / 32)), bit set where a token is allowed."""
    _TYPES or _types()
    device = _on(logits, "logits")
    code, strides = _rows(logits, "logits", 2, (F32, BF16, F16), device)
    rows, vocab = logits.shape
    if out is None:
        out = _torch().empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    code_out, out_strides = _rows(out, "out", 2, (code,), device)
    if out is not logits and out.shape != (rows, vocab):
        raise ValueError("out must have the shape and dtype of logits")
    h = n = p = longest = offsets = ids = values = count = m = m_rows = m_count = m_stride = 0
    if history is not None:
        if history.dim() != 2:
            raise ValueError("history must be (rows, longest)")
        longest = history.shape[1]
        h = _arg(history, "history", _I32, rows * longest, device)
        n = _arg(history_lengths, "history_lengths", _I32, rows, device)
        p = _arg(prompt_lengths, "prompt_lengths", _I32, rows, device)
    if bias_ids is not None and (count := bias_ids.numel()):
        offsets = _arg(bias_offsets, "bias_offsets", _I32, rows + 1, device)
        ids = _arg(bias_ids, "bias_ids", _I32, count, device)
        values = _arg(bias_values, "bias_values", _F32, count, device)
    if mask is not None:
        m, m_count, width, m_stride = _table(mask, "mask", device)
        if width * 32 < vocab:
            raise ValueError(f"mask has {width} words a row for {vocab} tokens")
        m_rows = _arg(mask_rows, "mask_rows", _I32, rows, device)
    controls = _CONTROLS.pack(
        h, n, p, longest, _arg(repetition, "repetition", _F32, rows, device), _arg(presence, "presence", _F32, rows, device),
        _arg(frequency, "frequency", _F32, rows, device), offsets, ids, values, count, m, m_rows, m_count, m_stride)
    _check(_lib.ninfer_logits_process(
        logits.data_ptr(), strides[0] if rows > 1 else vocab, out.data_ptr(), out_strides[0] if rows > 1 else vocab, code,
        rows, vocab, controls, _arg(status, "status", _I32, 1, device), _raw_stream(device)))
    return out


# ------------------------------------------------------------- layer's step ---
# The C argument structures of ninfer_layer.h as packed bytes.
_NORM = struct.Struct("=14Q2f6i")
_ROTARY = struct.Struct("=21Q3f3i")
_DELTA = struct.Struct("=27Q2f2i")
_SAMPLE = struct.Struct("=11Q2i")
_ANY = (F32, BF16, F16)


def _vector(t, name, count, device):
    """Address and library dtype of a contiguous tensor of `count` elements; (0, 0) for None."""
    if t is None:
        return 0, 0
    code = _TYPES.get(t.dtype, -1)
    if t.get_device() != device or code not in _ANY or not t.is_contiguous() or t.numel() != count:
        raise ValueError(f"{name} must be a contiguous tensor of {count} elements of a supported dtype on cuda:{device}, "
                         f"not {tuple(t.shape)} of {t.dtype} on {t.device}")
    return t.data_ptr(), code


def _matrix(t, name, shape, device):
    """Address, library dtype and row stride of a tensor of rows of a shape; zeros for None."""
    if t is None:
        return 0, 0, 0
    code, strides = _TYPES.get(t.dtype, E4M3), t.stride()
    if t.shape != shape or t.get_device() != device or code == E4M3 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be a tensor of {tuple(shape)} elements of a supported dtype on cuda:{device} with contiguous rows, "
                         f"not {tuple(t.shape)} of {t.dtype} on {t.device}")
    return t.data_ptr(), code, strides[0] if shape[0] > 1 else shape[1]


def ninfer_norm(x, weight=None, eps: float = 1e-6, residual=None, sum=None, gate=None, group=None, weight_offset: float = 0.0,
                out=None, out_dtype=None):
    """Root-mean-square norm of x (rows, cols), of x + residual where one is given (its sum goes to `sum`, which may be the
    residual itself), over groups of `group` neighbouring columns (all of them unless given), times weight + weight_offset
    (weight: `group` elements), times gate / (1 + e^-gate). All but weight are (rows, cols) with contiguous rows."""
    _TYPES or _types()
    device = _on(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be (rows, cols), not {tuple(shape)}")
    rows, cols = shape
    x_at, x_code, x_stride = _matrix(x, "x", shape, device)
    if out is None:
        out = _torch().empty(shape, dtype=out_dtype or x.dtype, device=x.device)
    r_at, r_code, r_stride = _matrix(residual, "residual", shape, device)
    s_at, s_code, s_stride = _matrix(sum, "sum", shape, device)
    if s_at and s_code != r_code:
        raise ValueError("sum must have the residual's dtype")
    g_at, g_code, g_stride = _matrix(gate, "gate", shape, device)
    o_at, o_code, o_stride = _matrix(out, "out", shape, device)
    group = cols if group is None else group
    w_at, w_code = _vector(weight, "weight", group, device)
    _check(_lib.ninfer_norm(_NORM.pack(x_at, r_at, g_at, w_at, s_at, o_at, rows, cols, group, x_stride, r_stride, g_stride,
                                       s_stride, o_stride, eps, weight_offset, x_code, r_code, g_code, w_code, o_code, 0),
                            _raw_stream(device)))
    return out


def ninfer_rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling="none", factor: float = 1.0, context: float = 0.0,
                              slow: float = 1.0, fast: float = 32.0):
    """The table that ninfer_rotary reads (numpy int64, rotary_dim / 2 turns a position times 2^64, as bits; copy it to the
    GPU) and the magnitude. scaling: "none", "linear", "dimensions" or "turns" (see ninfer_layer.h)."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(ROTARY_SCALINGS)}, not {scaling!r}")
    out, magnitude = np.empty(max(rotary_dim // 2, 0), np.uint64), C.c_float()
    _check(_lib.ninfer_rotary_frequencies(rotary_dim, base, ROTARY_SCALINGS[scaling], factor, context, slow, fast, _np_ptr(out),
                                          C.byref(magnitude)))
    return out.view(np.int64), magnitude.value


def _heads(t, name, tokens, code, device):
    """Address, library dtype, strides and shape of a (tokens, heads, elements) tensor; `code`: the dtype that it must have, or None."""
    found, strides, shape = _TYPES.get(t.dtype, E4M3), t.stride(), t.shape
    if len(shape) != 3 or shape[0] != tokens or t.get_device() != device or (found != code if code is not None else found == E4M3) or \
            (strides[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must be a tensor of ({tokens}, heads, elements) on cuda:{device} of a supported dtype, one for all, with the "
                         f"last dimension contiguous, not {tuple(shape)} of {t.dtype} on {t.device}")
    return t.data_ptr(), found, strides[0], strides[1], shape


def ninfer_rotary(q, k, positions, frequencies, magnitude: float = 1.0, interleaved: bool = False, q_weight=None, k_weight=None,
                  eps: float = 1e-6, weight_offset: float = 0.0, q_out=None, k_out=None):
    """Rotary positions of queries q (tokens, q_heads, head_dim) and keys k (tokens, kv_heads, head_dim; None: queries
    alone), in place unless q_out and k_out are given; the first 2 * len(frequencies) elements of a head turn. With
    weights (head_dim elements, one dtype) each head is normed first. Tokens of a negative position are left out."""
    _TYPES or _types()
    device = _on(q, "q")
    tokens = q.shape[0]
    q_at, code, q_token, q_head, shape = _heads(q, "q", tokens, None, device)
    q_heads, dim = shape[1], shape[2]
    o_at, o_token, o_head = q_at, q_token, q_head
    if q_out is not None:
        o_at, _, o_token, o_head, o_shape = _heads(q_out, "q_out", tokens, code, device)
        if o_shape != shape:
            raise ValueError("q_out must have the shape and dtype of q")
    k_at = k_token = k_head = kv_heads = p_at = p_token = p_head = 0
    if k is not None:
        k_at, _, k_token, k_head, k_shape = _heads(k, "k", tokens, code, device)
        kv_heads = k_shape[1]
        if k_shape[2] != dim:
            raise ValueError("q and k must have one dtype and head_dim")
        p_at, p_token, p_head = k_at, k_token, k_head
        if k_out is not None:
            p_at, _, p_token, p_head, p_shape = _heads(k_out, "k_out", tokens, code, device)
            if p_shape != k_shape:
                raise ValueError("k_out must have the shape and dtype of k")
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    turns = frequencies.numel()
    w_at, w_code = _vector(q_weight, "q_weight", dim, device)
    x_at, x_code = _vector(k_weight, "k_weight", dim, device)
    if w_at and x_at and w_code != x_code:
        raise ValueError("q_weight and k_weight must have one dtype")
    _check(_lib.ninfer_rotary(_ROTARY.pack(
        q_at, k_at, w_at, x_at, o_at, p_at, _arg(positions, "positions", _I32, tokens, device),
        _arg(frequencies, "frequencies", _I64, turns, device), tokens, q_heads, kv_heads, dim, 2 * turns, q_token, q_head, k_token,
        k_head, o_token, o_head, p_token, p_head, magnitude, eps, weight_offset, code, w_code or x_code, int(interleaved)),
        _raw_stream(device)))
    return (q if q_out is None else q_out), (k if k_out is None else k_out)


def ninfer_gated_delta_workspace(tokens: int, requests: int, k_heads: int, v_heads: int, k_dim: int, v_dim: int) -> int:
    b = C.c_uint64()
    _check(_lib.ninfer_gated_delta_workspace(tokens, requests, k_heads, v_heads, k_dim, v_dim, C.byref(b)))
    return b.value


def ninfer_gated_delta(q, k, v, log_decay, beta, state, offsets=None, slots=None, lengths=None, scale=None, norm_eps=None, out=None,
                       out_dtype=None, workspace=None, status=None):
    """The gated delta rule: q, k (tokens, k_heads, k_dim), v (tokens, v_heads, v_dim), log_decay and beta float32
    (tokens, v_heads), state float32 (slots, v_heads, k_dim, v_dim), updated in place. offsets (requests + 1): each
    request's tokens, as ninfer_kv_tables gives them; None: one token a request. slots: the state of each request (None: its
    index). lengths: tokens that each state has seen, 0 for one that begins with zeros (None: all are read). scale:
    k_dim ** -0.5 unless given; norm_eps: q and k are divided by sqrt(sum of squares + norm_eps), None: not."""
    _TYPES or _types()
    device = _on(q, "q")
    tokens = q.shape[0]
    q_at, code, q_token, q_head, shape = _heads(q, "q", tokens, None, device)
    k_at, _, k_token, k_head, k_shape = _heads(k, "k", tokens, code, device)
    v_at, _, v_token, v_head, v_shape = _heads(v, "v", tokens, code, device)
    _, k_heads, k_dim = shape
    _, v_heads, v_dim = v_shape
    if k_shape != shape:
        raise ValueError("q and k must have one shape")
    d_at, d_code, d_stride = _matrix(log_decay, "log_decay", (tokens, v_heads), device)
    b_at, b_code, b_stride = _matrix(beta, "beta", (tokens, v_heads), device)
    s_strides, s_shape, whole = state.stride(), state.shape, k_dim * v_dim
    if d_code or b_code or state.dtype is not _F32 or state.get_device() != device:
        raise ValueError(f"log_decay, beta and state must be float32 on cuda:{device}")
    # the strides of contiguous slots; a dimension of one element may have any
    if s_shape[1:] != (v_heads, k_dim, v_dim) or s_strides[1:] != (whole, v_dim, 1) and not state[:1].is_contiguous():
        raise ValueError(f"state must be (slots, {v_heads}, {k_dim}, {v_dim}) with contiguous slots")
    n = s_shape[0]
    requests = tokens if offsets is None else offsets.numel() - 1
    if slots is not None and offsets is None:
        requests = slots.numel()
    if out is None:
        out = _torch().empty(v_shape, dtype=out_dtype or v.dtype, device=v.device)
    w_at = w_bytes = 0
    if workspace is None and offsets is not None:       # single tokens need none
        workspace = _torch().empty(ninfer_gated_delta_workspace(tokens, requests, k_heads, v_heads, k_dim, v_dim), dtype=_torch().uint8, device=q.device)
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
        w_at, w_bytes = workspace.data_ptr(), workspace.nbytes
    o_dtype = out.dtype
    _check(_lib.ninfer_gated_delta(_DELTA.pack(
        q_at, k_at, v_at, d_at, b_at, state.data_ptr(), _arg(slots, "slots", _I32, requests, device),
        _arg(offsets, "offsets", _I32, requests + 1, device), _arg(lengths, "lengths", _I32, requests, device),
        _arg(out, "out", o_dtype, tokens * v_heads * v_dim, device), _arg(status, "status", _I32, 1, device), tokens, requests, n,
        k_heads, v_heads, k_dim, v_dim, q_token, q_head, k_token, k_head, v_token, v_head, d_stride, b_stride,
        s_strides[0] if n > 1 else v_heads * whole, k_dim ** -0.5 if scale is None else scale,
        -1.0 if norm_eps is None else norm_eps, code, _TYPES.get(o_dtype, -1)), w_at, w_bytes, _raw_stream(device)))
    return out


def ninfer_sample(logits, random, temperature=None, top_k=None, top_p=None, min_p=None, out=None, logprobs=None):
    """The next token of each row of logits (rows, vocab), int32 (rows,), by temperature (0: the largest logit), top_k
    (int32, 0: all), top_p and min_p (float32), each (rows,) or None, and random (float32 (rows,), in [0, 1)). logprobs:
    a float32 (rows,) tensor that gets the logarithm of the token's share of what is kept, or None."""
    _TYPES or _types()
    device = _on(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be (rows, vocab), not {tuple(logits.shape)}")
    rows, vocab = logits.shape
    at, code, stride = _matrix(logits, "logits", logits.shape, device)
    if out is None:
        out = _torch().empty(rows, dtype=_I32, device=logits.device)
    _check(_lib.ninfer_sample(_SAMPLE.pack(
        at, _arg(temperature, "temperature", _F32, rows, device), _arg(top_p, "top_p", _F32, rows, device),
        _arg(min_p, "min_p", _F32, rows, device), _arg(top_k, "top_k", _I32, rows, device),
        _arg(random, "random", _F32, rows, device) if random is not None else 0, _arg(out, "out", _I32, rows, device),
        _arg(logprobs, "logprobs", _F32, rows, device), rows, vocab, stride, code, 0), _raw_stream(device)))
    return out
