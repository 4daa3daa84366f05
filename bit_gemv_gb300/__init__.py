"""Python binding of libninfer_ternary.so (the GB300 Hadamard-rotated ternary
projection). Argument marshalling only: every step of the computation runs in
the library's CUDA kernels or its host C++ code. There is no fallback: if the
shared library is missing, importing this package raises ImportError.

Names match the C entry points of include/ninfer_ternary.h and
include/ninfer_decode.h. Host entry points take and return numpy arrays; device entry points take torch CUDA tensors and
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
