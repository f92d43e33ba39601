"""Layout-permuting tile copy for AMD MI355X (gfx950): Python binding of libtile_copy.so.

Thin ctypes marshalling over the C ABI declared in ``include/tile_copy.h``; every step of
the copy (planning, kernels) runs in the native library.  Names match the C entry points:
``tile_copy``, ``tile_copy_ex``, ``tc_plan``, ``tc_last_error``, ``tc_set_flags``,
``tc_get_flags``, ``tc_layout_slice``, ``tc_version``, ``tc_paged_append``, ``tc_paged_attention``,
``tc_paged_evict`` (these three take torch tensors and a ``PagedCache``).

Layouts are ``(shape, stride, offset)`` tuples in elements (TileLayout S[shape : stride]),
or ``TcLayout`` structs.  Source and destination are device pointers (ints) or torch
tensors (their ``data_ptr()`` is the base the layout offsets count from).
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple, Union

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtile_copy.so")

TC_MAX_RANK = 8

# dtypes (enum tc_dtype)
TC_U8, TC_I8, TC_F16, TC_BF16, TC_F32, TC_I32, TC_F64, TC_I64, TC_B128, TC_E4M3 = range(10)
ELEM_BYTES = {TC_E4M3: 1, TC_U8: 1, TC_I8: 1, TC_F16: 2, TC_BF16: 2, TC_F32: 4, TC_I32: 4, TC_F64: 8, TC_I64: 8, TC_B128: 16}
DTYPE_BY_NAME = {"uint8": TC_U8, "int8": TC_I8, "float16": TC_F16, "bfloat16": TC_BF16, "float32": TC_F32,
                 "int32": TC_I32, "float64": TC_F64, "int64": TC_I64, "int4vec": TC_B128, "float8_e4m3fn": TC_E4M3}

# status codes (enum tc_status)
TC_OK = 0
TC_E_NULL, TC_E_RANK, TC_E_EXTENT, TC_E_DTYPE, TC_E_ALIGN, TC_E_NONINJECTIVE, TC_E_ALIAS, \
    TC_E_DECLINED, TC_E_HIP, TC_E_RANGE, TC_E_ARG = range(-1, -12, -1)
STATUS_NAMES = {0: "TC_OK", -1: "TC_E_NULL", -2: "TC_E_RANK", -3: "TC_E_EXTENT", -4: "TC_E_DTYPE",
                -5: "TC_E_ALIGN", -6: "TC_E_NONINJECTIVE", -7: "TC_E_ALIAS", -8: "TC_E_DECLINED",
                -9: "TC_E_HIP", -10: "TC_E_RANGE", -11: "TC_E_ARG"}

# flags
TC_FLAG_STRICT = 0x01
TC_FLAG_FORCE_GUARDED = 0x02
TC_FLAG_FORCE_REGS = 0x04
TC_FLAG_FORCE_LDS = 0x08
TC_FLAG_NO_SWIZZLE = 0x10
TC_FLAG_NO_SHUFFLE = 0x20

# paths (enum tc_path)
TC_PATH_EMPTY, TC_PATH_TRANSPOSE, TC_PATH_ROWS, TC_PATH_ROUNDTRIP, TC_PATH_GUARDED_TILE, \
    TC_PATH_GUARDED_ROWS, TC_PATH_SHUFFLE, TC_PATH_INTERLEAVE = range(8)
PATH_NAMES = {0: "empty", 1: "transpose", 2: "rows", 3: "roundtrip", 4: "guarded_tile", 5: "guarded_rows",
              6: "shuffle", 7: "interleave"}


class TcLayout(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("reserved", ctypes.c_int32), ("offset", ctypes.c_int64),
                ("shape", ctypes.c_int64 * TC_MAX_RANK), ("stride", ctypes.c_int64 * TC_MAX_RANK)]

    def as_tuple(self):
        r = self.rank
        return tuple(self.shape[:r]), tuple(self.stride[:r]), int(self.offset)


class TcPlanInfo(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("elem_bytes", ctypes.c_int32), ("count", ctypes.c_int64),
                ("rank", ctypes.c_int32), ("declined", ctypes.c_int32),
                ("extent", ctypes.c_int64 * TC_MAX_RANK), ("src_stride", ctypes.c_int64 * TC_MAX_RANK),
                ("dst_stride", ctypes.c_int64 * TC_MAX_RANK), ("src_offset", ctypes.c_int64),
                ("dst_offset", ctypes.c_int64), ("threads", ctypes.c_int32), ("vec_bytes", ctypes.c_int32),
                ("load_outer", ctypes.c_int32), ("store_outer", ctypes.c_int32), ("mode_r", ctypes.c_int32),
                ("mode_c", ctypes.c_int32), ("mode_b", ctypes.c_int32), ("tile_r", ctypes.c_int32),
                ("tile_c", ctypes.c_int32), ("tile_b", ctypes.c_int32), ("workgroups", ctypes.c_int64),
                ("lds_bytes", ctypes.c_int32), ("xor_k", ctypes.c_int32), ("xor_shift", ctypes.c_int32),
                ("xor_mask", ctypes.c_int32), ("xor_tbit", ctypes.c_int32), ("xor_cshift", ctypes.c_int32),
                ("xor_cmask", ctypes.c_int32), ("grid_order", ctypes.c_int32), ("nontemporal", ctypes.c_int32),
                ("unaligned", ctypes.c_int32), ("src_step", ctypes.c_int32), ("wave_local", ctypes.c_int32),
                ("lds_write_bytes", ctypes.c_int32), ("lds_read_bytes", ctypes.c_int32), ("edge_tiles", ctypes.c_int32),
                ("loads_in_flight", ctypes.c_int32), ("super_rows", ctypes.c_int32), ("super_cols", ctypes.c_int32),
                ("src_view_bytes", ctypes.c_int32),
                ("write_conflicts", ctypes.c_int64),
                ("read_conflicts", ctypes.c_int64), ("reason", ctypes.c_char * 192)]

    def to_dict(self) -> dict:
        d = {}
        for name, _ in self._fields_:
            v = getattr(self, name)
            if name == "reason":
                v = v.decode()
            elif name in ("extent", "src_stride", "dst_stride"):
                v = tuple(v[: self.rank])
            d[name] = v
        d["path_name"] = PATH_NAMES.get(self.path, "?")
        return d


class TcPermuteInfo(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("elements_per_lane", ctypes.c_int32),
                ("extent", ctypes.c_int64 * TC_MAX_RANK), ("src_stride", ctypes.c_int64 * TC_MAX_RANK),
                ("dst_stride", ctypes.c_int64 * TC_MAX_RANK), ("k", ctypes.c_int32), ("shift", ctypes.c_int32),
                ("mask", ctypes.c_int32), ("reserved", ctypes.c_int32), ("read_conflicts", ctypes.c_int64),
                ("write_conflicts", ctypes.c_int64), ("reason", ctypes.c_char * 192)]

    def to_dict(self) -> dict:
        d = {}
        for name, _ in self._fields_:
            v = getattr(self, name)
            if name == "reason":
                v = v.decode()
            elif name in ("extent", "src_stride", "dst_stride"):
                v = tuple(v[: self.rank])
            d[name] = v
        return d


class TileCopyError(RuntimeError):
    def __init__(self, code: int, reason: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {reason}")
        self.code = code
        self.reason = reason


_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libtile_copy.so; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python layout_permuting_copy_amd/build.py` "
                          "(or __graft_entry__.build()); the copy has no non-native fallback")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.tile_copy.argtypes = [ctypes.c_void_p, P(TcLayout), ctypes.c_void_p, P(TcLayout), ctypes.c_int, ctypes.c_void_p]
    lib.tile_copy.restype = ctypes.c_int
    lib.tile_copy_ex.argtypes = [ctypes.c_void_p, P(TcLayout), ctypes.c_void_p, P(TcLayout), ctypes.c_int,
                                 ctypes.c_void_p, ctypes.c_int, P(TcPlanInfo)]
    lib.tile_copy_ex.restype = ctypes.c_int
    lib.tc_autotune.argtypes = [ctypes.c_void_p, P(TcLayout), ctypes.c_void_p, P(TcLayout), ctypes.c_int,
                                ctypes.c_void_p, ctypes.c_int, ctypes.c_int, P(TcPlanInfo), P(ctypes.c_float)]
    lib.tc_autotune.restype = ctypes.c_int
    lib.tc_plan_variants.argtypes = [P(TcLayout), P(TcLayout), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                     P(TcPlanInfo), ctypes.c_int]
    lib.tc_plan_variants.restype = ctypes.c_int
    lib.tc_plan.argtypes = [P(TcLayout), P(TcLayout), ctypes.c_int, ctypes.c_int, ctypes.c_int, P(TcPlanInfo)]
    lib.tc_plan.restype = ctypes.c_int
    lib.tc_last_error.argtypes = []
    lib.tc_last_error.restype = ctypes.c_char_p
    lib.tc_set_flags.argtypes = [ctypes.c_int]
    lib.tc_set_flags.restype = ctypes.c_int
    lib.tc_get_flags.argtypes = []
    lib.tc_get_flags.restype = ctypes.c_int
    i64p = P(ctypes.c_int64)
    lib.tc_layout_slice.argtypes = [P(TcLayout), i64p, i64p, i64p, P(TcLayout)]
    lib.tc_layout_slice.restype = ctypes.c_int
    lib.tc_version.argtypes = []
    lib.tc_version.restype = ctypes.c_int
    lib.tc_wave_permute_plan.argtypes = [P(TcLayout), P(TcLayout), ctypes.c_int, P(TcPermuteInfo)]
    lib.tc_wave_permute_plan.restype = ctypes.c_int
    vp, lp, i64, i32 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.tc_paged_append.argtypes = [vp, vp, lp, vp, lp, i32, vp, lp, vp, vp, vp, lp, vp]
    lib.tc_paged_append.restype = ctypes.c_int
    lib.tc_paged_attention_workspace.argtypes = [i64, i64, i64, i64, i64, i32]
    lib.tc_paged_attention_workspace.restype = ctypes.c_int64
    lib.tc_paged_attention.argtypes = [vp, vp, lp, vp, lp, i32, vp, lp, vp, i64, ctypes.c_float, vp, lp, vp, lp, vp, lp, vp,
                                       i64, vp]
    lib.tc_paged_attention.restype = ctypes.c_int
    lib.tc_paged_evict.argtypes = [vp, vp, lp, vp, i64, vp, lp, vp, vp, lp, i64, i64, vp, vp, lp, vp, lp, vp]
    lib.tc_paged_evict.restype = ctypes.c_int
    _lib = lib
    return lib


LayoutLike = Union[TcLayout, Tuple[Sequence[int], Sequence[int], int], Tuple[Sequence[int], Sequence[int]]]


def make_layout(shape: Sequence[int], stride: Optional[Sequence[int]] = None, offset: int = 0) -> TcLayout:
    """TileLayout S[shape : stride] with an element offset (row-major strides by default)."""
    shape = [int(e) for e in shape]
    if stride is None:
        stride, acc = [], 1
        for e in reversed(shape):
            stride.append(acc)
            acc *= e
        stride.reverse()
    if len(shape) != len(stride) or len(shape) > TC_MAX_RANK:
        raise ValueError("shape and stride must have the same length, at most 8")
    lay = TcLayout()
    lay.rank = len(shape)
    lay.offset = int(offset)
    for k, (e, s) in enumerate(zip(shape, stride)):
        lay.shape[k] = e
        lay.stride[k] = int(s)
    return lay


def _as_layout(x: LayoutLike) -> TcLayout:
    if isinstance(x, TcLayout):
        return x
    if len(x) == 2:
        return make_layout(x[0], x[1], 0)
    return make_layout(x[0], x[1], x[2])


def _ptr(x) -> int:
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    raise TypeError("expected a device pointer (int) or a tensor")


def _stream(stream) -> int:
    if stream is None:
        try:
            import torch
            if torch.cuda.is_available():
                return int(torch.cuda.current_stream().cuda_stream)
        except ImportError:
            pass
        return 0
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def tc_last_error() -> str:
    return load_library().tc_last_error().decode()


def _check(rc: int) -> int:
    if rc != TC_OK:
        raise TileCopyError(rc, tc_last_error())
    return rc


def tile_copy(src, src_layout: LayoutLike, dst, dst_layout: LayoutLike, dtype: int, stream=None) -> None:
    """dst[dst_layout(i)] = src[src_layout(i)] for every logical index i, on `stream`
    (default: torch's current stream).  Raises TileCopyError on a non-zero status."""
    lib = load_library()
    s, d = _as_layout(src_layout), _as_layout(dst_layout)
    _check(lib.tile_copy(_ptr(src), ctypes.byref(s), _ptr(dst), ctypes.byref(d), int(dtype), _stream(stream)))


def tile_copy_ex(src, src_layout: LayoutLike, dst, dst_layout: LayoutLike, dtype: int, stream=None,
                 flags: int = 0) -> dict:
    """tile_copy with explicit flags; returns the plan that ran (as a dict)."""
    lib = load_library()
    s, d = _as_layout(src_layout), _as_layout(dst_layout)
    info = TcPlanInfo()
    _check(lib.tile_copy_ex(_ptr(src), ctypes.byref(s), _ptr(dst), ctypes.byref(d), int(dtype), _stream(stream),
                            int(flags), ctypes.byref(info)))
    return info.to_dict()


def tc_autotune(src, src_layout: LayoutLike, dst, dst_layout: LayoutLike, dtype: int, stream=None, flags: int = 0,
                reps: int = 5) -> dict:
    """tile_copy_ex that times the copy on the library's candidate configurations and keeps the
    fastest as the cached plan of these layouts; returns that plan, with its mean time per launch
    in 'tuned_ms'.  Blocks until the timed launches end."""
    lib = load_library()
    s, d = _as_layout(src_layout), _as_layout(dst_layout)
    info = TcPlanInfo()
    ms = ctypes.c_float(0.0)
    _check(lib.tc_autotune(_ptr(src), ctypes.byref(s), _ptr(dst), ctypes.byref(d), int(dtype), _stream(stream),
                           int(flags), int(reps), ctypes.byref(info), ctypes.byref(ms)))
    out = info.to_dict()
    out["tuned_ms"] = float(ms.value)
    return out


def tc_plan(src_layout: LayoutLike, dst_layout: LayoutLike, dtype: int, flags: int = 0, ptr_align: int = 16,
            raise_on_error: bool = True) -> dict:
    """Host-only plan of a copy (no GPU).  With raise_on_error=False the dict carries
    'status' and 'error' instead of raising."""
    lib = load_library()
    s, d = _as_layout(src_layout), _as_layout(dst_layout)
    info = TcPlanInfo()
    rc = lib.tc_plan(ctypes.byref(s), ctypes.byref(d), int(dtype), int(flags), int(ptr_align), ctypes.byref(info))
    out = info.to_dict()
    out["status"] = rc
    out["error"] = tc_last_error() if rc != TC_OK else ""
    if rc != TC_OK and raise_on_error:
        raise TileCopyError(rc, out["error"])
    return out


def tc_plan_variants(src_layout: LayoutLike, dst_layout: LayoutLike, dtype: int, flags: int = 0,
                     ptr_align: int = 16, max_out: int = 64) -> list:
    """Host-only list of the plans tc_autotune would time (the planner's own first)."""
    lib = load_library()
    s, d = _as_layout(src_layout), _as_layout(dst_layout)
    arr = (TcPlanInfo * max_out)()
    n = lib.tc_plan_variants(ctypes.byref(s), ctypes.byref(d), int(dtype), int(flags), int(ptr_align), arr,
                             int(max_out))
    if n < 0:
        raise TileCopyError(n, tc_last_error())
    return [arr[i].to_dict() for i in range(min(n, max_out))]


def tc_set_flags(flags: int) -> int:
    rc = load_library().tc_set_flags(int(flags))
    if rc < 0:
        raise TileCopyError(rc, tc_last_error())
    return rc


def tc_get_flags() -> int:
    return load_library().tc_get_flags()


def tc_layout_slice(layout: LayoutLike, start: Sequence[int], stop: Sequence[int], step: Sequence[int]) -> TcLayout:
    lib = load_library()
    lay = _as_layout(layout)
    n = max(1, lay.rank)
    arr = lambda xs: (ctypes.c_int64 * n)(*[int(x) for x in xs])
    out = TcLayout()
    _check(lib.tc_layout_slice(ctypes.byref(lay), arr(start), arr(stop), arr(step), ctypes.byref(out)))
    return out


def tc_version() -> int:
    return load_library().tc_version()


def tc_wave_permute_plan(src_layout: LayoutLike, dst_layout: LayoutLike, dtype: int,
                         raise_on_error: bool = True) -> dict:
    """Host-only bank plan (k, shift, mask) of the wave-scope permute tcd::wave_permute."""
    lib = load_library()
    s, d = _as_layout(src_layout), _as_layout(dst_layout)
    info = TcPermuteInfo()
    rc = lib.tc_wave_permute_plan(ctypes.byref(s), ctypes.byref(d), int(dtype), ctypes.byref(info))
    out = info.to_dict()
    out["status"] = rc
    out["error"] = tc_last_error() if rc != TC_OK else ""
    if rc != TC_OK and raise_on_error:
        raise TileCopyError(rc, out["error"])
    return out


def torch_dtype_code(torch_dtype) -> int:
    """enum tc_dtype of a torch dtype (by width; the copy moves raw bytes)."""
    import torch
    table = {torch.uint8: TC_U8, torch.int8: TC_I8, torch.float16: TC_F16, torch.bfloat16: TC_BF16,
             torch.float32: TC_F32, torch.int32: TC_I32, torch.float64: TC_F64, torch.int64: TC_I64,
             torch.float8_e4m3fn: TC_E4M3, torch.int16: TC_F16, torch.uint16: TC_F16 if hasattr(torch, "uint16") else TC_F16}
    return table[torch_dtype]


def copy_tensor(dst, src, stream=None) -> dict:
    """dst[...] = src[...] for two device tensors of the same shape and element width, through
    their own strides (views: transposes, permutes, slices, expanded sources): the layouts are the
    tensors' shape and strides from their data pointers.  Returns the plan that ran."""
    if tuple(dst.shape) != tuple(src.shape):
        raise ValueError(f"shapes differ: {tuple(dst.shape)} and {tuple(src.shape)}")
    if dst.element_size() != src.element_size():
        raise ValueError("element widths differ")
    code = torch_dtype_code(src.dtype)
    shape = tuple(int(e) for e in src.shape)
    return tile_copy_ex(src, (shape, tuple(int(s) for s in src.stride()), 0), dst,
                        (shape, tuple(int(s) for s in dst.stride()), 0), code, stream)


# ---- paged key-value cache -------------------------------------------------------------------

class TcPagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_layout", TcLayout), ("v_layout", TcLayout),
                ("k_scale_layout", TcLayout), ("v_scale_layout", TcLayout), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class PagedCache:
    """A pool of pages of keys and values: torch tensors of logical shape (pages, page_size, heads,
    head_dim), any strides with an innermost 1 (transpose a head-major pool into this order), float16,
    bfloat16, or float8_e4m3fn with float32 ``k_scale`` and ``v_scale`` of shape (pages, page_size, heads).
    Holds the tensors; the layouts are read from them once."""

    __slots__ = ("_k", "_v", "_k_scale", "_v_scale", "_c", "_ref", "device", "pages", "page_size", "heads", "head_dim")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _import_torch()
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale
        if k.dtype != v.dtype:
            raise ValueError(f"keys are {k.dtype}, values {v.dtype}")
        self.device = k.device
        c = TcPagedCache()
        c.dtype = _paged_dtype(k)
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.k_layout, c.v_layout = make_layout(k.shape, k.stride()), make_layout(v.shape, v.stride())
        for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
            if (x is not None) != (c.dtype == TC_E4M3):
                raise ValueError("8-bit caches have k_scale and v_scale, others have none")
            if x is not None:
                _want(name, x, _T_F32)
                setattr(c, name, x.data_ptr())
                setattr(c, name + "_layout", make_layout(x.shape, x.stride()))
        _device_of(self, v, k_scale, v_scale)
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError(f"keys and values must have one shape (pages, page_size, heads, head_dim), got {tuple(k.shape)} "
                             f"and {tuple(v.shape)}")
        self.pages, self.page_size, self.heads, self.head_dim = k.shape
        self._c = c
        self._ref = ctypes.addressof(c)

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)


_torch = _here = _raw_stream = None
_T_I32 = _T_F32 = None
_PAGED_DTYPES = {}


def _import_torch():
    """torch and the types the paged entry points name, looked up once."""
    global _torch, _T_I32, _T_F32, _here, _raw_stream
    if _torch is None:
        import torch
        # the current device and stream without the public calls' wrappers (0.1 us each; current_stream() takes 2.5)
        _here = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                       or (lambda index: torch.cuda.current_stream(index).cuda_stream))
        _T_I32, _T_F32 = torch.int32, torch.float32
        _PAGED_DTYPES.update({torch.float16: TC_F16, torch.bfloat16: TC_BF16, torch.float8_e4m3fn: TC_E4M3})
        _torch = torch
    return _torch


def _paged_dtype(x) -> int:
    code = _PAGED_DTYPES.get(x.dtype)
    if code is None:
        raise ValueError(f"expected float16, bfloat16 or (a cache) float8_e4m3fn, got {x.dtype}")
    return code


def _want(name: str, x, dtype) -> None:
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")


def _device_of(cache, *tensors):
    dev = cache.device
    for x in tensors:
        if x is not None and x.device != dev:
            raise ValueError(f"tensors on {dev} and {x.device}")
    return dev


def _vector(name: str, x, n: int) -> int:
    if x.dtype != _T_I32 or x.dim() != 1 or x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{name} must be int32, contiguous, with {n} elements, got {x.dtype} {tuple(x.shape)}")
    return x.data_ptr()


_NONE = (None, None)
_layout_cache = {}


def _lay(x):
    """(address, owner) of the TcLayout of a tensor's shape and strides (made once per shape and strides)."""
    key = (x.shape, x.stride())
    at = _layout_cache.get(key)
    if at is None:
        if len(_layout_cache) >= 4096:
            _layout_cache.clear()
        lay = make_layout(key[0], key[1])
        at = _layout_cache[key] = (ctypes.addressof(lay), lay)
    return at


def _enter(dev):
    """Makes the tensors' device current; returns the one to go back to, or None."""
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not {dev}")
    here = _here()
    if here == dev.index:
        return None
    _torch.cuda.set_device(dev)
    return here


def _empty_on(handle, dev, shape, dtype):
    """Memory for this call, allocated on its stream: another stream's next use of it waits its turn."""
    if handle == _raw_stream(dev.index):
        return _torch.empty(shape, dtype=dtype, device=dev)
    with _torch.cuda.stream(_torch.cuda.ExternalStream(handle, device=dev)):
        return _torch.empty(shape, dtype=dtype, device=dev)


_workspace_cache = {}


def _workspace(lib, key) -> int:
    """tc_paged_attention_workspace of these sizes."""
    need = lib.tc_paged_attention_workspace(*key)
    if need < 0:
        _check(need)
    if len(_workspace_cache) >= 4096:
        _workspace_cache.clear()
    _workspace_cache[key] = need
    return need


def tc_paged_append(cache: PagedCache, k, v, block_table, seq_lens, token_starts=None, weights=None,
                    stream=None) -> None:
    """Copies new tokens' keys and values, (tokens, heads, head_dim) float16 or bfloat16 with any outer
    strides, into the cache: as they are, or rounded to e4m3 with a scale a row and head.

    ``block_table`` (batch, columns) int32 names each sequence's pages, ``seq_lens`` (batch) int32 counts its
    rows after the append.  Token b becomes the last row of sequence b; with ``token_starts`` (batch + 1) int32,
    tokens starts[b] .. starts[b + 1] - 1 become its last rows and tokens past starts[batch] are padding.
    ``weights`` (batch, heads, capacity) float32, if given, is zeroed for the new rows."""
    lib = _lib or load_library()
    dev = cache.device
    if k.device != dev or v.device != dev or block_table.device != dev or seq_lens.device != dev:
        _device_of(cache, k, v, block_table, seq_lens)
    if token_starts is not None or weights is not None:
        _device_of(cache, token_starts, weights)
    if k.dtype != v.dtype:
        raise ValueError(f"keys are {k.dtype}, values {v.dtype}")
    _want("block_table", block_table, _T_I32)
    batch = block_table.shape[0]
    lens = _vector("seq_lens", seq_lens, batch)
    starts = None if token_starts is None else _vector("token_starts", token_starts, batch + 1)
    wl, wp = _NONE, None
    if weights is not None:
        _want("weights", weights, _T_F32)
        wl, wp = _lay(weights), weights.data_ptr()
    kl, vl, tl = _lay(k), _lay(v), _lay(block_table)
    back = _enter(dev)
    try:
        rc = lib.tc_paged_append(cache._ref, k.data_ptr(), kl[0], v.data_ptr(), vl[0], _paged_dtype(k),
                                 block_table.data_ptr(), tl[0], lens, starts, wp, wl[0],
                                 _raw_stream(dev.index) if stream is None else _stream(stream))
    finally:
        if back is not None:
            _torch.cuda.set_device(back)
    if rc != TC_OK:
        _check(rc)


def tc_paged_attention(q, cache: PagedCache, block_table, seq_lens, scale: Optional[float] = None,
                       max_len: Optional[int] = None, out=None, lse=None, weights=None, weights_out=None,
                       stream=None):
    """Attention of one new token a sequence, ``q`` (batch, q_heads, head_dim), over its cached rows; returns ``out``.

    ``scale`` defaults to head_dim ** -0.5.  ``lse`` (batch, q_heads) float32 receives the log of the
    sums.  ``weights`` (batch, heads, capacity) float32: ``weights_out`` (default: ``weights`` itself) receives
    weights plus each row's attention weight summed over the query heads of its cache head.

    ``max_len`` bounds ``seq_lens`` (default: what the table's columns hold).  A tight one saves launches and memory,
    whatever the lengths are: from 513 on (1025 for large batches) rows are cut between workgroups and joined by a
    second kernel, and with ``weights`` the call takes batch * q_heads * max_len floats of scratch memory and a grid over
    max_len rows of every sequence (1.07 GB for 64 sequences of 32 heads under a table of 131072 rows).

    No gradient is formed: ``out`` is not part of ``q``'s graph, whether or not ``q`` requires a gradient."""
    lib = _lib or load_library()
    dev = cache.device
    if q.device != dev or block_table.device != dev or seq_lens.device != dev:
        _device_of(cache, q, block_table, seq_lens)
    if out is not None or lse is not None or weights is not None:
        _device_of(cache, out, lse, weights, weights_out)
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be (batch, q_heads, head_dim), block_table (batch, columns)")
    _want("block_table", block_table, _T_I32)
    batch, q_heads, dim = q.shape
    lens = _vector("seq_lens", seq_lens, batch)
    if max_len is None:
        max_len = block_table.shape[1] * cache.page_size
    if scale is None:
        scale = dim ** -0.5
    ll, wl, wol = _NONE, _NONE, _NONE
    lp = wp = wop = None
    if lse is not None:
        _want("lse", lse, _T_F32)
        ll, lp = _lay(lse), lse.data_ptr()
    if weights is not None:
        if weights_out is None:
            weights_out = weights
        _want("weights", weights, _T_F32)
        _want("weights_out", weights_out, _T_F32)
        wl, wol, wp, wop = _lay(weights), _lay(weights_out), weights.data_ptr(), weights_out.data_ptr()
    elif weights_out is not None:
        raise ValueError("weights_out without weights")
    code = _paged_dtype(q)
    ql, tl = _lay(q), _lay(block_table)
    back = _enter(dev)
    try:
        handle = _raw_stream(dev.index) if stream is None else _stream(stream)
        if out is None:
            out = _torch.empty_like(q) if stream is None else _empty_on(handle, dev, q.shape, q.dtype)
        elif out.dtype != q.dtype:
            raise ValueError(f"out is {out.dtype}, q {q.dtype}")
        ol = _lay(out)
        key = (batch, q_heads, cache.heads, dim, max_len, weights is not None)
        need = _workspace_cache.get(key)
        if need is None:
            need = _workspace(lib, key)
        work = _empty_on(handle, dev, need, _torch.uint8) if need else None
        rc = lib.tc_paged_attention(cache._ref, q.data_ptr(), ql[0], out.data_ptr(), ol[0], code, block_table.data_ptr(), tl[0],
                                    lens, max_len, scale, lp, ll[0], wp, wl[0], wop, wol[0],
                                    None if work is None else work.data_ptr(), need, handle)
    finally:
        if back is not None:
            _torch.cuda.set_device(back)
    if rc != TC_OK:
        _check(rc)
    return out


def tc_paged_evict(src: PagedCache, block_table, seq_lens, weights, dst: PagedCache, dst_table, budget: int,
                   recent: int = 0, max_len: Optional[int] = None, lens_out=None, weights_out=None, kept=None,
                   stream=None):
    """Shrinks every sequence to ``budget`` rows a head: the last ``recent`` and the heaviest others by
    ``weights`` (batch, heads, capacity) float32, in their order, copied into the pages that ``dst_table`` names
    in ``dst`` (another pool, or pages of the same one that hold none of the kept rows).  Returns
    ``(lens_out, kept)``: the new lengths, and the rows kept, (batch, heads, min(budget, max_len)) int32 with -1
    past the new length.  ``weights_out`` receives the kept rows' weights."""
    lib = _lib or load_library()
    dev = _device_of(src, block_table, seq_lens, weights, dst, dst_table, lens_out, weights_out, kept)
    if block_table.dim() != 2:
        raise ValueError("block_table must be (batch, columns)")
    batch = block_table.shape[0]
    _want("block_table", block_table, _T_I32)
    _want("dst_table", dst_table, _T_I32)
    _want("weights", weights, _T_F32)
    lens = _vector("seq_lens", seq_lens, batch)
    held = block_table.shape[1] * src.page_size
    max_len = held if max_len is None else min(max_len, held)
    wol, wop = _NONE, None
    if weights_out is not None:
        _want("weights_out", weights_out, _T_F32)
        wol, wop = _lay(weights_out), weights_out.data_ptr()
    tl, wl, dl = _lay(block_table), _lay(weights), _lay(dst_table)
    back = _enter(dev)
    try:
        handle = _raw_stream(dev.index) if stream is None else _stream(stream)
        if lens_out is None:
            lens_out = _empty_on(handle, dev, batch, _T_I32)
        if kept is None:
            kept = _empty_on(handle, dev, (batch, src.heads, max(0, min(budget, max_len))), _T_I32)
        _want("kept", kept, _T_I32)
        kl = _lay(kept)
        rc = lib.tc_paged_evict(src._ref, block_table.data_ptr(), tl[0], lens, max_len, weights.data_ptr(), wl[0],
                                dst._ref, dst_table.data_ptr(), dl[0], budget, recent,
                                _vector("lens_out", lens_out, batch), kept.data_ptr(), kl[0], wop, wol[0], handle)
    finally:
        if back is not None:
            _torch.cuda.set_device(back)
    if rc != TC_OK:
        _check(rc)
    return lens_out, kept
