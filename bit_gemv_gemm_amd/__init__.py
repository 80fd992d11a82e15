"""Python binding of libbgg.so (include/bgg.h), argument marshalling only.

Every function has the name of the C entry point it calls.  Host buffers are
numpy arrays; device buffers are torch tensors on the ROCm device (PyTorch is
used for device memory and streams, nothing else).  A non-OK status raises
BggError carrying the library's message.  There is no fallback: if
libbgg.so is missing, importing this package fails; without the module that
marshals the decoder-layer calls (_marshal, built against one torch) those
calls raise ImportError, and the others, which need libbgg.so alone, work.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct

import numpy as np

# PyTorch ships its own HIP runtime (libamdhip64.so.7, same soname as the
# system one).  libbgg.so must bind to the runtime PyTorch uses, so PyTorch
# is loaded first; loading libbgg.so first would pull the system runtime into
# the process and leave PyTorch running on a runtime it was not built for.
import torch  # noqa: F401  (load order matters, see above)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbgg.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
        "or `python bit_gemv_gemm_amd/build.py` (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)


class _Missing:
    """Stands for the marshalling module that could not be taken: any use
    raises an ImportError with the reason."""

    def __init__(self, why):
        self.why = why

    def __getattr__(self, name):
        raise ImportError(f"the _marshal module of {__name__} is needed for this call: {self.why}; build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'` or `python bit_gemv_gemm_amd/build.py`")


try:
    from . import _marshal
    # (it reads torch's tensors through that torch's own headers)
    _built_with = getattr(_marshal, "torch_version", "?")
    if _built_with != re.match(r"[\d.]*", torch.__version__)[0]:
        _marshal = _Missing(f"it was built with torch {_built_with}, this is {torch.__version__}")
except ImportError as e:
    _marshal = _Missing(str(e))

BGG_FMT_PQ2_0 = 1
BGG_FMT_PTQ1_0 = 2
BGG_FMT_Q1_0 = 3
BGG_FMT_Q2_0_G64 = 4
FORMATS = {"PQ2_0": BGG_FMT_PQ2_0, "PTQ1_0": BGG_FMT_PTQ1_0, "Q1_0": BGG_FMT_Q1_0,
           "Q2_0_G64": BGG_FMT_Q2_0_G64}
BGG_ROTATE_INPUT = 1
BGG_GROUP = 128
BGG_ROW_TILE = 64
BGG_CHUNK = 16
BGG_MAX_GEMV_M = 16
BGG_READ_SLACK = 8192
BGG_ACT_NONE = 0
BGG_ACT_RELU = 1
BGG_ACT_RELU2 = 2
BGG_ACT_SILU = 3
BGG_ACT_GELU = 4
BGG_ACT_GELU_TANH = 5
ACTIVATIONS = {"none": BGG_ACT_NONE, "relu": BGG_ACT_RELU, "relu2": BGG_ACT_RELU2, "silu": BGG_ACT_SILU,
               "gelu": BGG_ACT_GELU, "gelu_tanh": BGG_ACT_GELU_TANH}
BGG_TYPE_F16 = 1
BGG_TYPE_BF16 = 2
BGG_TYPE_E4M3 = 3
TYPES = {"f16": BGG_TYPE_F16, "bf16": BGG_TYPE_BF16, "e4m3": BGG_TYPE_E4M3}
BGG_ROTARY_HALF = 0
BGG_ROTARY_INTERLEAVED = 1
ROTARY_LAYOUTS = {"half": BGG_ROTARY_HALF, "interleaved": BGG_ROTARY_INTERLEAVED}
BGG_ROTARY_NONE = 0
BGG_ROTARY_LINEAR = 1
BGG_ROTARY_BASE = 2
BGG_ROTARY_PARTS = 3
ROTARY_SCALINGS = {"none": BGG_ROTARY_NONE, "linear": BGG_ROTARY_LINEAR, "base": BGG_ROTARY_BASE,
                   "parts": BGG_ROTARY_PARTS}
BGG_AXES_BLOCKS = 0
BGG_AXES_CYCLIC = 1
AXES_ARRANGEMENTS = {"blocks": BGG_AXES_BLOCKS, "cyclic": BGG_AXES_CYCLIC}
BGG_MAX_AXES = 4
STATUS = {0: "BGG_OK", 1: "BGG_ERR_NULL", 2: "BGG_ERR_FORMAT", 3: "BGG_ERR_SHAPE",
          4: "BGG_ERR_TRIT", 5: "BGG_ERR_PACKED_BYTE", 6: "BGG_ERR_BUFFER", 7: "BGG_ERR_DESC",
          8: "BGG_ERR_HIP", 9: "BGG_ERR_SCALE"}


class bgg_weights_desc(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("format", ctypes.c_int32), ("row_tile", ctypes.c_int32),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("row_tiles", ctypes.c_int64), ("row_bytes", ctypes.c_int64),
                ("chunks", ctypes.c_int64), ("trit_bytes", ctypes.c_uint64),
                ("scale_offset", ctypes.c_uint64), ("scale_bytes", ctypes.c_uint64),
                ("total_bytes", ctypes.c_uint64), ("format_bytes", ctypes.c_uint64),
                ("scale_group", ctypes.c_int64), ("scales", ctypes.c_int64)]

    def __repr__(self):
        return "bgg_weights_desc(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class bgg_cache_desc(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("type", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("page_bytes", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64)]

    def __repr__(self):
        return "bgg_cache_desc(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


# the argument structs of the epilogue and of the calls on a cache, in the
# field order of bgg.h, for calls of libbgg.so past _marshal (which fills the
# C structs themselves)
_EPILOGUE = struct.Struct("@iiPPPqq")
_ROTARY_ARGS = struct.Struct("@iiqqqPPPPqqqqPPPfiPPPP")
_ATTENTION_ARGS = struct.Struct("@ifqqqPPqqPPPPPPqqPPN")
_ROTARY_AXES_ARGS = struct.Struct("@qqP")
_SHARED_ARGS = struct.Struct("@qPP")
_ASSIGN_ARGS = struct.Struct("@qqPPPPqqPqPPPPPPP")


class BggError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.bgg_last_error().decode()
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")


_P = ctypes.POINTER(bgg_weights_desc)
_PC = ctypes.POINTER(bgg_cache_desc)
_f64 = ctypes.c_double
_vp, _i64, _u32, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int32, ctypes.c_size_t
_SIGS = {
    "bgg_describe": ([_i32, _i64, _i64, _P], _i32),
    "bgg_pack_weights": ([_P, _vp, _vp, _vp], _i32),
    "bgg_repack_canonical": ([_P, _vp, _vp, _vp], _i32),
    "bgg_validate_packed": ([_P, _vp], _i32),
    "bgg_unpack_weights": ([_P, _vp, _vp, _vp, _vp], _i32),
    "bgg_hadamard_rotate": ([_vp, _vp, _i64, _i64, _vp], _i32),
    "bgg_rotate_ternarize": ([_vp, _i64, _i64, _vp, _vp, _vp], _i32),
    "bgg_gemv_workspace_size": ([_P, _i64], _sz),
    "bgg_gemv_workspace_reset": ([_vp, _sz, _vp], _i32),
    "bgg_ternary_gemv": ([_P, _vp, _vp, _vp, _i64, _u32, _vp, _sz, _vp], _i32),
    "bgg_ternary_gemv_noalloc": ([_P, _vp, _vp, _vp, _i64, _u32, _vp], _i32),
    "bgg_gemv_prepare": ([_P, _vp, _i64, _u32, _vp, _sz, _vp], _i32),
    "bgg_gemv_run": ([_P, _vp, _vp, _i64, _vp, _sz, _vp], _i32),
    "bgg_gemv_kernel_name": ([_P, _i64, ctypes.c_char_p, _sz], _i32),
    "bgg_gemm_workspace_size": ([_P, _i64], _sz),
    "bgg_ternary_gemm": ([_P, _vp, _vp, _vp, _i64, _u32, _vp, _sz, _vp], _i32),
    "bgg_ternary_gemv_epilogue": ([_P, _vp, _vp, _vp, _i64, _u32, _vp, _vp, _sz, _vp], _i32),
    "bgg_gemv_run_epilogue": ([_P, _vp, _vp, _i64, _vp, _vp, _sz, _vp], _i32),
    "bgg_ternary_gemm_epilogue": ([_P, _vp, _vp, _vp, _i64, _u32, _vp, _vp, _sz, _vp], _i32),
    "bgg_cache_describe": ([_i32, _i64, _i64, _i64, _i64, _PC], _i32),
    "bgg_rotary_frequencies": ([_i64, _f64, _i32, _f64, _f64, _f64, _f64, _vp, _vp], _i32),
    "bgg_rotary_append": ([_PC, _vp, _vp], _i32),
    "bgg_rotary_axes": ([_vp, _i64, _i32, _vp], _i32),
    "bgg_rotary_append_axes": ([_PC, _vp, _vp, _vp], _i32),
    "bgg_cache_assign": ([_PC, _vp, _vp], _i32),
    "bgg_attention_workspace_size": ([_PC, _i64, _i64], _sz),
    "bgg_paged_attention": ([_PC, _vp, _vp], _i32),
    "bgg_shared_attention_workspace_size": ([_PC, _i64, _i64], _sz),
    "bgg_shared_attention": ([_PC, _vp, _vp, _vp], _i32),
    "bgg_status_string": ([_i32], ctypes.c_char_p),
    "bgg_last_error": ([], ctypes.c_char_p),
    "bgg_abi_version": ([], _u32),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = tuple(_SIGS)


def _ok(status: int, where: str):
    if status != 0:
        raise BggError(status, where)


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _host_ptr(a, dtype, shape=None):
    a = np.ascontiguousarray(a)
    if a.dtype == np.float16 and dtype == np.uint16:
        a = a.view(np.uint16)
    if a.dtype != dtype:
        raise TypeError(f"expected {np.dtype(dtype)}, got {a.dtype}")
    if shape is not None and tuple(a.shape) != tuple(shape):
        raise ValueError(f"expected shape {shape}, got {a.shape}")
    return a, a.ctypes.data


def _dev_ptr(t, min_bytes=0, what="buffer"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    nbytes = t.numel() * t.element_size()
    if nbytes < min_bytes:
        raise ValueError(f"{what} has {nbytes} bytes, needs {min_bytes}")
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------------------
# host calls
# ---------------------------------------------------------------------------
def bgg_describe(fmt, N: int, K: int) -> bgg_weights_desc:
    d = bgg_weights_desc()
    _ok(_lib.bgg_describe(_fmt(fmt), N, K, ctypes.byref(d)), "bgg_describe")
    return d


def bgg_pack_weights(desc: bgg_weights_desc, trits, scales) -> np.ndarray:
    """Host int8 trits [N][K] and fp16 scales [N][K/128] -> packed bytes (host)."""
    t, tp = _host_ptr(trits, np.int8, (desc.N, desc.K))
    s, sp = _host_ptr(scales, np.uint16, (desc.N, desc.scales))
    out = np.empty(desc.total_bytes, dtype=np.uint8)
    _ok(_lib.bgg_pack_weights(ctypes.byref(desc), tp, sp, out.ctypes.data), "bgg_pack_weights")
    return out


def bgg_repack_canonical(desc: bgg_weights_desc, canonical, scales) -> np.ndarray:
    c, cp = _host_ptr(canonical, np.uint8, (desc.N, desc.row_bytes))
    s, sp = _host_ptr(scales, np.uint16, (desc.N, desc.scales))
    out = np.empty(desc.total_bytes, dtype=np.uint8)
    _ok(_lib.bgg_repack_canonical(ctypes.byref(desc), cp, sp, out.ctypes.data), "bgg_repack_canonical")
    return out


def bgg_validate_packed(desc: bgg_weights_desc, packed) -> None:
    p, pp = _host_ptr(packed, np.uint8)
    if p.size < desc.total_bytes:
        raise ValueError("packed buffer too small")
    _ok(_lib.bgg_validate_packed(ctypes.byref(desc), pp), "bgg_validate_packed")


def bgg_status_string(status: int) -> str:
    return _lib.bgg_status_string(status).decode()


def bgg_last_error() -> str:
    return _lib.bgg_last_error().decode()


def bgg_abi_version() -> int:
    return int(_lib.bgg_abi_version())


def bgg_gemv_workspace_size(desc: bgg_weights_desc, M: int) -> int:
    return int(_lib.bgg_gemv_workspace_size(ctypes.byref(desc), M))


def bgg_gemv_kernel_name(desc: bgg_weights_desc, M: int) -> str:
    buf = ctypes.create_string_buffer(96)
    _ok(_lib.bgg_gemv_kernel_name(ctypes.byref(desc), M, buf, len(buf)), "bgg_gemv_kernel_name")
    return buf.value.decode()


def bgg_gemm_workspace_size(desc: bgg_weights_desc, M: int) -> int:
    return int(_lib.bgg_gemm_workspace_size(ctypes.byref(desc), M))


# ---------------------------------------------------------------------------
# device calls (torch tensors on the ROCm device)
# ---------------------------------------------------------------------------
def bgg_unpack_weights(desc, packed_dev, trits_dev, scales_dev, stream=None) -> None:
    _ok(_lib.bgg_unpack_weights(
        ctypes.byref(desc), _dev_ptr(packed_dev, desc.total_bytes, "packed"),
        _dev_ptr(trits_dev, desc.N * desc.K, "trits"),
        _dev_ptr(scales_dev, desc.N * desc.scales * 2, "scales"), _stream(stream)),
        "bgg_unpack_weights")


def bgg_hadamard_rotate(x_dev, xr_dev, M: int, K: int, stream=None) -> None:
    _ok(_lib.bgg_hadamard_rotate(_dev_ptr(x_dev, M * K * 2, "x"), _dev_ptr(xr_dev, M * K * 2, "xr"),
                                 M, K, _stream(stream)), "bgg_hadamard_rotate")


def bgg_rotate_ternarize(w_dev, N: int, K: int, trits_dev, scales_dev, stream=None) -> None:
    """Device float32 weights [N, K] -> device int8 trits [N, K] and fp16
    scales [N, K/128] in the layer's stored coordinates."""
    _ok(_lib.bgg_rotate_ternarize(_dev_ptr(w_dev, N * K * 4, "w"), N, K,
                                  _dev_ptr(trits_dev, N * K, "trits"),
                                  _dev_ptr(scales_dev, N * (K // 128) * 2, "scales"),
                                  _stream(stream)), "bgg_rotate_ternarize")


def bgg_ternary_gemv(desc, packed_dev, x_dev, y_dev, M: int, flags: int, workspace, stream=None) -> None:
    ws = _dev_ptr(workspace, 0, "workspace")
    wsb = workspace.numel() * workspace.element_size()
    _ok(_lib.bgg_ternary_gemv(ctypes.byref(desc), _dev_ptr(packed_dev, desc.total_bytes, "packed"),
                              _dev_ptr(x_dev, M * desc.K * 2, "x"), _dev_ptr(y_dev, M * desc.N * 2, "y"),
                              M, flags, ws, wsb, _stream(stream)), "bgg_ternary_gemv")


def bgg_gemv_workspace_reset(workspace, stream=None) -> None:
    wsb = workspace.numel() * workspace.element_size()
    _ok(_lib.bgg_gemv_workspace_reset(_dev_ptr(workspace, 0, "workspace"), wsb, _stream(stream)),
        "bgg_gemv_workspace_reset")


def bgg_ternary_gemv_noalloc(desc, packed_dev, x_dev, y_dev, M: int, flags: int, stream=None) -> None:
    _ok(_lib.bgg_ternary_gemv_noalloc(ctypes.byref(desc), _dev_ptr(packed_dev, desc.total_bytes, "packed"),
                                      _dev_ptr(x_dev, M * desc.K * 2, "x"), _dev_ptr(y_dev, M * desc.N * 2, "y"),
                                      M, flags, _stream(stream)), "bgg_ternary_gemv_noalloc")


def bgg_gemv_prepare(desc, x_dev, M: int, flags: int, workspace, stream=None) -> None:
    ws = _dev_ptr(workspace, 0, "workspace")
    wsb = workspace.numel() * workspace.element_size()
    _ok(_lib.bgg_gemv_prepare(ctypes.byref(desc), _dev_ptr(x_dev, M * desc.K * 2, "x"), M, flags, ws,
                              wsb, _stream(stream)), "bgg_gemv_prepare")


def bgg_gemv_run(desc, packed_dev, y_dev, M: int, workspace, stream=None) -> None:
    ws = _dev_ptr(workspace, 0, "workspace")
    wsb = workspace.numel() * workspace.element_size()
    _ok(_lib.bgg_gemv_run(ctypes.byref(desc), _dev_ptr(packed_dev, desc.total_bytes, "packed"),
                          _dev_ptr(y_dev, M * desc.N * 2, "y"), M, ws, wsb, _stream(stream)),
        "bgg_gemv_run")


def bgg_ternary_gemm(desc, packed_dev, x_dev, y_dev, M: int, flags: int, workspace, stream=None) -> None:
    ws = _dev_ptr(workspace, 0, "workspace") if workspace is not None else None
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _ok(_lib.bgg_ternary_gemm(ctypes.byref(desc), _dev_ptr(packed_dev, desc.total_bytes, "packed"),
                              _dev_ptr(x_dev, M * desc.K * 2, "x"), _dev_ptr(y_dev, M * desc.N * 2, "y"),
                              M, flags, ws, wsb, _stream(stream)), "bgg_ternary_gemm")


# the current stream's handle and the current device without building
# objects (1 us of a call's 8)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

# The calls below check and marshal their tensors in _marshal (C++: in Python
# that takes longer than most of the kernels) and then call libbgg.so.
if not isinstance(_marshal, _Missing):
    _marshal.bind(*(ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value for n in (
        "bgg_paged_attention", "bgg_rotary_append", "bgg_ternary_gemv_epilogue", "bgg_gemv_run_epilogue",
        "bgg_ternary_gemm_epilogue", "bgg_rotary_append_axes", "bgg_cache_assign", "bgg_shared_attention")))


def _run_on(where, on, stream, call, *args):
    """call(*args, stream) with the device of tensor `on` current."""
    dev = on.get_device()
    if dev < 0 or _current_device() == dev:
        st = call(*args, (_raw_stream(dev) if dev >= 0 else 0) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            st = call(*args, _raw_stream(dev) if stream is None else _stream(stream))
    if st != 0:
        raise BggError(st, where)


# ---------------------------------------------------------------------------
# products with an epilogue
# ---------------------------------------------------------------------------
def bgg_ternary_gemv_epilogue(desc, packed_dev, x_dev, y_dev, M: int, flags: int, workspace, activation="none",
                              bias=None, mul=None, residual=None, stream=None) -> None:
    """y = act(W x' + bias) * mul + residual, 1 <= M <= 16 tokens; bias [N],
    mul and residual [M, N] (rows of any stride), all float16 or None."""
    _run_on("bgg_ternary_gemv_epilogue", y_dev, stream, _marshal.product, 0, desc, packed_dev, x_dev, y_dev, M, flags,
            workspace, ACTIVATIONS[activation] if isinstance(activation, str) else activation, bias, mul, residual)


def bgg_gemv_run_epilogue(desc, packed_dev, y_dev, M: int, workspace, activation="none", bias=None, mul=None,
                          residual=None, stream=None) -> None:
    """bgg_gemv_run with an epilogue (see bgg_ternary_gemv_epilogue)."""
    _run_on("bgg_gemv_run_epilogue", y_dev, stream, _marshal.product, 1, desc, packed_dev, None, y_dev, M, 0, workspace,
            ACTIVATIONS[activation] if isinstance(activation, str) else activation, bias, mul, residual)


def bgg_ternary_gemm_epilogue(desc, packed_dev, x_dev, y_dev, M: int, flags: int, workspace, activation="none",
                              bias=None, mul=None, residual=None, stream=None) -> None:
    """y = act(W x' + bias) * mul + residual for a prompt of M tokens."""
    _run_on("bgg_ternary_gemm_epilogue", y_dev, stream, _marshal.product, 2, desc, packed_dev, x_dev, y_dev, M, flags,
            workspace, ACTIVATIONS[activation] if isinstance(activation, str) else activation, bias, mul, residual)


# ---------------------------------------------------------------------------
# the paged cache, rotary positions and attention
# ---------------------------------------------------------------------------
def bgg_cache_describe(type, pages: int, page_size: int, kv_heads: int, head_dim: int) -> bgg_cache_desc:
    d = bgg_cache_desc()
    _ok(_lib.bgg_cache_describe(TYPES[type] if isinstance(type, str) else int(type), pages, page_size, kv_heads,
                                head_dim, ctypes.byref(d)), "bgg_cache_describe")
    return d


def bgg_rotary_frequencies(rotary_dim: int, base: float, scaling="none", factor: float = 1.0,
                           trained_length: float = 0.0, low: float = 1.0, high: float = 32.0):
    """(float32 numpy [rotary_dim / 2] radians per position, magnitude)."""
    f = np.zeros(max(int(rotary_dim), 0) // 2 + 1, dtype=np.float32)
    m = ctypes.c_float()
    sc = ROTARY_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    _ok(_lib.bgg_rotary_frequencies(rotary_dim, base, sc, factor, trained_length, low, high, f.ctypes.data,
                                    ctypes.addressof(m)), "bgg_rotary_frequencies")
    return f[:rotary_dim // 2].copy(), m.value


def bgg_attention_workspace_size(cache: bgg_cache_desc, q_heads: int, batch: int) -> int:
    return int(_lib.bgg_attention_workspace_size(ctypes.byref(cache), q_heads, batch))


def bgg_rotary_append(cache: bgg_cache_desc, k_cache, v_cache, positions, slots, freqs, q=None, q_out=None, k=None,
                      v=None, layout="half", magnitude: float = 1.0, k_scale=None, v_scale=None, stream=None) -> None:
    """Rotate q into q_out, and k and v into their slots of the cache.  The
    rotated part of a head is 2 * len(freqs) values.  q, k and v: [T, heads *
    head_dim] (or [T, heads, head_dim]), rows of any stride; positions int32
    [T]; slots int64 [T]; freqs float32."""
    _run_on("bgg_rotary_append", positions, stream, _marshal.rotary_append, cache, k_cache, v_cache, positions, slots,
            freqs, q, q_out, k, v, ROTARY_LAYOUTS[layout] if isinstance(layout, str) else layout, magnitude, k_scale,
            v_scale)


def bgg_rotary_axes(sections, arrangement="blocks") -> np.ndarray:
    """uint8 [pairs]: the axis whose position turns each pair, with
    sections[a] pairs for axis a."""
    given = np.asarray(sections)
    if given.ndim != 1 or given.dtype.kind not in "iuf":
        raise ValueError("sections must be one whole number per axis")
    with np.errstate(invalid="ignore"):
        s = np.ascontiguousarray(given, dtype=np.int64)
    if (s != given).any():
        raise ValueError("sections must be one whole number per axis")
    out = np.zeros(128, dtype=np.uint8)
    kind = AXES_ARRANGEMENTS[arrangement] if isinstance(arrangement, str) else int(arrangement)
    _ok(_lib.bgg_rotary_axes(s.ctypes.data, s.size, kind, out.ctypes.data), "bgg_rotary_axes")
    return out[:int(s.sum())].copy()


def bgg_rotary_append_axes(cache: bgg_cache_desc, k_cache, v_cache, positions, axes, slots, freqs, q=None, q_out=None,
                           k=None, v=None, layout="half", magnitude: float = 1.0, k_scale=None, v_scale=None,
                           stream=None) -> None:
    """bgg_rotary_append for tokens with several positions: positions int32
    [A, T] (rows of any stride; one row expanded to A is one position on every
    axis), axes uint8 [len(freqs)], the row whose position turns each pair
    (bgg_rotary_axes)."""
    _run_on("bgg_rotary_append_axes", positions, stream, _marshal.rotary_append_axes, cache, k_cache, v_cache, positions,
            axes, slots, freqs, q, q_out, k, v, ROTARY_LAYOUTS[layout] if isinstance(layout, str) else layout, magnitude,
            k_scale, v_scale)


def bgg_cache_assign(cache: bgg_cache_desc, lengths, counts, page_table, free_pages, free_count, lengths_out,
                     free_count_out, past, starts, positions, slots, shared_pages=None, stream=None) -> None:
    """The bookkeeping of a batch's step: counts[b] new tokens for sequence b
    (below 0: that many given back) get pages from the stack free_pages, and
    every row of the step its position and slot.  lengths, counts,
    lengths_out, past, shared_pages: int32 [B]; page_table int32 [B, pages];
    free_pages int32; free_count, free_count_out int32 [1]; starts int32
    [B + 1]; positions int32 [T]; slots int64 [T].  lengths_out may be
    lengths, and free_count_out free_count."""
    _run_on("bgg_cache_assign", lengths, stream, _marshal.cache_assign, cache, lengths, counts, page_table, free_pages,
            free_count, lengths_out, free_count_out, past, starts, positions, slots, shared_pages)


def bgg_paged_attention(cache: bgg_cache_desc, k_cache, v_cache, page_table, lengths, q, out, workspace,
                        scale: float, window: int = 0, lse=None, k_scale=None, v_scale=None, stream=None) -> None:
    """Attention of one new token per sequence.  q and out: [B, heads *
    head_dim] (or [B, heads, head_dim]), rows of any stride; page_table int32
    [B, pages]; lengths int32 [B]; lse None or float32 [B, heads]."""
    _run_on("bgg_paged_attention", q, stream, _marshal.paged_attention, cache, k_cache, v_cache, page_table, lengths, q,
            out, workspace, scale, window, lse, k_scale, v_scale)


def bgg_shared_attention_workspace_size(cache: bgg_cache_desc, q_heads: int, batch: int) -> int:
    return int(_lib.bgg_shared_attention_workspace_size(ctypes.byref(cache), q_heads, batch))


def bgg_shared_attention(cache: bgg_cache_desc, k_cache, v_cache, page_table, lengths, group_starts, shared_pages, q, out,
                         workspace, scale: float, window: int = 0, lse=None, k_scale=None, v_scale=None,
                         stream=None) -> None:
    """bgg_paged_attention of a batch whose groups share their first pages,
    which are read once per group: sequences group_starts[g] ..
    group_starts[g + 1] - 1 share those of the first shared_pages[
    group_starts[g]] table entries.  group_starts int32 [G + 1], shared_pages
    int32 [B]."""
    _run_on("bgg_shared_attention", q, stream, _marshal.shared_attention, cache, k_cache, v_cache, page_table, lengths, q,
            out, workspace, scale, window, lse, k_scale, v_scale, group_starts, shared_pages)


# ---------------------------------------------------------------------------
# small conveniences over the calls above (allocation through torch)
# ---------------------------------------------------------------------------
def upload(host_bytes: np.ndarray, device="cuda"):
    """Copy a packed host buffer to a new device uint8 tensor."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(host_bytes)).to(device)


def workspace(nbytes: int, device="cuda"):
    """A zero-filled device workspace (the GEMV's split-K row sums must start
    at zero; every GEMV call leaves them so)."""
    import torch
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)
