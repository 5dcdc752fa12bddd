"""Python binding of libbitq (argument marshalling only).

Every function here forwards to the C ABI of the same name in
bit_plane_gemv_amd/libbitq.so (declared in include/bitq.h); all computation
happens in that library.  Device buffers are passed as torch tensors (their
data_ptr()) or raw integer addresses; PyTorch is used only to own device
memory and to name the current HIP stream.

Importing this package fails loudly if libbitq.so has not been built
(python bit_plane_gemv_amd/build.py); there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# BITQ_LIBRARY selects another build of the same library (the sanitizer
# build of build.py --sanitize); by default the in-tree libbitq.so
LIB_PATH = os.environ.get("BITQ_LIBRARY") or os.path.join(_HERE, "libbitq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libbitq.so not found at {LIB_PATH}; build it with "
                      "`python bit_plane_gemv_amd/build.py`")

# One HIP runtime per process: torch wheels bundle their own libamdhip64, and
# loading libbitq.so first would bind it to the system runtime while torch
# later loads a second one (device pointers and streams are then not shared).
# Importing torch first makes libbitq.so bind to the runtime torch uses.
try:
    import torch as _torch  # noqa: F401
except ImportError:
    _torch = None
_lib = ctypes.CDLL(LIB_PATH)


def _hip_runtimes() -> list:
    try:
        with open("/proc/self/maps") as f:
            return sorted({ln.split()[-1] for ln in f if "libamdhip64" in ln})
    except OSError:
        return []


if len(_hip_runtimes()) > 1:
    raise ImportError("two HIP runtimes are loaded in this process: " + ", ".join(_hip_runtimes()))

# ------------------------------------------------------------------ enums
OK, E_ARG, E_SHAPE, E_ALIGN, E_UNSUPPORTED, E_CAPACITY, E_DEVICE = 0, -1, -2, -3, -4, -5, -6
SIGN1, RABIT, TERNARY, W2A8, BVSR4, WNAM, HGF = 1, 2, 3, 4, 5, 6, 7
DT_F32, DT_BF16, DT_ACT, DT_BINARY = 0, 1, 2, 3
DT_ROW8 = 16       # bitq_block_norm: int8 rows with a scale each
KV_BF16, KV_INT8 = 0, 1
ROPE_HALF, ROPE_PAIRS = 0, 1                                     # the order of a rotated pair's elements
ROPE_PLAIN, ROPE_LINEAR, ROPE_RAMP, ROPE_BAND = 0, 1, 2, 3       # how frequencies are stretched
F_ACC_INT32 = 1
F_FUSE_QUANT = 2   # bitq_gemv: raw x, the activation quantizer runs in the GEMV kernel

FORMAT_NAMES = {SIGN1: "sign", RABIT: "rabit", TERNARY: "ternary", W2A8: "w2a8", BVSR4: "bvsr",
                WNAM: "wnam", HGF: "hgf"}
FORMATS = {v: k for k, v in FORMAT_NAMES.items()}
DEFAULT_PLANES = {SIGN1: 1, RABIT: 2, TERNARY: 2, W2A8: 2, BVSR4: 4, WNAM: 4, HGF: 2}
DEFAULT_GROUP = {SIGN1: 0, RABIT: 0, TERNARY: 0, W2A8: 128, BVSR4: 32, WNAM: 128, HGF: 0}
DEFAULT_ABITS = {SIGN1: 0, RABIT: 0, TERNARY: 8, W2A8: 8, BVSR4: 8, WNAM: 4, HGF: 8}
DEFAULT_RANK = {HGF: 32}


class BitqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"bitq status {status}: {message}")
        self.status = status


class WDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("planes", ctypes.c_int32), ("group", ctypes.c_int32), ("abits", ctypes.c_int32),
                ("rank", ctypes.c_int32)]


class QuantOpts(ctypes.Structure):
    _fields_ = [("rabit_svid_sweeps", ctypes.c_int32), ("wnam_bit_balance", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 6)]


class Logical(ctypes.Structure):
    _fields_ = [("sign", ctypes.c_void_p), ("tern", ctypes.c_void_p), ("code", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("g", ctypes.c_void_p), ("h", ctypes.c_void_p),
                ("gamma", ctypes.c_float), ("delta", ctypes.c_void_p), ("zero", ctypes.c_void_p),
                ("idx", ctypes.c_void_p), ("cache", ctypes.c_void_p), ("lora_a", ctypes.c_void_p),
                ("lora_b", ctypes.c_void_p), ("lora_alpha", ctypes.c_float)]


class KvDesc(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page", ctypes.c_int32),
                ("pages", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class KvPlanDesc(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_int32), ("page", ctypes.c_int32), ("table_stride", ctypes.c_int32),
                ("ring", ctypes.c_int32), ("tokens", ctypes.c_int32)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("kv", KvDesc), ("heads", ctypes.c_int32), ("requests", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("max_len", ctypes.c_int32), ("window", ctypes.c_int32),
                ("q_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("width", ctypes.c_int32), ("u_dtype", ctypes.c_int32),
                ("r_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("u_stride", ctypes.c_int64), ("r_stride", ctypes.c_int64), ("ro_stride", ctypes.c_int64),
                ("h_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("res_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("eps_post", ctypes.c_float), ("eps_pre", ctypes.c_float)]


class W8A8Desc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("lda", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldy", ctypes.c_int64), ("flags", ctypes.c_uint32)]


class PromptDesc(ctypes.Structure):
    _fields_ = [("kv", KvDesc), ("heads", ctypes.c_int32), ("requests", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("max_len", ctypes.c_int32), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("q_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class SharedDesc(ctypes.Structure):
    _fields_ = [("attn", AttnDesc), ("groups", ctypes.c_int32), ("max_prefix", ctypes.c_int32)]


class KvPagesDesc(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_int32), ("page", ctypes.c_int32), ("table_stride", ctypes.c_int32),
                ("pool", ctypes.c_int32), ("moves", ctypes.c_int32)]


class RopeFreq(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("kind", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("trained", ctypes.c_double), ("turns_keep", ctypes.c_double), ("turns_scale", ctypes.c_double)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("mscale", ctypes.c_float)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_I32 = ctypes.c_int32
_U32 = ctypes.c_uint32
_sigs = {
    "bitq_version": ([], _I32),
    "bitq_last_error": ([], ctypes.c_char_p),
    "bitq_packed_size": ([ctypes.POINTER(WDesc), ctypes.POINTER(_SZ)], _I32),
    "bitq_pack_weights": ([ctypes.POINTER(WDesc), ctypes.POINTER(Logical), _P, _SZ], _I32),
    "bitq_quantize_weights": ([ctypes.POINTER(WDesc), _P, _P, _SZ, _I32], _I32),
    "bitq_quantize_weights_opts": ([ctypes.POINTER(WDesc), _P, ctypes.POINTER(QuantOpts), _P, _SZ, _I32],
                                   _I32),
    "bitq_quantize_weights_hgf": ([ctypes.POINTER(WDesc), _P, _P, _P, ctypes.c_float, _P, _SZ, _I32], _I32),
    "bitq_act_size": ([_I32, _I32, ctypes.POINTER(_SZ)], _I32),
    "bitq_quantize_act": ([_P, _I32, _I32, _I32, _P, _SZ, _P], _I32),
    "bitq_quantize_act_bits": ([_P, _I32, _I32, _I32, _I32, _P, _SZ, _P], _I32),
    "bitq_hgf_act_size": ([ctypes.POINTER(WDesc), _I32, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)], _I32),
    "bitq_quantize_act_hgf": ([ctypes.POINTER(WDesc), _P, _P, _I32, _I32, _P, _SZ, _P, _SZ, _P], _I32),
    "bitq_quantize_act_hgf_noalloc": ([ctypes.POINTER(WDesc), _P, _P, _I32, _I32, _P, _SZ, _P], _I32),
    "bitq_binact_size": ([_I32, _I32, ctypes.POINTER(_SZ)], _I32),
    "bitq_binarize_act": ([_P, _I32, _I32, _I32, _P, _SZ, _P], _I32),
    "bitq_workspace_size": ([ctypes.POINTER(WDesc), _I32, ctypes.POINTER(_SZ)], _I32),
    "bitq_gemv": ([ctypes.POINTER(WDesc), _P, _P, _I32, _P, _P, _SZ, _U32, _P], _I32),
    "bitq_gemm_smallM": ([ctypes.POINTER(WDesc), _P, _P, _I32, _P, _P, _SZ, _U32, _P], _I32),
    # operators around the linear layers (include/bitq_lm.h)
    "bitq_kv_cache_size": ([ctypes.POINTER(KvDesc), ctypes.POINTER(_SZ)], _I32),
    "bitq_kv_plan_size": ([ctypes.POINTER(KvPlanDesc), ctypes.POINTER(_SZ)], _I32),
    "bitq_kv_plan": ([ctypes.POINTER(KvPlanDesc), _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "bitq_kv_write": ([ctypes.POINTER(KvDesc), _P, _P, _I32, _I64, _I64, _P, _I32, _P, _SZ, _P], _I32),
    "bitq_paged_attn_workspace": ([ctypes.POINTER(AttnDesc), ctypes.POINTER(_SZ)], _I32),
    "bitq_paged_attn": ([ctypes.POINTER(AttnDesc), _P, _I64, _P, _SZ, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "bitq_prompt_attn_workspace": ([ctypes.POINTER(PromptDesc), ctypes.POINTER(_SZ)], _I32),
    "bitq_prompt_attn": ([ctypes.POINTER(PromptDesc), _P, _I64, _P, _SZ, _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "bitq_shared_attn_workspace": ([ctypes.POINTER(SharedDesc), ctypes.POINTER(_SZ)], _I32),
    "bitq_shared_attn": ([ctypes.POINTER(SharedDesc), _P, _I64, _P, _SZ, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "bitq_kv_pages_size": ([ctypes.POINTER(KvPagesDesc), ctypes.POINTER(_SZ)], _I32),
    "bitq_kv_pages_workspace": ([ctypes.POINTER(KvPagesDesc), ctypes.POINTER(_SZ)], _I32),
    "bitq_kv_fork": ([ctypes.POINTER(KvPagesDesc), _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _SZ, _P], _I32),
    "bitq_kv_compact": ([ctypes.POINTER(KvPagesDesc), _P, _P, _P, _P, _P, _SZ, _P, _SZ, _P], _I32),
    "bitq_kv_copy": ([ctypes.POINTER(KvDesc), _P, _P, _I32, _P, _SZ, _P], _I32),
    "bitq_rope_table": ([ctypes.POINTER(RopeFreq), _P], _I32),
    "bitq_qk_rope": ([ctypes.POINTER(RopeDesc), _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _I64, _P, _I64, _P], _I32),
    "bitq_block_norm": ([ctypes.POINTER(NormDesc), _P, _P, _P, _P, _P, _P, _P, _P, _P], _I32),
    "bitq_w8a8_workspace": ([ctypes.POINTER(W8A8Desc), ctypes.POINTER(_SZ)], _I32),
    "bitq_gemm_w8a8": ([ctypes.POINTER(W8A8Desc), _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    # measurement context kernels (include/bitq_ctx.h)
    "bitq_ctx_empty": ([_I32, _P], _I32),
    "bitq_ctx_stream": ([_P, _SZ, _I32, _P, _I32, _P], _I32),
    "bitq_ctx_spin": ([_I32, _P], _I32),
    "bitq_ctx_launch_shape": ([ctypes.POINTER(WDesc), _I32, _I32, _U32, ctypes.POINTER(_I32), ctypes.POINTER(_I32)],
                              _I32),
}
for _name, (_args, _ret) in _sigs.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _ret

EXPORTED = tuple(_sigs)


def _check(status: int):
    if status != OK:
        raise BitqError(status, _lib.bitq_last_error().decode())


def _ptr(x) -> int | None:
    """Device/host address of a tensor, numpy array or raw int (None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)}")


def _current_stream() -> int:
    import torch
    return torch.cuda.current_stream().cuda_stream


# The current stream's handle straight from torch's C module where this torch
# has it (0.2 us against 2.9 us for building a Stream object on every call).
if _torch is not None and hasattr(_torch._C, "_cuda_getCurrentRawStream") and hasattr(_torch._C, "_cuda_getDevice"):
    _raw_stream_of, _device, _started = _torch._C._cuda_getCurrentRawStream, _torch._C._cuda_getDevice, False

    def _raw_stream() -> int:
        global _started
        if not _started:
            if not _torch.cuda.is_initialized():
                return _current_stream()
            _started = True
        return _raw_stream_of(_device())
else:
    _raw_stream = _current_stream


def _addr(x) -> int | None:
    """_ptr for the calls of a decode step: tensors first."""
    if x is None:
        return None
    try:
        return x.data_ptr()
    except AttributeError:
        return _ptr(x)


# What the calls of a decode step read is checked here, the ordinary tensor first (a check costs the host 0.1 to 0.3 us).
if _torch is not None:
    _INT, _WORDS = _torch.int32, frozenset((_torch.int32, _torch.uint32, _torch.uint8))
    _FLOATS = {DT_F32: frozenset((_torch.float32, _torch.int32, _torch.uint32)),             # (integers: bit patterns)
               DT_BF16: frozenset((_torch.bfloat16, _torch.int16, _torch.uint16))}


def _ints(x, n: int, name: str, stride: int = 0) -> int | None:
    """Address of n int32 values in a row; a tensor has to hold them (a table: in rows `stride` apart)."""
    try:
        if x.dtype is _INT and x.is_contiguous() and x.nbytes >= 4 * n:
            return x.data_ptr()
        at = x.data_ptr()
    except AttributeError:                       # (no tensor)
        return _ptr(x)
    if x.dtype not in _WORDS:
        raise TypeError(f"{name} must be int32, not {x.dtype}")
    if not x.is_contiguous():
        if not stride or x.dim() != 2 or x.stride(1) != 1 or x.stride(0) != stride or x.size(0) * stride < n:
            raise ValueError(f"{name} has shape {tuple(x.shape)} and strides {x.stride()}, the call reads {n} values in a row")
    elif x.nbytes < 4 * n:
        raise ValueError(f"{name} has {x.numel()} values, the call needs {n}")
    return at


def _longs(x, n: int, name: str) -> int | None:
    """Address of n 64-bit integers in a row."""
    try:
        at = x.data_ptr()
    except AttributeError:                       # (no tensor)
        return _ptr(x)
    if x.dtype not in (_torch.int64, _torch.uint64):
        raise TypeError(f"{name} must be int64 or uint64, not {x.dtype}")
    if not x.is_contiguous() or x.numel() < n:
        raise ValueError(f"{name} has shape {tuple(x.shape)} and strides {x.stride()}, the call reads {n} values in a row")
    return at


def _float(x, dtype: int, name: str, n: int = 0) -> int | None:
    """Address of x; a tensor has to have the type the call says (n > 0: and to hold n elements in a row)."""
    try:
        at = x.data_ptr()
    except AttributeError:                       # (no tensor)
        return _ptr(x)
    if dtype in _FLOATS and x.dtype not in _FLOATS[dtype]:
        raise TypeError(f"{name} is {x.dtype}, the call takes {'bf16' if dtype == DT_BF16 else 'fp32'}")
    if n and not (x.is_contiguous() and x.numel() >= n):
        raise ValueError(f"{name} has shape {tuple(x.shape)} and strides {x.stride()}, the call writes {n} elements in a row")
    return at


def _rows(x, rows: int, width: int, dtype: int, name: str, stride: int | None) -> tuple:
    """Address of x and the elements between its rows: `rows` or more, each `width` or more elements of the call's type
    next to each other.  An address comes with its stride, which is believed."""
    if stride is not None:
        return _float(x, dtype, name), stride
    shape, st = x.shape, x.stride()
    if len(st) == 3:
        n, h, d = shape
        a, b, c = st
        if c == 1 and b == d and n >= rows and n > 1 and h * d >= width and x.dtype in _FLOATS.get(dtype, ()):
            return x.data_ptr(), a
    size = 1
    for n, d in zip(shape[:0:-1], st[:0:-1]):
        if d != size and n != 1:
            raise ValueError(f"{name}: the elements of a row are not next to each other (shape {tuple(shape)}, strides {st})")
        size *= n
    if not st or shape[0] < rows or size < width:
        raise ValueError(f"{name} has shape {tuple(shape)}, the call reads {rows} rows of {width} elements")
    return _float(x, dtype, name), st[0] if shape[0] > 1 else size      # (the stride of a single row means nothing)


def _stream(stream) -> int | None:
    if stream is None:
        return _raw_stream()
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def wdesc(fmt, N: int, K: int, planes: int | None = None, group: int | None = None,
          abits: int | None = None, rank: int | None = None) -> WDesc:
    if isinstance(fmt, str):
        fmt = FORMATS[fmt]
    return WDesc(fmt, N, K, DEFAULT_PLANES[fmt] if planes is None else planes,
                 DEFAULT_GROUP[fmt] if group is None else group,
                 DEFAULT_ABITS[fmt] if abits is None else abits,
                 DEFAULT_RANK.get(fmt, 0) if rank is None else rank)


# -------------------------------------------------------------- host calls
def version() -> int:
    return _lib.bitq_version()


def last_error() -> str:
    return _lib.bitq_last_error().decode()


def packed_size(desc: WDesc) -> int:
    n = _SZ(0)
    _check(_lib.bitq_packed_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def _logical_shapes(desc: WDesc) -> dict:
    """Shape of each array field of bitq_logical that the descriptor's format
    reads (include/bitq.h, "Logical (unpacked) quantized form")."""
    N, K, P = desc.N, desc.K, desc.planes
    if desc.fmt == SIGN1:
        return {"sign": (N, K), "alpha": (N,)}
    if desc.fmt == RABIT:
        return {"sign": (P, N, K), "g": (P, N), "h": (P, K)}
    if desc.fmt == TERNARY:
        return {"tern": (N, K)}
    if desc.fmt in (W2A8, WNAM):
        return {"code": (N, K), "delta": (N, K // 128), "zero": (N, K // 128)}
    if desc.fmt == BVSR4:
        return {"code": (N, K), "idx": (N, K // 32), "cache": (256, 5)}
    if desc.fmt == HGF:
        return {"tern": (N, K), "lora_a": (K, desc.rank), "lora_b": (desc.rank, N)}
    return {}


def pack_weights(desc: WDesc, **fields) -> np.ndarray:
    """Pack a logical form (numpy arrays named as in bitq_logical) into a blob.
    Every array the format reads must be given, with the shape the header
    documents (ValueError otherwise): the C packer takes no lengths."""
    need = _logical_shapes(desc)
    for name, shape in need.items():
        if name not in fields or fields[name] is None:
            raise ValueError(f"{FORMAT_NAMES.get(desc.fmt, desc.fmt)} needs the field {name!r}")
        got = np.shape(fields[name])
        if tuple(got) != tuple(shape):
            raise ValueError(f"field {name!r} has shape {tuple(got)}, the descriptor needs {tuple(shape)}")
    keep = []
    lg = Logical()
    conv = {"sign": np.int8, "tern": np.int8, "code": np.uint8, "alpha": np.float32,
            "g": np.uint16, "h": np.uint16, "delta": np.uint16, "zero": np.uint16,
            "idx": np.uint8, "cache": np.float32, "lora_a": np.uint16, "lora_b": np.uint16}
    for name, val in fields.items():
        if name in ("gamma", "lora_alpha"):
            setattr(lg, name, float(val))
            continue
        arr = np.asarray(val)
        if arr.dtype == np.float16:
            arr = arr.view(np.uint16)
        arr = np.ascontiguousarray(arr, dtype=conv[name])
        keep.append(arr)
        setattr(lg, name, arr.ctypes.data)
    blob = np.zeros(packed_size(desc), dtype=np.uint8)
    _check(_lib.bitq_pack_weights(ctypes.byref(desc), ctypes.byref(lg), blob.ctypes.data, blob.nbytes))
    return blob


def quantize_weights(desc: WDesc, W: np.ndarray, nthreads: int = 0, svid_sweeps: int = 0,
                     bit_balance: bool = False) -> np.ndarray:
    """fp32 W [N, K] -> packed blob with the library's own offline quantizer
    (RABIT: svid_sweeps Gauss-Seidel refinement sweeps after the greedy pass;
    WNAM with 3 planes: bit_balance selects the symmetric five-level grid)."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    if W.shape != (desc.N, desc.K):
        raise ValueError(f"W has shape {W.shape}, descriptor says {(desc.N, desc.K)}")
    blob = np.zeros(packed_size(desc), dtype=np.uint8)
    if svid_sweeps or bit_balance:
        opts = QuantOpts(svid_sweeps, int(bit_balance))
        _check(_lib.bitq_quantize_weights_opts(ctypes.byref(desc), W.ctypes.data, ctypes.byref(opts),
                                               blob.ctypes.data, blob.nbytes, nthreads))
    else:
        _check(_lib.bitq_quantize_weights(ctypes.byref(desc), W.ctypes.data, blob.ctypes.data,
                                          blob.nbytes, nthreads))
    return blob


def quantize_weights_hgf(desc: WDesc, W: np.ndarray, lora_a, lora_b, lora_alpha: float,
                         nthreads: int = 0) -> np.ndarray:
    """fp32 W [N, K] -> HGF blob: the library's ternary quantizer for W plus
    the correction parameters A [K, r], B [r, N] (fp16 arrays or their bits)."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    if W.shape != (desc.N, desc.K):
        raise ValueError(f"W has shape {W.shape}, descriptor says {(desc.N, desc.K)}")
    a = np.ascontiguousarray(np.asarray(lora_a).view(np.uint16) if np.asarray(lora_a).dtype == np.float16
                             else lora_a, dtype=np.uint16)
    b = np.ascontiguousarray(np.asarray(lora_b).view(np.uint16) if np.asarray(lora_b).dtype == np.float16
                             else lora_b, dtype=np.uint16)
    if desc.fmt == HGF and (a.shape != (desc.K, desc.rank) or b.shape != (desc.rank, desc.N)):
        raise ValueError("lora_a must be [K, rank] and lora_b [rank, N]")
    blob = np.zeros(packed_size(desc), dtype=np.uint8)
    _check(_lib.bitq_quantize_weights_hgf(ctypes.byref(desc), W.ctypes.data, a.ctypes.data, b.ctypes.data,
                                          float(lora_alpha), blob.ctypes.data, blob.nbytes, nthreads))
    return blob


def act_size(M: int, K: int) -> int:
    n = _SZ(0)
    _check(_lib.bitq_act_size(M, K, ctypes.byref(n)))
    return n.value


def hgf_act_size(desc: WDesc, M: int) -> tuple:
    """(activation buffer bytes, workspace bytes) of an HGF layer's activation step."""
    a, w = _SZ(0), _SZ(0)
    _check(_lib.bitq_hgf_act_size(ctypes.byref(desc), M, ctypes.byref(a), ctypes.byref(w)))
    return a.value, w.value


def binact_size(M: int, K: int) -> int:
    n = _SZ(0)
    _check(_lib.bitq_binact_size(M, K, ctypes.byref(n)))
    return n.value


def binact_layout(M: int, K: int) -> dict:
    """Section offsets of a binary activation buffer (as include/bitq.h)."""
    Kp = (K + 127) // 128 * 128
    Kw = Kp // 32
    a = lambda v: (v + 255) // 256 * 256
    off_beta = a(4 * M * Kw)
    return dict(Kp=Kp, Kw=Kw, off_bits=0, off_beta=off_beta, total=a(off_beta + 4 * M))


def workspace_size(desc: WDesc, M: int = 1) -> int:
    n = _SZ(0)
    _check(_lib.bitq_workspace_size(ctypes.byref(desc), M, ctypes.byref(n)))
    return n.value


# ------------------------------------------------------------ device calls
def binarize_act(x, x_dtype: int, M: int, K: int, act, act_bytes: int | None = None, stream=None):
    nbytes = act.numel() * act.element_size() if act_bytes is None else act_bytes
    _check(_lib.bitq_binarize_act(_ptr(x), x_dtype, M, K, _ptr(act), nbytes, _stream(stream)))


def quantize_act(x, x_dtype: int, M: int, K: int, act, act_bytes: int | None = None, stream=None,
                 abits: int = 8):
    nbytes = act.numel() * act.element_size() if act_bytes is None else act_bytes
    if abits == 8:
        _check(_lib.bitq_quantize_act(_ptr(x), x_dtype, M, K, _ptr(act), nbytes, _stream(stream)))
    else:
        _check(_lib.bitq_quantize_act_bits(_ptr(x), x_dtype, M, K, abits, _ptr(act), nbytes,
                                           _stream(stream)))


def quantize_act_hgf(desc: WDesc, w, x, x_dtype: int, M: int, act, ws, act_bytes: int | None = None,
                     ws_bytes: int | None = None, stream=None):
    abytes = act.numel() * act.element_size() if act_bytes is None else act_bytes
    wbytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.bitq_quantize_act_hgf(ctypes.byref(desc), _ptr(w), _ptr(x), x_dtype, M, _ptr(act), abytes,
                                      _ptr(ws), wbytes, _stream(stream)))


def quantize_act_hgf_noalloc(desc: WDesc, w, x, x_dtype: int, M: int, act, act_bytes: int | None = None,
                             stream=None):
    """bitq_quantize_act_hgf without a workspace (the library's static device
    scratch holds the down projection's words; nothing is allocated)."""
    abytes = act.numel() * act.element_size() if act_bytes is None else act_bytes
    _check(_lib.bitq_quantize_act_hgf_noalloc(ctypes.byref(desc), _ptr(w), _ptr(x), x_dtype, M, _ptr(act), abytes,
                                              _stream(stream)))


def _nbytes(buf) -> int:
    """Size of a device buffer (0 for None: calls that need no workspace)."""
    return 0 if buf is None else buf.nbytes


def gemv(desc: WDesc, w, x, x_dtype: int, y, ws, ws_bytes: int | None = None, flags: int = 0,
         stream=None):
    nbytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check(_lib.bitq_gemv(ctypes.byref(desc), _ptr(w), _ptr(x), x_dtype, _ptr(y), _ptr(ws),
                          nbytes, flags, _stream(stream)))


def gemm_smallM(desc: WDesc, w, act, M: int, y, ws, ws_bytes: int | None = None, flags: int = 0,
                stream=None):
    nbytes = _nbytes(ws) if ws_bytes is None else ws_bytes
    _check(_lib.bitq_gemm_smallM(ctypes.byref(desc), _ptr(w), _ptr(act), M, _ptr(y), _ptr(ws),
                                 nbytes, flags, _stream(stream)))


# ------------------------------------- paged cache, norms, int8 products
def kvdesc(kv_heads: int, head_dim: int, page: int, pages: int, dtype: int = KV_BF16) -> KvDesc:
    return KvDesc(kv_heads, head_dim, page, pages, dtype)


def _size_of(fn, desc) -> int:
    n = _SZ(0)
    _check(fn(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def kv_cache_size(kv: KvDesc) -> int:
    return _size_of(_lib.bitq_kv_cache_size, kv)


def kv_cache_views(kv: KvDesc, cache) -> dict:
    """Sections of a cache buffer (a uint8 tensor) as tensors: K [pages, heads, page, Dp],
    V [pages, heads, page / 8, Dp, 8], and for int8 ks, vs [pages, heads, page]."""
    import torch
    Dp, P, H, n = (kv.head_dim + 31) // 32 * 32, kv.page, kv.kv_heads, kv.pages
    t, e = (torch.bfloat16, 2) if kv.dtype == KV_BF16 else (torch.int8, 1)
    size = n * H * P * Dp * e
    sec = (size + 255) // 256 * 256
    out = dict(K=cache[:size].view(t).view(n, H, P, Dp), V=cache[sec:sec + size].view(t).view(n, H, P // 8, Dp, 8))
    if kv.dtype == KV_INT8:
        sc = 4 * n * H * P
        at = 2 * sec
        out["ks"] = cache[at:at + sc].view(torch.float32).view(n, H, P)
        at += (sc + 255) // 256 * 256
        out["vs"] = cache[at:at + sc].view(torch.float32).view(n, H, P)
    return out


def kv_plan_desc(requests: int, page: int, table_stride: int, ring: int, tokens: int) -> KvPlanDesc:
    return KvPlanDesc(requests, page, table_stride, ring, tokens)


def kv_plan_size(desc: KvPlanDesc) -> int:
    return _size_of(_lib.bitq_kv_plan_size, desc)


def kv_plan_views(desc: KvPlanDesc, plan) -> dict:
    """Sections of a plan buffer (a uint8 tensor) as int32 tensors: state, len, start, slot, req, pos."""
    import torch
    out, at = {}, 0
    for name, n in (("state", 4), ("len", desc.requests), ("start", desc.requests + 1), ("slot", desc.tokens),
                    ("req", desc.tokens), ("pos", desc.tokens)):
        out[name] = plan[at:at + 4 * n].view(torch.int32)
        at += (4 * n + 255) // 256 * 256
    return out


def kv_plan(desc: KvPlanDesc, old_len, new_len, ring, state, table, plan, stream=None):
    """One scheduling step: pages from and to the ring, tables, slots (bitq_kv_plan).  Lengths, ring, state and table are
    int32 (TypeError otherwise) and as many as the descriptor says (ValueError)."""
    R, per = desc.requests, desc.table_stride
    _check(_lib.bitq_kv_plan(desc, _ints(old_len, R, "old_len"), _ints(new_len, R, "new_len"), _ints(ring, desc.ring, "ring"),
                             _ints(state, 2, "state"), _ints(table, R * per, "table", per), _addr(plan), _nbytes(plan),
                             _stream(stream)))


def kv_write(kv: KvDesc, k, v, x_dtype: int, slots, cache, tokens: int | None = None, k_stride: int | None = None,
             v_stride: int | None = None, stream=None):
    """Keys and values of new tokens into their slots (bitq_kv_write).  k, v: tensors [tokens, kv_heads,
    head_dim] whose last two dimensions are contiguous (or addresses, with the strides given); slots: int32.  k and v
    have a row for every slot of the list, the skipped ones too (ValueError otherwise)."""
    tokens = slots.numel() if tokens is None else tokens
    row = kv.kv_heads * kv.head_dim
    k_at, k_stride = _rows(k, tokens, row, x_dtype, "k", k_stride)
    v_at, v_stride = _rows(v, tokens, row, x_dtype, "v", v_stride)
    _check(_lib.bitq_kv_write(kv, k_at, v_at, x_dtype, k_stride, v_stride, _ints(slots, tokens, "slots"), tokens, _addr(cache),
                              _nbytes(cache), _stream(stream)))


def attn_desc(kv: KvDesc, heads: int, requests: int, table_stride: int, max_len: int, window: int = 0,
              q_dtype: int = DT_BF16, out_dtype: int = DT_BF16, scale: float | None = None) -> AttnDesc:
    return AttnDesc(kv, heads, requests, table_stride, max_len, window, q_dtype, out_dtype,
                    kv.head_dim ** -0.5 if scale is None else scale)


def paged_attn_workspace(desc: AttnDesc) -> int:
    return _size_of(_lib.bitq_paged_attn_workspace, desc)


def paged_attn(desc: AttnDesc, q, cache, table, lens, out, ws, lse=None, q_stride: int | None = None,
               ws_bytes: int | None = None, stream=None):
    """Attention of one new token per request over the paged cache (bitq_paged_attn).  q: a tensor [requests, heads,
    head_dim] whose last two dimensions are contiguous (rows may be longer); out and lse: contiguous; table and lens: int32."""
    R, per, A = desc.requests, desc.table_stride, desc.requests * desc.heads
    D = desc.kv.head_dim
    q_at, q_stride = _rows(q, R, desc.heads * D, desc.q_dtype, "q", q_stride)
    _check(_lib.bitq_paged_attn(desc, q_at, q_stride, _addr(cache), _nbytes(cache),
                                _ints(table, R * per, "table", per), _ints(lens, R, "lens"),
                                _float(out, desc.out_dtype, "out", A * D), _float(lse, DT_F32, "lse", A), _addr(ws),
                                _nbytes(ws) if ws_bytes is None else ws_bytes, _stream(stream)))


def prompt_desc(kv: KvDesc, heads: int, requests: int, tokens: int, table_stride: int, max_len: int, window: int = 0,
                sinks: int = 0, q_dtype: int = DT_BF16, out_dtype: int = DT_BF16, scale: float | None = None) -> PromptDesc:
    return PromptDesc(kv, heads, requests, tokens, table_stride, max_len, window, sinks, q_dtype, out_dtype,
                      kv.head_dim ** -0.5 if scale is None else scale)


def prompt_attn_workspace(desc: PromptDesc) -> int:
    return _size_of(_lib.bitq_prompt_attn_workspace, desc)


def prompt_attn(desc: PromptDesc, q, cache, table, start, lens, out, ws, lse=None, q_stride: int | None = None,
                ws_bytes: int | None = None, stream=None):
    """Attention of each request's new tokens, rows start[r] .. start[r + 1] - 1 of q, over the paged cache that holds them
    already (bitq_prompt_attn).  q: a tensor [tokens, heads, head_dim] whose last two dimensions are contiguous (rows may be
    longer); out and lse: contiguous; table, start and lens: int32."""
    R, per, A = desc.requests, desc.table_stride, desc.tokens * desc.heads
    D = desc.kv.head_dim
    q_at, q_stride = _rows(q, desc.tokens, desc.heads * D, desc.q_dtype, "q", q_stride)
    _check(_lib.bitq_prompt_attn(desc, q_at, q_stride, _addr(cache), _nbytes(cache), _ints(table, R * per, "table", per),
                                 _ints(start, R + 1, "start"), _ints(lens, R, "lens"),
                                 _float(out, desc.out_dtype, "out", A * D), _float(lse, DT_F32, "lse", A), _addr(ws),
                                 _nbytes(ws) if ws_bytes is None else ws_bytes, _stream(stream)))


def shared_desc(attn: AttnDesc, groups: int, max_prefix: int) -> SharedDesc:
    return SharedDesc(attn, groups, max_prefix)


def shared_attn_workspace(desc: SharedDesc) -> int:
    return _size_of(_lib.bitq_shared_attn_workspace, desc)


def shared_attn(desc: SharedDesc, q, cache, table, lens, start, prefix, out, ws, lse=None, q_stride: int | None = None,
                ws_bytes: int | None = None, stream=None):
    """paged_attn for groups of requests, start[g] .. start[g + 1] - 1, that have their first prefix[g] tokens in common:
    those are read once for the group (bitq_shared_attn).  Tensors as for paged_attn; start and prefix: int32."""
    a = desc.attn
    R, per, A = a.requests, a.table_stride, a.requests * a.heads
    D = a.kv.head_dim
    q_at, q_stride = _rows(q, R, a.heads * D, a.q_dtype, "q", q_stride)
    _check(_lib.bitq_shared_attn(desc, q_at, q_stride, _addr(cache), _nbytes(cache), _ints(table, R * per, "table", per),
                                 _ints(lens, R, "lens"), _ints(start, desc.groups + 1, "start"),
                                 _ints(prefix, desc.groups, "prefix"), _float(out, a.out_dtype, "out", A * D),
                                 _float(lse, DT_F32, "lse", A), _addr(ws), _nbytes(ws) if ws_bytes is None else ws_bytes,
                                 _stream(stream)))


def kv_pages_desc(requests: int, page: int, table_stride: int, pool: int, moves: int) -> KvPagesDesc:
    return KvPagesDesc(requests, page, table_stride, pool, moves)


def kv_pages_size(desc: KvPagesDesc) -> int:
    return _size_of(_lib.bitq_kv_pages_size, desc)


def kv_pages_workspace(desc: KvPagesDesc) -> int:
    return _size_of(_lib.bitq_kv_pages_workspace, desc)


def kv_pages_views(desc: KvPagesDesc, result) -> dict:
    """Sections of the result buffer (a uint8 tensor) of kv_fork and kv_compact as int32 tensors: state, len, frm, to."""
    import torch
    out, at = {}, 0
    for name, n in (("state", 4), ("len", desc.requests), ("frm", desc.moves), ("to", desc.moves)):
        out[name] = result[at:at + 4 * n].view(torch.int32)
        at += (4 * n + 255) // 256 * 256
    return out


def kv_fork(desc: KvPagesDesc, src, keep, lens, ring, state, table, table_out, result, ws, stream=None):
    """Request r becomes the first keep[r] tokens of request src[r]: forks, cuts, ends (bitq_kv_fork).  All int32; the
    copies of pages that result's frm and to list are the caller's to make, in every layer's cache (kv_copy)."""
    R, per = desc.requests, desc.table_stride
    _check(_lib.bitq_kv_fork(desc, _ints(src, R, "src"), _ints(keep, R, "keep"), _ints(lens, R, "lens"),
                             _ints(ring, desc.pool, "ring"), _ints(state, 2, "state"), _ints(table, R * per, "table", per),
                             _ints(table_out, R * per, "table_out", per), _addr(result), _nbytes(result), _addr(ws),
                             _nbytes(ws), _stream(stream)))


def kv_compact(desc: KvPagesDesc, lens, table, table_out, ring, result, ws, stream=None):
    """Held pages to the low end of the pool (bitq_kv_compact): tables, ring and the list of copies as for kv_fork."""
    R, per = desc.requests, desc.table_stride
    _check(_lib.bitq_kv_compact(desc, _ints(lens, R, "lens"), _ints(table, R * per, "table", per),
                                _ints(table_out, R * per, "table_out", per), _ints(ring, desc.pool, "ring"), _addr(result),
                                _nbytes(result), _addr(ws), _nbytes(ws), _stream(stream)))


def kv_copy(kv: KvDesc, frm, to, cache, moves: int | None = None, stream=None):
    """Pages frm[i] of a layer's cache to pages to[i] (bitq_kv_copy); pairs with an index outside the pool are skipped."""
    moves = to.numel() if moves is None else moves
    _check(_lib.bitq_kv_copy(kv, _ints(frm, moves, "frm"), _ints(to, moves, "to"), moves, _addr(cache), _nbytes(cache),
                             _stream(stream)))


def rope_table(rot: int, base: float = 10000.0, kind: int = ROPE_PLAIN, factor: float = 1.0, trained: float = 0.0,
               turns_keep: float = 0.0, turns_scale: float = 0.0) -> np.ndarray:
    """The rotation's turns per position as 64-bit fractions, uint64 [rot / 2] (bitq_rope_table); for qk_rope on the GPU:
    torch.from_numpy(table).cuda()."""
    out = np.empty(max(1, rot // 2), dtype=np.uint64)
    _check(_lib.bitq_rope_table(RopeFreq(rot, kind, base, factor, trained, turns_keep, turns_scale), out.ctypes.data))
    return out


def rope_desc(tokens: int, q_heads: int, k_heads: int, head_dim: int, rot: int | None = None, layout: int = ROPE_HALF,
              x_dtype: int = DT_F32, out_dtype: int = DT_BF16, w_dtype: int = DT_F32, eps: float = 1e-6,
              mscale: float = 1.0) -> RopeDesc:
    return RopeDesc(tokens, q_heads, k_heads, head_dim, head_dim if rot is None else rot, layout, x_dtype, out_dtype,
                    w_dtype, eps, mscale)


def qk_rope(desc: RopeDesc, q, k, q_w, k_w, table, pos, q_out, k_out, strides: tuple = (None,) * 4, stream=None):
    """Norms of queries and keys head by head, and their rotation (bitq_qk_rope).  q, k and the outputs: tensors [tokens,
    heads, head_dim] whose last two dimensions are contiguous (or addresses, with the four strides given), None without heads;
    q_w, k_w: [head_dim] or None; table: rope_table's values on the GPU; pos: int32."""
    T, D = desc.tokens, desc.head_dim
    row = []
    for x, heads, dtype, name, stride in ((q, desc.q_heads, desc.x_dtype, "q", strides[0]),
                                          (k, desc.k_heads, desc.x_dtype, "k", strides[1]),
                                          (q_out, desc.q_heads, desc.out_dtype, "q_out", strides[2]),
                                          (k_out, desc.k_heads, desc.out_dtype, "k_out", strides[3])):
        row += _rows(x, T, heads * D, dtype, name, stride) if x is not None and heads else (_addr(x), 0)
    _check(_lib.bitq_qk_rope(desc, *row[:4], _float(q_w, desc.w_dtype, "q_w", D), _float(k_w, desc.w_dtype, "k_w", D),
                             _longs(table, desc.rot // 2, "table"), _ints(pos, T, "pos"), *row[4:], _stream(stream)))


def norm_desc(rows: int, width: int, u_dtype: int = DT_F32, r_dtype: int = DT_F32, w_dtype: int = DT_F32,
              out_dtype: int = DT_F32, res_scale: float = 1.0, branch_scale: float = 1.0, eps_post: float = 1e-5,
              eps_pre: float = 1e-5, gate_stride: int = 0, u_stride: int | None = None, r_stride: int | None = None,
              ro_stride: int | None = None, h_stride: int | None = None) -> NormDesc:
    st = [width if s is None else s for s in (u_stride, r_stride, ro_stride, h_stride)]
    return NormDesc(rows, width, u_dtype, r_dtype, w_dtype, out_dtype, *st, gate_stride, res_scale, branch_scale,
                    eps_post, eps_pre)


def block_norm(desc: NormDesc, u, r, post, gate, pre, r_out, h, d=None, stream=None):
    """Residual update with the norms before and after it (bitq_block_norm); d: the rows' scales (DT_ROW8)."""
    _check(_lib.bitq_block_norm(desc, _addr(u), _addr(r), _addr(post), _addr(gate), _addr(pre), _addr(r_out), _addr(h),
                                _addr(d), _stream(stream)))


def w8a8_desc(M: int, N: int, K: int, y_dtype: int = DT_F32, lda: int | None = None, ldw: int | None = None,
              ldy: int | None = None, flags: int = 0) -> W8A8Desc:
    return W8A8Desc(M, N, K, y_dtype, K if lda is None else lda, K if ldw is None else ldw,
                    N if ldy is None else ldy, flags)


def w8a8_workspace(desc: W8A8Desc) -> int:
    return _size_of(_lib.bitq_w8a8_workspace, desc)


def gemm_w8a8(desc: W8A8Desc, a, a_scale, w, w_scale, y, ws=None, ws_bytes: int | None = None, stream=None):
    """y = diag(a_scale) a w^T diag(w_scale) on int8 rows (bitq_gemm_w8a8)."""
    _check(_lib.bitq_gemm_w8a8(desc, _addr(a), _addr(a_scale), _addr(w), _addr(w_scale), _addr(y), _addr(ws),
                               _nbytes(ws) if ws_bytes is None else ws_bytes, _stream(stream)))


# ------------------------------------------- measurement context kernels
def ctx_empty(grid: int, stream=None):
    """A launch of `grid` workgroups that does nothing (bitq_ctx_empty)."""
    _check(_lib.bitq_ctx_empty(grid, _stream(stream)))


def ctx_stream(src, nbytes: int, grid: int, out, nout: int, stream=None):
    """Read nbytes of src once with `grid` workgroups and write nout floats
    (bitq_ctx_stream): the streaming floor of a GEMV over those bytes."""
    _check(_lib.bitq_ctx_stream(_ptr(src), nbytes, grid, _ptr(out), nout, _stream(stream)))


def ctx_launch_shape(desc: WDesc, M: int, x_dtype: int, flags: int = 0) -> tuple:
    """(workgroups, lanes per workgroup) of the kernel bitq_gemv (M = 1) or
    bitq_gemm_smallM launches for these arguments."""
    g, b = _I32(0), _I32(0)
    _check(_lib.bitq_ctx_launch_shape(ctypes.byref(desc), M, x_dtype, flags, ctypes.byref(g), ctypes.byref(b)))
    return g.value, b.value


def ctx_spin(microseconds: int, stream=None):
    """One wave that waits the given wall-clock time (bitq_ctx_spin)."""
    _check(_lib.bitq_ctx_spin(microseconds, _stream(stream)))


def act_layout(M: int, K: int, rank: int = 0) -> dict:
    """Section offsets of an activation buffer (mirrors bitq_act_size; rank > 0:
    the HGF buffer of bitq_hgf_act_size with its h section)."""
    Kp = (K + 127) // 128 * 128
    Kw = Kp // 32

    def a256(v):
        return (v + 255) // 256 * 256
    off_S = a256(M * Kw * 32)
    off_q = a256(off_S + M * Kw * 4)
    off_qm = a256(off_q + M * Kp)
    off_d = a256(off_qm + 16 * ((M + 15) // 16) * Kp)   # qm: whole tiles of 16 tokens
    off_amax = a256(off_d + 4 * M)
    off_h = a256(off_amax + 4 * M)
    return dict(Kp=Kp, Kw=Kw, off_planes=0, off_S=off_S, off_q=off_q, off_qm=off_qm, off_d=off_d,
                off_amax=off_amax, off_h=off_h, total=a256(off_h + 4 * M * rank))
