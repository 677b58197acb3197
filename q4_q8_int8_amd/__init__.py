"""q4_K x q8_1 quantized matrix multiply (MMQ) on MI355X (gfx950).

A thin ctypes binding over libmmq.so, whose C ABI is declared in include/mmq.h (the integer
product), include/mmq_layer.h (its epilogue, the gated product, the mixture-of-experts layer),
include/mmq_q4g.h (matrix-vector products with group scales) and include/mmq_f16.h (the f16
comparator path). The functions here have the same
names and arguments as the C entry points and only marshal arguments: each tensor is checked
(a contiguous CUDA tensor on the current device, of the expected dtype and at least the size
the call reads or writes; MMQArgumentError otherwise) and passed as a device pointer, the
stream defaults to torch's current stream, and a nonzero status raises MMQError. Every step of the computation runs in the
library's HIP kernels; there is no fallback path. Importing this package fails loudly when
libmmq.so has not been built (python q4_q8_int8_amd/build.py).
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from operator import index as _int

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmmq.so")
INCLUDE_DIR = os.path.join(os.path.dirname(_PKG), "include")
HEADER_PATH = os.path.join(INCLUDE_DIR, "mmq.h")
HEADER_PATHS = (HEADER_PATH, os.path.join(INCLUDE_DIR, "mmq_layer.h"),
                os.path.join(INCLUDE_DIR, "mmq_q4g.h"), os.path.join(INCLUDE_DIR, "mmq_f16.h"))

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python q4_q8_int8_amd/build.py`")
# torch ships its own HIP runtime. Loading torch first makes libmmq.so's libamdhip64
# dependency resolve to that already-loaded runtime, so the process has a single HIP runtime
# and torch's device pointers and streams are valid in the library's calls. (Loaded the other
# way round, the process would hold two runtimes and the second sees no device.)
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)

MMQ_OK, MMQ_E_ARG, MMQ_E_SHAPE, MMQ_E_LDS, MMQ_E_DEVICE, MMQ_E_HIP = range(6)
(MMQ_TILE_AUTO, MMQ_TILE_LARGE, MMQ_TILE_SMALL, MMQ_TILE_SKINNY, MMQ_TILE_GEMV,
 MMQ_TILE_MEDIUM, MMQ_TILE_HALF) = range(7)
(MMQ_REASON_NONE, MMQ_REASON_LARGE, MMQ_REASON_SMALL_GRID, MMQ_REASON_LDS_FALLBACK,
 MMQ_REASON_FORCED, MMQ_REASON_NO_FIT, MMQ_REASON_FEW_TOKENS, MMQ_REASON_FUSED,
 MMQ_REASON_DECODE, MMQ_REASON_SPLIT_K) = range(10)
GEMV_MAX_M = 16  # largest M of the decode tile, which the guard chooses up to there
QK8, QK_K, Q4K_BLOCK_BYTES, REP_TILE_ROWS, REP_TILE_BYTES = 32, 256, 144, 32, 4608
Q6K_BLOCK_BYTES, REP6_TILE_BYTES = 210, 10240
(MMQ_ACT_NONE, MMQ_ACT_RELU, MMQ_ACT_SILU, MMQ_ACT_GELU, MMQ_ACT_GELU_TANH) = range(5)
ACTIVATIONS = {"none": MMQ_ACT_NONE, "relu": MMQ_ACT_RELU, "silu": MMQ_ACT_SILU,
               "gelu": MMQ_ACT_GELU, "gelu_tanh": MMQ_ACT_GELU_TANH}
MMQ_SCORE_SOFTMAX, MMQ_SCORE_SIGMOID = range(2)
SCORES = {"softmax": MMQ_SCORE_SOFTMAX, "sigmoid": MMQ_SCORE_SIGMOID}
MOE_MAX_TOKENS, MOE_MAX_PAIRS, MOE_MAX_EXPERTS, MOE_MAX_SLOTS = 64, 512, 512, 64
GROUP_MAX_PAIRS = 1 << 21
MMQ_F32, MMQ_F16, MMQ_BF16 = range(3)
TYPES = {torch.float32: MMQ_F32, torch.float16: MMQ_F16, torch.bfloat16: MMQ_BF16}
Q4G_MAX_TOKENS = 16
# The tokens up to which a program that does not look at the rows takes the products from float32
# activations (mmq_q4K_f32 and its forms: one launch, but every row block quantizes again) before
# quantize_q8_1 and the product. K = 4096, epilogue and gated alike (a gated product has 2 F rows): 1
# token is 1.6 to 2.1 us faster at 2048 to 22016 rows. 2 tokens are faster to 8192 rows (4096: 5.8
# against 7.3 us, 8192: 8.5 against 9.4) and slower above (11008: 11.4 against 10.6, 22016: 18.3 against
# 16.2), so a program with more rows does well to take them for 1 token only. 3 and 4 tokens are
# faster to 4096 rows (3: 6.9 against 8.0) and slower from 6144 (12.2 against 9.6).
FUSED_TOKENS = 2


class mmq_options(ctypes.Structure):
    _fields_ = [("force_tile", ctypes.c_int32), ("min_workgroups", ctypes.c_int32),
                ("lds_budget", ctypes.c_int64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64), ("splits", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class mmq_kernel_info(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int32), ("reason", ctypes.c_int32),
                ("block_m", ctypes.c_int32), ("block_n", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("fallback", ctypes.c_int32),
                ("lds_bytes", ctypes.c_int64), ("lds_budget", ctypes.c_int64),
                ("grid", ctypes.c_int64), ("splits", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("workspace_bytes", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class mmq_epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("act", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class mmq_q4G_format(ctypes.Structure):
    _fields_ = [("group", ctypes.c_int32), ("scale_type", ctypes.c_int32),
                ("zeros", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class mmq_q4G_epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("act", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MMQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        detail = _lib.mmq_last_error().decode()
        super().__init__(f"{fn}: {_lib.mmq_status_str(status).decode()}"
                         + (f" ({detail})" if detail else ""))


_i64, _vp, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
_i32c = ctypes.c_int32
_SIGS = {
    "mmq_q8_1_bytes": [_i64, _i64, ctypes.POINTER(_sz)],
    "mmq_q4K_bytes": [_i64, _i64, ctypes.POINTER(_sz)],
    "mmq_q4K_repacked_bytes": [_i64, _i64, ctypes.POINTER(_sz)],
    "quantize_q8_1": [_vp, _i64, _i64, _vp, _vp],
    "repack_q4_K": [_vp, _i64, _i64, _vp, _vp],
    "mmq_q4K_q8_1": [_i64, _i64, _i64, _vp, _vp, _vp, _vp],
    "mmq_q4K_q8_1_ex": [_i64, _i64, _i64, _vp, _vp, _vp, _vp, ctypes.POINTER(mmq_options)],
    "mmq_q4K_f32": [_i64, _i64, _i64, _vp, _vp, _vp, _vp],
    "mmq_workspace_bytes": [_i64, _i64, _i64, ctypes.POINTER(_sz)],
    "mmq_q6K_bytes": [_i64, _i64, ctypes.POINTER(_sz)],
    "mmq_q6K_repacked_bytes": [_i64, _i64, ctypes.POINTER(_sz)],
    "repack_q6_K": [_vp, _i64, _i64, _vp, _vp],
    "mmq_q6K_q8_1": [_i64, _i64, _i64, _vp, _vp, _vp, _vp],
    "mmq_q6K_q8_1_ex": [_i64, _i64, _i64, _vp, _vp, _vp, _vp, ctypes.POINTER(mmq_options)],
    "mmq_q6K_q8_1_blockdots": [_i64, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp,
                               ctypes.POINTER(mmq_options)],
    "mmq_q4K_q8_1_static": [_i64, _i64, _i64, _vp, _vp, _vp, _vp, ctypes.POINTER(mmq_options)],
    "mmq_q4K_q8_1_blockdots": [_i64, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp,
                               ctypes.POINTER(mmq_options)],
    "mmq_plan": [_i64, _i64, _i64, ctypes.POINTER(mmq_options), _i64,
                 ctypes.POINTER(mmq_kernel_info)],
    "mmq_last_kernel": [ctypes.POINTER(mmq_kernel_info)],
    "mmq_q4K_q8_1_epilogue": [_i64, _i64, _i64, _vp, _vp, _vp, _vp, ctypes.POINTER(mmq_epilogue),
                              ctypes.POINTER(mmq_options)],
    "mmq_q4K_f32_epilogue": [_i64, _i64, _i64, _vp, _vp, _vp, _vp, ctypes.POINTER(mmq_epilogue)],
    "mmq_q4K_pair_bytes": [_i64, _i64, ctypes.POINTER(_sz)],
    "repack_q4_K_pair": [_vp, _vp, _i64, _i64, _vp, _vp],
    "mmq_gated_workspace_bytes": [_i64, _i64, _i64, ctypes.POINTER(_sz)],
    "mmq_q4K_q8_1_gated": [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32c,
                           ctypes.POINTER(mmq_options)],
    "mmq_q4K_f32_gated": [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32c],
    "mmq_moe_plan_bytes": [_i64, _i64, _i64, ctypes.POINTER(_sz)],
    "mmq_moe_plan": [_i64, _i64, _i64, _vp, _vp, _vp],
    "mmq_moe_route": [_i64, _i64, _i64, _vp, _i32c, _i32c, _vp, _vp, _vp, _vp],
    "mmq_q4K_moe_gated": [_i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i32c, _vp],
    "mmq_q4K_moe_down": [_i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "mmq_moe_workspace_bytes": [_i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_sz)],
    "mmq_q4K_moe": [_i64, _i64, _i64, _i64, _i64, _vp, _vp, _i32c, _i32c, _vp, _i32c, _vp, _vp,
                    _vp, _vp, _sz, _vp],
    "mmq_moe_group_bytes": [_i64, _i64, _i64, ctypes.POINTER(_sz)],
    "mmq_moe_group": [_i64, _i64, _i64, _vp, _vp, _vp],
    "mmq_q4K_grouped": [_i64, _i64, _i64, _i64, _i64, _vp, _i32c, _vp, _vp, _vp, _vp, _i32c, _vp],
    "mmq_q4K_grouped_gated": [_i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i32c, _vp],
    "mmq_grouped_down_workspace_bytes": [_i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_sz)],
    "mmq_q4K_grouped_down": [_i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                             _vp],
    "mmq_grouped_moe_workspace_bytes": [_i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_sz)],
    "mmq_q4K_grouped_moe": [_i64, _i64, _i64, _i64, _i64, _vp, _vp, _i32c, _i32c, _vp, _i32c, _vp,
                            _vp, _vp, _vp, _sz, _vp],
    "mmq_q4G_repacked_bytes": [_i64, _i64, ctypes.POINTER(mmq_q4G_format), ctypes.POINTER(_sz)],
    "repack_q4_G": [_vp, _vp, _vp, _i64, _i64, ctypes.POINTER(mmq_q4G_format), _vp, _vp],
    "mmq_q4G": [_i64, _i64, _i64, _i32c, _vp, _vp, ctypes.POINTER(mmq_q4G_format), _i32c, _vp,
                ctypes.POINTER(mmq_q4G_epilogue), _vp],
    "mmq_f16_bytes": [_i64, _i64, ctypes.POINTER(_sz)],
    "convert_f32_f16": [_vp, _i64, _i64, _vp, _vp],
    "dequantize_q4_K_f16": [_vp, _i64, _i64, _vp, _vp],
    "gemm_f16": [_i64, _i64, _i64, _vp, _vp, _vp, _vp],
    "mmq_status_str": [ctypes.c_int],
    "mmq_last_error": [],
}
for _name, _args in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_char_p if _name in ("mmq_status_str", "mmq_last_error") else ctypes.c_int


def exported_symbols() -> list[str]:
    """Function names declared in the library's headers (include/*.h)."""
    names = []
    for path in HEADER_PATHS:
        with open(path) as f:
            text = f.read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        names += re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)
    return names


def _check(fn: str, status: int) -> None:
    if status != MMQ_OK:
        raise MMQError(fn, status)


class MMQArgumentError(ValueError):
    """A tensor handed to a wrapper does not fit the call (raised before any launch)."""


def _dev(t, name: str, nbytes: int, dtype=None, here: int | None = None) -> int:
    """Device pointer of tensor t after checking that the call may use it: a contiguous CUDA
    tensor on the current device, of `dtype` when given, holding at least `nbytes` bytes.
    The C ABI takes bare pointers and cannot check buffer sizes itself, so an undersized or
    mistyped buffer is refused here rather than read or written out of bounds. `here`: the current
    device, for a call that checks several tensors."""
    # the whole check in one expression: a decoding step makes tens of these calls, and the host
    # side of a call is longer than its kernel (0.4 us here against 0.8 us for the checks below)
    if (isinstance(t, torch.Tensor) and t.is_cuda and (dtype is None or t.dtype == dtype)
            and t.is_contiguous() and t.nbytes >= nbytes
            and t.get_device() == (_here() if here is None else here)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise MMQArgumentError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise MMQArgumentError(f"{name}: dtype must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise MMQArgumentError(f"{name}: must be contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise MMQArgumentError(f"{name}: holds {have} bytes, the call needs {nbytes}")
    if not t.is_cuda:
        raise MMQArgumentError(f"{name}: must be a CUDA tensor (got device {t.device})")
    if t.device.index != torch.cuda.current_device():
        raise MMQArgumentError(f"{name}: on {t.device}, but the current device is "
                               f"cuda:{torch.cuda.current_device()}")
    return t.data_ptr()


def _here() -> int | None:
    """The current device's index (0.1 us, a quarter of _dev: asked for once per call)."""
    try:
        return torch._C._cuda_getDevice()
    except RuntimeError:  # no GPU: then no tensor is on one
        return None


def _stream(stream, here: int | None = None) -> int | None:
    if stream is None:  # (torch.cuda.current_stream() makes a Stream object: 2.9 us against 0.2)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if here is None
                                                  else here)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _opts(force_tile: int = MMQ_TILE_AUTO, lds_budget: int = 0, min_workgroups: int = 0,
          workspace: int | None = None, workspace_bytes: int = 0, splits: int = 0):
    if (force_tile == MMQ_TILE_AUTO and lds_budget == 0 and min_workgroups == 0
            and workspace_bytes == 0 and splits == 0):
        return None
    return ctypes.byref(mmq_options(force_tile, min_workgroups, lds_budget, workspace,
                                    workspace_bytes, splits, 0))


@functools.lru_cache(maxsize=1024)
def _sized_ints(fn, *args) -> int:
    return fn(*args)


def _sized(fn, *args) -> int:
    """fn(*args) of a size query (host arithmetic on its arguments alone): the wrappers below ask
    for the same few sizes on every call. Only plain ints are remembered: what else passes for an
    integer (a 0-d tensor or array) can change, and a buffer must not be checked against a size that
    it had before."""
    for a in args:
        if type(a) is not int:
            return fn(*args)
    return _sized_ints(fn, *args)


def _workspace(workspace):
    """(pointer, bytes) of an optional split-K workspace tensor (a contiguous CUDA tensor)."""
    if workspace is None:
        return None, 0
    nbytes = workspace.numel() * workspace.element_size()
    return _dev(workspace, "workspace", 0), nbytes


# ---------------------------------------------------------------- sizes
def mmq_q8_1_bytes(M: int, K: int) -> int:
    n = _sz()
    _check("mmq_q8_1_bytes", _lib.mmq_q8_1_bytes(M, K, ctypes.byref(n)))
    return n.value


def mmq_q4K_bytes(N: int, K: int) -> int:
    n = _sz()
    _check("mmq_q4K_bytes", _lib.mmq_q4K_bytes(N, K, ctypes.byref(n)))
    return n.value


def mmq_q4K_repacked_bytes(N: int, K: int) -> int:
    n = _sz()
    _check("mmq_q4K_repacked_bytes", _lib.mmq_q4K_repacked_bytes(N, K, ctypes.byref(n)))
    return n.value


# ---------------------------------------------------------------- the hot path
# All buffer sizes of a call at once, for the calls of a decoding step: called with _int(...) of their
# arguments, so that they remember by value (three sizes 0.14 us, against 0.32 by _sized).
_sizes = functools.lru_cache(maxsize=256)


@_sizes
def _gemm_sizes(M, N, K):
    return mmq_q8_1_bytes(M, K), mmq_q4K_repacked_bytes(N, K), 4 * M * N


@_sizes
def _quantize_sizes(M, K):
    return 4 * M * K, mmq_q8_1_bytes(M, K)


@_sizes
def _f32_sizes(M, N, K):
    return 4 * M * K, mmq_q4K_repacked_bytes(N, K), 4 * M * N


def _gemm_ptrs(M: int, N: int, K: int, q8, w_rep, C, here: int | None = None):
    qn, rn, cn = _gemm_sizes(_int(M), _int(N), _int(K))
    return (_dev(q8, "q8", qn, here=here), _dev(w_rep, "w_rep", rn, here=here),
            _dev(C, "C", cn, torch.float32, here))


def quantize_q8_1(x, M: int, K: int, q8, stream=None) -> None:
    """x: f32 [M, K] device tensor; q8: device buffer of mmq_q8_1_bytes(M, K) bytes."""
    here = _here()
    xn, qn = _quantize_sizes(_int(M), _int(K))
    xp = _dev(x, "x", xn, torch.float32, here)
    qp = _dev(q8, "q8", qn, here=here)
    _check("quantize_q8_1", _lib.quantize_q8_1(xp, M, K, qp, _stream(stream, here)))


def repack_q4_K(w_q4K, N: int, K: int, w_rep, stream=None) -> None:
    """w_q4K: q4_K blocks (mmq_q4K_bytes); w_rep: mmq_q4K_repacked_bytes(N, K) bytes."""
    wp = _dev(w_q4K, "w_q4K", _sized(mmq_q4K_bytes, N, K))
    rp = _dev(w_rep, "w_rep", _sized(mmq_q4K_repacked_bytes, N, K))
    _check("repack_q4_K", _lib.repack_q4_K(wp, N, K, rp, _stream(stream)))


def mmq_q4K_q8_1(M: int, N: int, K: int, q8, w_rep, C, stream=None) -> None:
    """C[M, N] (f32 device tensor) = q8 (M x K) times repacked q4_K weights (N x K)^T."""
    qp, rp, cp = _gemm_ptrs(M, N, K, q8, w_rep, C)
    _check("mmq_q4K_q8_1", _lib.mmq_q4K_q8_1(M, N, K, qp, rp, cp, _stream(stream)))


def mmq_q4K_q8_1_ex(M: int, N: int, K: int, q8, w_rep, C, stream=None,
                    force_tile: int = MMQ_TILE_AUTO, lds_budget: int = 0,
                    min_workgroups: int = 0, workspace=None, splits: int = 0) -> None:
    """As mmq_q4K_q8_1 with options; `workspace` (any contiguous CUDA tensor, its whole byte
    size usable) lets the guard split K over workgroups, `splits` forces a split count."""
    qp, rp, cp = _gemm_ptrs(M, N, K, q8, w_rep, C)
    wp, wb = _workspace(workspace)
    _check("mmq_q4K_q8_1_ex",
           _lib.mmq_q4K_q8_1_ex(M, N, K, qp, rp, cp, _stream(stream),
                                _opts(force_tile, lds_budget, min_workgroups, wp, wb, splits)))


def mmq_q4K_q8_1_static(M: int, N: int, K: int, q8, w_rep, C, stream=None,
                        force_tile: int = MMQ_TILE_AUTO, lds_budget: int = 0,
                        min_workgroups: int = 0, splits: int = 0) -> None:
    """As mmq_q4K_q8_1_ex, the split-K workspace being the library's own 32 MiB device array
    (for callers that cannot allocate); calls that overlap on one GPU race."""
    qp, rp, cp = _gemm_ptrs(M, N, K, q8, w_rep, C)
    _check("mmq_q4K_q8_1_static",
           _lib.mmq_q4K_q8_1_static(M, N, K, qp, rp, cp, _stream(stream),
                                    _opts(force_tile, lds_budget, min_workgroups, None, 0,
                                          splits)))


def mmq_workspace_bytes(M: int, N: int, K: int) -> int:
    """Split-K workspace the guard would use for M x N x K given an unlimited one (0: none)."""
    n = _sz()
    _check("mmq_workspace_bytes", _lib.mmq_workspace_bytes(M, N, K, ctypes.byref(n)))
    return n.value


def mmq_q4K_f32(M: int, N: int, K: int, x, w_rep, C, stream=None) -> None:
    """Few tokens (M <= 128): C[M, N] from f32 activations x [M, K], quantized in the GEMM."""
    here = _here()
    xn, rn, cn = _f32_sizes(_int(M), _int(N), _int(K))
    xp = _dev(x, "x", xn, torch.float32, here)
    rp = _dev(w_rep, "w_rep", rn, here=here)
    cp = _dev(C, "C", cn, torch.float32, here)
    _check("mmq_q4K_f32", _lib.mmq_q4K_f32(M, N, K, xp, rp, cp, _stream(stream, here)))


def _dots_bytes(K, per, i0, i1, j0, j1) -> int:
    return 4 * (_int(K) // per) * max(_int(i1) - _int(i0), 0) * max(_int(j1) - _int(j0), 0)


def mmq_q4K_q8_1_blockdots(M: int, N: int, K: int, q8, w_rep, i0: int, i1: int, j0: int,
                           j1: int, S, stream=None, force_tile: int = MMQ_TILE_AUTO,
                           lds_budget: int = 0) -> None:
    """S: int32 device tensor [K/32, i1-i0, j1-j0] of per-block integer dot products."""
    qp = _dev(q8, "q8", _sized(mmq_q8_1_bytes, M, K))
    rp = _dev(w_rep, "w_rep", _sized(mmq_q4K_repacked_bytes, N, K))
    sp = _dev(S, "S", _dots_bytes(K, QK8, i0, i1, j0, j1), torch.int32)
    _check("mmq_q4K_q8_1_blockdots",
           _lib.mmq_q4K_q8_1_blockdots(M, N, K, qp, rp, i0, i1, j0, j1, sp,
                                       _stream(stream), _opts(force_tile, lds_budget)))


# ---------------------------------------------------------------- the product's epilogue
def _epi(M: int, N: int, bias, residual, act: int, here: int):
    M, N = _int(M), _int(N)
    bp = None if bias is None else _dev(bias, "bias", 4 * N, torch.float32, here)
    rp = None if residual is None else _dev(residual, "residual", 4 * M * N, torch.float32, here)
    return ctypes.byref(mmq_epilogue(bp, rp, act, 0))


def mmq_q4K_q8_1_epilogue(M: int, N: int, K: int, q8, w_rep, C, bias=None, residual=None,
                          act: int = MMQ_ACT_NONE, stream=None, force_tile: int = MMQ_TILE_AUTO,
                          lds_budget: int = 0, min_workgroups: int = 0, workspace=None,
                          splits: int = 0) -> None:
    """C[M, N] = act(product + bias[N]) + residual[M, N] (f32 tensors; residual may be C)."""
    here = _here()
    qp, rp, cp = _gemm_ptrs(M, N, K, q8, w_rep, C, here)
    wp, wb = _workspace(workspace)
    _check("mmq_q4K_q8_1_epilogue",
           _lib.mmq_q4K_q8_1_epilogue(M, N, K, qp, rp, cp, _stream(stream, here),
                                      _epi(M, N, bias, residual, act, here),
                                      _opts(force_tile, lds_budget, min_workgroups, wp, wb,
                                            splits)))


def mmq_q4K_f32_epilogue(M: int, N: int, K: int, x, w_rep, C, bias=None, residual=None,
                         act: int = MMQ_ACT_NONE, stream=None) -> None:
    """Few tokens (M <= 128): the same from f32 activations x [M, K]."""
    here = _here()
    xn, rn, cn = _f32_sizes(_int(M), _int(N), _int(K))
    xp = _dev(x, "x", xn, torch.float32, here)
    rp = _dev(w_rep, "w_rep", rn, here=here)
    cp = _dev(C, "C", cn, torch.float32, here)
    _check("mmq_q4K_f32_epilogue",
           _lib.mmq_q4K_f32_epilogue(M, N, K, xp, rp, cp, _stream(stream, here),
                                     _epi(M, N, bias, residual, act, here)))


# ---------------------------------------------------------------- the gated product
def mmq_q4K_pair_bytes(F: int, K: int) -> int:
    n = _sz()
    _check("mmq_q4K_pair_bytes", _lib.mmq_q4K_pair_bytes(F, K, ctypes.byref(n)))
    return n.value


def repack_q4_K_pair(w_gate, w_up, F: int, K: int, w_pair, stream=None) -> None:
    """w_gate, w_up: q4_K blocks (mmq_q4K_bytes(F, K)); w_pair: mmq_q4K_pair_bytes(F, K) bytes."""
    gp = _dev(w_gate, "w_gate", _sized(mmq_q4K_bytes, F, K))
    up = _dev(w_up, "w_up", _sized(mmq_q4K_bytes, F, K))
    pp = _dev(w_pair, "w_pair", _sized(mmq_q4K_pair_bytes, F, K))
    _check("repack_q4_K_pair", _lib.repack_q4_K_pair(gp, up, F, K, pp, _stream(stream)))


def mmq_gated_workspace_bytes(M: int, F: int, K: int) -> int:
    """Split-K workspace mmq_q4K_q8_1_gated would use given an unlimited one (0: none)."""
    n = _sz()
    _check("mmq_gated_workspace_bytes",
           _lib.mmq_gated_workspace_bytes(M, F, K, ctypes.byref(n)))
    return n.value


@_sizes
def _gated_sizes(M, F, K):
    return mmq_q8_1_bytes(M, K), mmq_q4K_pair_bytes(F, K), 4 * M * F


@_sizes
def _f32_gated_sizes(M, F, K):
    return 4 * M * K, mmq_q4K_pair_bytes(F, K), 4 * M * F


def mmq_q4K_q8_1_gated(M: int, F: int, K: int, q8, w_pair, H, act: int = MMQ_ACT_SILU,
                       stream=None, force_tile: int = MMQ_TILE_AUTO, lds_budget: int = 0,
                       min_workgroups: int = 0, workspace=None, splits: int = 0) -> None:
    """H[M, F] (f32) = act(x Wg^T) * (x Wu^T), q8 (M x K) and a repacked pair (F x K)."""
    here = _here()
    qn, pn, hn = _gated_sizes(_int(M), _int(F), _int(K))
    qp = _dev(q8, "q8", qn, here=here)
    pp = _dev(w_pair, "w_pair", pn, here=here)
    hp = _dev(H, "H", hn, torch.float32, here)
    wp, wb = _workspace(workspace)
    _check("mmq_q4K_q8_1_gated",
           _lib.mmq_q4K_q8_1_gated(M, F, K, qp, pp, hp, _stream(stream, here), act,
                                   _opts(force_tile, lds_budget, min_workgroups, wp, wb, splits)))


def mmq_q4K_f32_gated(M: int, F: int, K: int, x, w_pair, H, act: int = MMQ_ACT_SILU,
                      stream=None) -> None:
    """Few tokens (M <= 128): the same from f32 activations x [M, K]."""
    here = _here()
    xn, pn, hn = _f32_gated_sizes(_int(M), _int(F), _int(K))
    xp = _dev(x, "x", xn, torch.float32, here)
    pp = _dev(w_pair, "w_pair", pn, here=here)
    hp = _dev(H, "H", hn, torch.float32, here)
    _check("mmq_q4K_f32_gated",
           _lib.mmq_q4K_f32_gated(M, F, K, xp, pp, hp, _stream(stream, here), act))


# ---------------------------------------------------------------- mixture of experts
def mmq_moe_plan_bytes(M: int, E: int, k: int) -> int:
    n = _sz()
    _check("mmq_moe_plan_bytes", _lib.mmq_moe_plan_bytes(M, E, k, ctypes.byref(n)))
    return n.value


def mmq_moe_plan(M: int, E: int, k: int, ids, plan, stream=None) -> None:
    """plan (int32, mmq_moe_plan_bytes) from ids int32 [M, k]; an id outside [0, E) is no expert."""
    here = _here()
    ip = _dev(ids, "ids", 4 * _int(M) * _int(k), torch.int32, here)
    pp = _dev(plan, "plan", _sized(mmq_moe_plan_bytes, M, E, k), torch.int32, here)
    _check("mmq_moe_plan", _lib.mmq_moe_plan(M, E, k, ip, pp, _stream(stream, here)))


@_sizes
def _route_sizes(M, E, k, planned):
    return 4 * M * E, 4 * M * k, mmq_moe_plan_bytes(M, E, k) if planned else 0


@_sizes
def _moe_gated_sizes(M, E, k, F, D):
    return (4 * M * D, mmq_moe_plan_bytes(M, E, k), E * mmq_q4K_pair_bytes(F, D), 4 * M * k * F,
            mmq_q8_1_bytes(M, D))


@_sizes
def _moe_down_sizes(M, E, k, D, F):
    return (4 * M * k * F, mmq_moe_plan_bytes(M, E, k), 4 * M * k,
            E * mmq_q4K_repacked_bytes(D, F), 4 * M * D, mmq_q8_1_bytes(M * k, F))


@_sizes
def _moe_sizes(M, E, k, D, F):
    return (4 * M * D, 4 * M * E, E * mmq_q4K_pair_bytes(F, D), E * mmq_q4K_repacked_bytes(D, F),
            mmq_moe_workspace_bytes(M, E, k, D, F))


def mmq_moe_route(M: int, E: int, k: int, logits, ids, weights, plan=None,
                  score: int = MMQ_SCORE_SOFTMAX, renorm: bool = True, stream=None) -> None:
    """The k experts of the greatest logits [M, E] (f32): ids int32 [M, k], weights f32 [M, k] and,
    for at most 64 tokens, the plan of the experts' products (int32, mmq_moe_plan_bytes)."""
    here = _here()
    ln, kn, pn = _route_sizes(_int(M), _int(E), _int(k), plan is not None)
    lp = _dev(logits, "logits", ln, torch.float32, here)
    ip = _dev(ids, "ids", kn, torch.int32, here)
    wp = _dev(weights, "weights", kn, torch.float32, here)
    pp = None if plan is None else _dev(plan, "plan", pn, torch.int32, here)
    _check("mmq_moe_route",
           _lib.mmq_moe_route(M, E, k, lp, score, int(renorm), ip, wp, pp, _stream(stream, here)))


def mmq_q4K_moe_gated(M: int, E: int, k: int, F: int, D: int, x, plan, w_pairs, H, q8,
                      act: int = MMQ_ACT_SILU, stream=None) -> None:
    """H[M*k, F] (f32): per (token, slot) pair of the plan the gated product of its expert.
    w_pairs: E repacked pairs (mmq_q4K_pair_bytes(F, D) each); q8: scratch, mmq_q8_1_bytes(M, D)."""
    here = _here()
    xn, pn, wn, hn, qn = _moe_gated_sizes(_int(M), _int(E), _int(k), _int(F), _int(D))
    xp = _dev(x, "x", xn, torch.float32, here)
    pp = _dev(plan, "plan", pn, torch.int32, here)
    wp = _dev(w_pairs, "w_pairs", wn, here=here)
    hp = _dev(H, "H", hn, torch.float32, here)
    qp = _dev(q8, "q8", qn, here=here)
    _check("mmq_q4K_moe_gated",
           _lib.mmq_q4K_moe_gated(M, E, k, F, D, xp, pp, wp, hp, qp, act, _stream(stream, here)))


def mmq_q4K_moe_down(M: int, E: int, k: int, D: int, F: int, H, plan, weights, w_down, out, q8,
                     residual=None, stream=None) -> None:
    """out[M, D] (f32) = residual + per token the weighted sum over its slots of H[p] W(expert)^T.
    w_down: E repacked matrices (mmq_q4K_repacked_bytes(D, F) each); q8: scratch of
    mmq_q8_1_bytes(M*k, F) bytes; residual may be out."""
    here = _here()
    hn, pn, gn, wn, on, qn = _moe_down_sizes(_int(M), _int(E), _int(k), _int(D), _int(F))
    hp = _dev(H, "H", hn, torch.float32, here)
    pp = _dev(plan, "plan", pn, torch.int32, here)
    gp = _dev(weights, "weights", gn, torch.float32, here)
    wp = _dev(w_down, "w_down", wn, here=here)
    op = _dev(out, "out", on, torch.float32, here)
    rp = None if residual is None else _dev(residual, "residual", on, torch.float32, here)
    qp = _dev(q8, "q8", qn, here=here)
    _check("mmq_q4K_moe_down",
           _lib.mmq_q4K_moe_down(M, E, k, D, F, hp, pp, gp, wp, rp, op, qp, _stream(stream, here)))


def mmq_moe_workspace_bytes(M: int, E: int, k: int, D: int, F: int) -> int:
    n = _sz()
    _check("mmq_moe_workspace_bytes",
           _lib.mmq_moe_workspace_bytes(M, E, k, D, F, ctypes.byref(n)))
    return n.value


def mmq_q4K_moe(M: int, E: int, k: int, D: int, F: int, x, logits, w_pairs, w_down, out,
                workspace, score: int = MMQ_SCORE_SOFTMAX, renorm: bool = True,
                act: int = MMQ_ACT_SILU, residual=None, stream=None) -> None:
    """The whole layer for a few tokens: out[M, D] = residual + experts of x [M, D] chosen by the
    router's logits [M, E]. workspace: mmq_moe_workspace_bytes(M, E, k, D, F) bytes."""
    here = _here()
    xn, ln, gn, dn, sn = _moe_sizes(_int(M), _int(E), _int(k), _int(D), _int(F))
    xp = _dev(x, "x", xn, torch.float32, here)
    lp = _dev(logits, "logits", ln, torch.float32, here)
    gp = _dev(w_pairs, "w_pairs", gn, here=here)
    dp = _dev(w_down, "w_down", dn, here=here)
    op = _dev(out, "out", xn, torch.float32, here)
    rp = None if residual is None else _dev(residual, "residual", xn, torch.float32, here)
    sp = _dev(workspace, "workspace", sn, here=here)
    sb = workspace.numel() * workspace.element_size()
    _check("mmq_q4K_moe",
           _lib.mmq_q4K_moe(M, E, k, D, F, xp, lp, score, int(renorm), gp, act, dp, rp, op, sp, sb,
                            _stream(stream, here)))


# ---------------------------------------------------------------- products grouped by expert
def mmq_moe_group_bytes(M: int, E: int, k: int) -> int:
    n = _sz()
    _check("mmq_moe_group_bytes", _lib.mmq_moe_group_bytes(M, E, k, ctypes.byref(n)))
    return n.value


@_sizes
def _group_sizes(M, E, k):
    return 4 * M * k, mmq_moe_group_bytes(M, E, k)


def mmq_moe_group(M: int, E: int, k: int, ids, groups, stream=None) -> None:
    """groups (int32, mmq_moe_group_bytes): the pairs of ids int32 [M, k] sorted by expert; an id
    outside [0, E) is no expert. moe_groups gives its parts."""
    here = _here()
    n, gn = _group_sizes(_int(M), _int(E), _int(k))
    ip = _dev(ids, "ids", n, torch.int32, here)
    gp = _dev(groups, "groups", gn, torch.int32, here)
    _check("mmq_moe_group", _lib.mmq_moe_group(M, E, k, ip, gp, _stream(stream, here)))


def moe_groups(groups, M: int, E: int, k: int):
    """Views (offsets [E + 1], order [M*k], place [M*k]) of what mmq_moe_group wrote."""
    M, E, k = _int(M), _int(E), _int(k)
    need = _group_sizes(M, E, k)[1]
    if (not isinstance(groups, torch.Tensor) or groups.dtype != torch.int32
            or not groups.is_contiguous() or groups.nbytes < need):
        raise MMQArgumentError(f"groups: must be a contiguous int32 tensor of {need} bytes or more")
    P, at = M * k, groups.storage_offset()
    a = (E + 1 + 3) // 4 * 4
    b = a + (P + 3) // 4 * 4
    one = (1,)
    return (groups.as_strided((E + 1,), one, at), groups.as_strided((P,), one, at + a),
            groups.as_strided((P,), one, at + b))


@_sizes
def _grouped_sizes(M, E, k, N, K, per_pair):
    rows = M * k if per_pair else M
    return (4 * rows * K, mmq_moe_group_bytes(M, E, k), E * mmq_q4K_repacked_bytes(N, K),
            4 * M * k * N, mmq_q8_1_bytes(rows, K))


@_sizes
def _grouped_gated_sizes(M, E, k, F, D):
    return (4 * M * D, mmq_moe_group_bytes(M, E, k), E * mmq_q4K_pair_bytes(F, D), 4 * M * k * F,
            mmq_q8_1_bytes(M, D))


@_sizes
def _grouped_down_sizes(M, E, k, D, F):
    return (4 * M * k * F, mmq_moe_group_bytes(M, E, k), 4 * M * k,
            E * mmq_q4K_repacked_bytes(D, F), 4 * M * D,
            mmq_grouped_down_workspace_bytes(M, E, k, D, F))


@_sizes
def _grouped_moe_sizes(M, E, k, D, F):
    return (4 * M * D, 4 * M * E, E * mmq_q4K_pair_bytes(F, D), E * mmq_q4K_repacked_bytes(D, F),
            mmq_grouped_moe_workspace_bytes(M, E, k, D, F))


def mmq_q4K_grouped(M: int, E: int, k: int, N: int, K: int, x, groups, w_rep, C, q8,
                    per_pair: bool = False, act: int = MMQ_ACT_NONE, stream=None) -> None:
    """C[M*k, N] (f32) = act(x[r] W(expert)^T) per pair p of the groups, r = p // k (x [M, K]) or, with
    per_pair, p (x [M*k, K]). w_rep: E repacked matrices; q8: scratch, mmq_q8_1_bytes(rows of x, K)."""
    here = _here()
    xn, gn, wn, cn, qn = _grouped_sizes(_int(M), _int(E), _int(k), _int(N), _int(K),
                                        bool(per_pair))
    xp = _dev(x, "x", xn, torch.float32, here)
    gp = _dev(groups, "groups", gn, torch.int32, here)
    wp = _dev(w_rep, "w_rep", wn, here=here)
    cp = _dev(C, "C", cn, torch.float32, here)
    qp = _dev(q8, "q8", qn, here=here)
    _check("mmq_q4K_grouped",
           _lib.mmq_q4K_grouped(M, E, k, N, K, xp, int(bool(per_pair)), gp, wp, cp, qp, act,
                                _stream(stream, here)))


def mmq_q4K_grouped_gated(M: int, E: int, k: int, F: int, D: int, x, groups, w_pairs, H, q8,
                          act: int = MMQ_ACT_SILU, stream=None) -> None:
    """H[M*k, F] (f32): per pair of the groups the gated product of its expert, for any number of
    tokens. w_pairs: E repacked pairs; q8: scratch, mmq_q8_1_bytes(M, D)."""
    here = _here()
    xn, gn, wn, hn, qn = _grouped_gated_sizes(_int(M), _int(E), _int(k), _int(F), _int(D))
    xp = _dev(x, "x", xn, torch.float32, here)
    gp = _dev(groups, "groups", gn, torch.int32, here)
    wp = _dev(w_pairs, "w_pairs", wn, here=here)
    hp = _dev(H, "H", hn, torch.float32, here)
    qp = _dev(q8, "q8", qn, here=here)
    _check("mmq_q4K_grouped_gated",
           _lib.mmq_q4K_grouped_gated(M, E, k, F, D, xp, gp, wp, hp, qp, act,
                                      _stream(stream, here)))


def mmq_grouped_down_workspace_bytes(M: int, E: int, k: int, D: int, F: int) -> int:
    n = _sz()
    _check("mmq_grouped_down_workspace_bytes",
           _lib.mmq_grouped_down_workspace_bytes(M, E, k, D, F, ctypes.byref(n)))
    return n.value


def mmq_q4K_grouped_down(M: int, E: int, k: int, D: int, F: int, H, groups, weights, w_down, out,
                         workspace, residual=None, stream=None) -> None:
    """out[M, D] (f32) = residual + per token the weighted sum over its slots of H[p] W(expert)^T.
    workspace: mmq_grouped_down_workspace_bytes(M, E, k, D, F) bytes; residual may be out."""
    here = _here()
    hn, gn, tn, wn, on, sn = _grouped_down_sizes(_int(M), _int(E), _int(k), _int(D), _int(F))
    hp = _dev(H, "H", hn, torch.float32, here)
    gp = _dev(groups, "groups", gn, torch.int32, here)
    tp = _dev(weights, "weights", tn, torch.float32, here)
    wp = _dev(w_down, "w_down", wn, here=here)
    op = _dev(out, "out", on, torch.float32, here)
    rp = None if residual is None else _dev(residual, "residual", on, torch.float32, here)
    sp = _dev(workspace, "workspace", sn, here=here)
    _check("mmq_q4K_grouped_down",
           _lib.mmq_q4K_grouped_down(M, E, k, D, F, hp, gp, tp, wp, rp, op, sp, workspace.nbytes,
                                     _stream(stream, here)))


def mmq_grouped_moe_workspace_bytes(M: int, E: int, k: int, D: int, F: int) -> int:
    n = _sz()
    _check("mmq_grouped_moe_workspace_bytes",
           _lib.mmq_grouped_moe_workspace_bytes(M, E, k, D, F, ctypes.byref(n)))
    return n.value


def mmq_q4K_grouped_moe(M: int, E: int, k: int, D: int, F: int, x, logits, w_pairs, w_down, out,
                        workspace, score: int = MMQ_SCORE_SOFTMAX, renorm: bool = True,
                        act: int = MMQ_ACT_SILU, residual=None, stream=None) -> None:
    """The whole layer for any number of tokens: out[M, D] = residual + experts of x [M, D] chosen by
    the router's logits [M, E]. workspace: mmq_grouped_moe_workspace_bytes(M, E, k, D, F) bytes."""
    here = _here()
    xn, ln, gn, dn, sn = _grouped_moe_sizes(_int(M), _int(E), _int(k), _int(D), _int(F))
    xp = _dev(x, "x", xn, torch.float32, here)
    lp = _dev(logits, "logits", ln, torch.float32, here)
    gp = _dev(w_pairs, "w_pairs", gn, here=here)
    dp = _dev(w_down, "w_down", dn, here=here)
    op = _dev(out, "out", xn, torch.float32, here)
    rp = None if residual is None else _dev(residual, "residual", xn, torch.float32, here)
    sp = _dev(workspace, "workspace", sn, here=here)
    _check("mmq_q4K_grouped_moe",
           _lib.mmq_q4K_grouped_moe(M, E, k, D, F, xp, lp, score, int(renorm), gp, act, dp, rp, op,
                                    sp, workspace.nbytes, _stream(stream, here)))


# ---------------------------------------------------------------- group scales (q4_G)
def q4G_format(group: int, scale_dtype, zeros: bool) -> mmq_q4G_format:
    """How the weights of a q4_G matrix are scaled: `group` values share a scale (and, with zeros, a
    zero) of scale_dtype, torch.float16 or torch.bfloat16."""
    if scale_dtype not in (torch.float16, torch.bfloat16):
        raise MMQArgumentError(f"scale_dtype: must be float16 or bfloat16, got {scale_dtype}")
    group = _int(group)
    if not -2 ** 31 <= group < 2 ** 31:  # the structure would keep its low 32 bits
        raise MMQArgumentError(f"group: {group} does not fit 32 bits")
    return mmq_q4G_format(group, TYPES[scale_dtype], int(bool(zeros)), 0)


@_sizes
def _q4G_bytes(N, K, group, scale_type, zeros, reserved):
    n = _sz()
    _check("mmq_q4G_repacked_bytes",
           _lib.mmq_q4G_repacked_bytes(N, K, mmq_q4G_format(group, scale_type, zeros, reserved),
                                       ctypes.byref(n)))
    return n.value


def _q4G_size(N, K, f):
    if not isinstance(f, mmq_q4G_format):
        raise MMQArgumentError(f"format: expected an mmq_q4G_format, got {type(f).__name__}")
    return _q4G_bytes(N, K, f.group, f.scale_type, f.zeros, f.reserved)


def mmq_q4G_repacked_bytes(N: int, K: int, format: mmq_q4G_format) -> int:
    return _q4G_size(_int(N), _int(K), format)


def repack_q4_G(w, scales, zeros, N: int, K: int, format: mmq_q4G_format, w_rep,
                stream=None) -> None:
    """w: uint8 [N, K/2], the even value of two in the low four bits; scales and zeros (None where the
    format has none): [N, ceil(K/group)] of the format's type; w_rep: mmq_q4G_repacked_bytes."""
    here = _here()
    N, K = _int(N), _int(K)  # the sizes below in Python's integers, which do not wrap
    rn = _q4G_size(N, K, format)
    dtype = torch.float16 if format.scale_type == MMQ_F16 else torch.bfloat16
    n = 2 * N * -(-K // format.group)
    wp = _dev(w, "w", N * K // 2, torch.uint8, here)
    sp = _dev(scales, "scales", n, dtype, here)
    zp = None if zeros is None else _dev(zeros, "zeros", n, dtype, here)
    rp = _dev(w_rep, "w_rep", rn, here=here)
    _check("repack_q4_G", _lib.repack_q4_G(wp, sp, zp, N, K, ctypes.byref(format), rp,
                                           _stream(stream, here)))


def mmq_q4G(M: int, N: int, K: int, x, w_rep, format: mmq_q4G_format, y, bias=None, residual=None,
            act: int = MMQ_ACT_NONE, stream=None) -> None:
    """y[M, N] = act(x[M, K] W^T + bias[N]) + residual[M, N] for 1 <= M <= 16 tokens. x and y: float32,
    float16 or bfloat16 each; residual of y's type (it may be y), bias float32."""
    here = _here()
    M, N, K = _int(M), _int(N), _int(K)
    rn = _q4G_size(N, K, format)
    xt, yt = TYPES.get(getattr(x, "dtype", None)), TYPES.get(getattr(y, "dtype", None))
    if xt is None or yt is None:
        raise MMQArgumentError("x and y: must be float32, float16 or bfloat16 tensors")
    yn = M * N * (4 if yt == MMQ_F32 else 2)
    xp = _dev(x, "x", M * K * (4 if xt == MMQ_F32 else 2), None, here)
    rp = _dev(w_rep, "w_rep", rn, here=here)
    yp = _dev(y, "y", yn, None, here)
    epi = None
    if bias is not None or residual is not None or act != MMQ_ACT_NONE:
        epi = ctypes.byref(mmq_q4G_epilogue(
            None if bias is None else _dev(bias, "bias", 4 * N, torch.float32, here),
            None if residual is None else _dev(residual, "residual", yn, y.dtype, here), act, 0))
    _check("mmq_q4G", _lib.mmq_q4G(M, N, K, xt, xp, rp, ctypes.byref(format), yt, yp, epi,
                                   _stream(stream, here)))


# ---------------------------------------------------------------- the q6_K variant
def mmq_q6K_bytes(N: int, K: int) -> int:
    n = _sz()
    _check("mmq_q6K_bytes", _lib.mmq_q6K_bytes(N, K, ctypes.byref(n)))
    return n.value


def mmq_q6K_repacked_bytes(N: int, K: int) -> int:
    n = _sz()
    _check("mmq_q6K_repacked_bytes", _lib.mmq_q6K_repacked_bytes(N, K, ctypes.byref(n)))
    return n.value


def repack_q6_K(w_q6K, N: int, K: int, w_rep, stream=None) -> None:
    """w_q6K: q6_K blocks (mmq_q6K_bytes); w_rep: mmq_q6K_repacked_bytes(N, K) bytes."""
    wp = _dev(w_q6K, "w_q6K", _sized(mmq_q6K_bytes, N, K))
    rp = _dev(w_rep, "w_rep", _sized(mmq_q6K_repacked_bytes, N, K))
    _check("repack_q6_K", _lib.repack_q6_K(wp, N, K, rp, _stream(stream)))


@_sizes
def _gemm6_sizes(M, N, K):
    return mmq_q8_1_bytes(M, K), mmq_q6K_repacked_bytes(N, K), 4 * M * N


def _gemm6_ptrs(M: int, N: int, K: int, q8, w_rep, C):
    qn, rn, cn = _gemm6_sizes(_int(M), _int(N), _int(K))
    return (_dev(q8, "q8", qn), _dev(w_rep, "w_rep", rn), _dev(C, "C", cn, torch.float32))


def mmq_q6K_q8_1(M: int, N: int, K: int, q8, w_rep, C, stream=None) -> None:
    """C[M, N] (f32) = q8 (M x K) times repacked q6_K weights (N x K)^T."""
    qp, rp, cp = _gemm6_ptrs(M, N, K, q8, w_rep, C)
    _check("mmq_q6K_q8_1", _lib.mmq_q6K_q8_1(M, N, K, qp, rp, cp, _stream(stream)))


def mmq_q6K_q8_1_ex(M: int, N: int, K: int, q8, w_rep, C, stream=None,
                    force_tile: int = MMQ_TILE_AUTO, lds_budget: int = 0,
                    min_workgroups: int = 0, workspace=None, splits: int = 0) -> None:
    qp, rp, cp = _gemm6_ptrs(M, N, K, q8, w_rep, C)
    wp, wb = _workspace(workspace)
    _check("mmq_q6K_q8_1_ex",
           _lib.mmq_q6K_q8_1_ex(M, N, K, qp, rp, cp, _stream(stream),
                                _opts(force_tile, lds_budget, min_workgroups, wp, wb, splits)))


def mmq_q6K_q8_1_blockdots(M: int, N: int, K: int, q8, w_rep, i0: int, i1: int, j0: int,
                           j1: int, S, stream=None, force_tile: int = MMQ_TILE_AUTO) -> None:
    """S: int32 device tensor [K/16, i1-i0, j1-j0] of per-group integer dot products."""
    qp = _dev(q8, "q8", _sized(mmq_q8_1_bytes, M, K))
    rp = _dev(w_rep, "w_rep", _sized(mmq_q6K_repacked_bytes, N, K))
    sp = _dev(S, "S", _dots_bytes(K, 16, i0, i1, j0, j1), torch.int32)
    _check("mmq_q6K_q8_1_blockdots",
           _lib.mmq_q6K_q8_1_blockdots(M, N, K, qp, rp, i0, i1, j0, j1, sp, _stream(stream),
                                       _opts(force_tile)))


# ---------------------------------------------------------------- the guard
def mmq_plan(M: int, N: int, K: int, lds_budget: int, force_tile: int = MMQ_TILE_AUTO,
             opt_lds_budget: int = 0, min_workgroups: int = 0, workspace_bytes: int = 0,
             splits: int = 0) -> dict:
    info = mmq_kernel_info()
    _check("mmq_plan", _lib.mmq_plan(M, N, K, _opts(force_tile, opt_lds_budget, min_workgroups,
                                                    None, workspace_bytes, splits),
                                     lds_budget, ctypes.byref(info)))
    return info.as_dict()


# ---------------------------------------------------------------- the f16 comparator path
def mmq_f16_bytes(rows: int, K: int) -> int:
    n = _sz()
    _check("mmq_f16_bytes", _lib.mmq_f16_bytes(rows, K, ctypes.byref(n)))
    return n.value


def convert_f32_f16(x, M: int, K: int, x_f16, stream=None) -> None:
    """x: f32 [M, K] device tensor; x_f16: device buffer of mmq_f16_bytes(M, K) bytes."""
    xp = _dev(x, "x", 4 * _int(M) * _int(K), torch.float32)
    hp = _dev(x_f16, "x_f16", _sized(mmq_f16_bytes, M, K))
    _check("convert_f32_f16", _lib.convert_f32_f16(xp, M, K, hp, _stream(stream)))


def dequantize_q4_K_f16(w_q4K, N: int, K: int, w_f16, stream=None) -> None:
    """w_q4K: q4_K blocks (mmq_q4K_bytes); w_f16: mmq_f16_bytes(N, K) bytes."""
    wp = _dev(w_q4K, "w_q4K", _sized(mmq_q4K_bytes, N, K))
    hp = _dev(w_f16, "w_f16", _sized(mmq_f16_bytes, N, K))
    _check("dequantize_q4_K_f16", _lib.dequantize_q4_K_f16(wp, N, K, hp, _stream(stream)))


def gemm_f16(M: int, N: int, K: int, x_f16, w_f16, C, stream=None) -> None:
    """C[M, N] (f32 device tensor) = x_f16 [M, K] times w_f16 [N, K]^T, f32 accumulation."""
    xp = _dev(x_f16, "x_f16", _sized(mmq_f16_bytes, M, K))
    wp = _dev(w_f16, "w_f16", _sized(mmq_f16_bytes, N, K))
    cp = _dev(C, "C", 4 * _int(M) * _int(N), torch.float32)
    _check("gemm_f16", _lib.gemm_f16(M, N, K, xp, wp, cp, _stream(stream)))


def mmq_last_kernel() -> dict:
    info = mmq_kernel_info()
    _check("mmq_last_kernel", _lib.mmq_last_kernel(ctypes.byref(info)))
    return info.as_dict()


def mmq_status_str(status: int) -> str:
    return _lib.mmq_status_str(status).decode()


def mmq_last_error() -> str:
    return _lib.mmq_last_error().decode()


def raw_call(name: str, *args) -> int:
    """Call a C entry point by name with raw ctypes-compatible arguments; returns the status."""
    return getattr(_lib, name)(*args)
