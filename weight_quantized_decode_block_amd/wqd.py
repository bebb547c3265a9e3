"""Python binding of libwqd.so: argument marshalling only.

Every function here forwards to the C ABI declared in ``include/wqd.h`` with
the same name.  Device arguments may be torch tensors (their ``data_ptr()`` is
passed) or raw integer device addresses; ``stream`` defaults to torch's current
stream on the current device.  A non-zero status raises :class:`WqdError` with
the library's message.  The library must be built first
(``python -m weight_quantized_decode_block_amd.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libwqd.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "wqd.h")

WQD_OK, WQD_EINVAL, WQD_ENULL, WQD_EALIGN, WQD_EUNSUPPORTED, WQD_ENODEV, WQD_EHIP = range(7)
Q2_0_GROUP = 128
Q2_0_BLOCK_BYTES = 34
Q2_0_BATCHM_MAX_M = 8
W8A16_MAX_M = 16
MXFP4, MXFP8 = 4, 8  # WQD_MXFP4, WQD_MXFP8
TYPE_BF16, TYPE_FP16, TYPE_FP32 = range(3)  # WQD_TYPE_*
I4_BY_ROW = 0x100  # WQD_I4_BY_ROW
MOE_SOFTMAX, MOE_SIGMOID = range(2)  # WQD_MOE_*
Q2_0_TIER_WIDTHS = (1, 2, 4, 6, 8)  # WQD_Q2_0_TIER_WIDTHS, narrowest first

_lib = None


class WqdError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with status {code}: {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libwqd.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m weight_quantized_decode_block_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, u32, sz = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_size_t
    L.q2_0_gemv.argtypes = [vp, vp, vp, u32, u32, u32, vp]
    L.q2_0_gemv_batchm.argtypes = [vp, vp, vp, u32, u32, u32, u32, vp]
    L.w8a16_gemm_m16.argtypes = [vp, vp, vp, vp, u32, u32, u32, vp]
    L.w8a16_gemm_m16_n64.argtypes = [vp, vp, vp, vp, u32, u32, u32, vp]
    L.w8a16_gemm_m16_strided.argtypes = [vp, vp, vp, vp, u32, u32, u32, u32, u32, vp]
    L.w8a16_gemv_batch16.argtypes = [vp, vp, vp, vp, u32, u32, u32, vp]
    L.w8a16_gemv_batch16_strided.argtypes = [vp, vp, vp, vp, u32, u32, u32, u32, u32, vp]
    for f in (L.q2_0_gemv, L.q2_0_gemv_batchm, L.w8a16_gemm_m16, L.w8a16_gemm_m16_n64,
              L.w8a16_gemm_m16_strided, L.w8a16_gemv_batch16, L.w8a16_gemv_batch16_strided):
        f.restype = ctypes.c_int
    L.mx_quantize.argtypes = [vp, u32, vp, vp, u32, u32, u32, u32, vp]
    L.mx_dequantize.argtypes = [vp, vp, u32, vp, u32, u32, u32, u32, vp]
    L.add_rmsnorm_mx8.argtypes = [vp, vp, vp, vp, vp, vp, vp, u32, u32, u32, u32, ctypes.c_float, vp]
    L.w4a16_gemm.argtypes = [vp, vp, vp, vp, u32, u32, u32, u32, u32, vp]
    L.w4a16_gated.argtypes = [vp, vp, vp, vp, vp, vp, u32, u32, u32, u32, u32, vp]
    for f in (L.w4a8_gemm, L.w4a4_gemm):
        f.argtypes = [vp, vp, vp, vp, vp, u32, u32, u32, u32, vp]
    for f in (L.w4a8_gated, L.w4a4_gated):
        f.argtypes = [vp, vp, vp, vp, vp, vp, vp, u32, u32, u32, u32, vp]
    for f in (L.mx_quantize, L.mx_dequantize, L.add_rmsnorm_mx8, L.w4a16_gemm, L.w4a8_gemm, L.w4a4_gemm,
              L.w4a16_gated, L.w4a8_gated, L.w4a4_gated):
        f.restype = ctypes.c_int
    i32, f32 = ctypes.c_int, ctypes.c_float
    L.i4_pack.argtypes = [vp] * 6 + [u32] * 4 + [vp]
    L.i4a16_gemm.argtypes = [vp] * 5 + [u32] * 7 + [vp]
    L.i4a16_gated.argtypes = [vp] * 8 + [u32] * 7 + [vp]
    L.moe_route.argtypes = [vp, u32, vp, vp, vp] + [u32] * 8 + [i32, f32, vp]
    L.moe_lists.argtypes = [vp, vp, vp, u32, u32, u32, vp]
    L.i4a16_experts_gated.argtypes = [vp] * 11 + [u32] * 8 + [vp]
    L.i4a16_experts_down.argtypes = [vp] * 10 + [u32] * 8 + [vp]
    for f in (L.i4_pack, L.i4a16_gemm, L.i4a16_gated, L.moe_route, L.moe_lists, L.i4a16_experts_gated, L.i4a16_experts_down):
        f.restype = ctypes.c_int
    L.i4_packed_rows.argtypes = [u32]
    L.i4_packed_rows.restype = u32
    L.q2_0_packed_bytes.argtypes = [u32, u32]
    L.q2_0_packed_bytes.restype = sz
    L.q2_0_pack.argtypes = [vp, vp, u32, u32, vp]
    L.q2_0_pack.restype = ctypes.c_int
    L.q2_0_batchm_chunks.argtypes = [u32, u32, u32, ctypes.POINTER(ctypes.c_uint64), u32]
    L.q2_0_batchm_chunks.restype = u32
    L.q2_0_select_tier.argtypes = [u32, u32, ctypes.c_int]
    L.q2_0_select_tier.restype = ctypes.c_int
    L.q2_0_tier_width.argtypes = [u32]
    L.q2_0_tier_width.restype = u32
    L.q2_0_exact_m_tiers_enabled.argtypes = []
    L.q2_0_exact_m_tiers_enabled.restype = ctypes.c_int
    L.wqd_last_error.argtypes = []
    L.wqd_last_error.restype = ctypes.c_char_p
    _lib = L
    return L


def header_functions() -> list[str]:
    """Names of the functions include/wqd.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*([a-z][a-z0-9_]*)\s*\(", text, flags=re.M)


def last_error() -> str:
    return lib().wqd_last_error().decode()


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


_current_raw_stream = None


def _stream(stream) -> int | None:
    global _current_raw_stream
    if stream is None:
        if _current_raw_stream is None:
            import torch
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            if raw is not None:
                _current_raw_stream = lambda: raw(torch.cuda.current_device())
            else:
                _current_raw_stream = lambda: int(torch.cuda.current_stream().cuda_stream)
        return _current_raw_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(fn: str, rc: int) -> None:
    if rc != WQD_OK:
        raise WqdError(fn, rc, last_error())


# -------------------------------------------------------------- GPU calls
def q2_0_gemv(A, B, C, N: int, K: int, group: int = Q2_0_GROUP, stream=None) -> None:
    _check("q2_0_gemv", lib().q2_0_gemv(_ptr(A), _ptr(B), _ptr(C), N, K, group, _stream(stream)))


def q2_0_gemv_batchm(A, B, C, N: int, K: int, group: int = Q2_0_GROUP, M: int = 1, stream=None) -> None:
    _check("q2_0_gemv_batchm",
           lib().q2_0_gemv_batchm(_ptr(A), _ptr(B), _ptr(C), N, K, group, M, _stream(stream)))


def w8a16_gemm_m16(A, W, S, C, M: int, N: int, K: int, stream=None) -> None:
    _check("w8a16_gemm_m16",
           lib().w8a16_gemm_m16(_ptr(A), _ptr(W), _ptr(S), _ptr(C), M, N, K, _stream(stream)))


def w8a16_gemm_m16_n64(A, W, S, C, M: int, N: int, K: int, stream=None) -> None:
    _check("w8a16_gemm_m16_n64",
           lib().w8a16_gemm_m16_n64(_ptr(A), _ptr(W), _ptr(S), _ptr(C), M, N, K, _stream(stream)))


def w8a16_gemm_m16_strided(A, W, S, C, M: int, N: int, K: int, a_row_stride: int, c_row_stride: int,
                           stream=None) -> None:
    _check("w8a16_gemm_m16_strided",
           lib().w8a16_gemm_m16_strided(_ptr(A), _ptr(W), _ptr(S), _ptr(C), M, N, K, a_row_stride,
                                        c_row_stride, _stream(stream)))


def w8a16_gemv_batch16(A, W, S, C, M: int, N: int, K: int, stream=None) -> None:
    _check("w8a16_gemv_batch16",
           lib().w8a16_gemv_batch16(_ptr(A), _ptr(W), _ptr(S), _ptr(C), M, N, K, _stream(stream)))


def w8a16_gemv_batch16_strided(A, W, S, C, M: int, N: int, K: int, a_row_stride: int, c_row_stride: int,
                               stream=None) -> None:
    _check("w8a16_gemv_batch16_strided",
           lib().w8a16_gemv_batch16_strided(_ptr(A), _ptr(W), _ptr(S), _ptr(C), M, N, K, a_row_stride,
                                            c_row_stride, _stream(stream)))


# ---------------------------------------------------- microscaled operators
_MX_FORMATS = {"mxfp4": MXFP4, "mxfp8": MXFP8, MXFP4: MXFP4, MXFP8: MXFP8}
_types: dict = {}  # torch's types of values: WQD_TYPE_*
# torch's types that a kind of operand may have: its own, and integers of its size for plain bits (_here fills them)
_VALUES, _BF16, _SCALES = set(), set(), set()
_CODES: dict = {MXFP4: set(), MXFP8: set()}
_BYTES, _I4_SCALES, _INT32, _FP32 = set(), set(), set(), set()


def _sizes(fn: str, bits: int, K: int) -> None:
    """`bits`: the sizes and pitches of a call or-ed together; each must fit the C ABI's 32 bits.
    A K that is not whole blocks is refused here, with the library's status, as a tensor's rows
    cannot be held against it."""
    if bits >> 32:
        raise ValueError(f"{fn}: sizes and strides must be from 0 to 2^32 - 1")
    if K % 32 or not K:
        raise WqdError(fn, WQD_EINVAL, f"{fn}: K={K} is not a positive multiple of 32")


def _span(rows: int, pitch: int, width: int, size: int) -> int:
    """Bytes from the first row's start to the last row's end."""
    return ((rows - 1) * pitch + width) * size if rows > 0 else 0


def _rows_apart(x, pitch: int) -> bool:
    """Whether the rows of x, all its leading dimensions counted through, are `pitch` elements apart."""
    for n, step in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
        if n > 1 and step != pitch:
            return False
        pitch *= n
    return True


def _check_rows(fn: str, name: str, x, nbytes: int, pitch: int) -> None:
    """_arg's checks of a tensor that is not contiguous and just as large as the call reaches."""
    if x.dim() and x.stride(-1) != 1 and x.shape[-1] > 1:
        raise ValueError(f"{fn}: {name}'s last dimension must be contiguous")
    apart = f"{fn}: {name}'s rows are not {pitch} elements apart"
    whole = x.is_contiguous()
    if not whole and not _rows_apart(x, pitch):
        raise ValueError(apart)
    if x.untyped_storage().nbytes() - x.storage_offset() * x.element_size() < nbytes:
        raise ValueError(f"{fn}: {name} holds fewer than the {nbytes} bytes the call reaches")
    if whole and x.dim() > 1 and 0 < pitch < nbytes // x.element_size():  # more than one row
        if x.numel() != x.shape[-1] and pitch % x.shape[-1]:
            raise ValueError(apart)


def _arg(fn: str, name: str, x, nbytes: int, device: int, kind: set, pitch: int = 0) -> int | None:
    """Device address of an operand.  A tensor must live on `device`, the current
    one (the call goes to its stream), be of one of the types of its `kind` and its
    last dimension contiguous, and its memory must reach `nbytes` past its first
    element.  Rows lie `pitch` elements apart: those of a view with gaps, and those
    of a contiguous tensor that is not just as large as the call reaches, where its
    last dimension is a row or divides one (flat memory and a single row are any
    shape).  An integer is taken as it is."""
    if x is None or isinstance(x, int):
        return x
    if x.get_device() != device:
        raise ValueError(f"{fn}: {name} is not on the current GPU")
    if x.dtype not in kind:
        size = max(t.itemsize for t in kind)
        raise ValueError(f"{fn}: {name} must have {size}-byte elements of type "
                         f"{', '.join(sorted(str(t)[6:] for t in kind))}, not {str(x.dtype)[6:]}")
    n = x.nbytes
    if not (x.is_contiguous() and (n == nbytes or (n > nbytes and x.dim() and x.shape[-1] == pitch))):
        _check_rows(fn, name, x, nbytes, pitch)  # perhaps rows of a wider buffer
    return x.data_ptr()


_no_gpu = -2  # no tensor's device
_raw_device = _raw_stream = None


def _here(fn: str, stream) -> tuple[int, int | None]:
    """Index of torch's current GPU and the stream of a call: `stream`, which must
    be that GPU's (an integer, or an object that names no GPU, is taken as it is),
    or its current one."""
    global _raw_device, _raw_stream
    if _raw_device is None:
        import torch
        _types.update({torch.bfloat16: TYPE_BF16, torch.float16: TYPE_FP16, torch.float32: TYPE_FP32})
        _VALUES.update(_types)  # mx_quantize and mx_dequantize tell the library which
        _BF16.update((torch.bfloat16, torch.int16, torch.uint16))
        _SCALES.update((torch.float8_e8m0fnu, torch.uint8, torch.int8))
        _CODES[MXFP8].update((torch.float8_e4m3fn, torch.uint8, torch.int8))
        _CODES[MXFP4].update((torch.float4_e2m1fn_x2, torch.uint8, torch.int8))
        _BYTES.update((torch.uint8, torch.int8))
        _I4_SCALES.update((torch.float16, torch.bfloat16))
        _INT32.add(torch.int32)
        _FP32.add(torch.float32)
        gpu = torch.cuda.is_available()
        if gpu:
            torch.cuda.init()
        _raw_device = torch._C._cuda_getDevice if gpu else lambda: _no_gpu
        _raw_stream = torch._C._cuda_getCurrentRawStream if gpu else lambda device: None
    device = _raw_device()
    if stream is None:
        return device, _raw_stream(device)
    if not isinstance(stream, int):
        gpu = getattr(getattr(stream, "device", None), "index", None)
        if gpu not in (None, device):
            raise ValueError(f"{fn}: the stream is not the current GPU's")
    return device, _stream(stream)


def _type_of(fn: str, x, given: int | None) -> int:
    """WQD_TYPE_* of a tensor's values (an address comes with its type)."""
    if isinstance(x, int) or x is None:
        return TYPE_BF16 if given is None else given
    t = _types.get(x.dtype)
    if t is None or given not in (None, t):
        raise ValueError(f"{fn}: values must be BF16, FP16 or FP32, as their tensor is ({x.dtype})")
    return t


def _mx_format(fn: str, fmt) -> int:
    try:
        return _MX_FORMATS[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"{fn}: format {fmt!r} is neither 'mxfp4' nor 'mxfp8'") from None


def _code_bytes(fmt: int, n: int) -> int:
    return n // 2 if fmt == MXFP4 else n


def mx_quantize(X, Q, S, fmt, M: int, K: int, x_row_stride: int | None = None, x_type: int | None = None,
                stream=None) -> None:
    """Rows of X to `fmt` ("mxfp4" or "mxfp8") codes Q and scale bytes S.  The
    type is the tensor's; with an address pass `x_type` (default BF16)."""
    fn, ld = "mx_quantize", K if x_row_stride is None else x_row_stride
    _sizes(fn, M | K | ld, K)
    d, st = _here(fn, stream)
    f, t = _mx_format(fn, fmt), _type_of(fn, X, x_type)
    w = 4 if t == TYPE_FP32 else 2
    _check(fn, (_lib or lib()).mx_quantize(_arg(fn, "X", X, _span(M, ld, K, w), d, _VALUES, ld), t,
                                           _arg(fn, "Q", Q, _code_bytes(f, M * K), d, _CODES[f], _code_bytes(f, K)),
                                           _arg(fn, "S", S, M * K // 32, d, _SCALES, K // 32), f, M, K, ld, st))


def mx_dequantize(Q, S, Y, fmt, M: int, K: int, y_row_stride: int | None = None, y_type: int | None = None,
                  stream=None) -> None:
    """The values of `fmt` rows, in Y's type."""
    fn, ld = "mx_dequantize", K if y_row_stride is None else y_row_stride
    _sizes(fn, M | K | ld, K)
    d, st = _here(fn, stream)
    f, t = _mx_format(fn, fmt), _type_of(fn, Y, y_type)
    w = 4 if t == TYPE_FP32 else 2
    _check(fn, (_lib or lib()).mx_dequantize(_arg(fn, "Q", Q, _code_bytes(f, M * K), d, _CODES[f], _code_bytes(f, K)),
                                             _arg(fn, "S", S, M * K // 32, d, _SCALES, K // 32), f,
                                             _arg(fn, "Y", Y, _span(M, ld, K, w), d, _VALUES, ld), t,
                                             M, K, ld, st))


def add_rmsnorm_mx8(X, R, G, H, Y, Q, S, M: int, K: int, eps: float, x_row_stride: int | None = None,
                    r_row_stride: int | None = None, stream=None) -> None:
    """h = X + R (R and H may be None), its root-mean-square norm times G in
    MXFP8 (Q, S) and, unless Y is None, in BF16."""
    fn = "add_rmsnorm_mx8"
    lx, lr = K if x_row_stride is None else x_row_stride, K if r_row_stride is None else r_row_stride
    _sizes(fn, M | K | lx | lr, K)
    rows = _span(M, lr, K, 2)
    d, st = _here(fn, stream)
    _check(fn, (_lib or lib()).add_rmsnorm_mx8(_arg(fn, "X", X, _span(M, lx, K, 2), d, _BF16, lx),
                                               _arg(fn, "R", R, rows, d, _BF16, lr),
                                               _arg(fn, "G", G, 2 * K, d, _BF16), _arg(fn, "H", H, rows, d, _BF16, lr),
                                               _arg(fn, "Y", Y, 2 * M * K, d, _BF16, K),
                                               _arg(fn, "Q", Q, M * K, d, _CODES[MXFP8], K),
                                               _arg(fn, "S", S, M * K // 32, d, _SCALES, K // 32), M, K, lx, lr, eps, st))


def _gemm(call, fn: str, fmt: int | None, A, AS, W, WS, C, M, N, K, lda, ldc, stream) -> None:
    """A product with MXFP4 weights; fmt is that of the activations, None for BF16 rows of pitch lda."""
    ldc = N if ldc is None else ldc
    lda = K if lda is None else lda
    _sizes(fn, M | N | K | lda | ldc, K)
    d, st = _here(fn, stream)
    a = (_arg(fn, "A", A, _span(M, lda, K, 2), d, _BF16, lda) if fmt is None else
         _arg(fn, "A", A, _code_bytes(fmt, M * K), d, _CODES[fmt], _code_bytes(fmt, K)))
    w, ws = _arg(fn, "W", W, N * K // 2, d, _CODES[MXFP4], K // 2), _arg(fn, "WS", WS, N * K // 32, d, _SCALES, K // 32)
    c = _arg(fn, "C", C, _span(M, ldc, N, 2), d, _BF16, ldc)
    if fmt is None:
        rc = call(a, w, ws, c, M, N, K, lda, ldc, st)
    else:
        rc = call(a, _arg(fn, "AS", AS, M * K // 32, d, _SCALES, K // 32), w, ws, c, M, N, K, ldc, st)
    _check(fn, rc)


def _gated(call, fn: str, fmt: int | None, A, AS, WG, WGS, WU, WUS, C, M, N, K, lda, ldc, stream) -> None:
    """The same for the pair of products of a gated block."""
    ldc = N if ldc is None else ldc
    lda = K if lda is None else lda
    _sizes(fn, M | N | K | lda | ldc, K)
    d, st = _here(fn, stream)
    a = (_arg(fn, "A", A, _span(M, lda, K, 2), d, _BF16, lda) if fmt is None else
         _arg(fn, "A", A, _code_bytes(fmt, M * K), d, _CODES[fmt], _code_bytes(fmt, K)))
    w = (_arg(fn, "WG", WG, N * K // 2, d, _CODES[MXFP4], K // 2), _arg(fn, "WGS", WGS, N * K // 32, d, _SCALES, K // 32),
         _arg(fn, "WU", WU, N * K // 2, d, _CODES[MXFP4], K // 2), _arg(fn, "WUS", WUS, N * K // 32, d, _SCALES, K // 32))
    c = _arg(fn, "C", C, _span(M, ldc, N, 2), d, _BF16, ldc)
    if fmt is None:
        rc = call(a, *w, c, M, N, K, lda, ldc, st)
    else:
        rc = call(a, _arg(fn, "AS", AS, M * K // 32, d, _SCALES, K // 32), *w, c, M, N, K, ldc, st)
    _check(fn, rc)


def w4a16_gemm(A, W, WS, C, M: int, N: int, K: int, a_row_stride: int | None = None,
               c_row_stride: int | None = None, stream=None) -> None:
    _gemm((_lib or lib()).w4a16_gemm, "w4a16_gemm", None, A, None, W, WS, C, M, N, K, a_row_stride, c_row_stride, stream)


def w4a8_gemm(A, AS, W, WS, C, M: int, N: int, K: int, c_row_stride: int | None = None, stream=None) -> None:
    _gemm((_lib or lib()).w4a8_gemm, "w4a8_gemm", MXFP8, A, AS, W, WS, C, M, N, K, None, c_row_stride, stream)


def w4a4_gemm(A, AS, W, WS, C, M: int, N: int, K: int, c_row_stride: int | None = None, stream=None) -> None:
    _gemm((_lib or lib()).w4a4_gemm, "w4a4_gemm", MXFP4, A, AS, W, WS, C, M, N, K, None, c_row_stride, stream)


def w4a16_gated(A, WG, WGS, WU, WUS, C, M: int, N: int, K: int, a_row_stride: int | None = None,
                c_row_stride: int | None = None, stream=None) -> None:
    _gated((_lib or lib()).w4a16_gated, "w4a16_gated", None, A, None, WG, WGS, WU, WUS, C, M, N, K, a_row_stride,
           c_row_stride, stream)


def w4a8_gated(A, AS, WG, WGS, WU, WUS, C, M: int, N: int, K: int, c_row_stride: int | None = None,
               stream=None) -> None:
    _gated((_lib or lib()).w4a8_gated, "w4a8_gated", MXFP8, A, AS, WG, WGS, WU, WUS, C, M, N, K, None, c_row_stride, stream)


def w4a4_gated(A, AS, WG, WGS, WU, WUS, C, M: int, N: int, K: int, c_row_stride: int | None = None,
               stream=None) -> None:
    _gated((_lib or lib()).w4a4_gated, "w4a4_gated", MXFP4, A, AS, WG, WGS, WU, WUS, C, M, N, K, None, c_row_stride, stream)


# ------------------------- 4-bit integer weights, routed experts
_SCORING = {"softmax": MOE_SOFTMAX, "sigmoid": MOE_SIGMOID, MOE_SOFTMAX: MOE_SOFTMAX, MOE_SIGMOID: MOE_SIGMOID}


def _i4_sizes(fn: str, bits: int, K: int, group: int) -> None:
    """As _sizes, for K in whole tiles of 128 and a group that divides them."""
    if bits < 0 or bits >> 32:
        raise ValueError(f"{fn}: sizes and strides must be from 0 to 2^32 - 1")
    if K % 128 or not K:
        raise WqdError(fn, WQD_EINVAL, f"{fn}: K={K} is not a positive multiple of 128")
    if group not in (32, 64, 128):
        raise WqdError(fn, WQD_EINVAL, f"{fn}: group={group} is not 32, 64 or 128")


def _i4_by_row(shape, E: int, N: int, K: int, group: int) -> bool | None:
    """Whether scales or zero points of E matrices lie row by row and not in tiles.  Both are as many bytes where N is a multiple
    of 16, so the shape has to tell: [N, K / group] ([E, N, K / group], or with the first two as one) is row by row; flat
    memory, whole matrices that are flat and [..., K / 128, 16, 128 / group] are tiles.  None: neither."""
    n = len(shape)
    if n < 2:
        return False
    last, g = shape[-1], K // group
    if n > 2 and shape[-2] == 16 and last * group == 128 and shape[-3] * 128 == K:
        return False
    if last == g and (shape[-2] >= N if E == 1 else shape[-2] == (N if n > 2 else E * N)):
        return True
    return None if last % ((N + 15 & -16) * g or 1) else False


def _i4_scales(fn: str, given: int | None, E: int, N: int, K: int, group: int, *matrices) -> int:
    """scale_type of a call: `matrices` are the names, scales and zero points of each.  An address comes with its type, FP16
    and in tiles unless told (TYPE_*, plus I4_BY_ROW where it is row by row)."""
    t = by_row = seen = None
    if given is not None:
        t, by_row = given & ~I4_BY_ROW, True if given & I4_BY_ROW else None
    for name, s, z in matrices:
        if not (s is None or isinstance(s, int)):
            own = _types.get(s.dtype)
            if own != t:
                if t is not None or own not in (TYPE_FP16, TYPE_BF16):
                    raise ValueError(f"{fn}: scales must all be FP16 or all BF16, as their tensors are ({str(s.dtype)[6:]})")
                t = own
        for x in (s, z):
            if x is None or isinstance(x, int):
                continue
            shape = x.shape
            if shape == seen:
                continue
            seen, rows = shape, _i4_by_row(shape, E, N, K, group)
            if rows is None:
                raise ValueError(f"{fn}: {name}{'S' if x is s else 'Z'} of shape {list(shape)} is neither row by row, "
                                 f"{[E, N, K // group]}, nor in tiles as i4_pack writes them, flat or [..., {K // 128}, 16, {128 // group}]")
            if rows is not by_row:
                if by_row is not None:
                    raise ValueError(f"{fn}: scales and zero points must all lie row by row or all in tiles, and not "
                                     f"{name}{'S' if x is s else 'Z'} alone")
                by_row = rows
    return (TYPE_FP16 if t is None else t) | (I4_BY_ROW if by_row else 0)


def _i4_matrix(fn: str, name: str, W, S, Z, E: int, N: int, K: int, group: int, d: int, by_row: int = 0) -> tuple:
    """Addresses of E matrices' laid-out codes, scales and zero points."""
    n = E * (N + 15 & -16) * K
    m, g = (E * N * K // group, K // group) if by_row else (n // group, 0)
    return (_arg(fn, name, W, n // 2, d, _BYTES), _arg(fn, name + "S", S, m * 2, d, _I4_SCALES, g),
            None if Z is None else _arg(fn, name + "Z", Z, m, d, _BYTES, g))


def i4_packed_rows(N: int) -> int:
    """Rows of a laid-out matrix: N rounded up to a multiple of 16."""
    return int(lib().i4_packed_rows(N))


def i4_pack(Q, S, Z, W, WS, WZ, N: int, K: int, group: int, count: int = 1, stream=None) -> None:
    """`count` matrices to the layout that the products read: codes Q, two a byte with
    the even k in the low nibble, scales S and zero points Z (or None, and WZ too; S, Z, WS
    and WZ None lays out the codes alone, and scales and zero points stay row by row).  WS
    and WZ are tiles, and their shape says so: flat, or [..., K / 128, 16, 128 / group]."""
    fn = "i4_pack"
    _i4_sizes(fn, N | K | count, K, group)
    d, st = _here(fn, stream)
    n, g = count * N * K, K // group
    if not isinstance(S, int) and not isinstance(WS, int) and S is not None and WS is not None and S.dtype != WS.dtype:
        raise ValueError(f"{fn}: S and WS must have the same type")
    for name, x in ("WS", WS), ("WZ", WZ):
        if x is not None and not isinstance(x, int) and _i4_by_row(x.shape, count, N, K, group) is not False:
            raise ValueError(f"{fn}: {name} of shape {list(x.shape)} is not in tiles: make it flat")
    _check(fn, (_lib or lib()).i4_pack(_arg(fn, "Q", Q, n // 2, d, _BYTES, K // 2), _arg(fn, "S", S, n // group * 2, d, _I4_SCALES, g),
                                       _arg(fn, "Z", Z, n // group, d, _BYTES, g),
                                       *_i4_matrix(fn, "W", W, WS, WZ, count, N, K, group, d), N, K, group, count, st))


def i4a16_gemm(A, W, WS, WZ, C, M: int, N: int, K: int, group: int, a_row_stride: int | None = None,
               c_row_stride: int | None = None, scale_type: int | None = None, stream=None) -> None:
    """C = A W^T, W in laid-out codes W, scales WS and zero points WZ (None: 8).  Scales and
    zero points lie in tiles, as i4_pack writes them, or row by row, [N, K / group]: their
    tensors' shape tells (_i4_by_row); with addresses pass `scale_type`, for rows plus I4_BY_ROW."""
    fn = "i4a16_gemm"
    lda, ldc = K if a_row_stride is None else a_row_stride, N if c_row_stride is None else c_row_stride
    _i4_sizes(fn, M | N | K | lda | ldc, K, group)
    d, st = _here(fn, stream)
    t = _i4_scales(fn, scale_type, 1, N, K, group, ("W", WS, WZ))
    _check(fn, (_lib or lib()).i4a16_gemm(_arg(fn, "A", A, _span(M, lda, K, 2), d, _BF16, lda),
                                          *_i4_matrix(fn, "W", W, WS, WZ, 1, N, K, group, d, t & I4_BY_ROW),
                                          _arg(fn, "C", C, _span(M, ldc, N, 2), d, _BF16, ldc), M, N, K, group, t, lda, ldc, st))


def i4a16_gated(A, WG, WGS, WGZ, WU, WUS, WUZ, C, M: int, N: int, K: int, group: int, a_row_stride: int | None = None,
                c_row_stride: int | None = None, scale_type: int | None = None, stream=None) -> None:
    """C = silu(A WG^T) * (A WU^T); scales and zero points as for i4a16_gemm."""
    fn = "i4a16_gated"
    lda, ldc = K if a_row_stride is None else a_row_stride, N if c_row_stride is None else c_row_stride
    _i4_sizes(fn, M | N | K | lda | ldc, K, group)
    d, st = _here(fn, stream)
    t = _i4_scales(fn, scale_type, 1, N, K, group, ("WG", WGS, WGZ), ("WU", WUS, WUZ))
    _check(fn, (_lib or lib()).i4a16_gated(_arg(fn, "A", A, _span(M, lda, K, 2), d, _BF16, lda),
                                           *_i4_matrix(fn, "WG", WG, WGS, WGZ, 1, N, K, group, d, t & I4_BY_ROW),
                                           *_i4_matrix(fn, "WU", WU, WUS, WUZ, 1, N, K, group, d, t & I4_BY_ROW),
                                           _arg(fn, "C", C, _span(M, ldc, N, 2), d, _BF16, ldc), M, N, K, group, t, lda, ldc, st))


def moe_route(logits, bias, ids, weights, T: int, E: int, top_k: int, scoring="softmax", groups: int = 1,
              top_groups: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
              row_stride: int | None = None, logits_type: int | None = None, stream=None) -> None:
    """Each token's experts and their weights from its logits; `scoring` is "softmax"
    or "sigmoid", bias [E] or None.  The type of the logits is the tensor's; with
    an address pass `logits_type` (default BF16)."""
    fn, ld = "moe_route", E if row_stride is None else row_stride
    _moe_sizes(fn, T, E, top_k, ld, groups, top_groups, group_top)
    if not isinstance(scoring, (str, int)) or scoring not in _SCORING:
        raise ValueError(f"{fn}: scoring {scoring!r} is neither 'softmax' nor 'sigmoid'")
    d, st = _here(fn, stream)
    t = _type_of(fn, logits, logits_type)
    _check(fn, (_lib or lib()).moe_route(_arg(fn, "logits", logits, _span(T, ld, E, 4 if t == TYPE_FP32 else 2), d, _VALUES, ld), t,
                                         _arg(fn, "bias", bias, 4 * E, d, _FP32), _arg(fn, "ids", ids, 4 * T * top_k, d, _INT32, top_k),
                                         _arg(fn, "weights", weights, 4 * T * top_k, d, _FP32, top_k), T, E, top_k, ld,
                                         _SCORING[scoring], groups, top_groups, group_top, bool(renormalize), scale, st))


def _moe_sizes(fn: str, *sizes: int) -> None:
    for n in sizes:
        if n >> 32:
            raise ValueError(f"{fn}: sizes and strides must be from 0 to 2^32 - 1")


def moe_lists(ids, order, offsets, T: int, top_k: int, E: int, stream=None) -> None:
    """Each expert's pairs (token * top_k + slot), expert by expert."""
    fn = "moe_lists"
    _moe_sizes(fn, T, top_k, E)
    d, st = _here(fn, stream)
    _check(fn, (_lib or lib()).moe_lists(_arg(fn, "ids", ids, 4 * T * top_k, d, _INT32, top_k),
                                         _arg(fn, "order", order, 4 * T * top_k, d, _INT32),
                                         _arg(fn, "offsets", offsets, 4 * (E + 1), d, _INT32), T, top_k, E, st))


def i4a16_experts_gated(A, ids, order, offsets, WG, WGS, WGZ, WU, WUS, WUZ, H, T: int, top_k: int, E: int, N: int, K: int,
                        group: int, a_row_stride: int | None = None, scale_type: int | None = None, stream=None) -> None:
    """A row of H per pair: the gated product of the token's row with its expert's
    matrices.  order and offsets are moe_lists', or both None for a few tokens."""
    fn, lda = "i4a16_experts_gated", K if a_row_stride is None else a_row_stride
    _i4_sizes(fn, T | top_k | E | N | K | lda, K, group)
    d, st = _here(fn, stream)
    t = _i4_scales(fn, scale_type, E, N, K, group, ("WG", WGS, WGZ), ("WU", WUS, WUZ))
    pairs = T * top_k
    _check(fn, (_lib or lib()).i4a16_experts_gated(
        _arg(fn, "A", A, _span(T, lda, K, 2), d, _BF16, lda), _arg(fn, "ids", ids, 4 * pairs, d, _INT32, top_k),
        _arg(fn, "order", order, 4 * pairs, d, _INT32), _arg(fn, "offsets", offsets, 4 * (E + 1), d, _INT32),
        *_i4_matrix(fn, "WG", WG, WGS, WGZ, E, N, K, group, d, t & I4_BY_ROW),
        *_i4_matrix(fn, "WU", WU, WUS, WUZ, E, N, K, group, d, t & I4_BY_ROW),
        _arg(fn, "H", H, 2 * pairs * N, d, _BF16, N), T, top_k, E, N, K, group, t, lda, st))


def i4a16_experts_down(H, ids, weights, order, offsets, W, WS, WZ, Y, C, T: int, top_k: int, E: int, N: int, K: int,
                       group: int, c_row_stride: int | None = None, scale_type: int | None = None, stream=None) -> None:
    """The weighted sum over each token's experts of its pairs' rows of H times their
    matrices.  With lists Y is scratch, fp32 [T * top_k][N]; without it may be None."""
    fn, ldc = "i4a16_experts_down", N if c_row_stride is None else c_row_stride
    _i4_sizes(fn, T | top_k | E | N | K | ldc, K, group)
    d, st = _here(fn, stream)
    t = _i4_scales(fn, scale_type, E, N, K, group, ("W", WS, WZ))
    pairs = T * top_k
    _check(fn, (_lib or lib()).i4a16_experts_down(
        _arg(fn, "H", H, 2 * pairs * K, d, _BF16, K), _arg(fn, "ids", ids, 4 * pairs, d, _INT32, top_k),
        _arg(fn, "weights", weights, 4 * pairs, d, _FP32, top_k), _arg(fn, "order", order, 4 * pairs, d, _INT32),
        _arg(fn, "offsets", offsets, 4 * (E + 1), d, _INT32), *_i4_matrix(fn, "W", W, WS, WZ, E, N, K, group, d, t & I4_BY_ROW),
        _arg(fn, "Y", Y, 4 * pairs * N, d, _FP32, N), _arg(fn, "C", C, _span(T, ldc, N, 2), d, _BF16, ldc),
        T, top_k, E, N, K, group, t, ldc, st))


# ------------------------------------------------------------ host helpers
def q2_0_packed_bytes(N: int, K: int) -> int:
    return int(lib().q2_0_packed_bytes(N, K))


def q2_0_pack(codes: np.ndarray, d_f16: np.ndarray) -> np.ndarray:
    """Pack codes u8 [N,K] and fp16 scale bits [N,K/128] into block_q2_0 bytes."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    d = np.ascontiguousarray(d_f16, dtype=np.uint16)
    N, K = codes.shape
    if d.shape != (N, K // 128):
        raise ValueError(f"d_f16 shape {d.shape} != {(N, K // 128)}")
    out = np.empty(max(q2_0_packed_bytes(N, K), 1), np.uint8)
    rc = lib().q2_0_pack(codes.ctypes.data, d.ctypes.data, N, K, out.ctypes.data)
    if rc != WQD_OK:
        raise WqdError("q2_0_pack", rc, "codes must be 0..2 and K a positive multiple of 128")
    return out[:q2_0_packed_bytes(N, K)]


def q2_0_batchm_chunks(M: int, K: int, N: int) -> list[tuple[int, int, int]]:
    L = lib()
    count = int(L.q2_0_batchm_chunks(M, K, N, None, 0))
    buf = (ctypes.c_uint64 * max(3 * count, 1))()
    L.q2_0_batchm_chunks(M, K, N, buf, count)
    return [(int(buf[3 * i]), int(buf[3 * i + 1]), int(buf[3 * i + 2])) for i in range(count)]


def q2_0_select_tier(m: int, present_mask: int, exact_m: bool) -> int | None:
    """Index into Q2_0_TIER_WIDTHS of the tier that serves m rows, or None."""
    i = int(lib().q2_0_select_tier(m, present_mask, 1 if exact_m else 0))
    return None if i < 0 else i


def q2_0_tier_width(m: int) -> int:
    """Row width the Q2_0 matrix-core kernel runs m rows on in this process (0: none)."""
    return int(lib().q2_0_tier_width(m))


def q2_0_exact_m_tiers_enabled() -> bool:
    return bool(lib().q2_0_exact_m_tiers_enabled())
