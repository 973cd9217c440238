"""Thin Python binding of libmxq (ctypes).

Argument marshalling only: every function here allocates its outputs with torch
on the input's device, passes raw device pointers and torch's current HIP stream
to the C ABI in include/mxq.h, and raises MxqError on a non-zero status. No
step of the quantize / GEMM path runs in Python, and there is no fallback: if
libmxq.so is missing the first call raises. MXQ_LIBRARY, when set, names another
build of the same library to load instead (the host-sanitizer build that the ABI
tests run under).
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MXQ_LIBRARY") or os.path.join(_HERE, "libmxq.so")

MXFP8, NVFP4, BF16, MXFP4 = 1, 2, 3, 4
BF16_NVFP4T = 5                    # grouped only: BF16 A x stacked NVFP4 weights (K, N) read transposed
_PACKED4 = (NVFP4, MXFP4)          # formats with two elements per byte
OUT_BF16, OUT_F32 = 0, 1
SCOPE = {"row": 0, "token": 0, "tensor": 1, "group": 2}
OP_QUANTIZE_NVFP4, OP_GROUPED_GEMM, OP_NORM_BACKWARD, OP_ROUTE, OP_DECODE_DOWN, OP_GEMM_SWIGLU = 1, 2, 3, 4, 5, 6
OP_GROUPED_SWIGLU = 7
GATE = {"none": 0, "token": 1, "channel": 2, "full": 3}

_c_void_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_size = ctypes.c_size_t
_f32 = ctypes.c_float
_f64 = ctypes.c_double

_SIGS = {
    "quantize_mxfp8": [_c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "quantize_mxfp8_multi": [_c_void_p, _int, _c_void_p],
    "quantize_mxfp4": [_c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "quantize_mxfp4_multi": [_c_void_p, _int, _c_void_p],
    "quantize_fp8_block_act": [_c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "quantize_fp8_block_weight": [_c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "gemm_block_scaled_batch": [_int, _c_void_p, _int, _c_void_p],
    "gemm_fp8_blockwise": [_i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _i64,
                           _c_void_p],
    "gemm_fp8_blockwise_batch": [_c_void_p, _int, _c_void_p],
    "quantize_nvfp4_per_token": [_c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "quantize_nvfp4": [_c_void_p, _i64, _i64, _i64, _int, _i64, _int, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                       _c_void_p, _size, _c_void_p],
    "quantize_nvfp4_stochastic": [_c_void_p, _i64, _i64, _i64, _int, _i64, _int, _c_void_p, ctypes.c_uint64,
                                  _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p],
    "quantize_nvfp4_2d": [_c_void_p, _i64, _i64, _i64, _int, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                          _c_void_p, _c_void_p, _size, _c_void_p],
    "dequantize": [_int, _c_void_p, _c_void_p, _c_void_p, _int, _i64, _i64, _i64, _c_void_p, _int, _c_void_p],
    "dequantize_transposed": [_int, _c_void_p, _c_void_p, _c_void_p, _int, _i64, _i64, _i64, _c_void_p, _i64,
                              _c_void_p, _i64, _c_void_p],
    "gemm_block_scaled": [_int, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p,
                          _c_void_p, _int, _c_void_p, _i64, _c_void_p],
    "gemm_mxfp8_matrix_core": [_i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64,
                               _c_void_p],
    "grouped_gemm_block_scaled": [_int, _i64, _c_void_p, _int, _i64, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p,
                                  _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p,
                                  _c_void_p, _size, _c_void_p],
    "grouped_gemm_block_scaled_noalloc": [_int, _i64, _c_void_p, _int, _i64, _i64, _i64, _i64, _c_void_p, _i64,
                                          _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p,
                                          _int, _c_void_p, _c_void_p],
    "moe_swiglu_quantize_nvfp4": [_c_void_p, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "moe_combine": [_c_void_p, _i64, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p],
    "rmsnorm_quantize": [_int, _c_void_p, _int, _i64, _i64, _i64, _c_void_p, _f64, _c_void_p, _c_void_p, _c_void_p,
                         _c_void_p, _c_void_p, _c_void_p],
    "rmsnorm_backward": [_c_void_p, _c_void_p, _int, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p, _f32, _i64, _i64,
                         _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p],
    "rmsnorm_gate_residual": [_c_void_p, _int, _c_void_p, _int, _c_void_p, _c_void_p, _int, _f64, _f32, _f32, _i64, _i64,
                              _c_void_p, _c_void_p, _c_void_p],
    "rmsnorm_gate_residual_backward": [_c_void_p, _int, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p, _int, _f32,
                                       _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p],
    "moe_route": [_c_void_p, _c_void_p, _i64, _i64, _i64, _i64, _i64, _i64, _f32, _c_void_p, _c_void_p, _c_void_p,
                  _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p],
    "moe_route_backward": [_c_void_p, _i64, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                           _f32, _c_void_p, _int, _c_void_p],
    "moe_combine_backward": [_c_void_p, _int, _c_void_p, _i64, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p,
                             _c_void_p, _c_void_p, _c_void_p],
    "gemm_swiglu": [_int, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p, _int,
                    _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p],
    "gemm_swiglu_backward": [_int, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _int,
                             _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p],
    "grouped_gemm_swiglu": [_int, _i64, _c_void_p, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p,
                            _int, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p, _size,
                            _c_void_p],
    "grouped_gemm_swiglu_backward": [_int, _i64, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                     _c_void_p, _int, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p],
    "gemv_block_scaled": [_int, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _int,
                          _i64, _c_void_p],
    "gemv_swiglu": [_int, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _int, _c_void_p, _i64,
                    _c_void_p],
    "moe_decode_gate_up": [_int, _i64, _i64, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p,
                           _c_void_p, _int, _c_void_p, _c_void_p],
    "moe_decode_down": [_int, _i64, _i64, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                        _c_void_p, _int, _c_void_p, _int, _c_void_p, _size, _c_void_p],
    "mxq_route_slots": [_i64, _i64, _i64, _i64],
    "mxq_scale_bytes": [_int, _i64, _i64],
    "mxq_workspace_bytes": [_int, _i64, _i64, _i64],
    "mxq_status_string": [_int],
    "mxq_abi_version": [],
}
_RESTYPES = {"mxq_scale_bytes": _size, "mxq_workspace_bytes": _size, "mxq_route_slots": _i64,
             "mxq_status_string": ctypes.c_char_p}

_lib = None


class MxqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed with status {status}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """Load libmxq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m microscaling_precision_quantization_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = _RESTYPES.get(name, _int)
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().mxq_status_string(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise MxqError(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    """The raw handle of dev's current stream (20 times cheaper than building a Stream object); dev
    as torch names devices: a torch.device, a string or an index."""
    if type(dev) is not torch.device:
        dev = torch.device(dev)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev.index is None else dev.index)


def _call(fn: str, dev, *args):
    """One C-ABI call on dev's current stream (the last argument), with dev the current device:
    a kernel is launched on the device that is current, whatever its stream. dev: a tensor's."""
    if dev.index == torch._C._cuda_getDevice():
        _check(fn, getattr(lib(), fn)(*args, _stream(dev)))
    else:
        with torch.cuda.device(dev):
            _check(fn, getattr(lib(), fn)(*args, _stream(dev)))


def _bf16(x):
    if x.dtype != torch.bfloat16:
        raise TypeError("expected a bfloat16 tensor")
    if not x.is_cuda:
        raise TypeError("expected a device tensor")
    return x


def _u8(shape, dev):
    return torch.empty(*shape, dtype=torch.uint8, device=dev)


class _Checks:
    """Host-side checks of the tensors handed to one C-ABI call: dtype, exact shape, unit
    inner stride and a dense layout (ld=True: rows may be padded, row stride >= the row
    length) for each tensor as it is named, then, in done(), that all of them live on the
    one GPU the call runs on. Every mismatch raises ValueError before anything reaches
    the library, so a wrong buffer can never be read or written past its end."""

    def __init__(self, dev):
        self.dev = dev
        self.index = dev.index
        self.seen = []

    def need(self, t, name: str, dtype, shape, ld: bool = False):
        # what nearly every call hands in, in one comparison each; anything else is looked at below
        if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == self.index and not (ld and t.stride(0) < shape[1])):
            return t
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")
        if t.dtype != dtype:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
        shape = tuple(int(v) for v in shape)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
        if t.numel():
            if t.dim() and t.stride(-1) != 1:
                raise ValueError(f"{name}: the innermost dimension must be contiguous")
            if ld:
                if t.dim() != 2 or t.stride(0) < t.shape[1]:
                    raise ValueError(f"{name}: expected a 2-D tensor with row stride >= {t.shape[1]}")
            elif not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous tensor")
        self.seen.append((name, t))
        return t

    def opt(self, t, *a, **kw):
        return None if t is None else self.need(t, *a, **kw)

    def operand(self, fmt: int, name: str, t, rows: int, K: int, s=None):
        """A K-contiguous GEMM operand of `rows` rows and K elements (+ its block scales)."""
        width = K if fmt == BF16 else K // _elems_per_byte(fmt)
        self.need(t, name, _operand_dtype(fmt), (rows, width))
        if fmt != BF16:
            if s is None:
                raise ValueError(f"s{name}: block scales are required for this format")
            self.need(s, "s" + name, torch.uint8, (rows, K // _scale_block(fmt)))

    def outer_scale(self, name: str, t, scope: str, rows: int):
        if t is None:
            raise ValueError(f"{name}: NVFP4 needs its FP32 scale")
        self.need(t, name, torch.float32, (rows if SCOPE[scope] == 0 else 1,))

    def done(self):
        for name, t in self.seen:
            if not t.is_cuda:
                raise ValueError(f"{name}: expected a GPU tensor, got one on {t.device}")
            if t.device != self.dev:
                raise ValueError(f"{name}: on {t.device}, expected {self.dev}")


def _elems_per_byte(fmt: int) -> int:
    return 2 if fmt in _PACKED4 else 1


def _operand_dtype(fmt: int):
    return torch.bfloat16 if fmt == BF16 else torch.uint8


def _scale_block(fmt: int) -> int:
    return 16 if fmt == NVFP4 else 32


# ---------------------------------------------------------------------------
# Quantizers
# ---------------------------------------------------------------------------

def quantize_mxfp8(x: torch.Tensor, rowwise: bool = True, colwise: bool = True, out=None):
    """MXFP8 rowwise (R, C) + columnwise-transposed (C, R) copies of BF16 x.

    Returns (q_row, s_row, q_colT, s_colT); skipped copies are None. `out` may
    supply preallocated (q_row, s_row, q_colT, s_colT) buffers.
    """
    _bf16(x)
    R, C = x.shape
    dev = x.device
    if out is not None:
        q_row, s_row, q_col, s_col = out
        _mx_check_out("quantize_mxfp8", x, out, 1)
    else:
        q_row = _u8((R, C), dev) if rowwise else None
        s_row = _u8((R, C // 32), dev) if rowwise else None
        q_col = _u8((C, R), dev) if colwise else None
        s_col = _u8((C, R // 32), dev) if colwise else None
    _call("quantize_mxfp8", dev, _ptr(x), R, C, x.stride(0), _ptr(q_row), _ptr(s_row), _ptr(q_col), _ptr(s_col))
    return q_row, s_row, q_col, s_col


def quantize_mxfp4(x: torch.Tensor, rowwise: bool = True, colwise: bool = True, out=None):
    """MXFP4 rowwise (R, C/2) + columnwise-transposed (C, R/2) packed copies of BF16 x.

    Returns (q_row, s_row, q_colT, s_colT); skipped copies are None.
    """
    _bf16(x)
    R, C = x.shape
    dev = x.device
    if out is not None:
        q_row, s_row, q_col, s_col = out
        _mx_check_out("quantize_mxfp4", x, out, 2)
    else:
        q_row = _u8((R, C // 2), dev) if rowwise else None
        s_row = _u8((R, C // 32), dev) if rowwise else None
        q_col = _u8((C, R // 2), dev) if colwise else None
        s_col = _u8((C, R // 32), dev) if colwise else None
    _call("quantize_mxfp4", dev, _ptr(x), R, C, x.stride(0), _ptr(q_row), _ptr(s_row), _ptr(q_col), _ptr(s_col))
    return q_row, s_row, q_col, s_col


def quantize_fp8_block_act(x: torch.Tensor, rowwise: bool = True, colwise: bool = False, out=None):
    """Blockwise FP8 of an activation / gradient: (q_row (R, C), s_row (R, C/128)) with 1 x 128
    tiles along rows and (q_colT (C, R), s_colT (C, R/128)) with tiles of 128 down columns,
    stored transposed; skipped copies are None."""
    _bf16(x)
    R, C = x.shape
    dev = x.device
    f32 = lambda *sh: torch.empty(sh, dtype=torch.float32, device=dev)
    if out is not None:
        q_row, s_row, q_col, s_col = out
    else:
        q_row, s_row = (_u8((R, C), dev), f32(R, C // 128)) if rowwise else (None, None)
        q_col, s_col = (_u8((C, R), dev), f32(C, R // 128)) if colwise else (None, None)
    _call("quantize_fp8_block_act", dev, _ptr(x), R, C, x.stride(0), _ptr(q_row), _ptr(s_row), _ptr(q_col), _ptr(s_col))
    return q_row, s_row, q_col, s_col


def quantize_fp8_block_weight(x: torch.Tensor, rowwise: bool = True, colwise: bool = True, out=None):
    """Blockwise FP8 of a weight (128 x 128 blocks): (q_row (R, C), s_row (R/128, C/128),
    q_colT (C, R), s_colT (C/128, R/128)); skipped copies are None."""
    _bf16(x)
    R, C = x.shape
    dev = x.device
    f32 = lambda *sh: torch.empty(sh, dtype=torch.float32, device=dev)
    if out is not None:
        q_row, s_row, q_col, s_col = out
    else:
        q_row = _u8((R, C), dev) if rowwise else None
        s_row = f32(R // 128, C // 128) if rowwise else None
        q_col = _u8((C, R), dev) if colwise else None
        s_col = f32(C // 128, R // 128) if colwise else None
    _call("quantize_fp8_block_weight", dev, _ptr(x), R, C, x.stride(0), _ptr(q_row), _ptr(s_row), _ptr(q_col),
          _ptr(s_col))
    return q_row, s_row, q_col, s_col


class _Mxfp8Tensor(ctypes.Structure):
    _fields_ = [("x", _c_void_p), ("rows", _i64), ("cols", _i64), ("ld_x", _i64), ("q_row", _c_void_p),
                ("s_row", _c_void_p), ("q_colT", _c_void_p), ("s_colT", _c_void_p)]


def _mx_check_out(fn: str, x, out, per_byte: int):
    """Output buffers of an MXFP8 / MXFP4 quantize: (R, C/per_byte) + (R, C/32) rowwise,
    (C, R/per_byte) + (C, R/32) columnwise; a skipped copy is (None, None)."""
    R, C = x.shape
    q_row, s_row, q_col, s_col = out
    if (q_row is None) != (s_row is None) or (q_col is None) != (s_col is None):
        raise ValueError(f"{fn}: a copy needs both its element and its scale buffer")
    c = _Checks(x.device)
    c.opt(q_row, "q_row", torch.uint8, (R, C // per_byte))
    c.opt(s_row, "s_row", torch.uint8, (R, C // 32))
    c.opt(q_col, "q_colT", torch.uint8, (C, R // per_byte))
    c.opt(s_col, "s_colT", torch.uint8, (C, R // 32))
    c.done()


def _mx_multi(fn: str, xs, outs):
    n = len(xs)
    if len(outs) != n:
        raise ValueError(f"{fn}: {n} inputs but {len(outs)} output tuples")
    arr = (_Mxfp8Tensor * n)()
    for i, (x, o) in enumerate(zip(xs, outs)):
        _mx_check_out(fn, x, o, 2 if fn.startswith("quantize_mxfp4") else 1)
        _bf16(x)
        q_row, s_row, q_col, s_col = o
        arr[i] = _Mxfp8Tensor(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0),
                              *(None if t is None else t.data_ptr() for t in (q_row, s_row, q_col, s_col)))
    _call(fn, xs[0].device, ctypes.cast(arr, _c_void_p), n)
    return outs


def quantize_mxfp8_multi(xs, outs):
    """quantize_mxfp8 of several BF16 tensors in one launch; outs[i] = (q_row, s_row,
    q_colT, s_colT) preallocated (a skipped copy is (None, None) in its slots)."""
    return _mx_multi("quantize_mxfp8_multi", xs, outs)


def quantize_mxfp4_multi(xs, outs):
    """quantize_mxfp4 of several BF16 tensors in one launch; outs as quantize_mxfp8_multi
    with packed (R, C/2) / (C, R/2) element buffers."""
    return _mx_multi("quantize_mxfp4_multi", xs, outs)


def quantize_nvfp4_per_token(x: torch.Tensor):
    """Per-token NVFP4 of BF16 x (T, H): (packed (T, H/2), E4M3 scales (T, H/16), t (T,))."""
    _bf16(x)
    T, H = x.shape
    dev = x.device
    q, s = _u8((T, H // 2), dev), _u8((T, H // 16), dev)
    t = torch.empty(T, dtype=torch.float32, device=dev)
    _call("quantize_nvfp4_per_token", dev, _ptr(x), T, H, x.stride(0), _ptr(q), _ptr(s), _ptr(t))
    return q, s, t


def quantize_nvfp4(x: torch.Tensor, scope: str = "tensor", group_rows: int = 0, transpose: bool = False,
                   rht_signs=None, workspace: torch.Tensor | None = None, sr_seed: int | None = None):
    """General NVFP4 quantizer (see include/mxq.h). rht_signs: 16 ints in {-1, +1} or None.
    sr_seed: None = round-to-nearest-even; an int = stochastic rounding of the elements
    (quantize_nvfp4_stochastic) with that seed."""
    _bf16(x)
    R, C = x.shape
    dev = x.device
    out_rows, out_cols = (C, R) if transpose else (R, C)
    sc = SCOPE[scope]
    n_scopes = out_rows if sc == 0 else 1 if sc == 1 else (out_rows // group_rows if group_rows else 0)
    q, s = _u8((out_rows, out_cols // 2), dev), _u8((out_rows, out_cols // 16), dev)
    t = torch.empty(max(n_scopes, 1), dtype=torch.float32, device=dev)
    signs = None
    if rht_signs is not None:
        signs = (ctypes.c_int8 * 16)(*[int(v) for v in rht_signs])
    ws_bytes = lib().mxq_workspace_bytes(OP_QUANTIZE_NVFP4, out_rows, out_cols, n_scopes) if sc != 0 else 0
    if workspace is None and ws_bytes:
        workspace = _u8((ws_bytes,), dev)
    wsn = workspace.numel() if workspace is not None else 0
    if sr_seed is None:
        _call("quantize_nvfp4", dev, _ptr(x), R, C, x.stride(0), sc, group_rows, int(transpose), signs, _ptr(q),
              _ptr(s), _ptr(t), _ptr(workspace), wsn)
    else:
        _call("quantize_nvfp4_stochastic", dev, _ptr(x), R, C, x.stride(0), sc, group_rows, int(transpose), signs,
              int(sr_seed), _ptr(q), _ptr(s), _ptr(t), _ptr(workspace), wsn)
    return q, s, t


def quantize_nvfp4_2d(x: torch.Tensor, scope: str = "tensor", group_rows: int = 0, rowwise: bool = True,
                      colwise: bool = True, out=None, workspace: torch.Tensor | None = None):
    """NVFP4 with 16x16 block scales: (q_row, s_row, q_colT, s_colT, t); skipped copies are None.
    The transposed copy is per scope group: (groups * cols, group_rows / 2)."""
    _bf16(x)
    R, C = x.shape
    dev = x.device
    n_scopes = 1 if scope == "tensor" else (R // group_rows if group_rows else 0)
    if out is not None:
        q_row, s_row, q_col, s_col, t = out
    else:
        q_row = _u8((R, C // 2), dev) if rowwise else None
        s_row = _u8((R, C // 16), dev) if rowwise else None
        gr = R if scope == "tensor" else group_rows
        q_col = _u8((max(n_scopes, 1) * C, gr // 2), dev) if colwise else None
        s_col = _u8((max(n_scopes, 1) * C, gr // 16), dev) if colwise else None
        t = torch.empty(max(n_scopes, 1), dtype=torch.float32, device=dev)
    ws_bytes = lib().mxq_workspace_bytes(OP_QUANTIZE_NVFP4, R, C, n_scopes)
    if workspace is None:
        workspace = _u8((max(ws_bytes, 4),), dev)
    _call("quantize_nvfp4_2d", dev, _ptr(x), R, C, x.stride(0), SCOPE[scope], group_rows, _ptr(q_row), _ptr(s_row),
          _ptr(q_col), _ptr(s_col), _ptr(t), _ptr(workspace), workspace.numel())
    return q_row, s_row, q_col, s_col, t


def dequantize(fmt: int, q: torch.Tensor, s: torch.Tensor, t: torch.Tensor | None = None, t_scope: str = "row",
               group_rows: int = 0, out_dtype: torch.dtype = torch.bfloat16):
    rows = q.shape[0]
    cols = q.shape[1] * (2 if fmt in _PACKED4 else 1)
    out = torch.empty((rows, cols), dtype=out_dtype, device=q.device)
    od = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    _call("dequantize", q.device, fmt, _ptr(q), _ptr(s), _ptr(t), SCOPE[t_scope], group_rows, rows, cols, _ptr(out), od)
    return out


def dequantize_transposed(fmt: int, q: torch.Tensor, s=None, t=None, t_scope: str = "row", groups: int = 1,
                          group_rows: int | None = None, cols: int | None = None, src_row=None,
                          out_cols: int | None = None, out=None):
    """BF16 (groups, cols, out_cols): out[g, c, j] = dequantized input (g * group_rows + src(j), c)."""
    rows = q.shape[0]
    if cols is None:
        cols = q.shape[1] * (2 if fmt == NVFP4 else 1)
    if group_rows is None:
        group_rows = rows // max(groups, 1)
    if out_cols is None:
        out_cols = src_row.numel() if src_row is not None else group_rows
    if out is None:
        out = torch.empty((groups, cols, out_cols), dtype=torch.bfloat16, device=q.device)
    elif (out.dtype != torch.bfloat16 or out.dim() != 3 or tuple(out.shape[:2]) != (groups, cols)
          or out.shape[2] < out_cols or out.stride(-1) != 1 or out.stride(0) != cols * out.stride(1)
          or out.device != q.device):
        raise ValueError(f"out: expected BF16 (groups={groups}, cols={cols}, >= {out_cols}) rows on {q.device}")
    _call("dequantize_transposed", q.device, fmt, _ptr(q), _ptr(s), _ptr(t), SCOPE[t_scope], groups, group_rows, cols,
          _ptr(src_row), out_cols, _ptr(out), out.stride(-2))
    return out


# ---------------------------------------------------------------------------
# GEMMs
# ---------------------------------------------------------------------------

def _gemm_args(fmt: int, A, sA, B, sB, tA, tB, tA_scope, tB_scope, out):
    """Validate one TN GEMM's operands and output; returns (M, N, K)."""
    if fmt not in (MXFP8, NVFP4, BF16, MXFP4):
        raise ValueError(f"unknown format {fmt}")
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D (rows, K-contiguous bytes or elements)")
    M, N = A.shape[0], B.shape[0]
    K = A.shape[1] * _elems_per_byte(fmt)
    c = _Checks(A.device)
    c.operand(fmt, "A", A, M, K, sA)
    c.operand(fmt, "B", B, N, K, sB)
    if fmt == NVFP4:
        c.outer_scale("tA", tA, tA_scope, M)
        c.outer_scale("tB", tB, tB_scope, N)
    if out is not None:
        c.need(out, "out", torch.float32, (M, N), ld=True)
    c.done()
    return M, N, K


def gemm_block_scaled(fmt: int, A, sA, B, sB, tA=None, tB=None, tA_scope="row", tB_scope="tensor", out=None):
    """C = A_hat B_hat^T in FP32; A (M, K-bytes) and B (N, K-bytes) K-contiguous."""
    M, N, K = _gemm_args(fmt, A, sA, B, sB, tA, tB, tA_scope, tB_scope, out)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _call("gemm_block_scaled", A.device, fmt, M, N, K, _ptr(A), _ptr(sA), _ptr(tA), SCOPE[tA_scope], _ptr(B),
          _ptr(sB), _ptr(tB), SCOPE[tB_scope], _ptr(out), out.stride(0))
    return out


class _GemmProblem(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("A", _c_void_p), ("sA", _c_void_p), ("tA", _c_void_p),
                ("tA_scope", _int), ("B", _c_void_p), ("sB", _c_void_p), ("tB", _c_void_p), ("tB_scope", _int),
                ("C", _c_void_p), ("ldc", _i64)]


def gemm_block_scaled_batch(fmt: int, problems):
    """Several gemm_block_scaled problems of one format in one launch. problems: list of
    dicts with A, sA, B, sB, out and optionally tA, tB, tA_scope, tB_scope."""
    n = len(problems)
    arr = (_GemmProblem * n)()
    dev = problems[0]["A"].device
    for i, q in enumerate(problems):
        A, B_, out = q["A"], q["B"], q["out"]
        if A.device != dev:
            raise ValueError(f"problem {i}: operands on {A.device}, the batch runs on {dev}")
        _, _, K = _gemm_args(fmt, A, q.get("sA"), B_, q.get("sB"), q.get("tA"), q.get("tB"),
                             q.get("tA_scope", "row"), q.get("tB_scope", "tensor"), out)
        ptr = lambda t: None if t is None else t.data_ptr()
        arr[i] = _GemmProblem(A.shape[0], B_.shape[0], K, A.data_ptr(), ptr(q.get("sA")), ptr(q.get("tA")),
                              SCOPE[q.get("tA_scope", "row")], B_.data_ptr(), ptr(q.get("sB")), ptr(q.get("tB")),
                              SCOPE[q.get("tB_scope", "tensor")], out.data_ptr(), out.stride(0))
    _call("gemm_block_scaled_batch", dev, fmt, ctypes.cast(arr, _c_void_p), n)
    return [q["out"] for q in problems]


def _fp8_block_args(A, sA, B, sB, b_blocks: bool, out):
    """Validate a blockwise-FP8 GEMM; returns (M, N, K)."""
    M, K = A.shape
    N = B.shape[0]
    c = _Checks(A.device)
    c.need(A, "A", torch.uint8, (M, K))
    c.need(sA, "sA", torch.float32, (M, K // 128))
    c.need(B, "B", torch.uint8, (N, K))
    c.need(sB, "sB", torch.float32, ((N + 127) // 128, K // 128) if b_blocks else (N, K // 128))
    if out is not None:
        c.need(out, "out", torch.float32, (M, N), ld=True)
    c.done()
    return M, N, K


def gemm_fp8_blockwise(A, sA, B, sB, b_blocks: bool = True, out=None):
    """Blockwise FP8 GEMM C = A_hat B_hat^T (FP32); sB per 128 x 128 block (b_blocks) or per row."""
    M, N, K = _fp8_block_args(A, sA, B, sB, b_blocks, out)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _call("gemm_fp8_blockwise", A.device, M, N, K, _ptr(A), _ptr(sA), _ptr(B), _ptr(sB), int(b_blocks), _ptr(out),
          out.stride(0))
    return out


class _Fp8BlockProblem(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("A", _c_void_p), ("sA", _c_void_p), ("B", _c_void_p),
                ("sB", _c_void_p), ("b_blocks", _int), ("C", _c_void_p), ("ldc", _i64)]


def gemm_fp8_blockwise_batch(problems):
    """Several gemm_fp8_blockwise problems in one launch. problems: list of dicts with A, sA,
    B, sB, b_blocks and out."""
    n = len(problems)
    arr = (_Fp8BlockProblem * n)()
    dev = problems[0]["A"].device
    for i, q in enumerate(problems):
        A, B_, out = q["A"], q["B"], q["out"]
        if A.device != dev:
            raise ValueError(f"problem {i}: operands on {A.device}, the batch runs on {dev}")
        _fp8_block_args(A, q["sA"], B_, q["sB"], q["b_blocks"], out)
        arr[i] = _Fp8BlockProblem(A.shape[0], B_.shape[0], A.shape[1], A.data_ptr(), q["sA"].data_ptr(), B_.data_ptr(),
                                  q["sB"].data_ptr(), int(q["b_blocks"]), out.data_ptr(), out.stride(0))
    _call("gemm_fp8_blockwise_batch", dev, ctypes.cast(arr, _c_void_p), n)
    return [q["out"] for q in problems]


def gemm_mxfp8_matrix_core(A, sA, B, sB, out=None):
    """MXFP8 GEMM on the native scaled-FP8 matrix core (see include/mxq.h for its accumulation)."""
    M, N, K = _gemm_args(MXFP8, A, sA, B, sB, None, None, "row", "tensor", out)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _call("gemm_mxfp8_matrix_core", A.device, M, N, K, _ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(out), out.stride(0))
    return out


def _grouped_args(fmt, offsets, A, B, N, K, sA, sB, tA, tB, tA_scope, tB_scope, a_row_index, vary_k, M, total,
                  a_rows, out):
    """Validate a grouped GEMM's host-visible shapes (the offsets' values are checked on
    the device)."""
    c = _Checks(A.device)
    c.need(offsets, "offsets", torch.int64, (offsets.numel(),))
    G = offsets.numel() - 1
    if G < 0:
        raise ValueError("offsets: needs groups + 1 entries")
    if fmt == BF16_NVFP4T:
        if vary_k or a_row_index is not None:
            raise ValueError("BF16_NVFP4T: row-grouped only, no gather")
        c.need(A, "A", torch.bfloat16, (total, K))
        c.need(B.reshape(-1, B.shape[-1]) if B.dim() == 3 else B, "B", torch.uint8, (G * K, N // 2))
        if sB is None or tB is None:
            raise ValueError("BF16_NVFP4T: sB and tB (one FP32 scale per group) are required")
        c.need(sB.reshape(-1, sB.shape[-1]) if sB.dim() == 3 else sB, "sB", torch.uint8, (G * K, N // 16))
        c.need(tB, "tB", torch.float32, (G,))
        if out is not None:
            c.need(out, "out", torch.float32, (total, N))
        c.done()
        return
    if vary_k:
        if a_row_index is not None:
            raise ValueError("a_row_index is not supported with vary_k")
        if vary_k == 2:                                     # K-major A: (total, M), BF16 only
            if fmt != BF16:
                raise ValueError("vary_k=2 (K-major A) is BF16 only")
            c.operand(fmt, "A", A, total, M, None)
        else:
            c.operand(fmt, "A", A, M, total, sA)
        c.operand(fmt, "B", B, N, total, sB)
        if out is not None:
            c.need(out, "out", torch.float32, (G, M, N))
        c.done()
        return
    rows = A.shape[0]
    if a_row_index is not None:
        c.need(a_row_index, "a_row_index", torch.int32, (total,))
        if a_rows is not None and a_rows != rows:
            raise ValueError(f"a_rows = {a_rows} but A has {rows} rows")
    elif rows != total:
        raise ValueError(f"A: {rows} rows, expected total = {total} (no gather)")
    c.operand(fmt, "A", A, rows, K, sA)
    width = K if fmt == BF16 else K // _elems_per_byte(fmt)
    if B.shape[-1] != width or B.numel() != G * N * width:
        raise ValueError(f"B: shape {tuple(B.shape)}, expected {G} stacked ({N}, {width}) operands")
    if not B.is_contiguous():
        raise ValueError("B: expected a contiguous tensor")
    c.operand(fmt, "B", B.reshape(G * N, width), G * N, K, None if sB is None else sB.reshape(-1, sB.shape[-1]))
    if fmt == NVFP4:
        c.outer_scale("tA", tA, tA_scope, rows)
        if tB is None:
            raise ValueError("tB: NVFP4 needs its FP32 scale")
        c.need(tB, "tB", torch.float32, (G if SCOPE[tB_scope] == 2 else G * N if SCOPE[tB_scope] == 0 else 1,))
    if out is not None:
        c.need(out, "out", torch.float32, (total, N))
    c.done()


def grouped_gemm_block_scaled(fmt: int, offsets, A, B, N: int, K: int, sA=None, sB=None, tA=None, tB=None,
                              tA_scope="row", tB_scope="group", a_row_index=None, vary_k=False, M: int = 0,
                              total: int | None = None, a_rows: int | None = None, out=None, workspace=None):
    """One GEMM per group; see include/mxq.h for the two modes.

    vary_k=False: out (total_slots, N); vary_k=True: out (groups, M, N); vary_k=2: as True
    with A given K-major, (total, M).
    """
    groups = offsets.numel() - 1
    dev = A.device
    if total is None:
        total = int(offsets[-1].item())
    _grouped_args(fmt, offsets, A, B, N, K, sA, sB, tA, tB, tA_scope, tB_scope, a_row_index, vary_k, M, total,
                  a_rows, out)
    if out is None:
        shape = (groups, M, N) if vary_k else (total, N)
        out = torch.empty(shape, dtype=torch.float32, device=dev)
    ws_bytes = lib().mxq_workspace_bytes(OP_GROUPED_GEMM, groups, 0, 0)
    if workspace is None:
        workspace = _u8((max(ws_bytes, 1),), dev)
    elif workspace.numel() < ws_bytes:
        raise ValueError(f"workspace: {workspace.numel()} bytes, the call needs {ws_bytes}")
    _call("grouped_gemm_block_scaled", dev, fmt, groups, _ptr(offsets), int(vary_k), total, M, N, K,
          _ptr(a_row_index), a_rows if a_rows is not None else (A.shape[0] if a_row_index is not None else 0),
          _ptr(A), _ptr(sA), _ptr(tA), SCOPE[tA_scope], _ptr(B), _ptr(sB), _ptr(tB), SCOPE[tB_scope], _ptr(out),
          _ptr(workspace), workspace.numel())
    return out


def grouped_gemm_block_scaled_noalloc(fmt: int, offsets, A, B, N: int, K: int, sA=None, sB=None, tA=None, tB=None,
                                      tA_scope="row", tB_scope="group", a_row_index=None, vary_k=False, M: int = 0,
                                      total: int | None = None, a_rows: int | None = None, out=None):
    """grouped_gemm_block_scaled with the scheduler scratch in the library's static device
    array (no workspace): for callers that cannot allocate. `out` must be given (this
    call allocates nothing)."""
    if out is None:
        raise ValueError("out: the no-allocation call needs a preallocated output")
    if total is None:
        raise ValueError("total: pass it explicitly (reading it from the device offsets would synchronize)")
    _grouped_args(fmt, offsets, A, B, N, K, sA, sB, tA, tB, tA_scope, tB_scope, a_row_index, vary_k, M, total,
                  a_rows, out)
    _call("grouped_gemm_block_scaled_noalloc", A.device, fmt, offsets.numel() - 1, _ptr(offsets), int(vary_k), total,
          M, N, K, _ptr(a_row_index),
          a_rows if a_rows is not None else (A.shape[0] if a_row_index is not None else 0), _ptr(A), _ptr(sA),
          _ptr(tA), SCOPE[tA_scope], _ptr(B), _ptr(sB), _ptr(tB), SCOPE[tB_scope], _ptr(out))
    return out


# ---------------------------------------------------------------------------
# MoE glue
# ---------------------------------------------------------------------------

def moe_swiglu_quantize_nvfp4(gate_up: torch.Tensor, keep_h: bool = True):
    """SwiGLU of (rows, 2*inter) FP32 gate_up, then per-row NVFP4: (h_bf16 | None, q, s, t)."""
    rows, two_i = gate_up.shape
    inter = two_i // 2
    dev = gate_up.device
    c = _Checks(dev)
    c.need(gate_up, "gate_up", torch.float32, (rows, 2 * inter))
    c.done()
    h = torch.empty((rows, inter), dtype=torch.bfloat16, device=dev) if keep_h else None
    q, s = _u8((rows, inter // 2), dev), _u8((rows, inter // 16), dev)
    t = torch.empty(rows, dtype=torch.float32, device=dev)
    _call("moe_swiglu_quantize_nvfp4", dev, _ptr(gate_up), rows, inter, _ptr(h), _ptr(q), _ptr(s), _ptr(t))
    return h, q, s, t


def moe_combine(o_slots: torch.Tensor, slot_of: torch.Tensor, weights: torch.Tensor, out=None):
    T, k = slot_of.shape
    H = o_slots.shape[1]
    c = _Checks(o_slots.device)
    c.need(o_slots, "o_slots", torch.float32, tuple(o_slots.shape))
    c.need(slot_of, "slot_of", torch.int64, (T, k))
    c.need(weights, "weights", torch.float32, (T, k))
    c.opt(out, "out", torch.float32, (T, H))
    c.done()
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=o_slots.device)
    _call("moe_combine", o_slots.device, _ptr(o_slots), o_slots.shape[0], T, k, H, _ptr(slot_of), _ptr(weights),
          _ptr(out))
    return out


# ---------------------------------------------------------------------------
# Gated feed-forward block
# ---------------------------------------------------------------------------

def _gated_out(c, out, names, rows: int, inter: int, keep: bool, dev):
    """(h, gate_up) or (d_gate_up, h) BF16: the caller's (the second may be None), or new ones.
    names: which of them is 2 inter wide ends in "gate_up"."""
    width = lambda n: 2 * inter if n.endswith("gate_up") else inter
    if out is not None:
        first, second = out
        c.need(first, names[0], torch.bfloat16, (rows, width(names[0])))
        c.opt(second, names[1], torch.bfloat16, (rows, width(names[1])))
        c.done()
        return first, second
    c.done()
    new = lambda n: torch.empty(rows, width(n), dtype=torch.bfloat16, device=dev)
    return new(names[0]), new(names[1]) if keep else None


def _two_d(t, name: str):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    return t


def gemm_swiglu(fmt: int, A, sA, B, sB, tA=None, tB=None, tA_scope="row", tB_scope="tensor", keep_gate_up: bool = False,
                out=None, workspace=None):
    """h = silu(g) u in BF16, (g | u) = A_hat B_hat^T, in one kernel: (h (M, inter), gate_up (M, 2 inter) | None).
    fmt: MXFP8, NVFP4 or BF16; B (2 inter, K): the gate rows, then the up rows. `out` may supply
    (h, gate_up); gate_up None there = not written."""
    if fmt not in (MXFP8, NVFP4, BF16):
        raise ValueError(f"gemm_swiglu: format {fmt} is not supported")
    M, N, K = _gemm_args(fmt, _two_d(A, "A"), sA, _two_d(B, "B"), sB, tA, tB, tA_scope, tB_scope, None)
    if N % 2:
        raise ValueError(f"B: {N} rows, expected as many up rows as gate rows")
    c = _Checks(A.device)
    h, gate_up = _gated_out(c, out, ("h", "gate_up"), M, N // 2, keep_gate_up, A.device)
    ws = _workspace(OP_GEMM_SWIGLU, M, N, workspace, A.device, K)
    _call("gemm_swiglu", A.device, fmt, M, N // 2, K, _ptr(A), _ptr(sA), _ptr(tA), SCOPE[tA_scope], _ptr(B), _ptr(sB),
          _ptr(tB), SCOPE[tB_scope], _ptr(h), _ptr(gate_up), _ptr(ws), ws.numel())
    return h, gate_up


def _gate_up_dtype(gate_up) -> int:
    if not isinstance(gate_up, torch.Tensor) or gate_up.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("gate_up: expected a bfloat16 or float32 tensor")
    return OUT_F32 if gate_up.dtype == torch.float32 else OUT_BF16


def gemm_swiglu_backward(fmt: int, A, sA, B, sB, gate_up, keep_h: bool = True, out=None, workspace=None):
    """The gradient A (M, K) of a gated block's output through W_d and SwiGLU: (d_gate_up BF16 (M, 2 inter),
    h BF16 (M, inter) | None). B (inter, K): W_d^T, K-contiguous; fmt BF16 or MXFP8 (the columnwise copy
    of W_d). gate_up: as gemm_swiglu kept it, or FP32. `out` may supply (d_gate_up, h)."""
    if fmt not in (MXFP8, BF16):
        raise ValueError(f"gemm_swiglu_backward: format {fmt} is not supported")
    gd = _gate_up_dtype(gate_up)
    M, inter, K = _gemm_args(fmt, _two_d(A, "A"), sA, _two_d(B, "B"), sB, None, None, "row", "tensor", None)
    c = _Checks(A.device)
    c.need(gate_up, "gate_up", gate_up.dtype, (M, 2 * inter))
    d_gate_up, h = _gated_out(c, out, ("d_gate_up", "h"), M, inter, keep_h, A.device)
    ws = _workspace(OP_GEMM_SWIGLU, M, inter, workspace, A.device, K)
    _call("gemm_swiglu_backward", A.device, fmt, M, inter, K, _ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(gate_up), gd,
          _ptr(d_gate_up), _ptr(h), _ptr(ws), ws.numel())
    return d_gate_up, h


def grouped_gemm_swiglu(fmt: int, offsets, A, B, inter: int, K: int, sA=None, sB=None, tA=None, tB=None, tA_scope="row",
                        tB_scope="group", a_row_index=None, total: int | None = None, keep_gate_up: bool = False,
                        out=None, workspace=None):
    """gemm_swiglu per expert: (h (total, inter), gate_up (total, 2 inter) | None), BF16. fmt: NVFP4 or BF16;
    offsets, a_row_index, total and the operands as grouped_gemm_block_scaled's with N = 2 inter."""
    if fmt not in (NVFP4, BF16):
        raise ValueError(f"grouped_gemm_swiglu: format {fmt} is not supported")
    if total is None:
        total = int(offsets[-1].item())
    _two_d(A, "A")
    _grouped_args(fmt, offsets, A, B, 2 * inter, K, sA, sB, tA, tB, tA_scope, tB_scope, a_row_index, False, 0, total,
                  None, None)
    dev, groups = A.device, offsets.numel() - 1
    c = _Checks(dev)
    h, gate_up = _gated_out(c, out, ("h", "gate_up"), total, inter, keep_gate_up, dev)
    ws = _workspace(OP_GROUPED_SWIGLU, groups, 0, workspace, dev)
    _call("grouped_gemm_swiglu", dev, fmt, groups, _ptr(offsets), total, inter, K, _ptr(a_row_index),
          A.shape[0] if a_row_index is not None else 0, _ptr(A), _ptr(sA), _ptr(tA), SCOPE[tA_scope], _ptr(B), _ptr(sB),
          _ptr(tB), SCOPE[tB_scope], _ptr(h), _ptr(gate_up), _ptr(ws), ws.numel())
    return h, gate_up


def grouped_gemm_swiglu_backward(fmt: int, offsets, A, B, inter: int, K: int, gate_up, sB=None, tB=None,
                                 total: int | None = None, keep_h: bool = True, out=None, workspace=None):
    """gemm_swiglu_backward per expert: (d_gate_up (total, 2 inter), h (total, inter) | None), BF16. A BF16
    (total, K); fmt BF16 (B: the experts' (inter, K) stacked) or BF16_NVFP4T (B, sB, tB: the forward's
    NVFP4 W_d as it is, (experts K, inter / 2))."""
    if fmt not in (BF16, BF16_NVFP4T):
        raise ValueError(f"grouped_gemm_swiglu_backward: format {fmt} is not supported")
    if total is None:
        total = int(offsets[-1].item())
    gd = _gate_up_dtype(gate_up)
    _two_d(A, "A")
    _grouped_args(fmt, offsets, A, B, inter, K, None, sB, None, tB, "row", "group", None, False, 0, total, None, None)
    dev, groups = A.device, offsets.numel() - 1
    c = _Checks(dev)
    c.need(gate_up, "gate_up", gate_up.dtype, (total, 2 * inter))
    d_gate_up, h = _gated_out(c, out, ("d_gate_up", "h"), total, inter, keep_h, dev)
    ws = _workspace(OP_GROUPED_SWIGLU, groups, 0, workspace, dev)
    _call("grouped_gemm_swiglu_backward", dev, fmt, groups, _ptr(offsets), total, inter, K, _ptr(A), _ptr(B), _ptr(sB),
          _ptr(tB), _ptr(gate_up), gd, _ptr(d_gate_up), _ptr(h), _ptr(ws), ws.numel())
    return d_gate_up, h


# ---------------------------------------------------------------------------
# Matrix-vector products with 4-bit weights
# ---------------------------------------------------------------------------

def _weights4(c, fmt: int, W, sW, tW, t_scope: str, rows: int, K: int, groups: int, wide: str):
    """4-bit weights of `rows` rows in all; NVFP4: one FP32 scale a row, or (t_scope == wide) a group."""
    if fmt not in _PACKED4:
        raise ValueError(f"format {fmt}: expected NVFP4 or MXFP4 weights")
    c.need(W, "W", torch.uint8, (rows, K // 2))
    c.need(sW, "sW", torch.uint8, (rows, K // _scale_block(fmt)))
    if fmt == NVFP4:
        if t_scope not in ("row", wide):
            raise ValueError(f"t_scope: {t_scope!r}, expected 'row' or {wide!r}")
        if tW is None:
            raise ValueError("tW: NVFP4 needs its FP32 scale")
        c.need(tW, "tW", torch.float32, (rows if t_scope == "row" else groups,))


def _decode_rows(x, name: str, dim: int):
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != dim:
        raise ValueError(f"{name}: expected a {dim}-D bfloat16 tensor")
    return x.shape


def _gemv_args(fmt: int, x, W, sW, tW, t_scope: str, gated: bool, out_dtype, out):
    """The output and the C call's arguments up to it."""
    rows, K = _decode_rows(x, "x", 2)
    N = _two_d(W, "W").shape[0]
    if gated and N % 2:
        raise ValueError(f"W: {N} rows, expected as many up rows as gate rows")
    n = N // 2 if gated else N
    dev = x.device
    c = _Checks(dev)
    c.need(x, "x", torch.bfloat16, (rows, K), ld=True)
    _weights4(c, fmt, W, sW, tW, t_scope, N, K, 1, "tensor")
    if out is not None:
        c.need(out, "out", out.dtype if not gated and _float_dtype(out, "out") is not None else torch.bfloat16,
               (rows, n), ld=True)
    c.done()
    if out is None:
        out = torch.empty(rows, n, dtype=out_dtype, device=dev)
    return out, (fmt, rows, n, K, _ptr(x), max(x.stride(0), K), _ptr(W), _ptr(sW), _ptr(tW), SCOPE[t_scope], _ptr(out))


def gemv_block_scaled(fmt: int, x, W, sW, tW=None, t_scope: str = "tensor", out_dtype: torch.dtype = torch.float32,
                      out=None):
    """y = x W_hat^T of a few BF16 rows x (rows <= 64, K; rows may be strided) and 4-bit weights W (N, K/2):
    (rows, N) in FP32 or BF16 (`out`'s type where given). fmt: NVFP4 (tW, t_scope "tensor" or "row") or MXFP4."""
    if out is None and out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype: {out_dtype}, expected float32 or bfloat16")
    out, args = _gemv_args(fmt, x, W, sW, tW, t_scope, False, out_dtype, out)
    _call("gemv_block_scaled", x.device, *args, OUT_F32 if out.dtype == torch.float32 else OUT_BF16,
          max(out.stride(0), out.shape[1]))
    return out


def gemv_swiglu(fmt: int, x, W, sW, tW=None, t_scope: str = "tensor", out=None):
    """h = silu(x Wg_hat^T) (x Wu_hat^T) in BF16 (rows, inter), W (2 inter, K/2): gate rows, then up rows;
    otherwise as gemv_block_scaled."""
    out, args = _gemv_args(fmt, x, W, sW, tW, t_scope, True, torch.bfloat16, out)
    _call("gemv_swiglu", x.device, *args, max(out.stride(0), out.shape[1]))
    return out


def _stacked(W, experts: int) -> int:
    """Rows an expert of a stacked weight (experts n, K/2)."""
    rows = _two_d(W, "W").shape[0]
    if experts < 1 or rows % experts:
        raise ValueError(f"W: {rows} rows for {experts} experts")
    return rows // experts


def moe_decode_gate_up(fmt: int, x, topk_idx, W, sW, tW=None, experts: int = 0, t_scope: str = "group", out=None):
    """h (tokens, topk, inter) BF16 of a decoding step: each token (x (tokens <= 64, K) BF16, rows may be
    strided) through gate_up and SwiGLU of the experts topk_idx (tokens, topk) int32 names; zeros for a
    choice of -1. W: (experts 2 inter, K/2), inter <= 65520, NVFP4 or MXFP4, as quantize_nvfp4(scope="group") and
    quantize_mxfp4 store the stacked weights."""
    T, K = _decode_rows(x, "x", 2)
    n = _stacked(W, experts)
    if n % 2:
        raise ValueError(f"W: {n} rows an expert, expected as many up rows as gate rows")
    dev = x.device
    c = _Checks(dev)
    c.need(x, "x", torch.bfloat16, (T, K), ld=True)
    k = _two_d(topk_idx, "topk_idx").shape[1]
    c.need(topk_idx, "topk_idx", torch.int32, (T, k))
    _weights4(c, fmt, W, sW, tW, t_scope, W.shape[0], K, experts, "group")
    c.opt(out, "out", torch.bfloat16, (T, k, n // 2))
    c.done()
    if out is None:
        out = torch.empty(T, k, n // 2, dtype=torch.bfloat16, device=dev)
    _call("moe_decode_gate_up", dev, fmt, T, k, experts, n // 2, K, _ptr(x), max(x.stride(0), K), _ptr(topk_idx), _ptr(W),
          _ptr(sW), _ptr(tW), SCOPE[t_scope], _ptr(out))
    return out


def moe_decode_down(fmt: int, h, topk_idx, weights, W, sW, tW=None, experts: int = 0, t_scope: str = "group",
                    out_dtype: torch.dtype = torch.float32, out=None, workspace=None):
    """y (tokens, hidden) = sum over j of weights[t, j] (h[t, j] W_hat_e^T), FP32 or BF16 (`out`'s type where
    given): the down projection and the combine of a decoding step. h (tokens, topk, inter) BF16 as
    moe_decode_gate_up gives it, W: (experts hidden, inter / 2), hidden <= 65520."""
    T, k, K = _decode_rows(h, "h", 3)
    n = _stacked(W, experts)
    if out is None and out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype: {out_dtype}, expected float32 or bfloat16")
    dev = h.device
    c = _Checks(dev)
    c.need(h, "h", torch.bfloat16, (T, k, K))
    c.need(topk_idx, "topk_idx", torch.int32, (T, k))
    c.need(weights, "weights", torch.float32, (T, k))
    _weights4(c, fmt, W, sW, tW, t_scope, W.shape[0], K, experts, "group")
    if out is not None:
        c.need(out, "out", torch.float32 if out.dtype == torch.float32 else torch.bfloat16, (T, n))
    c.done()
    if out is None:
        out = torch.empty(T, n, dtype=out_dtype, device=dev)
    ws = _workspace(OP_DECODE_DOWN, T, n, workspace, dev, k)
    _call("moe_decode_down", dev, fmt, T, k, experts, n, K, _ptr(h), _ptr(topk_idx), _ptr(weights), _ptr(W), _ptr(sW),
          _ptr(tW), SCOPE[t_scope], _ptr(out), OUT_F32 if out.dtype == torch.float32 else OUT_BF16, _ptr(ws), ws.numel())
    return out


# ---------------------------------------------------------------------------
# Norms around a block
# ---------------------------------------------------------------------------

def _float_dtype(t, name: str) -> int:
    """MXQ_OUT_* code of a BF16 or FP32 tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name}: expected a bfloat16 or float32 tensor")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor (rows, cols)")
    if t.shape[1] == 0:                                      # the mean over a row is undefined
        raise ValueError(f"{name}: rows without elements")
    return OUT_F32 if t.dtype == torch.float32 else OUT_BF16


def _need_gate(c, gate, gate_mode: str, name: str, rows: int, cols: int) -> int:
    if gate_mode not in GATE:
        raise ValueError(f"gate_mode: {gate_mode!r}, expected one of {sorted(GATE)}")
    mode = GATE[gate_mode]
    if mode == 0 and gate is not None:
        raise ValueError(f"{name}: gate_mode is 'none'")
    if mode:
        c.need(gate, name, torch.float32, {1: (rows,), 2: (cols,), 3: (rows, cols)}[mode])
    return mode


_NOTHING = torch.empty(0, dtype=torch.uint8)              # NULL, no bytes: spares an allocation a call


def _workspace(op: int, a: int, b: int, workspace, dev, c: int = 0):
    """The call's scratch: allocated here, or the caller's, checked for size and device."""
    need = lib().mxq_workspace_bytes(op, a, b, c)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else _NOTHING
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError(f"workspace: expected contiguous uint8 memory on {dev}")
    if workspace.numel() < need:
        raise ValueError(f"workspace: {workspace.numel()} bytes, the call needs {need}")
    return workspace


def rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, fmt: int = NVFP4,
                     keep_n: bool = True, out=None):
    """RMSNorm of BF16 or FP32 x (T, H), rounded to BF16 and quantized row by row in one pass:
    (n | None, q | None, s | None, t | None, rstd). fmt: MXFP8, MXFP4, NVFP4 (per token) or
    BF16 (n only). x's rows may be strided (rmsnorm_backward takes dense ones). `out` may supply
    preallocated (n, q, s, t, rstd); n or rstd None there = not written."""
    xd = _float_dtype(x, "x")
    if fmt not in (MXFP8, NVFP4, BF16, MXFP4):
        raise ValueError(f"unknown format {fmt}")
    T, H = x.shape
    dev = x.device
    c = _Checks(dev)
    c.need(x, "x", x.dtype, (T, H), ld=True)
    c.opt(weight, "weight", torch.float32, (H,))
    if out is not None:
        n, q, s, t, rstd = out
        (c.need if fmt == BF16 else c.opt)(n, "n", torch.bfloat16, (T, H))
        if fmt != BF16:
            c.need(q, "q", torch.uint8, (T, H // _elems_per_byte(fmt)))
            c.need(s, "s", torch.uint8, (T, H // _scale_block(fmt)))
        if fmt == NVFP4:
            c.need(t, "t", torch.float32, (T,))
        c.opt(rstd, "rstd", torch.float32, (T,))
    c.done()
    if out is None:
        n = torch.empty(T, H, dtype=torch.bfloat16, device=dev) if keep_n or fmt == BF16 else None
        q = s = t = None
        if fmt != BF16:
            q, s = _u8((T, H // _elems_per_byte(fmt)), dev), _u8((T, H // _scale_block(fmt)), dev)
        if fmt == NVFP4:
            t = torch.empty(T, dtype=torch.float32, device=dev)
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
    _call("rmsnorm_quantize", dev, fmt, _ptr(x), xd, T, H, max(x.stride(0), H), _ptr(weight), eps, _ptr(n), _ptr(q),
          _ptr(s), _ptr(t), _ptr(rstd))
    return n, q, s, t, rstd


def rmsnorm_backward(dn: torch.Tensor, x: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor | None = None,
                     dn2: torch.Tensor | None = None, d_res: torch.Tensor | None = None, res_scale: float = 1.0,
                     out=None, workspace: torch.Tensor | None = None):
    """Gradients of rmsnorm_quantize's n: (dx in x's type, dw FP32 | None). dn2 is a second
    gradient of n, d_res the residual branch's gradient (added times res_scale). `out` may
    supply (dx, dw); dw None there = not wanted."""
    dd, xd = _float_dtype(dn, "dn"), _float_dtype(x, "x")
    T, H = x.shape
    dev = x.device
    c = _Checks(dev)
    c.need(x, "x", x.dtype, (T, H))
    c.need(dn, "dn", dn.dtype, (T, H))
    c.opt(dn2, "dn2", dn.dtype, (T, H))
    c.need(rstd, "rstd", torch.float32, (T,))
    c.opt(weight, "weight", torch.float32, (H,))
    c.opt(d_res, "d_res", x.dtype, (T, H))
    if out is not None:
        dx, dw = out
        c.need(dx, "dx", x.dtype, (T, H))
        c.opt(dw, "dw", torch.float32, (H,))
    c.done()
    if out is None:
        dx, dw = torch.empty_like(x), None if weight is None else torch.empty_like(weight)
    ws = _workspace(OP_NORM_BACKWARD, T, H, workspace, dev) if dw is not None else None
    _call("rmsnorm_backward", dev, _ptr(dn), _ptr(dn2), dd, _ptr(x), xd, _ptr(rstd), _ptr(weight), _ptr(d_res),
          res_scale, T, H, _ptr(dx), _ptr(dw), _ptr(ws), 0 if ws is None else ws.numel())
    return dx, dw


def rmsnorm_gate_residual(x: torch.Tensor, y: torch.Tensor, weight: torch.Tensor | None = None,
                          gate: torch.Tensor | None = None, gate_mode: str = "none", eps: float = 1e-6,
                          branch_scale: float = 1.0, res_scale: float = 1.0, out=None):
    """res_scale x + branch_scale gate RMSNorm(y): (out in x's type, rstd). gate is FP32, (T,) for
    gate_mode "token", (H,) for "channel", (T, H) for "full". `out` may supply (out, rstd)."""
    xd, yd = _float_dtype(x, "x"), _float_dtype(y, "y")
    T, H = x.shape
    dev = x.device
    c = _Checks(dev)
    c.need(x, "x", x.dtype, (T, H))
    c.need(y, "y", y.dtype, (T, H))
    c.opt(weight, "weight", torch.float32, (H,))
    mode = _need_gate(c, gate, gate_mode, "gate", T, H)
    if out is not None:
        o, rstd = out
        c.need(o, "out", x.dtype, (T, H))
        c.opt(rstd, "rstd", torch.float32, (T,))
    c.done()
    if out is None:
        o, rstd = torch.empty_like(x), torch.empty(T, dtype=torch.float32, device=dev)
    _call("rmsnorm_gate_residual", dev, _ptr(x), xd, _ptr(y), yd, _ptr(weight), _ptr(gate), mode, eps, branch_scale,
          res_scale, T, H, _ptr(o), _ptr(rstd))
    return o, rstd


def rmsnorm_gate_residual_backward(d_out: torch.Tensor, y: torch.Tensor, rstd: torch.Tensor,
                                   weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                                   gate_mode: str = "none", branch_scale: float = 1.0, out=None,
                                   workspace: torch.Tensor | None = None):
    """Gradients of rmsnorm_gate_residual: (dy in y's type, dw FP32 | None, dgate FP32 | None); the
    residual's own is res_scale d_out. `out` may supply (dy, dw, dgate); None there = not wanted."""
    dd, yd = _float_dtype(d_out, "d_out"), _float_dtype(y, "y")
    T, H = y.shape
    dev = y.device
    c = _Checks(dev)
    c.need(d_out, "d_out", d_out.dtype, (T, H))
    c.need(y, "y", y.dtype, (T, H))
    c.need(rstd, "rstd", torch.float32, (T,))
    c.opt(weight, "weight", torch.float32, (H,))
    mode = _need_gate(c, gate, gate_mode, "gate", T, H)
    if out is not None:
        dy, dw, dgate = out
        c.need(dy, "dy", y.dtype, (T, H))
        c.opt(dw, "dw", torch.float32, (H,))
        if dgate is not None:
            _need_gate(c, dgate, gate_mode, "dgate", T, H)
    c.done()
    if out is None:
        dy = torch.empty_like(y)
        dw = None if weight is None else torch.empty_like(weight)
        dgate = None if gate is None else torch.empty_like(gate)
    sums = dw is not None or (dgate is not None and mode == GATE["channel"])
    ws = _workspace(OP_NORM_BACKWARD, T, H, workspace, dev) if sums else None
    _call("rmsnorm_gate_residual_backward", dev, _ptr(d_out), dd, _ptr(y), yd, _ptr(rstd), _ptr(weight), _ptr(gate),
          mode, branch_scale, T, H, _ptr(dy), _ptr(dw), _ptr(dgate), _ptr(ws), 0 if ws is None else ws.numel())
    return dy, dw, dgate


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------

class RoutePlan:
    """A routing on the device: topk_idx, weights, counts, offsets, row_index, slot_of and the
    balance loss (None if not wanted), as moe_route writes them (include/mxq.h), with `slots`
    (the total), `groups` (the experts) and the call's scratch, all in one allocation. Made once
    for a batch size, it serves every call."""

    def __init__(self, tokens: int, experts: int, topk: int, pad: int = 1, total: int | None = None,
                 loss: bool = False, dev="cuda"):
        need = route_slots(tokens, experts, topk, pad)
        total = need if total is None else total
        if total < need or total % pad or total > 0x7FFFFFFF:
            raise ValueError(f"total: {total} slots, expected a multiple of {pad} and at least {need}")
        self.tokens, self.groups, self.topk, self.pad, self.slots = tokens, experts, topk, pad, total
        ws = (lib().mxq_workspace_bytes(OP_ROUTE, tokens, experts, 0) + 15) // 16 * 4
        n = tokens * topk
        sizes = (ws, 2 * experts + 2, 2 * n, n, n, experts + 1, total, 1)          # in dwords, 8-byte values first
        (self.workspace, offsets, slot_of, topk_idx, weights, self.counts, self.row_index, loss_) = torch.empty(
            sum(sizes), dtype=torch.int32, device=dev).split_with_sizes(sizes)
        self.offsets = offsets.view(torch.int64)
        self.slot_of = slot_of.view(torch.int64).view(tokens, topk)
        self.topk_idx = topk_idx.view(tokens, topk)
        self.weights = weights.view(torch.float32).view(tokens, topk)
        self.loss = loss_.view(torch.float32) if loss else None


def route_slots(tokens: int, experts: int, topk: int, pad: int = 1) -> int:
    """Slots that hold every routing of this size, each expert's range a multiple of pad."""
    n = lib().mxq_route_slots(tokens, experts, topk, pad)
    if n < 0:
        raise ValueError(f"no routing of {tokens} tokens, {experts} experts, top-{topk}, pad {pad}")
    return n


def moe_route(logits: torch.Tensor, topk: int, pad: int = 1, valid: torch.Tensor | None = None,
              balance_coef: float | None = None, total: int | None = None,
              out: RoutePlan | None = None) -> RoutePlan:
    """Top-k routing of FP32 logits (T, G) with its slots, counts and (balance_coef given) balance
    loss. valid: bool or uint8 (T,), False = a padding token that is not routed. `out`: a plan
    of the same sizes to write into, made with a loss if balance_coef is given and without one if
    not."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits: expected a 2-D tensor (tokens, experts)")
    T, G = logits.shape
    dev = logits.device
    c = _Checks(dev)
    c.need(logits, "logits", torch.float32, (T, G), ld=True)
    if valid is not None:
        if isinstance(valid, torch.Tensor) and valid.dtype == torch.bool:
            valid = valid.view(torch.uint8)
        c.need(valid, "valid", torch.uint8, (T,))
    plan = out
    if plan is None:
        plan = RoutePlan(T, G, topk, pad, total, balance_coef is not None, dev)
    elif (plan.tokens, plan.groups, plan.topk, plan.pad) != (T, G, topk, pad) or (total or plan.slots) != plan.slots:
        raise ValueError("out: a plan of other sizes")
    elif balance_coef is not None and plan.loss is None:
        raise ValueError("out: a plan without a loss")
    elif balance_coef is None and plan.loss is not None:     # it would keep an earlier call's
        raise ValueError("out: a plan with a loss, which a call without balance_coef does not write")
    c.need(plan.offsets, "out", torch.int64, (G + 1,))
    c.done()
    ws = plan.workspace
    loss = None if balance_coef is None else plan.loss
    _call("moe_route", dev, _ptr(logits), _ptr(valid), T, G, max(logits.stride(0), G), topk, pad, plan.slots,
          0.0 if balance_coef is None else balance_coef, _ptr(plan.topk_idx), _ptr(plan.weights), _ptr(plan.counts),
          _ptr(plan.offsets), _ptr(plan.row_index), _ptr(plan.slot_of), _ptr(loss), _ptr(ws), 4 * ws.numel())
    return plan


def moe_route_backward(logits: torch.Tensor, topk_idx: torch.Tensor, weights: torch.Tensor, counts: torch.Tensor,
                       d_weights: torch.Tensor | None = None, d_loss: torch.Tensor | None = None,
                       balance_coef: float = 0.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """d_logits (T, G) from the gradients of the combine weights (T, k) and of the balance loss
    (1,), either None; topk_idx, weights and counts from moe_route. FP32, or `out`'s type (FP32
    or BF16)."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("logits, topk_idx: expected 2-D tensors")
    T, G = logits.shape
    k = topk_idx.shape[1]
    dev = logits.device
    c = _Checks(dev)
    c.need(logits, "logits", torch.float32, (T, G), ld=True)
    c.need(topk_idx, "topk_idx", torch.int32, (T, k))
    c.need(weights, "weights", torch.float32, (T, k))
    c.need(counts, "counts", torch.int32, (G + 1,))
    c.opt(d_weights, "d_weights", torch.float32, (T, k))
    c.opt(d_loss, "d_loss", torch.float32, (1,))
    od = OUT_F32 if out is None else _float_dtype(out, "out")
    if out is not None:
        c.need(out, "out", out.dtype, (T, G))
    c.done()
    if out is None:
        out = torch.empty(T, G, dtype=torch.float32, device=dev)
    _call("moe_route_backward", dev, _ptr(logits), T, G, max(logits.stride(0), G), k, _ptr(topk_idx), _ptr(weights),
          _ptr(d_weights), _ptr(counts), _ptr(d_loss), balance_coef, _ptr(out), od)
    return out


def moe_combine_backward(dy: torch.Tensor, o_slots: torch.Tensor, slot_of: torch.Tensor, weights: torch.Tensor,
                         row_index: torch.Tensor, out=None):
    """Gradients of moe_combine: (d_o BF16 (slots, H), padding slots cleared, d_weights FP32 (T, k)).
    `out` may supply both."""
    dd = _float_dtype(dy, "dy")
    T, k = slot_of.shape
    S, H = o_slots.shape
    dev = o_slots.device
    c = _Checks(dev)
    c.need(dy, "dy", dy.dtype, (T, H))
    c.need(o_slots, "o_slots", torch.float32, (S, H))
    c.need(slot_of, "slot_of", torch.int64, (T, k))
    c.need(weights, "weights", torch.float32, (T, k))
    c.need(row_index, "row_index", torch.int32, (S,))
    if out is not None:
        d_o, d_w = out
        c.need(d_o, "d_o", torch.bfloat16, (S, H))
        c.need(d_w, "d_weights", torch.float32, (T, k))
    c.done()
    if out is None:
        d_o, d_w = torch.empty(S, H, dtype=torch.bfloat16, device=dev), torch.empty_like(weights)
    _call("moe_combine_backward", dev, _ptr(dy), dd, _ptr(o_slots), S, T, k, H, _ptr(slot_of), _ptr(weights),
          _ptr(row_index), _ptr(d_o), _ptr(d_w))
    return d_o, d_w


def scale_bytes(fmt: int, rows: int, cols: int) -> int:
    return lib().mxq_scale_bytes(fmt, rows, cols)


def abi_version() -> int:
    return lib().mxq_abi_version()
