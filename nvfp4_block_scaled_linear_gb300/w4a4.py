"""ctypes binding of the NVFP4 x NVFP4 operators (include/nvfp4_w4a4.h).

A layer whose activations are NVFP4 as well as its weights:

    gate_up = Fp4Weight(w_packed, w_scale, [gs_gate, gs_up], [inner, inner])   # once, at load
    down = Fp4Weight(w_packed, w_scale, gs)
    a, residual = add_rms_norm_quantize(x, residual, norm_weight, eps, input_scale)
    h = linear_w4a4_swiglu_quantize(a, gate_up, inner_scale)
    y = linear_w4a4(h, down)

and, where rows come as bf16 (attention's output) or leave as bf16 (for the
linear layer of bf16 activations),

    y = linear_w4a4(quantize_rows(x, input_scale), o)
    y, residual = add_rms_norm(x, residual, norm_weight, eps)

Argument marshalling only, as in ``_lib``: every step runs in the library's
kernels, on the current CUDA stream unless one is given (a ``torch.cuda.Stream``
or a raw handle).  What a call makes itself belongs to the stream that it runs on,
as under ``torch.cuda.stream(stream)``.
"""
import ctypes
import os
import re
import struct

import torch

from . import _lib
from ._lib import OK, Nvfp4Error
from .attention import _empty

W4A4_HEADER = os.path.join(os.path.dirname(_lib.HEADER), "nvfp4_w4a4.h")

W4A4_TIMEOUT = 1
MAX_SEGMENTS = 8

# The C structures, packed into bytes (which a pointer argument takes as they are).
_pack_rows = struct.Struct("@PPf4x").pack                  # nvfp4_rows
_pack_weight = struct.Struct("@PPqqi8f8q").pack            # nvfp4_weight

_ready = None


def _library():
    global _ready
    if _ready is None:
        lib = _lib.load_library()
        P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        signatures = {
            "nvfp4_w4a4_scale_layout": [P, i64, i64, P, P, P],
            "nvfp4_quantize_rows": [P, i64, i64, i64, P, P],
            "nvfp4_add_rms_norm": [P, i64, P, i64, P, f32, i64, i64, P, i64, P, i64, P, P],
            "nvfp4_linear_w4a4": [P, i64, P, i32, P, P, P],
            "nvfp4_w4a4_status": [P, ctypes.c_int],
        }
        for name, args in signatures.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = ctypes.c_int, args
        lib.nvfp4_w4a4_scale_bytes.restype = i64
        lib.nvfp4_w4a4_scale_bytes.argtypes = [i64, i64]
        _ready = lib
    return _ready


def w4a4_header_functions():
    """Names of the functions declared in include/nvfp4_w4a4.h."""
    text = open(W4A4_HEADER).read()
    return sorted(set(re.findall(r"^(?:int|int64_t) (nvfp4_\w+)\(", text, re.M)))


def w4a4_error(clear: bool = True) -> int:
    """These operators' device error word (W4A4_TIMEOUT); synchronises."""
    bits = ctypes.c_uint(0)
    st = _library().nvfp4_w4a4_status(ctypes.byref(bits), 1 if clear else 0)
    if st != OK:
        raise Nvfp4Error(st, "nvfp4_w4a4_status")
    return bits.value


_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _call(name, device, stream, *args):
    """One library call on `stream` (the device's current one by default)."""
    index = device.index
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    f = getattr(_ready or _library(), name)
    if index == _current_device():
        st = f(*args, stream)
    else:
        with torch.cuda.device(device):
            st = f(*args, stream)
    if st:
        raise Nvfp4Error(st, name)


def _scale(value, name):
    value = float(value)
    # (what fp32 rounds neither to zero nor to infinity)
    if not 2.0 ** -150 < value < 2.0 ** 128 - 2.0 ** 103:
        raise ValueError("%s must be positive and finite in fp32, got %s" % (name, value))
    return value


class Fp4Rows:
    """NVFP4 rows [M, K], K a multiple of 256, on one device.

    codes         uint8 [M, K/2], the low nibble holding the even k.
    scales        uint8 [ceil(M/128), K/64, 512]: the e4m3 scales in the order
                  that the product reads (include/nvfp4_w4a4.h).
    global_scale  the values are codes times scales divided by it.

    What rows are is fixed when they are made: another scale or other memory are
    other Fp4Rows.  Copies (``copy.deepcopy``, ``torch.save``) have memory of their own.
    """
    __slots__ = ("_codes", "_scales", "_global_scale", "_shape", "_device", "_c")

    def __init__(self, codes, scales, global_scale=1.0):
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8, got %s and %s" % (codes.dtype, scales.dtype))
        if not codes.is_cuda or codes.device != scales.device:
            raise ValueError("codes and scales must be CUDA tensors on one device")
        if codes.dim() != 2 or codes.shape[1] == 0 or codes.shape[1] % 128:
            raise ValueError("codes must be [M, K/2], K a multiple of 256, got %s" % (tuple(codes.shape),))
        m, k = codes.shape[0], codes.shape[1] * 2
        if scales.shape != (-(-m // 128), k // 64, 512):
            raise ValueError("scales must have shape %s, got %s"
                             % ((-(-m // 128), k // 64, 512), tuple(scales.shape)))
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        # (tensors of its own: the memory whose addresses _c holds stays, whatever the caller's are set to)
        self._codes, self._scales = codes.detach(), scales.detach()
        self._global_scale = _scale(global_scale, "global_scale")
        self._shape, self._device = (m, k), codes.device
        self._c = _pack_rows(codes.data_ptr(), scales.data_ptr(), self._global_scale)

    global_scale = property(lambda self: self._global_scale)
    shape = property(lambda self: self._shape)
    device = property(lambda self: self._device)

    # (rows that a call makes are one allocation, in _codes; the views of it cost
    # as much as a small kernel, and no call needs them)
    @property
    def codes(self):
        if self._scales is None:
            m, k = self._shape
            return self._codes[:m * (k // 2)].view(m, k // 2)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            m, k = self._shape
            return self._codes[m * (k // 2):].view(-(-m // 128), k // 64, 512)
        return self._scales

    def __reduce__(self):
        return type(self), (self.codes, self.scales, self._global_scale)


def new_fp4_rows(m, k, global_scale=1.0, device="cuda", stream=None):
    """Fp4Rows of fresh memory (one allocation), to be written by a call."""
    if m < 0 or k <= 0 or k % 256:
        raise ValueError("rows must be [M, K], K a positive multiple of 256, got [%d, %d]" % (m, k))
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("rows are of a CUDA device, got %s" % device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return _new_rows(m, k, _scale(global_scale, "global_scale"), device, stream)


def _new_rows(m, k, global_scale, device, stream):
    split = m * (k >> 1)                                   # a multiple of 128: both parts are aligned
    size = split + (m + 127 >> 7) * 8 * k
    if stream is None:
        raw = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        raw = _empty(size, torch.uint8, device, stream)
    rows = Fp4Rows.__new__(Fp4Rows)
    rows._codes, rows._scales, rows._global_scale, rows._shape, rows._device = raw, None, global_scale, (m, k), device
    p = raw.data_ptr()
    rows._c = _pack_rows(p, p + split, global_scale)
    return rows


class Fp4Weight:
    """An NVFP4 weight [N, K] as ``linear_w4a4`` takes it, kept as long as the
    layer: N a multiple of 128, K of 256.

    w_packed      uint8 [N, K/2], as ``linear`` takes it; referred to, not copied, and
                  read before the kernel ahead of a call has ended: neither that kernel
                  nor, where it is one of this library's, one of those that it follows
                  directly may write it.
    w_scale       uint8 (or float8_e4m3fn) [N, K/16], as ``linear`` takes it; its
                  scales are laid out anew once, here, which synchronises.  None may
                  be negative or NaN.
    global_scale  the weight's, or a list of one for each of up to 8 stacked segments
                  of segment_rows rows (multiples of 16).

    Its scales and segments are fixed when it is made; what is copied into ``codes`` later
    is read by later calls.  Copies (``copy.deepcopy``, ``torch.save``) have memory of
    their own.
    """

    def __init__(self, w_packed, w_scale, global_scale, segment_rows=None):
        w_packed, w_scale = _lib._as_u8(w_packed, "w_packed"), _lib._as_u8(w_scale, "w_scale")
        if not w_packed.is_cuda or w_packed.device != w_scale.device:
            raise ValueError("w_packed and w_scale must be CUDA tensors on one device")
        if w_packed.dim() != 2 or w_scale.dim() != 2:
            raise ValueError("w_packed and w_scale must be 2-D")
        n, k = w_packed.shape[0], w_packed.shape[1] * 2
        if n == 0 or n % 128 or k == 0 or k % 256:
            raise ValueError("a weight is [N, K], N a multiple of 128 and K of 256, got [%d, %d]" % (n, k))
        if tuple(w_scale.shape) != (n, k // 16):
            raise ValueError("w_scale must have shape %s, got %s" % ((n, k // 16), tuple(w_scale.shape)))
        if not (w_packed.is_contiguous() and w_scale.is_contiguous()):
            raise ValueError("w_packed and w_scale must be contiguous")
        several = isinstance(global_scale, (list, tuple))
        scales = [_scale(s, "global_scale") for s in (global_scale if several else [global_scale])]
        rows = [n] if segment_rows is None else [int(r) for r in segment_rows]
        if len(rows) != len(scales) or not 1 <= len(rows) <= MAX_SEGMENTS:
            raise ValueError("%d global scales for %d segments (1 to %d)" % (len(scales), len(rows), MAX_SEGMENTS))
        if sum(rows) != n or any(r <= 0 or r % 16 for r in rows):
            raise ValueError("segment_rows must be positive multiples of 16 that sum to %d, got %s" % (n, rows))
        dev = w_packed.device
        blocked = torch.empty((n // 128, k // 64, 512), dtype=torch.uint8, device=dev)
        refused = torch.zeros(1, dtype=torch.int32, device=dev)
        _call("nvfp4_w4a4_scale_layout", dev, None, w_scale.data_ptr(), n, k, blocked.data_ptr(),
              refused.data_ptr())
        if int(refused):
            raise ValueError("w_scale holds a negative scale or a NaN")
        self._set(w_packed.detach(), blocked, scales, rows)

    def _set(self, codes, blocked, scales, rows):
        """Fill in from checked arguments, the scales in the product's order."""
        # (tensors of its own: the memory whose addresses _c holds stays, whatever the caller's are set to)
        n, k = codes.shape[0], codes.shape[1] * 2
        self._codes, self._scales, self._global_scales, self._segment_rows = codes, blocked, scales, rows
        self._shape, self._device = (n, k), codes.device
        pad = MAX_SEGMENTS - len(rows)
        self._c = _pack_weight(codes.data_ptr(), blocked.data_ptr(), n, k, len(rows), *scales,
                               *[0.0] * pad, *rows, *[0] * pad)

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    global_scales = property(lambda self: list(self._global_scales))
    segment_rows = property(lambda self: list(self._segment_rows))
    shape = property(lambda self: self._shape)
    device = property(lambda self: self._device)

    def __reduce__(self):
        own = {"_codes", "_scales", "_global_scales", "_segment_rows", "_shape", "_device", "_c"}
        rest = {name: value for name, value in self.__dict__.items() if name not in own}
        return _copied_weight, (type(self), self._codes, self._scales, self.global_scales, self.segment_rows), rest or None


def _copied_weight(kind, codes, blocked, scales, rows):
    """The Fp4Weight of a copy's tensors."""
    if not (codes.is_cuda and codes.device == blocked.device and codes.is_contiguous() and blocked.is_contiguous()):
        raise ValueError("an Fp4Weight's codes and scales must be contiguous CUDA tensors on one device")
    w = kind.__new__(kind)
    w._set(codes, blocked, scales, rows)
    return w


def _matrix(t, name, shape, device):
    """Address and row stride of bfloat16 [M, K]."""
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be bfloat16, got %s" % (name, t.dtype))
    if t.shape != shape or t.device != device:
        raise ValueError("%s must have shape %s on %s, got %s on %s"
                         % (name, tuple(shape), device, tuple(t.shape), t.device))
    row, one = t.stride()
    if one != 1:
        raise ValueError("the rows of %s must be dense" % name)
    return t.data_ptr(), row


def _input(x):
    """Device, rows, width, address and row stride of the input that decides them."""
    if not x.is_cuda or x.ndim != 2:
        raise ValueError("x must be a CUDA tensor [M, K]")
    if x.dtype is not torch.bfloat16:
        raise TypeError("x must be bfloat16, got %s" % x.dtype)
    m, k = x.shape
    row, one = x.stride()
    if one != 1:
        raise ValueError("the rows of x must be dense")
    return x.device, m, k, x.data_ptr(), row


def _rows_out(out, m, k, global_scale, device, stream):
    if out is None:
        return _new_rows(m, k, _scale(global_scale, "global_scale"), device, stream)
    if not isinstance(out, Fp4Rows):
        raise TypeError("out must be Fp4Rows, got %s" % type(out).__name__)
    if out._shape != (m, k) or out._device != device:
        raise ValueError("out must hold rows %s on %s, got %s on %s" % ((m, k), device, out.shape, out.device))
    if out._global_scale != global_scale:
        raise ValueError("out has the global scale %s, the call %s" % (out.global_scale, global_scale))
    return out


def quantize_rows(x, global_scale=1.0, out=None, stream=None):
    """x (bfloat16 [M, K], rows may be strided, K a multiple of 256) as NVFP4 rows
    with the given global scale (a checkpoint's input_global_scale; 1 keeps what
    lies between about 0.1 and 2688).  Returns Fp4Rows."""
    dev, m, k, p, stride = _input(x)
    if k == 0 or k % 256:
        raise ValueError("K must be a positive multiple of 256, got %d" % k)
    out = _rows_out(out, m, k, global_scale, dev, stream)
    _call("nvfp4_quantize_rows", dev, stream, p, stride, m, k, out._c)
    return out


def _norm(given, x, residual, weight, eps, residual_out, y, rows, stream):
    """The call on `given`, the _input of x; makes the sum's tensor where that is missing.  Returns the sum."""
    dev, m, k, px, sx = given
    shape = x.shape
    pr, sr = (None, 0) if residual is None else _matrix(residual, "residual", shape, dev)
    if weight.dtype is not torch.bfloat16:
        raise TypeError("weight must be bfloat16, got %s" % weight.dtype)
    if weight.shape != (k,) or weight.device != dev or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous tensor of shape %s on %s, got %s on %s"
                         % ((k,), dev, tuple(weight.shape), weight.device))
    py, sy = (None, 0) if y is None else _matrix(y, "out", shape, dev)
    if residual_out is not None:
        po, so = _matrix(residual_out, "residual_out", shape, dev)
        total = residual_out
    elif residual is not None or (m and py == px):
        # (without a residual the sum is x, unless that is written over)
        total = _like(shape, dev, stream)
        po, so = total.data_ptr(), k
    else:
        po, so, total = None, 0, x
    _call("nvfp4_add_rms_norm", dev, stream, px, sx, pr, sr, weight.data_ptr(), eps, m, k, po, so, py, sy,
          None if rows is None else rows._c)
    return total


def _like(shape, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    return _empty(shape, torch.bfloat16, device, stream)


def add_rms_norm(x, residual, weight, eps=1e-6, out=None, residual_out=None, stream=None):
    """r = x + residual (rounded to bfloat16) and its RMS norm, r * rsqrt(mean(r^2)
    + eps) * weight: x, residual bfloat16 [M, K] (rows may be strided, K a multiple
    of 16), weight bfloat16 [K].  Without a residual (None) r is x, or a copy of it
    where the normed rows go over x.  Returns (normed, r); either may be written over
    one of the inputs (``out``, ``residual_out``)."""
    given = _input(x)
    if out is None:
        out = _like(x.shape, given[0], stream)
    return out, _norm(given, x, residual, weight, eps, residual_out, out, None, stream)


def add_rms_norm_quantize(x, residual, weight, eps=1e-6, global_scale=1.0, out=None, residual_out=None,
                          stream=None):
    """As ``add_rms_norm``, with the normed rows rounded once, to NVFP4 with the
    given global scale (K a multiple of 256).  Returns (Fp4Rows, r)."""
    given = dev, m, k, _, _ = _input(x)
    if k == 0 or k % 256:
        raise ValueError("K must be a positive multiple of 256, got %d" % k)
    out = _rows_out(out, m, k, global_scale, dev, stream)
    return out, _norm(given, x, residual, weight, eps, residual_out, None, out, stream)


def _check_product(a, w):
    if not (isinstance(a, Fp4Rows) and isinstance(w, Fp4Weight)):
        raise TypeError("a product is of Fp4Rows and an Fp4Weight, got %s and %s" % (type(a).__name__, type(w).__name__))
    if a._shape[1] != w._shape[1] or a._device != w._device:
        raise ValueError("rows %s on %s do not fit a weight %s on %s" % (a.shape, a.device, w.shape, w.device))


def _product(a, w, swiglu, out, stream):
    _check_product(a, w)
    shape = (a._shape[0], w._shape[0] // 2 if swiglu else w._shape[0])
    if out is None:
        out = _like(shape, a._device, stream)
    elif out.dtype != torch.bfloat16 or out.shape != shape or not out.is_contiguous() or out.device != a._device:
        raise ValueError("out must be a contiguous bfloat16 tensor of shape %s on %s" % (shape, a._device))
    _call("nvfp4_linear_w4a4", a._device, stream, a._c, a._shape[0], w._c, swiglu, out.data_ptr(), None)
    return out


def linear_w4a4(a, w, out=None, stream=None):
    """y[M, N] bfloat16 = the rows a (Fp4Rows [M, K]) through the weight w
    (Fp4Weight [N, K]); of a stacked weight the segments' outputs side by side."""
    return _product(a, w, 0, out, stream)


def linear_w4a4_swiglu(a, w, out=None, stream=None):
    """y[M, N/2] bfloat16 = silu(gate) * up, w holding the gate's rows and then the
    up projection's (N a multiple of 256)."""
    return _product(a, w, 1, out, stream)


def linear_w4a4_swiglu_quantize(a, w, global_scale=1.0, out=None, stream=None):
    """As ``linear_w4a4_swiglu``, its fp32 results rounded once, to NVFP4 with the
    given global scale (N a multiple of 512).  Returns Fp4Rows [M, N/2]."""
    _check_product(a, w)
    n = w._shape[0]
    if n % 512:
        raise ValueError("N must be a multiple of 512, got %d" % n)
    out = _rows_out(out, a._shape[0], n // 2, global_scale, a._device, stream)
    _call("nvfp4_linear_w4a4", a._device, stream, a._c, a._shape[0], w._c, 1, None, out._c)
    return out
