"""The NVFP4 x NVFP4 operators' C ABI on the host: every declared function is exported, the packed structures
have the C layout, and bad arguments are rejected before a device is touched (no call here gets past validation)."""
import ctypes

import pytest

from nvfp4_block_scaled_linear_gb300 import _lib, w4a4
from nvfp4_block_scaled_linear_gb300 import build as cuda_build

A = 0x10000           # fake, 16-byte aligned, never dereferenced
INVALID, MISALIGNED, SHAPE = -1, -2, -3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    _lib.load_library()
    return w4a4._library()


class _Rows(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("global_scale", ctypes.c_float)]


class _Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("segments", ctypes.c_int32), ("global_scale", ctypes.c_float * 8), ("segment_rows", ctypes.c_int64 * 8)]


def rows(codes=A, scales=A, gs=1.0):
    return ctypes.byref(_Rows(codes, scales, gs))


def weight(codes=A, scales=A, n=512, k=512, gs=(1.0,), parts=None):
    parts = [n] if parts is None else parts
    w = _Weight(codes, scales, n, k, len(parts))
    for i, (s, r) in enumerate(zip(gs, parts)):
        w.global_scale[i], w.segment_rows[i] = s, r
    return w


def test_exports_and_constants(lib):
    names = w4a4.w4a4_header_functions()
    assert len(names) == 6, names
    for n in names:
        assert hasattr(lib, n)
    text = open(w4a4.W4A4_HEADER).read()
    assert "#define NVFP4_W4A4_TIMEOUT %du" % w4a4.W4A4_TIMEOUT in text


def test_packed_structures_have_the_c_layout():
    a = w4a4._pack_rows(1, 2, 3.5)
    assert len(a) == ctypes.sizeof(_Rows) and a[:20] == bytes(_Rows(1, 2, 3.5))[:20]
    w = weight(1, 2, 96, 256, (1.5, 2.5), [32, 64])
    b = w4a4._pack_weight(1, 2, 96, 256, 2, 1.5, 2.5, *[0.0] * 6, 32, 64, *[0] * 6)
    assert len(b) == ctypes.sizeof(_Weight)
    for name, _ in _Weight._fields_:
        f = getattr(_Weight, name)
        assert b[f.offset:f.offset + f.size] == bytes(w)[f.offset:f.offset + f.size], name


def test_scale_bytes(lib):
    f = lib.nvfp4_w4a4_scale_bytes
    assert f(1, 256) == 128 * 16 and f(128, 256) == 128 * 16 and f(129, 512) == 256 * 32 and f(0, 256) == 0
    assert f(1, 0) == 0 and f(1, 128) == 0 and f(-1, 256) == 0 and f(1, -256) == 0 and f(1 << 31, 256) == 0


def test_scale_layout_rejects(lib):
    def call(s=A, n=128, k=256, b=A, r=A):
        return lib.nvfp4_w4a4_scale_layout(s, n, k, b, r, None)
    assert call(s=None) == INVALID and call(b=None) == INVALID and call(r=None) == INVALID
    assert call(n=0) == INVALID and call(n=-128) == INVALID and call(k=0) == INVALID
    assert call(n=64) == SHAPE and call(k=128) == SHAPE and call(n=(1 << 30) + 128) == SHAPE
    assert call(s=A + 8) == MISALIGNED and call(b=A + 4) == MISALIGNED and call(r=A + 2) == MISALIGNED


def test_quantize_rows_rejects(lib):
    def call(x=A, stride=256, m=2, k=256, out=rows()):
        return lib.nvfp4_quantize_rows(x, stride, m, k, out, None)
    assert call(x=None) == INVALID and call(out=None) == INVALID
    assert call(out=rows(codes=None)) == INVALID and call(out=rows(scales=None)) == INVALID
    for gs in (0.0, -1.0, NAN, INF, -INF):
        assert call(out=rows(gs=gs)) == INVALID
    assert call(x=A + 8) == MISALIGNED and call(out=rows(codes=A + 8)) == MISALIGNED and call(out=rows(scales=A + 4)) == MISALIGNED
    assert call(m=-1) == INVALID and call(k=0) == INVALID and call(k=128) == SHAPE and call(k=257) == SHAPE
    assert call(m=(1 << 30) + 1) == SHAPE
    assert call(stride=248) == INVALID and call(stride=260) == MISALIGNED and call(stride=1 << 31) == SHAPE
    assert call(stride=-256) == INVALID
    assert call(m=0, x=None, out=None) == 0


def test_add_rms_norm_rejects(lib):
    def call(x=A, xs=256, r=A, rs=256, w=A, eps=1e-6, m=2, k=256, ro=A, ros=256, y=A, ys=256, out=None):
        return lib.nvfp4_add_rms_norm(x, xs, r, rs, w, eps, m, k, ro, ros, y, ys, out, None)
    assert call(x=None) == INVALID and call(w=None) == INVALID and call(y=None) == INVALID
    assert call(out=rows()) == INVALID                              # y and rows
    assert call(y=None, out=rows(gs=0.0)) == INVALID and call(y=None, out=rows(codes=A + 8)) == MISALIGNED
    for eps in (-1e-6, NAN, INF):
        assert call(eps=eps) == INVALID
    for name, stride in (("x", "xs"), ("r", "rs"), ("ro", "ros"), ("y", "ys")):
        assert call(**{name: A + 8}) == MISALIGNED
        assert call(**{stride: 255}) == INVALID and call(**{stride: 260}) == MISALIGNED and call(**{stride: 1 << 31}) == SHAPE
    assert call(w=A + 2) == MISALIGNED
    assert call(k=24) == SHAPE and call(k=0) == INVALID and call(m=-1) == INVALID and call(k=32768 + 16) == SHAPE
    assert call(k=272, y=None, out=rows()) == SHAPE                 # bf16 rows may have it
    assert call(m=0, x=None, y=None, r=None, ro=None) == 0


def test_linear_rejects(lib):
    def call(a=rows(), m=2, w=weight(), swiglu=0, y=A, out=None):
        return lib.nvfp4_linear_w4a4(a, m, None if w is None else ctypes.byref(w), swiglu, y, out, None)
    assert call(a=None) == INVALID and call(w=None) == INVALID and call(y=None) == INVALID
    assert call(m=-1) == INVALID and call(m=(1 << 30) + 1) == SHAPE
    assert call(a=rows(gs=NAN)) == INVALID and call(a=rows(codes=A + 8)) == MISALIGNED and call(a=rows(scales=None)) == INVALID
    assert call(w=weight(codes=None)) == INVALID and call(w=weight(scales=None)) == INVALID
    assert call(w=weight(codes=A + 4)) == MISALIGNED and call(w=weight(scales=A + 8)) == MISALIGNED
    assert call(w=weight(n=0)) == INVALID and call(w=weight(n=64)) == SHAPE and call(w=weight(n=192)) == SHAPE
    assert call(w=weight(k=128)) == SHAPE and call(w=weight(k=0)) == INVALID
    for gs in (0.0, -2.0, NAN, INF):
        assert call(w=weight(gs=(gs,))) == INVALID
    assert call(w=weight(parts=[496])) == INVALID and call(w=weight(parts=[500])) == SHAPE and call(w=weight(gs=(1, 1), parts=[256, 128])) == INVALID
    assert call(w=weight(gs=(1, 1), parts=[504, 8])) == SHAPE and call(w=weight(gs=(1, 1), parts=[512, 0])) == INVALID
    assert call(w=weight(gs=(), parts=[])) == INVALID
    assert call(a=rows(gs=1e-30), w=weight(gs=(1e-30,))) == INVALID and call(a=rows(gs=1e30), w=weight(gs=(1e30,))) == INVALID
    w = weight()
    w.segments = 9
    assert call(w=w) == INVALID
    assert call(w=weight(n=384), swiglu=1) == SHAPE                 # gate and up of 192 rows
    assert call(out=rows(), y=None) == INVALID                      # NVFP4 rows are of the gated product
    assert call(w=weight(n=768), swiglu=1, y=None, out=rows()) == SHAPE
    assert call(swiglu=1, out=rows()) == INVALID                    # y and rows
    assert call(swiglu=1, y=None, out=rows(gs=INF)) == INVALID
    assert call(y=A + 8) == MISALIGNED
    assert call(m=0, a=None, y=None) == 0


def test_status_rejects(lib):
    assert lib.nvfp4_w4a4_status(None, 0) == INVALID


def test_no_multicast_copy():
    """Every CTA copies its own tiles; what is multicast is a commit's arrival on the pair's barriers."""
    import glob
    import os
    here = os.path.join(os.path.dirname(os.path.abspath(w4a4.__file__)), "csrc_w4a4")
    sources = glob.glob(os.path.join(here, "*.cu*"))
    assert len(sources) > 5
    for f in sources:
        for line in open(f):
            assert "cp.async.bulk" not in line or "multicast" not in line
