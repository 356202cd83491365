"""Outputs over inputs and over one another: refused on the host before a device is touched, and nothing else is.

The addresses are made up: what is let through ends at the missing device, so those tests are for machines without one.
"""
import ctypes
import random

import pytest
import torch

from test_w4a4_abi import INVALID, lib, rows, weight  # noqa: F401

DEVICE = -5
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses, let through")

X, R, W, O, Y, Z = (0x10000000 * i for i in range(1, 7))           # far apart


def norm(lib, x=X, xs=512, r=R, rs=512, w=W, m=40, k=512, ro=O, ros=512, y=Y, ys=512, out=None):
    return lib.nvfp4_add_rms_norm(x, xs, r, rs, w, 1e-6, m, k, ro, ros, y, ys, out, None)


def test_norm_refuses(lib):
    for other in (dict(y=X + 16), dict(y=X, ys=1024), dict(y=X + 1024), dict(ro=X + 1024), dict(ro=R - 1024), dict(ro=R, ros=520),
                  dict(y=O), dict(y=O + 39 * 1024), dict(ro=Y, ros=1024), dict(y=W), dict(y=W - 39 * 1024), dict(ro=W + 512),
                  dict(m=1, y=X + 512), dict(m=1, y=O), dict(r=X + 1024, y=X), dict(r=None, ro=None, y=X + 16)):
        assert norm(lib, **other) == INVALID, other
    for other in (rows(X, Z), rows(X + 39 * 1024 + 1008, Z), rows(R, Z), rows(O, Z), rows(W, Z), rows(Z, X), rows(Z, O + 1024),
                  rows(Z, Z + 40 * 256 - 16)):
        assert norm(lib, y=None, out=other) == INVALID


@no_gpu
def test_norm_lets_through(lib):
    for other in (dict(), dict(y=X), dict(y=R), dict(ro=X), dict(ro=R), dict(y=X, ro=R), dict(y=R, ro=X), dict(r=X), dict(r=X, y=X),
                  dict(m=1, y=X, ys=9), dict(y=X + 40 * 1024), dict(y=X - 40 * 1024), dict(xs=1024, y=X + 1024, ys=1024),
                  dict(xs=2048, y=X + 1024, ys=2048, ro=X + 2048, ros=2048), dict(xs=2048, y=X + 1024, ys=4096),
                  dict(r=None, ro=None, y=X), dict(r=None, ro=X)):
        assert norm(lib, **other) == DEVICE, other
    assert norm(lib, y=None, out=rows(Z, Z + 40 * 256)) == DEVICE


@no_gpu
def test_strided_views_exactly(lib):
    """Random pairs of strided matrices, byte by byte."""
    rng = random.Random(4)
    seen = set()
    for _ in range(4000):
        m, k = rng.randint(1, 6), 16 * rng.randint(1, 4)
        sx, sy = (k + 8 * rng.randint(0, 24) for _ in range(2))
        if rng.random() < 0.4:
            sy = sx
        y = X + 16 * rng.randint(-70, 70)
        a = {X + 2 * (i * sx + j) for i in range(m) for j in range(k)}
        b = {y + 2 * (i * sy + j) for i in range(m) for j in range(k)}
        same = y == X and (m == 1 or sx == sy)
        want = INVALID if (a & b) and not same else DEVICE
        assert norm(lib, x=X, xs=sx, r=None, ro=None, m=m, k=k, y=y, ys=sy) == want, (m, k, sx, sy, y - X)
        seen.add((want, sx == sy, y > X, m > 1))
    assert len(seen) == 16


def test_quantize_refuses(lib):
    def call(x=X, stride=512, m=40, k=512, out=rows(Y, Z)):
        return lib.nvfp4_quantize_rows(x, stride, m, k, out, None)
    for other in (rows(X, Z), rows(Y, X), rows(X + 39 * 1024 + 1008, Z), rows(X - 40 * 256 + 16, Z), rows(Y, Y + 40 * 256 - 16)):
        assert call(out=other) == INVALID
    assert call(stride=4096, out=rows(X + 1024 - 16, Z), m=2) == INVALID
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(out=rows(Y, Y + 40 * 256)) == DEVICE
        # one row's codes in the gap of two strided rows
        assert call(stride=4096, out=rows(X + 1024, Z), m=2) == DEVICE


def test_linear_refuses(lib):
    m, n, k = 40, 512, 512

    def call(a=rows(X, R), w=None, swiglu=0, y=Y, out=None):
        w = weight(W, O, n, k) if w is None else w
        return lib.nvfp4_linear_w4a4(a, m, ctypes.byref(w), swiglu, y, out, None)
    codes, y_bytes = m * k // 2, m * n * 2
    for at in (X, X + codes - 16, X - y_bytes + 16, R, R + 16, W, W + n * k // 2 - 16, O, O + n * k // 16 - 16):
        assert call(y=at) == INVALID, hex(at)
        if at != X - y_bytes + 16:                                 # (which is the last of y's bytes, beyond the rows')
            assert call(swiglu=1, y=None, out=rows(at, Z)) == INVALID
            assert call(swiglu=1, y=None, out=rows(Z, at)) == INVALID
    assert call(swiglu=1, y=None, out=rows(Y, Y)) == INVALID       # codes over scales
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(y=X + codes) == DEVICE and call(y=X - y_bytes) == DEVICE
        assert call(a=rows(W, O)) == DEVICE                        # inputs may be the same
        assert call(swiglu=1, y=None, out=rows(Y, Y + m * n // 4)) == DEVICE


def test_layout_refuses(lib):
    n, k = 256, 512

    def call(s=X, b=Y, r=Z):
        return lib.nvfp4_w4a4_scale_layout(s, n, k, b, r, None)
    size = n * k // 16
    for other in (dict(b=X), dict(b=X + size - 16), dict(b=X - size + 16), dict(r=Y), dict(r=Y + size - 4)):
        assert call(**other) == INVALID, other
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(b=X + size) == DEVICE and call(r=Y + size) == DEVICE
