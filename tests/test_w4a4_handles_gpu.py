"""Fp4Rows and Fp4Weight as objects: what they say is what the kernels take, whatever becomes of them or of the tensors
that they were made of."""
import copy
import io

import pytest
import torch

import _w4a4_ref as ref
from test_w4a4_gpu import BF16, DEV, hidden, no_device_error, pkg, weight  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rows_do_not_change():
    x = hidden(4, 512, 1).to(DEV)
    made = pkg.quantize_rows(x, 2.0)
    given = pkg.Fp4Rows(made.codes, made.scales, 2.0)
    for rows in (made, given):
        for name, value in (("global_scale", 3.0), ("codes", made.codes), ("scales", made.scales), ("shape", (4, 256)),
                            ("device", DEV)):
            with pytest.raises(AttributeError):
                setattr(rows, name, value)
        assert rows.global_scale == 2.0 and rows.shape == (4, 512) and rows.device == x.device
    with pytest.raises(ValueError):
        pkg.quantize_rows(x, 3.0, out=made)


def test_a_weight_does_not_change():
    w = weight(256, 512, 2, gs=[3.0, 4.0], rows=[128, 128])[0]
    for name, value in (("codes", w.codes.clone()), ("scales", w.scales.clone()), ("global_scales", [1.0, 1.0]),
                        ("segment_rows", [256]), ("shape", (128, 512)), ("device", DEV)):
        with pytest.raises(AttributeError):
            setattr(w, name, value)
    w.global_scales[0], w.segment_rows[0] = 7.0, 16                # (lists of the caller's own)
    assert w.global_scales == [3.0, 4.0] and w.segment_rows == [128, 128]


def duplicates(thing):
    f = io.BytesIO()
    torch.save(thing, f)
    f.seek(0)
    return [copy.deepcopy(thing), torch.load(f, weights_only=False), copy.deepcopy({"layer": [thing]})["layer"][0]]


def test_copies_have_memory_of_their_own():
    """A copy works on after the original's memory is gone and written over, and does not see what is done to it."""
    x = hidden(5, 512, 3).to(DEV)
    made = pkg.quantize_rows(x, 20.0)
    given = pkg.Fp4Rows(made.codes.clone(), made.scales.clone(), 20.0)
    w = weight(256, 512, 4, gs=[30.0, 40.0], rows=[128, 128])[0]
    w.name = "layer 0"
    want = pkg.linear_w4a4(made, w)
    torch.cuda.synchronize()
    rows, weights = duplicates(made) + duplicates(given), duplicates(w)
    for c in rows:
        assert c._c != made._c and c._c != given._c
        assert c.codes.data_ptr() not in (made.codes.data_ptr(), given.codes.data_ptr())
        assert c.shape == (5, 512) and c.global_scale == 20.0
        assert torch.equal(c.codes, made.codes) and torch.equal(ref.plain_scales(c), ref.plain_scales(made))
    for c in weights:
        assert c._c != w._c and c.codes.data_ptr() != w.codes.data_ptr() and c.scales.data_ptr() != w.scales.data_ptr()
        assert c.global_scales == [30.0, 40.0] and c.segment_rows == [128, 128] and c.name == "layer 0"
    for t in (made.codes, made.scales, given.codes, given.scales, w.codes, w.scales):
        t.zero_()
    del made, given, w, t
    for c in rows:
        for v in weights:
            assert torch.equal(pkg.linear_w4a4(c, v), want)


def test_a_shallow_copy_shares_the_memory():
    x = hidden(5, 512, 5).to(DEV)
    a, w = pkg.quantize_rows(x, 20.0), weight(128, 512, 6)[0]
    b, v = copy.copy(a), copy.copy(w)
    assert b.codes.data_ptr() == a.codes.data_ptr() and v.codes.data_ptr() == w.codes.data_ptr()
    want = pkg.linear_w4a4(a, w)
    del a, w
    assert torch.equal(pkg.linear_w4a4(b, v), want)


def test_the_memory_stays_where_the_callers_tensors_move():
    packed = torch.randint(0, 256, (128, 256), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).to(DEV)
    scale = torch.full((128, 32), 0x38, dtype=torch.uint8, device=DEV)
    w = pkg.Fp4Weight(packed, scale, 4.0)
    a = pkg.quantize_rows(hidden(3, 512, 7).to(DEV), 20.0)
    b = pkg.Fp4Rows(a.codes, a.scales, 20.0)
    want = pkg.linear_w4a4(b, w)
    at = w.codes.data_ptr()
    packed.data = torch.zeros_like(packed)
    del a
    assert w.codes.data_ptr() == at
    for _ in range(8):
        torch.zeros((128, 256), dtype=torch.uint8, device=DEV)
    assert torch.equal(pkg.linear_w4a4(b, w), want)
    # what is copied into the weight's memory is what later calls read
    w.codes.zero_()
    torch.cuda.synchronize()
    assert bool((pkg.linear_w4a4(b, w) == 0).all())
