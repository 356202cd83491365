"""Global scales at the ends of fp32, on the host (made-up addresses: what is let through ends at the missing device)."""
import ctypes
import struct

import pytest
import torch

from test_w4a4_abi import INVALID, lib, rows, weight  # noqa: F401
from nvfp4_block_scaled_linear_gb300 import w4a4

DEVICE = -5
X, R, W, O, Y = (0x10000000 * i for i in range(1, 6))


def product(lib, gs_a, gs_w):
    w = weight(W, O, 512, 512, gs_w, [512 // len(gs_w)] * len(gs_w))
    return lib.nvfp4_linear_w4a4(rows(X, R, gs_a), 4, ctypes.byref(w), 0, Y, None, None)


def test_reciprocals_below_the_normal_range(lib):
    for a, w in ((2.0 ** 64, 2.0 ** 63), (3e20, 3e20), (2.0 ** 100, 2.0 ** 48), (3e38, 1.0)):
        assert product(lib, a, [w]) == INVALID and product(lib, a, [1e-3, w]) == INVALID
    if not torch.cuda.is_available():
        for a, w in ((2.0 ** 63, 2.0 ** 63), (1.0, 8e37), (2.0 ** -64, 2.0 ** -63), (1e-20, 3e-19)):
            assert product(lib, a, [w]) == DEVICE, (a, w)


@pytest.mark.parametrize("value", [0.0, -1.0, float("nan"), float("inf"), float("-inf"), 1e39, 3.4028236e38, 1e300, 1e-46, 7e-46, 5e-324])
def test_the_binding_refuses_what_fp32_does_not_hold(value):
    with pytest.raises(ValueError):
        w4a4._scale(value, "global_scale")
    with pytest.raises(ValueError):
        w4a4.new_fp4_rows(1, 256, value, device="cuda:0")


@pytest.mark.parametrize("value", [3.4028234663852886e38, 3.40282352e38, 1.4e-45, 7.1e-46, 1, 448.0])
def test_the_binding_takes_what_fp32_holds(value):
    assert w4a4._scale(value, "global_scale") == value
    gs = struct.unpack("f", w4a4._pack_rows(X, R, value)[16:20])[0]
    assert 0.0 < gs < float("inf")


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_rows_are_of_a_cuda_device(device):
    with pytest.raises(ValueError):
        w4a4.new_fp4_rows(4, 256, device=device)


def test_out_is_rows():
    for out in (torch.empty((4, 256)), (1, 2), "rows"):
        with pytest.raises(TypeError):
            w4a4._rows_out(out, 4, 256, 1.0, torch.device("cuda:0"), None)
