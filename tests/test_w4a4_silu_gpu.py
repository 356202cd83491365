"""silu of the gated products far below zero, where it ends slowly: fp32 holds it down to about -92.

One k of a row and of a weight is not zero, so that each sum is a single exact product: gate = -36 a b for block
scales a (of the row) in [1, 2) and b (of the weight) in [1, 4), from -36 to -253, exact in fp32.
"""
import pytest
import torch

from test_w4a4_gpu import BF16, DEV, no_device_error, pkg  # noqa: F401

pytestmark = pytest.mark.gpu

K = 256


def mantissas(count):
    """e4m3 bytes of 1 + j/8, for 8 and more of twice that as well, in turn, and their values."""
    j = torch.arange(count) % 16
    return (0x38 + j).to(torch.uint8), (1.0 + (j % 8).double() / 8) * 2.0 ** (j // 8)


def tail(m, n, up_gs):
    """Rows [m, K], a pair [2n, K] and the exact gate and up [m, n]: the gate the same over 16 outputs."""
    byte, a = mantissas(8)
    byte, a = byte.repeat(m // 8 + 1)[:m], a.repeat(m // 8 + 1)[:m]
    rows = pkg.new_fp4_rows(m, K, 1.0)
    rows.codes.zero_()
    rows.codes[:, 0] = 0x07                                         # 6 at k = 0
    rows.scales.fill_(0x38)
    r = torch.arange(m)
    rows.scales.view(-1)[((r // 128) * (K // 64) * 512 + (r % 32) * 16 + (r // 32) % 4 * 4).to(DEV)] = byte.to(DEV)
    packed = torch.zeros((2 * n, K // 2), dtype=torch.uint8)
    scale = torch.full((2 * n, K // 16), 0x38, dtype=torch.uint8)
    packed[:n, 0], packed[n:, 0] = 0x0F, 0x02                       # gate -6, up 1
    byte, b = mantissas(n // 16)
    scale[:n, 0] = byte.repeat_interleave(16)
    w = pkg.Fp4Weight(packed.to(DEV), scale.to(DEV), [1.0, up_gs], [n, n])
    gate = -36.0 * a[:, None] * b.repeat_interleave(16)[None, :]
    up = (6.0 * a / up_gs)[:, None].expand(m, n)
    return rows, w, gate, up


def sizes():
    """Rows for the kernels of up to 32, of 33 and more, and of many rows (more tiles of 128 rows by 128 outputs
    than SMs), whatever the device."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return [3, 32, 100, 128 * (sms // 2 + 1) + 5]


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("up_gs", [1.0, 2.0 ** -30])
def test_the_tail_of_silu(which, up_gs):
    m, n = sizes()[which], 256
    rows, w, gate, up = tail(m, n, up_gs)
    want = gate * torch.exp(gate) / (1 + torch.exp(gate)) * up
    y = pkg.linear_w4a4_swiglu(rows, w).cpu().double()
    # the rounding to bf16 (below its normal range half of 2^-133); an exponential of the fp32 product g log2 e,
    # off by 2^-18 of its value near g = -100, its constant by 2^-18 more, the rest a few 2^-23; where the
    # exponential is below fp32's normal range a few 2^-149, times g and up
    bound = want.abs() * (2.0 ** -8 + 2.0 ** -16) + 2.0 ** -134 + 4 * 2.0 ** -149 * gate.abs() * up.abs()
    off = (y - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    assert bool((y[(gate > -92)] != 0).all())


@pytest.mark.parametrize("which", range(4))
def test_the_tail_of_silu_quantised(which):
    m, n = sizes()[which], 256
    rows, w, gate, up = tail(m, n, 2.0 ** -100)
    want = gate * torch.exp(gate) / (1 + torch.exp(gate)) * up
    gs = 2.0 ** 20
    h = pkg.linear_w4a4_swiglu_quantize(rows, w, gs)
    r, b = torch.arange(m)[:, None], torch.arange(n // 16)[None, :]
    at = ((r // 128) * (n // 64) + b // 4) * 512 + (r % 32) * 16 + (r // 32) % 4 * 4 + b % 4
    s = h.scales.cpu().view(-1)[at].view(torch.float8_e4m3fn).double()
    codes = h.codes.cpu()
    # 16 equal values: codes of 6 (7, or negative 15) beside a scale within half an e4m3 step of a sixth of them
    top = want[:, ::16].abs() * gs / 6
    normal = (top >= 2.0 ** -6) & (top <= 440.0)
    assert bool(((gate[:, ::16] < -88) & normal).any()) and bool(((gate[:, ::16] > -86) & normal).any())
    assert bool(((s - top).abs() <= top * (2.0 ** -4 + 2.0 ** -12))[normal].all())
    eight = codes.view(m, n // 16, 8)
    assert bool((eight[normal] == 0xFF).all())


def test_far_beyond_and_not_finite():
    """Gates whose exponential is zero, infinite ones, NaN: as g / (1 + exp(-g)) has them."""
    m, n = 2, 256
    rows, w, _, _ = tail(m, n, 1.0)
    far = pkg.Fp4Weight(w.codes, torch.full((2 * n, K // 16), 0x7E, dtype=torch.uint8, device=DEV), [1.0, 1.0], [n, n])
    y = pkg.linear_w4a4_swiglu(rows, far).cpu()
    assert bool((y == 0).all())                                    # g = -16128
    rows.scales.fill_(0x7F)
    assert bool(torch.isnan(pkg.linear_w4a4_swiglu(rows, far)).all())
    # up = 6 x 448 x 448 x 1e35, infinite in fp32: -0 times infinity
    rows.scales.fill_(0x7E)
    huge = pkg.Fp4Weight(w.codes, torch.full((2 * n, K // 16), 0x7E, dtype=torch.uint8, device=DEV), [1.0, 1e-35], [n, n])
    assert bool(torch.isnan(pkg.linear_w4a4_swiglu(rows, huge)).all())
