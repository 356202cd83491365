"""The NVFP4 x NVFP4 operators against 64-bit forms."""
import pytest
import torch

import _w4a4_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("nvfp4_block_scaled_linear_gb300")
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert pkg.w4a4_error() == 0


def hidden(m, k, seed, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g) * torch.exp(spread * torch.randn((m, 1), generator=g))
    x[:, torch.randint(0, k, (2,), generator=g)] *= 7.0
    return x.to(BF16)


def weight(n, k, seed, gs=None, rows=None):
    """(handle, codes times scales fp64 [n, k], global scale of each row)."""
    g = torch.Generator().manual_seed(seed)
    packed = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scale = torch.randint(0x20, 0x51, (n, k // 16), generator=g, dtype=torch.uint8)
    gs = [8.0 * k ** 0.5] if gs is None else gs
    rows = [n] if rows is None else rows
    w = pkg.Fp4Weight(packed.to(DEV), scale.to(DEV), gs, rows)
    per_row = torch.cat([torch.full((r,), s, dtype=torch.float64) for r, s in zip(rows, gs)])
    return w, ref.values_of(packed, scale), per_row


def check_quantized(rows, x, gs):
    want, byte = ref.quantize(x, gs)
    assert torch.equal(ref.plain_scales(rows), byte)
    assert torch.equal(ref.E2M1[ref.unpack(rows.codes)], want)     # (-0 equals 0)


@pytest.mark.parametrize("m, k", [(1, 256), (3, 512), (31, 1280), (127, 256), (128, 256), (129, 768), (300, 5120),
                                  (5, 17408)])
@pytest.mark.parametrize("gs", [1.0, 336.0, 0.37])
def test_quantize_rows_by_bits(m, k, gs):
    x = hidden(m, k, m * k)
    check_quantized(pkg.quantize_rows(x.to(DEV), gs), x.float(), gs)


def test_quantize_rows_extremes():
    """Blocks of zeros, of values whose scale rounds to zero or is subnormal, of one spike, beyond the largest
    scale, and values on the borders between codes."""
    x = torch.randn((40, 256), generator=torch.Generator().manual_seed(1))
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= 1e-30
    x[3] = 2.0 ** -8
    x[4] = 6 * 2.0 ** -10                                          # a scale of half its smallest
    x[5, ::16] = 3e4
    x[6] *= 1e20
    x[7] = 3.3e38
    x[8:24] = torch.arange(16.0)[:, None] * 0.25 * torch.tensor([1.0, -1.0]).repeat(128)
    x[8:24, ::16] = 6.0                                            # the scale is 1: every quarter
    x[24:40] *= 2.0 ** torch.arange(-12.0, 4.0)[:, None]
    x = x.to(BF16)
    check_quantized(pkg.quantize_rows(x.to(DEV), 1.0), x.float(), 1.0)


def test_quantize_rows_not_finite():
    x = hidden(6, 512, 3)
    x[1, 17], x[2, 40], x[3, 511] = float("nan"), float("inf"), float("-inf")
    rows = pkg.quantize_rows(x.to(DEV), 2.0)
    check_quantized(rows, x.float(), 2.0)
    w, _, _ = weight(128, 512, 4)
    y = pkg.linear_w4a4(rows, w).cpu()
    assert torch.equal(torch.isnan(y).any(1), torch.tensor([False, True, True, True, False, False]))
    assert torch.isnan(y[1:4]).all()
    # a finite value that the scale takes beyond fp32
    x = hidden(2, 256, 4)
    x[1, 5] = 3e38
    check_quantized(pkg.quantize_rows(x.to(DEV), 1e3), x.float(), 1e3)


def test_quantize_rows_strided_and_padding():
    base = hidden(70, 1024, 5).to(DEV)
    x = base[3:63, 256:768]
    out = pkg.new_fp4_rows(60, 512, 3.0)
    out.scales.fill_(0xAB)
    assert pkg.quantize_rows(x, 3.0, out=out) is out
    check_quantized(out, x.float().cpu(), 3.0)
    left = torch.ones(out.scales.numel(), dtype=torch.bool)
    left[ref.scale_index(60, 512).flatten()] = False
    assert bool((out.scales.cpu().flatten()[left] == 0xAB).all())


# ------------------------------------------------------------------ the norm
def norm64(r, w, eps):
    f = r.double()
    return f / (f.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


# fp32 steps around the one rounding to bf16: the sum's tree and rsqrt, three products
FP32 = 2.0 ** -18


@pytest.mark.parametrize("m, k", [(1, 16), (2, 48), (7, 256), (33, 5120), (3, 8208), (2, 16400), (2, 32768), (300, 2048)])
@pytest.mark.parametrize("add", [True, False])
def test_add_rms_norm(m, k, add):
    x, res = hidden(m, k, k + m), hidden(m, k, k + m + 1)
    w = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(2))).to(BF16)
    y, r = pkg.add_rms_norm(x.to(DEV), res.to(DEV) if add else None, w.to(DEV), 1e-5)
    want_r = (x.float() + res.float()).to(BF16) if add else x
    assert torch.equal(r.cpu(), want_r)
    want = norm64(want_r, w, 1e-5)
    assert bool(((y.cpu().double() - want).abs() <= want.abs() * (2.0 ** -8 + FP32)).all())


@pytest.mark.parametrize("m, k", [(1, 256), (5, 5120), (130, 768), (2, 32768)])
def test_add_rms_norm_quantize(m, k):
    gs = 200.0
    x, res = hidden(m, k, 3 * k + m), hidden(m, k, 3 * k + m + 1)
    w = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(2))).to(BF16)
    rows, r = pkg.add_rms_norm_quantize(x.to(DEV), res.to(DEV), w.to(DEV), 1e-6, gs)
    want_r = (x.float() + res.float()).to(BF16)
    assert torch.equal(r.cpu(), want_r)
    want = norm64(want_r, w, 1e-6).unflatten(1, (-1, 16)) * gs
    s = ref.e4m3(ref.plain_scales(rows))
    # (a row's largest can be sqrt(k) before the weight: times gs / 6 that passes 448, where scales end)
    top = (want.abs().amax(-1) / 6).clamp(max=448.0)
    # the scale: half an e4m3 step from the largest, a step of 2^-9 below its normal range
    assert bool(((s - top).abs() <= (top * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + FP32) + top * FP32).all())
    code = ref.E2M1[ref.unpack(rows.codes)].unflatten(1, (-1, 16))
    q = want / s.clamp(min=2.0 ** -9)[:, :, None]
    half = torch.where(q.abs() <= 2, 0.25, torch.where(q.abs() <= 4, 0.5, 1.0))
    over = torch.where(top[:, :, None] == 448.0, (q.abs() - 6).clamp(min=0.0), torch.zeros_like(q))
    assert bool(((code - q).abs()[s > 0] <= (half * (1 + FP32) + q.abs() * FP32 + over)[s > 0]).all())


def test_norm_in_place_and_strided():
    base = hidden(50, 1536, 9).to(DEV)
    x, res = base[:40, 256:768].clone(), base[5:45, 1024:1536]
    w = torch.ones(512, dtype=BF16, device=DEV)
    want_y, want_r = pkg.add_rms_norm(x, res.contiguous(), w)
    other = base.clone()
    res = other[5:45, 1024:1536]
    y, r = pkg.add_rms_norm(x, res, w, out=x, residual_out=res)
    assert y is x and r is res and torch.equal(y, want_y) and torch.equal(r, want_r)
    other[5:45, 1024:1536] = base[5:45, 1024:1536]
    assert torch.equal(other, base)                                # nothing around it was written


@pytest.mark.parametrize("m, k", [(1, 512), (40, 1536), (700, 4096)])
def test_outputs_over_either_input(m, k):
    x, res = hidden(m, k, 14).to(DEV), hidden(m, k, 15).to(DEV)
    w = (1 + 0.1 * torch.randn(k, generator=torch.Generator().manual_seed(3))).to(BF16).to(DEV)
    want_y, want_r = pkg.add_rms_norm(x, res, w)
    rows, _ = pkg.add_rms_norm_quantize(x, res, w, 1e-6, 150.0)
    for swap in (False, True):
        a, b = x.clone(), res.clone()
        y, r = pkg.add_rms_norm(a, b, w, out=b if swap else a, residual_out=a if swap else b)
        assert torch.equal(y, want_y) and torch.equal(r, want_r)
        a, b = x.clone(), res.clone()
        q, r = pkg.add_rms_norm_quantize(a, b, w, 1e-6, 150.0, residual_out=a if swap else b)
        assert torch.equal(r, want_r) and torch.equal(q.codes, rows.codes)
        assert torch.equal(ref.plain_scales(q), ref.plain_scales(rows))
    a = x.clone()
    y, r = pkg.add_rms_norm(a, None, w, out=a, residual_out=res)    # no residual: the sum is x, copied
    assert torch.equal(r, x) and torch.equal(y, pkg.add_rms_norm(x, None, w)[0])


def test_norm_not_finite_rows_stay_apart():
    x = hidden(4, 512, 11)
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    w = torch.ones(512, dtype=BF16)
    y, _ = pkg.add_rms_norm(x.to(DEV), None, w.to(DEV))
    want = norm64(x[[0, 3]], w, 1e-6)
    assert bool(((y.cpu()[[0, 3]].double() - want).abs() <= want.abs() * (2.0 ** -8 + FP32)).all())
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 5])
    rows, _ = pkg.add_rms_norm_quantize(x.to(DEV), None, w.to(DEV))
    byte = ref.plain_scales(rows)
    assert bool((byte[1] == 0x7F).all()) and byte[2, 0] == 0x7F and bool((byte[[0, 3]] < 0x7F).all())


# ------------------------------------------------------------------ the products
def product64(rows, w64, per_row, gs):
    a = ref.values_of(rows.codes, ref.plain_scales(rows)).to(DEV)
    w = w64.to(DEV)
    scale = (1.0 / (gs * per_row)).to(DEV)
    return (a @ w.T) * scale, (a.abs() @ w.abs().T) * scale


SHAPES = [(1, 128, 256), (1, 5120, 6144), (2, 256, 512), (7, 640, 1280), (8, 8192, 5120), (9, 128, 17408), (32, 384, 2560),
          (64, 1024, 2048), (65, 128, 256), (100, 2560, 3840), (127, 256, 768), (128, 256, 512), (129, 128, 512),
          (255, 512, 1024), (256, 256, 256), (257, 768, 1536), (300, 2560, 5120), (515, 640, 2048), (1111, 8192, 1024),
          (2048, 5120, 512), (600, 5504, 256), (1300, 3968, 768), (1030, 8064, 1536), (900, 128, 256), (3500, 384, 512),
          (16, 128, 256), (17, 1024, 4352), (24, 640, 1024), (31, 256, 17408), (33, 640, 1024), (32, 16640, 256), (40, 20608, 512)]


@pytest.mark.parametrize("m, n, k", SHAPES, ids=str)
def test_linear(m, n, k):
    rows = pkg.quantize_rows(hidden(m, k, m + n + k).to(DEV), 64.0)
    w, w64, per_row = weight(n, k, n)
    y = pkg.linear_w4a4(rows, w)
    want, total = product64(rows, w64, per_row, 64.0)
    off = (y.double() - want).abs()
    assert bool((off <= want.abs() * 2.0 ** -8 + total * ref.product_bound(k)).all()), float((off / total).max())


def test_linear_segments():
    rows = pkg.quantize_rows(hidden(37, 512, 8).to(DEV), 10.0)
    w, w64, per_row = weight(1280, 512, 9, gs=[100.0, 3.0, 1e4, 55.5], rows=[16, 48, 960, 256])
    y = pkg.linear_w4a4(rows, w)
    want, total = product64(rows, w64, per_row, 10.0)
    assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + total * ref.product_bound(512)).all())


def test_every_scale_and_code():
    """Each finite scale with each code, on both sides: a row of the weight has one value, a row of activations a one."""
    k = 256
    scale = (torch.arange(128) % 127).to(torch.uint8)[:, None].repeat(1, k // 16)
    byte = torch.arange(16, dtype=torch.uint8).repeat(8)
    packed = (byte | byte << 4)[:, None].repeat(1, k // 2)
    w = pkg.Fp4Weight(packed.to(DEV), scale.to(DEV), 1.0)
    x = torch.zeros((128, k))
    x[torch.arange(128), torch.arange(128) * 2] = torch.arange(128) + 1.0
    rows = pkg.quantize_rows(x.to(BF16).to(DEV), 1.0)
    y = pkg.linear_w4a4(rows, w)
    want, _ = product64(rows, ref.values_of(packed, scale), torch.ones(128, dtype=torch.float64), 1.0)
    assert torch.equal(y.double(), want.to(BF16).double())         # single products: exact before the rounding
    # and the other way round
    rows = pkg.Fp4Rows(w.codes, w.scales, 1.0)
    g = ref.values_of(packed, scale)
    one = torch.full((128, k // 2), 0, dtype=torch.uint8)
    one[torch.arange(128), torch.arange(128)] = 2
    v = pkg.Fp4Weight(one.to(DEV), torch.full((128, k // 16), 0x38, dtype=torch.uint8, device=DEV), 1.0)
    y = pkg.linear_w4a4(rows, v)
    assert torch.equal(y.double().cpu(), (g @ ref.values_of(one, torch.full((128, k // 16), 0x38, dtype=torch.uint8)).T).to(BF16).double())


def gated64(rows, w64, per_row, gs, k):
    y, t = product64(rows, w64, per_row, gs)
    n = y.shape[1] // 2
    g, u = y[:, :n], y[:, n:]
    eg, eu = t[:, :n] * ref.product_bound(k), t[:, n:] * ref.product_bound(k)
    silu = g * torch.sigmoid(g)
    # |silu'| < 1.1; the fast exponential and division are off by a few 2^-23
    return silu * u, 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (silu * u).abs() * 2.0 ** -19 + 1e-30


GATED = [(1, 512, 256), (1, 34816, 512), (3, 1024, 2560), (32, 512, 5120), (100, 2048, 512), (128, 512, 512),
         (129, 1024, 256), (515, 1536, 1024), (700, 512, 3840),
         (8, 512, 17408), (17, 1536, 1024), (32, 34816, 512), (33, 1024, 1024), (40, 512, 256), (2, 40960, 256), (32, 40960, 1280), (9, 39424, 768), (90, 20480, 768)]


@pytest.mark.parametrize("m, n, k", GATED + [(5, 256, 512), (200, 768, 512)], ids=str)
def test_linear_swiglu(m, n, k):
    rows = pkg.quantize_rows(hidden(m, k, m + n + k).to(DEV), 30.0)
    w, w64, per_row = weight(n, k, n + 1, gs=[3.0 * k ** 0.5, 5.0 * k ** 0.5], rows=[n // 2, n // 2])
    y = pkg.linear_w4a4_swiglu(rows, w)
    want, err = gated64(rows, w64, per_row, 30.0, k)
    assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + err * (1 + 2.0 ** -8)).all())


@pytest.mark.parametrize("m, n, k", GATED, ids=str)
def test_linear_swiglu_quantize(m, n, k):
    out_gs = 40.0
    rows = pkg.quantize_rows(hidden(m, k, m + n + k).to(DEV), 30.0)
    w, w64, per_row = weight(n, k, n + 1, gs=[3.0 * k ** 0.5, 5.0 * k ** 0.5], rows=[n // 2, n // 2])
    h = pkg.linear_w4a4_swiglu_quantize(rows, w, out_gs)
    assert h.shape == (m, n // 2) and h.global_scale == out_gs
    want, err = gated64(rows, w64, per_row, 30.0, k)
    want, err = (want * out_gs).cpu().unflatten(1, (-1, 16)), (err * out_gs).cpu().unflatten(1, (-1, 16))
    s = ref.e4m3(ref.plain_scales(h))
    top, slack = (want.abs().amax(-1) / 6).clamp(max=448.0), err.amax(-1) / 6
    assert bool(((s - top).abs() <= ((top + slack) * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + FP32) + slack).all())
    code = ref.E2M1[ref.unpack(h.codes)].unflatten(1, (-1, 16))
    v = code * s[:, :, None]
    q = want.abs() + err
    # half a code's step, what exceeds the largest code, and the product's own error
    half = torch.where(q <= 2 * s[:, :, None], 0.25, torch.where(q <= 4 * s[:, :, None], 0.5, 1.0)) * s[:, :, None]
    over = (q - 6 * s[:, :, None]).clamp(min=0.0)
    some = (s > 0)[:, :, None].expand_as(v)
    assert bool(((v - want).abs() <= half * (1 + FP32) + over + err)[some].all())


def test_feed_forward_block():
    """norm -> gate and up -> down, as a layer runs them, against 64 bits over the rows that each step left."""
    m, k, inner = 45, 1024, 1536
    x, res = hidden(m, k, 21, 0.2).to(DEV), hidden(m, k, 22, 0.2).to(DEV)
    nw = torch.ones(k, dtype=BF16, device=DEV)
    gu, gu64, gu_gs = weight(2 * inner, k, 23)
    dn, dn64, dn_gs = weight(k, inner, 24)
    a, r = pkg.add_rms_norm_quantize(x, res, nw, 1e-6, 300.0)
    h = pkg.linear_w4a4_swiglu_quantize(a, gu, 90.0)
    y = pkg.linear_w4a4(h, dn)
    want, total = product64(h, dn64, dn_gs, 90.0)
    assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + total * ref.product_bound(inner)).all())
    # the whole against no quantisation of the activations: two roundings to 3 bits, 2^-4 of a block's largest each
    f = norm64(r.cpu(), nw.cpu(), 1e-6).to(DEV)
    z = f @ gu64.to(DEV).T / gu_gs.to(DEV)
    z = torch.nn.functional.silu(z[:, :inner]) * z[:, inner:]
    z = z @ dn64.to(DEV).T / dn_gs.to(DEV)
    assert float((y.double() - z).norm() / z.norm()) < 0.3


def test_no_rows():
    w, _, _ = weight(512, 256, 1)
    x = torch.empty((0, 256), dtype=BF16, device=DEV)
    nw = torch.ones(256, dtype=BF16, device=DEV)
    rows = pkg.quantize_rows(x)
    assert pkg.linear_w4a4(rows, w).shape == (0, 512)
    assert pkg.linear_w4a4_swiglu(rows, w).shape == (0, 256)
    assert pkg.linear_w4a4_swiglu_quantize(rows, w).shape == (0, 256)
    y, r = pkg.add_rms_norm(x, x, nw)
    assert y.shape == r.shape == (0, 256)
    assert pkg.add_rms_norm_quantize(x, None, nw)[0].shape == (0, 256)
