"""Plain forms of the NVFP4 x NVFP4 operators, on the CPU: the quantisation in the fp32 steps of
include/nvfp4_w4a4.h, everything else in 64 bits."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def e4m3(byte):
    return byte.contiguous().view(torch.float8_e4m3fn).double()


def scale_index(rows, k):
    """Byte of the scale of row r and 16-block b in the blocked order, int64 [rows, k/16]."""
    r, b = torch.arange(rows)[:, None], torch.arange(k // 16)[None, :]
    return ((r // 128) * (k // 64) + b // 4) * 512 + (r % 32) * 16 + (r // 32) % 4 * 4 + b % 4


def unpack(codes):
    c = codes.cpu()
    return torch.stack([c & 15, c >> 4], -1).flatten(1).long()


def values_of(codes, scales):
    """codes [m, k/2], scales [m, k/16] (plain order) -> codes times scales, fp64 [m, k]."""
    v = E2M1[unpack(codes)]
    return (v.unflatten(1, (-1, 16)) * e4m3(scales.cpu())[:, :, None]).flatten(1)


def plain_scales(rows):
    """The scales of Fp4Rows (or of a weight's handle) in plain order, uint8 [m, k/16]."""
    m, k = rows.shape
    return rows.scales.cpu().flatten()[scale_index(m, k)]


def nearest_e2m1(q):
    """Code magnitudes (0..7) of |q|, fp32, ties to even, saturating."""
    a = q.abs().double()
    v = E2M1[:8]
    mid = (v[1:] + v[:-1]) / 2
    low, high = torch.searchsorted(mid, a.contiguous()), torch.searchsorted(mid, a.contiguous(), right=True)
    return torch.where(low % 2 == 0, low, high)


def quantize(x, gs):
    """fp32 [m, k] on the CPU -> (signed code values fp64 [m, k], scale bytes [m, k/16])."""
    gs = torch.tensor(gs, dtype=torch.float32)
    t = x.unflatten(1, (-1, 16))
    top = t.abs().amax(-1) * gs
    scale = (top / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[:, :, None]
    q = (t * gs) / torch.where(s > 0, s, torch.ones_like(s))
    v = E2M1[nearest_e2m1(q)] * torch.where(q < 0, -1.0, 1.0)
    v = torch.where(s > 0, v, torch.zeros_like(v))
    bad = ~torch.isfinite(top)
    v[bad] = 0.0
    byte = scale.view(torch.uint8).clone()
    byte[bad] = 0x7F
    return v.flatten(1), byte


def product_bound(k):
    """The accumulation's error relative to the sum of |a w|: one fp32 rounding (possibly a truncation, 2^-23)
    for each MMA of 64 k, and as many again for the terms of one MMA aligned to its largest."""
    return (k / 64 + 64) * 2.0 ** -23
