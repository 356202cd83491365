"""One product that takes longer than the limit of a pipeline wait (2^31 clocks, about a second): the limit is of a
wait, not of a call."""
import pytest
import torch

from test_w4a4_gpu import DEV, no_device_error, pkg  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_product_of_seconds():
    m, n, k = 1 << 18, 3 << 16, 1 << 17                            # 1.4e16 operations, some 6e9 clocks; 52 GB
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB")
    g = torch.Generator(device=DEV).manual_seed(1)

    def fill(t, lo, hi):
        for part in t.flatten().split(1 << 30):
            part.random_(lo, hi, generator=g)
        return t
    rows = pkg.new_fp4_rows(m, k, 64.0)
    fill(rows.codes, 0, 256), fill(rows.scales, 0x20, 0x51)
    packed = fill(torch.empty((n, k // 2), dtype=torch.uint8, device=DEV), 0, 256)
    scale = fill(torch.empty((n, k // 16), dtype=torch.uint8, device=DEV), 0x20, 0x51)
    w = pkg.Fp4Weight(packed, scale, 8.0 * k ** 0.5)
    del scale
    out = pkg.new_fp4_rows(m, n // 2, 4.0)
    fill(out.codes, 0, 256)
    pkg.linear_w4a4_swiglu_quantize(rows, w, 4.0, out=out)
    torch.cuda.synchronize()
    assert pkg.w4a4_error(clear=False) == 0
    # the last rows, of the last tiles, and the first ones against a product of theirs alone
    for at in (0, m // 2, m - 1024):
        part = pkg.Fp4Rows(rows.codes[at:at + 1024], rows.scales[at // 128:at // 128 + 8], 64.0)
        want = pkg.linear_w4a4_swiglu_quantize(part, w, 4.0)
        assert torch.equal(out.codes[at:at + 1024], want.codes)
        assert torch.equal(out.scales[at // 128:at // 128 + 8], want.scales)
        assert bool((want.codes & 7 != 0).any())
    del rows, packed, w, out, part, want
    torch.cuda.empty_cache()
