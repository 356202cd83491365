"""The norm's mean square is the sum divided by the width, rounded once."""
import pytest
import torch

import _w4a4_ref as ref
from test_w4a4_gpu import BF16, DEV, no_device_error, pkg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gs", [6.375, 7.125, 7.875])
def test_the_mean_is_exact_where_it_can_be(gs):
    """Rows of one magnitude a of 5 bits: every partial sum of squares is exact in fp32, and so is the mean, a^2,
    whatever the width.  A row's normed values are 1 up to the root's rounding, and times gs / 6 on the border between
    two scales, so that one step of fp32 in the mean shows: the scale is that of the same row at a width of 256, where
    a product with the width's reciprocal would be exact as well."""
    a = torch.tensor([(16 + i) * 2.0 ** e for i in range(16) for e in range(-4, 0)])

    def scales(k):
        x = a[:, None].repeat(1, k).to(BF16).to(DEV)
        rows, _ = pkg.add_rms_norm_quantize(x, None, torch.ones(k, dtype=BF16, device=DEV), 0.0, gs)
        s = ref.plain_scales(rows)
        assert bool((s == s[:, :1]).all())
        return s[:, 0]
    want = scales(256)
    for j in range(3, 129, 2):
        assert torch.equal(scales(256 * j), want), j
