"""Results over the inputs: what a call returns where one tensor is given twice."""
import pytest
import torch

from test_w4a4_gpu import BF16, DEV, hidden, no_device_error, pkg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m, k", [(1, 512), (40, 1536), (700, 4096)])
@pytest.mark.parametrize("view", [False, True])
def test_norm_over_its_only_input(m, k, view):
    """No residual, no tensor for the sum, the normed rows over x: the sum returned is what x held."""
    x = hidden(m, k, 14).to(DEV)
    w = (1 + 0.1 * torch.randn(k, generator=torch.Generator().manual_seed(3))).to(BF16).to(DEV)
    want, same = pkg.add_rms_norm(x, None, w)
    assert same is x
    a = x.clone()
    out = a[:] if view else a
    for stream in (None, torch.cuda.current_stream()):
        a.copy_(x)
        y, r = pkg.add_rms_norm(a, None, w, out=out, stream=stream)
        assert y is out and torch.equal(a, want) and torch.equal(r, x)
