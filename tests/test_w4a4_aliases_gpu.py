"""Results over the inputs: what a call returns where one tensor is given twice."""
import pytest
import torch

from test_w4a4_gpu import BF16, DEV, hidden, no_device_error, pkg, weight  # noqa: F401

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


def test_views_between_one_another():
    """x, the residual and both results as columns of one tensor; results of one row over the other's gap."""
    m, k = 70, 512
    base = hidden(m, 4 * k, 21).to(DEV)
    w = torch.ones(k, dtype=BF16, device=DEV)
    want_y, want_r = pkg.add_rms_norm(base[:, :k].contiguous(), base[:, k:2 * k].contiguous(), w)
    t = base.clone()
    y, r = pkg.add_rms_norm(t[:, :k], t[:, k:2 * k], w, out=t[:, 2 * k:3 * k], residual_out=t[:, 3 * k:])
    assert torch.equal(y, want_y) and torch.equal(r, want_r) and torch.equal(t[:, :2 * k], base[:, :2 * k])
    # every other row against every row
    t = base.clone()
    x, out = t[::2, :k], t[:m // 2, k:2 * k]
    y, _ = pkg.add_rms_norm(x, None, w, out=out)
    assert torch.equal(y, pkg.add_rms_norm(base[::2, :k].contiguous(), None, w)[0])


def test_results_over_inputs_are_refused():
    m, k = 40, 512
    base = hidden(m, 2 * k, 22).to(DEV)
    x, w = base[:, :k], torch.ones(k, dtype=BF16, device=DEV)
    flat = base.view(-1)
    shifted = flat[k // 2:k // 2 + m * k].view(m, k)
    before = base.clone()
    for kw in (dict(out=shifted), dict(residual_out=shifted), dict(out=base[:, 8:k + 8]), dict(residual_out=base[:, 256:k + 256])):
        with pytest.raises(RuntimeError):
            pkg.add_rms_norm(x, None, w, **kw)
    y = torch.empty((m, k), dtype=BF16, device=DEV)
    with pytest.raises(RuntimeError):
        pkg.add_rms_norm(x, y, w, out=y, residual_out=y)
    a = pkg.quantize_rows(x, 20.0)
    square = weight(k, k, 23)[0]
    pair = weight(2 * k, k, 24)[0]
    with pytest.raises(RuntimeError):
        pkg.linear_w4a4_swiglu_quantize(a, pair, 20.0, out=a)
    with pytest.raises(RuntimeError):
        pkg.linear_w4a4(a, square, out=square.codes.view(BF16).view(-1)[:m * k].view(m, k))
    torch.cuda.synchronize()
    assert torch.equal(base, before)
