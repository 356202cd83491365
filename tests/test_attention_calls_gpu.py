"""Calls at the edges of the attention block's operators."""
import pytest
import torch

from test_attention_gpu import BF16, DEV, E4M3, Batch, att, no_device_error  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hint", [0, 1, 400])
def test_mass_of_no_tokens(dtype, hint):
    """Nothing is received: what was received before stays, and the rest is 0."""
    kv_lens, room = [70, 0, 33], 80
    b = Batch(kv_lens, [0, 0, 0], 8, 2, 128, dtype=dtype, seed=41, width=5)
    before = torch.rand(3, 2, room, generator=torch.Generator().manual_seed(1))
    args = b.args[:-1] + (hint,)
    q, lse = b.q.to(DEV), torch.empty(0, 8, device=DEV)
    held = torch.arange(room)[None, :] < torch.tensor(kv_lens)[:, None]
    for start in (None, before.to(DEV)):
        out = torch.full((3, 2, room), 9.0, device=DEV)
        got = att.attention_mass(q, *args, lse, start, out=out).cpu()
        want = torch.zeros_like(before) if start is None else before * held[:, None]
        assert torch.equal(got, want)
