"""The same calls by either of an operator's kernels: the most tokens that a
sequence may have, which the caller states, decides, so that a larger figure
moves a small batch to the kernel for many rows.  Both are held against the
64-bit form with test_attention_gpu.py's bounds.  And NaN in values that only
the later tokens see, at every place of a block that a copying warp may look
over."""
import pytest
import torch

import _attention_ref as ref
from test_attention_gpu import BF16, DEV, E4M3, SHAPES, Batch, att, check_attention, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hint", [5, 400])
def test_either_kernel(dtype, hq, hk, dim, page, hint):
    kv_lens, q_lens = [259, 5, 384], [5, 1, 3]
    b = Batch(kv_lens, q_lens, hq, hk, dim, page=page, dtype=dtype, seed=page + dim)
    b.args = b.args[:-1] + (hint,)
    want = b.reference()
    out, lse = run_attention(b)
    check_attention(out, lse, want)
    room = 400
    l32 = want[1].float()
    mass, tol = ref.mass(b.q, b.k, b.ks, b.table, kv_lens, q_lens, b.scale, l32, None, room)
    got = att.attention_mass(b.q.to(DEV), *b.args, l32.to(DEV), out=torch.empty(3, hk, room, device=DEV))
    assert ((got.double().cpu() - mass).abs() <= tol).all()
    assert att.attention_error() == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_nan_values_that_later_tokens_see(dtype, hq, hk, dim, page):
    n, m = 300, 140
    b = Batch([n], [m], hq, hk, dim, page=page, dtype=dtype, seed=3 * page + dim)
    # key j is seen from token j - (n - m) on: NaN in one column of keys 1, 4, 7 ... of the new ones
    keys = list(range(n - m + 1, n, 3))
    hit = torch.zeros(m, hk, dim, dtype=torch.bool)
    raw = b.v.view(torch.uint8) if dtype == E4M3 else b.v
    for i, j in enumerate(keys):
        p, at, h, c = int(b.table[0, j // page]), j % page, i % hk, (11 * i) % dim
        raw[p, at, h, c] = 0                            # the 64-bit form goes without it
        hit[j - (n - m):, h, c] = True
    want = b.reference()
    for i, j in enumerate(keys):
        raw[int(b.table[0, j // page]), j % page, i % hk, (11 * i) % dim] = 0x7F if dtype == E4M3 else float("nan")
    dev = b.cache.v.view(torch.uint8) if dtype == E4M3 else b.cache.v
    dev.copy_(raw)
    out, lse = run_attention(b)
    heads = hit.repeat_interleave(hq // hk, dim=1)
    assert torch.equal(torch.isnan(out.cpu()), heads)
    out = torch.where(heads.to(DEV), want[0].to(DEV).to(out.dtype), out)
    check_attention(out, lse, want)
