"""One strong key and a long tail of keys whose weights lie near 2^-26 of its
own, over e4m3 pages and by either attention kernel.  The strong keys' values
are zero, so that the output is the tail's share alone: what the 16-bit weights
drop, the output lacks.

Tolerance: f16 holds a weight of 2^-27 of the largest, shifted up by 2^11 at
least, to 2^-9 of itself (the subnormal step is 2^-24); a weight's score adds
twice its fp32 rounding error, and the output's own rounding 2^-8 of itself, as
in test_attention_gpu.py."""
import math

import pytest
import torch

import _attention_ref as ref
from test_attention_gpu import BF16, DEV, E4M3, att, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk,dim", [(24, 4, 256), (8, 2, 128), (7, 1, 64)])
@pytest.mark.parametrize("kv_lens,q_lens,hint", [([3000], [1], 1), ([3000, 700], [5, 2], 5), ([3000, 700], [5, 2], 400),
                                                 ([1500], [150], 150)], ids=str)
def test_a_long_tail_behind_strong_keys(hq, hk, dim, kv_lens, q_lens, hint):
    g = torch.Generator().manual_seed(dim + sum(q_lens))
    page = 64
    table, n = ref.table_for(kv_lens, page, g)
    # codes of 1 in every dimension of each 61st key, 0 elsewhere; values 0 there, 1 to 2 elsewhere
    k = torch.zeros(n, page, hk, dim)
    v = 1 + torch.rand((n, page, hk, dim), generator=g)
    for s, m in enumerate(kv_lens):
        at = torch.arange(0, m, 61)
        k[table[s].long()[at // page], at % page] = 1.0
        v[table[s].long()[at // page], at % page] = 0.0
    k, v = k.to(E4M3), v.to(E4M3)
    t = sum(q_lens)
    # a strong key's score above a tail key's: between 25 and 27 in log2
    gap = (26 + (torch.rand((t, hq, 1), generator=g) * 1.8 - 0.9)) * math.log(2.0) / dim ** 0.5
    q = gap.expand(t, hq, dim).to(BF16).contiguous()
    starts = torch.tensor([sum(q_lens[:i]) for i in range(len(q_lens) + 1)], dtype=torch.int32)
    cache = att.KVCache(*(x.view(torch.uint8).to(DEV).view(E4M3) for x in (k, v)))

    class Call:
        args = (cache, table.to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV), starts.to(DEV), hint)
    out, lse = run_attention(Call, q.to(DEV))
    assert att.attention_error() == 0
    o, l, _, err = ref.attention(q, k, v, None, None, table, kv_lens, q_lens, dim ** -0.5)
    tol = o * (2.0 ** -8 + 2.0 ** -9 + 2 * err[..., None] + 2.0 ** -17)
    off = (out.double().cpu() - o).abs()
    assert (o > 0).all() and (off <= tol).all(), float((off / o).max())
    assert ((lse.double().cpu() - l).abs() <= err + 2.0 ** -18 * (1 + l.abs())).all()
