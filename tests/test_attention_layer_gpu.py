"""The layer that runs the attention block's operators together: against the
same steps in plain torch, chunk by chunk and token by token, and over a cache
that was cut."""
import pytest
import torch

import _attention_ref as ref
from nvfp4_block_scaled_linear_gb300 import _lib
from nvfp4_block_scaled_linear_gb300 import attention as att
from nvfp4_block_scaled_linear_gb300.attention_layer import seeded_layer, serve

pytestmark = pytest.mark.gpu


def test_layer_in_chunks_matches_the_plain_steps():
    """The layer's projections in fp32 around the operators' plain forms."""
    layer = seeded_layer(hidden=512, q_heads=6, kv_heads=2, head_dim=128, rotary_dim=64, positions=200, seed=3)
    dev, hq, hk, d, page = "cuda", 6, 2, 128, 16
    g = torch.Generator().manual_seed(1)
    n = 150
    x = torch.randn((n, 512), generator=g).to(torch.bfloat16).to(dev)
    cache = att.new_kv_cache(12, page, hk, d)
    table = torch.randperm(12, generator=g).to(torch.int32).to(dev).view(1, -1)
    mass = torch.zeros(1, hk, 12 * page, device=dev)
    out, a = [], 0
    for m in (100, 1, 1, 7, 41):
        place = torch.arange(a, a + m, device=dev)
        out.append(layer(x[a:a + m], cache, table[0].long()[place // page] * page + place % page, place, table,
                         torch.tensor([a + m], dtype=torch.int32, device=dev),
                         torch.tensor([0, m], dtype=torch.int32, device=dev), m, mass))
        a += m
    torch.cuda.synchronize()
    assert att.attention_error() == 0 and _lib.device_error() == 0
    out = torch.cat(out)

    w, s, gs = layer.qkv
    rows = [hq * d, hk * d, hk * d]
    y = _lib.linear_segmented(x, w, s, gs, rows).cpu()
    q, k, v = (t.unflatten(1, (-1, d)) for t in y.split(rows, 1))
    pos, cs = torch.arange(n), layer.cos_sin.cpu()
    q = ref.norm_rope(q, layer.q_weight.cpu(), cs, pos, 1e-6)
    k = ref.norm_rope(k, layer.k_weight.cpu(), cs, pos, 1e-6)
    v = v.double()
    sc = torch.einsum("qgrd,kgd->grqk", q.view(n, hk, -1, d), k) * d ** -0.5
    sc.masked_fill_(torch.ones(n, n, dtype=torch.bool).triu(1), float("-inf"))
    p = torch.softmax(sc, -1)
    o = torch.einsum("grqk,kgd->qgrd", p, v).reshape(n, hq * d)
    want = _lib.linear_f32(o.to(torch.bfloat16).to(dev), *layer.o).double().cpu()
    # bf16 queries, keys, values, weights and outputs between exact steps: each
    # rounding is 2^-9 of its value at random, six of them in a row
    err = (out.double().cpu() - want).norm() / want.norm()
    assert err < 6 ** 0.5 * 2.0 ** -8, float(err)
    got = mass[0, :, :n].double().cpu()
    received = p.sum((1, 2))
    assert ((got - received).norm() / received.norm()) < 2.0 ** -7
    assert (mass[0, :, n:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
def test_serving_over_a_cut_cache(dtype):
    """Nothing is cut where all keys are kept: the same keys in other pages give
    the same outputs up to the order of the sums; a real cut changes them."""
    layer = seeded_layer(hidden=512, q_heads=8, kv_heads=2, head_dim=64, rotary_dim=32, positions=400, seed=4)
    whole, short, held, cut = serve(layer, 200, 64, 5, keep=300, recent=8, page=16, dtype=dtype)
    assert (held, cut) == (205, 205)
    assert (whole.float() - short.float()).norm() / whole.float().norm() < 2.0 ** -7
    whole, short, held, cut = serve(layer, 200, 64, 5, keep=60, recent=8, page=16, dtype=dtype)
    assert (held, cut) == (205, 60) and torch.isfinite(short).all()
    assert (whole.float() - short.float()).norm() / whole.float().norm() > 2.0 ** -7
    assert att.attention_error() == 0
