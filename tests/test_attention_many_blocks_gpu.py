"""The attention kernels over thousands of keys, against the 64-bit form: many
key blocks to a CTA, maxima that rise along the sequence, so that accumulators
are rescaled late.  Bounds are those of test_attention_gpu.py."""
import pytest
import torch

from test_attention_gpu import BF16, DEV, E4M3, Batch, att, check_attention, run_attention, to_dev

pytestmark = pytest.mark.gpu
SHAPES = [(24, 4, 256), (12, 2, 128), (8, 2, 64), (6, 1, 256)]


def reference(b):
    """_attention_ref.attention's (out, lse, mag, err), all heads of a sequence at a time."""
    q = b.q.to(DEV).double()
    T, Hq, D = q.shape
    page, Hk = b.k.shape[1:3]
    k, v = (to_dev(x).float() for x in (b.k, b.v))
    scales = [None if c is None else c.to(DEV).double()[:, None, None] for c in (b.ks, b.vs)]
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((T, Hq), float("-inf"), dtype=torch.float64, device=DEV)
    err = torch.zeros(T, Hq, dtype=torch.float64, device=DEV)
    a = 0
    for s, (n, m) in enumerate(zip(b.kv_lens, b.q_lens)):
        skip = max(0, m - n)                       # tokens that see no key
        if n == 0 or m == 0:
            a += m
            continue
        at = torch.arange(n)
        where = (b.table[s].long()[at // page].to(DEV), (at % page).to(DEV))
        kk, vv = (x[where].double().transpose(0, 1) * (1.0 if c is None else c) for x, c in zip((k, v), scales))
        for t in range(skip, m, 128):
            e = min(m, t + 128)
            x = q[a + t:a + e].view(e - t, Hk, -1, D).permute(1, 2, 0, 3).reshape(Hk, -1, D)
            hidden = torch.arange(n, device=DEV)[None, :] > torch.arange(n - m + t, n - m + e, device=DEV)[:, None]
            hidden = hidden.repeat(Hq // Hk, 1)
            sc = (x @ kk.transpose(1, 2) * b.scale).masked_fill_(hidden, float("-inf"))
            l = torch.logsumexp(sc, 2, keepdim=True)
            p = torch.exp(sc - l)
            top = (x.abs() @ kk.abs().transpose(1, 2)).masked_fill_(hidden, 0.0).amax(2, keepdim=True) * b.scale

            def put(to, y):
                to[a + t:a + e] = y.view(Hk, Hq // Hk, e - t, -1).permute(2, 0, 1, 3).reshape(to[a + t:a + e].shape)
            put(out, p @ vv)
            put(mag, p @ vv.abs())
            put(lse, l)
            put(err, (D + 4) * 2.0 ** -23 * top)
        a += m
    return out.cpu(), lse.cpu(), mag.cpu(), err.cpu()


def batch(kv_lens, q_lens, hq, hk, dim, dtype, page, amp, rise, seed):
    b = Batch(kv_lens, q_lens, hq, hk, dim, page=page, dtype=dtype, seed=seed, order="heads" if seed % 2 else "tokens")
    b.q = (b.q.float() * amp).to(BF16)
    if rise != 1.0:
        for s, n in enumerate(kv_lens):
            at = torch.arange(n)
            where = (b.table[s].long()[at // page], at % page)
            up = b.k.float()[where] * torch.linspace(1.0, rise, n)[:, None, None]
            if dtype == E4M3:
                b.k.view(torch.uint8)[where] = up.clamp(-448, 448).to(E4M3).view(torch.uint8)
            else:
                b.k[where] = up.to(dtype)
        b.cache = att.KVCache(to_dev(b.k), to_dev(b.v), b.cache.k_scale, b.cache.v_scale)
        b.args = (b.cache,) + b.args[1:]
    return b


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("amp,rise", [(6.0, 1.0), (2.0, 5.0)])
def test_maxima_that_rise_in_an_items_last_block(dtype, hq, hk, dim, amp, rise):
    """The two groups of a tile's softmax agree on the row's last maximum: sums
    that are right, and the same bits on every run."""
    b = batch([3000, 260], [200, 90], hq, hk, dim, dtype, 64, amp, rise, seed=25)
    out, lse = run_attention(b)
    for _ in range(20):
        again, lse2 = run_attention(b)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    want = reference(b)
    _, l, _, err = want
    assert ((lse.double().cpu() - l).abs() <= err + 2.0 ** -18 * (1 + l.abs())).all()
    if dtype == BF16:
        check_attention(out, lse, want)
    assert att.attention_error() == 0
