"""Either attention kernel against the 64-bit form where a CTA has dozens of key
blocks or many items, so that every ring turns several times: thousands of keys,
maxima that rise along them, hundreds of ragged sequences, NaN in late values.

Bounds over bf16 pages are those of test_attention_gpu.py.  Over e4m3 pages,
where the weights are f16, per element:
  2^-11 of the weighted sum of |v| (a weight's rounding), and 2^-36 of the plain
  sum of |v| over the keys seen (weights too small for that: half f16's subnormal
  step, 2^-25, with the row's largest weight at 2^11 or more);
  2^-14 of the weighted sum for its accumulation (a step of 2^-23 for each 16 of
  at most 8192 keys);
  the score's error, the exponential's and the output's rounding as over bf16."""
import pytest
import torch

from test_attention_gpu import BF16, DEV, E4M3, att, check_attention, run_attention, to_dev
from test_attention_many_blocks_gpu import SHAPES, batch, reference

pytestmark = pytest.mark.gpu


def seen_values(b):
    """The sum of |v| over the keys that each token sees, [T, Hq, D]."""
    page, Hk, D = b.v.shape[1:]
    v = to_dev(b.v).float().abs()
    out = torch.zeros(b.q.shape, dtype=torch.float64, device=DEV)
    a = 0
    for s, (n, m) in enumerate(zip(b.kv_lens, b.q_lens)):
        skip = max(0, m - n)
        if n and m:
            at = torch.arange(n)
            x = v[b.table[s].long()[at // page].to(DEV), (at % page).to(DEV)].double()
            if b.vs is not None:
                x = x * b.vs.to(DEV).double()[:, None]
            upto = x.cumsum(0)[n - m + skip:]
            out[a + skip:a + m] = upto.repeat_interleave(b.q.shape[1] // Hk, dim=1)
        a += m
    return out.cpu()


def check(b, out, lse, want):
    if b.k.dtype == BF16:
        return check_attention(out, lse, want)
    o, l, mag, err = want
    got, got_lse = out.double().cpu(), lse.double().cpu()
    tol = mag * (2.0 ** -11 * 1.01 + 2.0 ** -14 + 2 * err[..., None] + 2.0 ** -17) + 2.0 ** -36 * seen_values(b)
    tol = tol + 2.0 ** -8 * o.abs() + 1e-30
    bad = ((got - o).abs() > tol) | torch.isnan(got)
    assert not bad.any(), "out: %d of %d off, worst %.3g of its bound" % (bad.sum(), bad.numel(), ((got - o).abs() / tol).max())
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(got_lse) & (got_lse < 0), empty)
    assert ((got_lse - l).abs() <= err + 2.0 ** -18 * (1 + l.abs()))[~empty].all()


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("amp,rise", [(6.0, 1.0), (2.0, 5.0)])
@pytest.mark.parametrize("kv_lens,q_lens", [([6011, 2500], [150, 333]), ([7001, 3000, 129], [5, 4, 3])], ids=str)
def test_many_blocks(dtype, hq, hk, dim, amp, rise, kv_lens, q_lens):
    b = batch(kv_lens, q_lens, hq, hk, dim, dtype, 64, amp, rise, seed=dim + sum(q_lens))
    out, lse = run_attention(b)
    check(b, out, lse, reference(b))
    again, lse2 = run_attention(b)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert att.attention_error() == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("longest", [3, 40])
def test_many_items(dtype, hq, hk, dim, longest):
    """Items of none to five blocks, odd and even, many to a CTA."""
    g = torch.Generator().manual_seed(dim + longest)
    kv_lens = torch.randint(0, 600, (400,), generator=g).tolist()
    q_lens = torch.randint(0, longest + 1, (400,), generator=g).tolist()
    q_lens[0] = longest
    b = batch(kv_lens, q_lens, hq, hk, dim, dtype, 48, 6.0, 1.0, seed=dim + longest)
    out, lse = run_attention(b)
    check(b, out, lse, reference(b))
    again, lse2 = run_attention(b)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert att.attention_error() == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("m", [4, 400])
def test_nan_late_in_a_long_sequence(dtype, hq, hk, dim, m):
    n = 5000
    b = batch([n], [m], hq, hk, dim, dtype, 64, 3.0, 1.0, seed=dim)
    keys = list(range(n - m + 1, n, max(1, m // 11)))
    hit = torch.zeros(m, hk, dim, dtype=torch.bool)
    raw = b.v.view(torch.uint8) if dtype == E4M3 else b.v
    for i, j in enumerate(keys):
        raw[int(b.table[0, j // 64]), j % 64, i % hk, (11 * i) % dim] = 0
        hit[j - (n - m):, i % hk, (11 * i) % dim] = True
    want = reference(b)
    for i, j in enumerate(keys):
        raw[int(b.table[0, j // 64]), j % 64, i % hk, (11 * i) % dim] = 0x7F if dtype == E4M3 else float("nan")
    b.args = (att.KVCache(b.cache.k, to_dev(b.v), b.cache.k_scale, b.cache.v_scale),) + b.args[1:]
    out, lse = run_attention(b)
    heads = hit.repeat_interleave(hq // hk, dim=1)
    assert torch.equal(torch.isnan(out.cpu()), heads)
    for i, j in enumerate(keys):
        raw[int(b.table[0, j // 64]), j % 64, i % hk, (11 * i) % dim] = 0
    check(b, torch.where(heads.to(DEV), want[0].to(DEV).to(out.dtype), out), lse, want)
    assert att.attention_error() == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("kv_lens,q_lens", [([4100], [1000]), ([3000, 700], [40, 333]), ([2100, 600], [3, 1])], ids=str)
def test_mass_of_many_blocks(dtype, hq, hk, dim, kv_lens, q_lens):
    """Many query tiles past each key; per key twice the score's error and 2^-18 for
    each weight, and 2^-18 of the sum and 2^-24 of it for each addition in a row."""
    b = batch(kv_lens, q_lens, hq, hk, dim, dtype, 64, 2.0, 1.0, seed=dim + 2)
    _, l, _, err = reference(b)
    q, lse = b.q.to(DEV), l.float().to(DEV)
    got = att.attention_mass(q, *b.args, lse).double()
    page, a = 64, 0
    for s, (n, m) in enumerate(zip(kv_lens, q_lens)):
        at = torch.arange(n)
        k = to_dev(b.k).float()[b.table[s].long()[at // page].to(DEV), (at % page).to(DEV)].double().transpose(0, 1)
        if b.ks is not None:
            k = k * b.ks.to(DEV).double()[:, None, None]
        x = q[a:a + m].double().view(m, hk, -1, dim).permute(1, 2, 0, 3).reshape(hk, -1, dim)
        hidden = torch.arange(n, device=DEV)[None, :] > torch.arange(n - m, n, device=DEV)[:, None]
        ls, e = (y[a:a + m].to(DEV).double().view(m, hk, -1).permute(1, 2, 0).reshape(hk, -1, 1) for y in (l.float(), err))
        w = torch.exp((x @ k.transpose(1, 2)) * b.scale - ls).masked_fill_(hidden.repeat(hq // hk, 1), 0.0)
        want = w.sum(1)
        tol = (w * (2 * e + 2.0 ** -18 + 2.0 ** -23 * ls.abs())).sum(1) + want * (2.0 ** -18 + 2.0 ** -24 * w.shape[1])
        assert ((got[s, :, :n] - want).abs() <= tol).all(), float(((got[s, :, :n] - want).abs() / tol).max())
        assert (got[s, :, n:] == 0).all()
        a += m
    assert att.attention_error() == 0
