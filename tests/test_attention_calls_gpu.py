"""Calls at the edges of the attention block's operators."""
import pytest
import torch

import _attention_ref as ref
from test_attention_gpu import BF16, DEV, E4M3, Batch, att, check_attention, no_device_error, to_dev  # noqa: F401

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


@pytest.mark.parametrize("which", ["other", "none_to_some", "some_to_none", "equal"])
@pytest.mark.parametrize("page,order", [(16, "heads"), (48, "tokens")])
def test_evict_between_caches_of_different_scales(which, page, order):
    """A row keeps the values it stands for: its codes are taken over where the
    head's scales are equal, and rounded once to the new scale where not."""
    g = torch.Generator().manual_seed(page)
    n, hk, dim, keep = 300, 3, 128, 64
    table, pages = ref.table_for([n], page, g)
    k, v = (ref.pages(pages, page, hk, dim, E4M3, order, g, 40.0) for _ in range(2))
    k.view(torch.uint8)[:, :, 0, 5] = 0x7F                       # NaN stays NaN
    some = [(0.5 + torch.rand(hk, generator=g)) / 16 for _ in range(4)]
    one = torch.ones(hk)
    a, b = {"other": (some[:2], some[2:]), "none_to_some": ([None] * 2, some[2:]), "some_to_none": (some[:2], [None] * 2),
            "equal": (some[:2], [x.clone() for x in some[:2]])}[which]
    if which == "other":
        b[0][1] = a[0][1]                                        # one head alike
    width = -(-keep // page)
    to = att.new_kv_cache(width, page, hk, dim, E4M3, *(x if x is None else x.to(DEV) for x in b))
    cache = att.KVCache(to_dev(k), to_dev(v), *(x if x is None else x.to(DEV) for x in a))
    mass = torch.rand(1, hk, n, generator=g)
    to_table = torch.arange(width, dtype=torch.int32).view(1, width)
    _, index, _ = att.evict(cache, table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV), mass.to(DEV), keep, 7, to,
                            to_table.to(DEV))
    r = torch.arange(keep)
    for src, dst, x, y in ((k, to.k, a[0], b[0]), (v, to.v, a[1], b[1])):
        x, y = (one if s is None else s for s in (x, y))
        got = dst.view(torch.uint8).cpu()
        for h in range(hk):
            at = index[0, h].cpu().long()
            codes = src.view(torch.uint8)[table[0].long()[at // page], at % page, h]
            want = codes
            if x[h] != y[h]:
                want = (codes.view(E4M3).float() * x[h] / y[h]).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
            here = got[to_table[0].long()[r // page], r % page, h]
            nan = (want & 0x7F) == 0x7F
            assert torch.equal(here[~nan], want[~nan]) and ((here[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("hq,hk,dim", [(24, 4, 256), (12, 4, 128), (7, 1, 64)])
@pytest.mark.parametrize("hint", [1, 400])
@pytest.mark.parametrize("q_len", [1, 150])
def test_mass_of_a_key_whose_scores_are_minus_infinity(hq, hk, dim, hint, q_len):
    """Groups of 3, 6 and 7 leave rows of a 128-row tile without a token: a key
    with an infinite element, whose score is -inf for every query, receives
    nothing from them either."""
    n, room = 300, 320
    b = Batch([n], [q_len], hq, hk, dim, seed=dim + q_len, width=20)
    b.q[..., 3] = b.q[..., 3].abs() + 0.5
    keys = [0, 17, 100]
    at = torch.tensor(keys)
    _, lse, _, _ = b.reference()
    lse = lse.float()
    want, tol = ref.mass(b.q, b.k, None, b.table, [n], [q_len], b.scale, lse, None, room)
    want[..., keys] = tol[..., keys] = 0.0
    b.cache.k[b.table[0].long()[at // 16].to(DEV), (at % 16).to(DEV), :, 3] = float("-inf")
    args = b.args[:-1] + (hint,)
    got = att.attention_mass(b.q.to(DEV), *args, lse.to(DEV), out=torch.empty(1, hk, room, device=DEV)).double().cpu()
    assert not torch.isnan(got).any()
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("hq,hk,dim", [(24, 4, 256), (8, 2, 128)])
@pytest.mark.parametrize("hint", [1, 400])
def test_mass_of_rows_without_a_weight(hq, hk, dim, hint):
    """A query whose every score is -inf has lse -inf and an output of zeros;
    no key receives anything from it, by either kernel."""
    n, q_len = 130, 4
    b = Batch([n], [q_len], hq, hk, dim, seed=dim, width=9)
    b.cache.k[..., 3] = float("-inf")
    b.q[..., 3] = b.q[..., 3].abs() + 0.5
    q = b.q.to(DEV)
    args = b.args[:-1] + (hint,)
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = att.paged_attention(q, *args, lse=lse)
    assert (out == 0).all() and (lse == float("-inf")).all()
    got = att.attention_mass(q, *args, lse)
    assert (got == 0).all()


def test_a_workspace_elsewhere_is_refused():
    """Memory of the host, or less memory than the tensor's size says."""
    b = Batch([70], [2], 8, 2, 128, seed=44)
    q = b.q.to(DEV)
    n = att.attention_workspace(b.cache).numel()
    for workspace in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device=DEV).expand(n),
                      torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            att.paged_attention(q, *b.args, workspace=workspace)


@pytest.mark.parametrize("hint", [1, 300])
@pytest.mark.parametrize("starts", [[0, 4, 0, 4], [0, 4, 2, 4], [4, 0, 4, 4]], ids=str)
def test_starts_that_descend(hint, starts):
    """Sequences that would overlap: the error bit, and nothing is written."""
    b = Batch([90, 64, 33], [2, 1, 1], 4, 2, 128, seed=45)
    cache, table, kv, good, _ = b.args
    q, want = b.q.to(DEV), b.reference()
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 7.0, device=DEV)
    att.paged_attention(q, cache, table, kv, torch.tensor(starts, dtype=torch.int32, device=DEV), hint, out=out, lse=lse)
    torch.cuda.synchronize()
    assert att.attention_error() == att.ATTENTION_BAD_INDEX
    assert (out == 3.0).all() and (lse == 7.0).all()
    att.paged_attention(q, cache, table, kv, good, hint, out=out, lse=lse)
    check_attention(out, lse, want)


def test_norm_rope_values_at_the_edges_of_keys_and_queries():
    """Rows of zeros, of one large or small value and with a NaN: the same of keys
    as of queries, and each row to itself."""
    x = torch.zeros(4, 2, 128, dtype=BF16)
    x[1, 0, 5], x[2, 1, 7], x[3, 0, 9] = 1e18, float("nan"), 1e-30
    w = torch.ones(128, dtype=BF16, device=DEV)
    q, k = (t.float().cpu() for t in att.qk_norm_rope(x.to(DEV), x.to(DEV), w, w, None, None))
    nan = torch.zeros(4, 2, 128, dtype=torch.bool)
    nan[2, 1] = True
    for got in (q, k):
        assert torch.equal(torch.isnan(got), nan)
        want = ref.norm_rope(torch.where(nan, torch.zeros_like(x), x), w.cpu(), None, None, 1e-6)
        off = (got.double() - want).abs()
        assert (off <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * want.abs().amax(-1, keepdim=True))[~nan].all()
    assert torch.equal(q.nan_to_num(), k.nan_to_num())


def test_the_example_at_small_sizes(capsys):
    """One token after a short prompt, cut to fewer keys than are kept as recent by default."""
    from nvfp4_block_scaled_linear_gb300 import attention_layer
    attention_layer.main(["100", "64", "1", "32"])
    assert "cache cut from 101 to 32 keys" in capsys.readouterr().out
    assert att.attention_error() == 0
