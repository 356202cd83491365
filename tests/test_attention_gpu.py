"""The attention block's operators against plain forms in 64 bits, at the
sizes and masks where they can go wrong.

Tolerances, derived per element:
  attention  a weight's relative error is its rounding to the operand type
             (bf16: 2^-8; f16 over an e4m3 cache is finer) plus twice its
             score's fp32 rounding error e (and 2^-18 for the exponential and
             the sums), so the weighted sum of |v| times those bounds the sum;
             the output's own rounding adds 2^-8 of itself.
  lse        the score's error plus 2^-18 (1 + |lse|).
  mass       each weight's 2 e + 2^-18, and 2^-18 of the sum.
  norm_rope  2^-8 of the value (bf16), or half an e4m3 step (2^-4 of the value,
             2^-10 below the normal range), plus 2^-18 of the pair's size.
  evict      equal.
"""
import math

import pytest
import torch

import _attention_ref as ref
from nvfp4_block_scaled_linear_gb300 import attention as att

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def no_device_error():
    assert att.attention_error() == 0
    yield
    assert att.attention_error() == 0


def to_dev(x):
    """On the device with the same strides (float8 has no strided copy)."""
    if x.dtype == E4M3:
        return to_dev(x.view(torch.uint8)).view(E4M3)
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEV)
    y.copy_(x)
    return y


class Batch:
    """A random batch: lengths, pages, queries; host and device copies."""

    def __init__(self, kv_lens, q_lens, hq, hk, dim, page=16, dtype=BF16, order="heads", seed=0, scales=True,
                 poison=True, width=0):
        g = torch.Generator().manual_seed(seed)
        self.kv_lens, self.q_lens = list(kv_lens), list(q_lens)
        self.table, n = ref.table_for(kv_lens, page, g, width=width)
        amp = 16.0 if dtype == E4M3 else 1.0
        self.k = ref.pages(n, page, hk, dim, dtype, order, g, amp)
        self.v = ref.pages(n, page, hk, dim, dtype, order, g, amp)
        self.ks = self.vs = None
        if dtype == E4M3 and scales:
            self.ks, self.vs = ((0.5 + torch.rand(hk, generator=g)) / 16 for _ in range(2))
        if poison:
            # NaN in every row that no sequence holds
            bad = torch.ones(n, page, dtype=torch.bool)
            for s, m in enumerate(kv_lens):
                at = torch.arange(m)
                bad[self.table[s].long()[at // page], at % page] = False
            for x in (self.k, self.v):
                raw = x.view(torch.uint8) if dtype == E4M3 else x
                raw[bad] = 0x7F if dtype == E4M3 else float("nan")
        t = sum(q_lens)
        self.q = (1.5 * torch.randn((t, hq, dim), generator=g)).to(BF16)
        self.starts = torch.tensor([sum(q_lens[:i]) for i in range(len(q_lens) + 1)], dtype=torch.int32)
        self.scale = dim ** -0.5
        self.cache = att.KVCache(to_dev(self.k), to_dev(self.v), None if self.ks is None else self.ks.to(DEV),
                                 None if self.vs is None else self.vs.to(DEV))
        self.args = (self.cache, self.table.to(DEV), torch.tensor(self.kv_lens, dtype=torch.int32, device=DEV),
                     self.starts.to(DEV), max(q_lens + [0]))

    def reference(self):
        return ref.attention(self.q, self.k, self.v, self.ks, self.vs, self.table, self.kv_lens, self.q_lens,
                             self.scale)


def check_attention(out, lse, want):
    o, l, mag, err = want
    got, got_lse = out.float().double().cpu(), lse.double().cpu()
    tol = mag * (2.0 ** -8 * 1.01 + 2 * err[..., None] + 2.0 ** -17) + 2.0 ** -8 * o.abs() + 1e-30
    bad = ((got - o).abs() > tol) | torch.isnan(got)
    assert not bad.any(), "out: %d of %d off, worst %.3g" % (bad.sum(), bad.numel(), (got - o).abs().max())
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(got_lse) & (got_lse < 0), empty)
    assert (got[empty] == 0).all()
    off = (got_lse - l).abs()[~empty]
    assert (off <= (err + 2.0 ** -18 * (1 + l.abs()))[~empty]).all(), float(off.max())


def run_attention(b, q=None, **kw):
    q = b.q.to(DEV) if q is None else q
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = att.paged_attention(q, *b.args, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


SHAPES = [(24, 4, 256), (8, 2, 128), (7, 1, 64)]


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("kv_lens,q_lens", [
    ([1], [1]), ([15, 16, 17], [1, 1, 1]), ([300, 1, 129, 64], [1, 1, 1, 1]), ([700], [7]), ([333, 77], [5, 9]),
    ([130], [130]), ([200, 31], [64, 31])], ids=str)
def test_attention(dtype, hq, hk, dim, kv_lens, q_lens):
    b = Batch(kv_lens, q_lens, hq, hk, dim, dtype=dtype, seed=sum(kv_lens) + dim)
    out, lse = run_attention(b)
    check_attention(out, lse, b.reference())


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page,order", [(16, "tokens"), (48, "heads"), (64, "tokens"), (112, "tokens"), (128, "heads"),
                                        (256, "heads")])
@pytest.mark.parametrize("q_lens", [[1, 1], [3, 40]], ids=str)
def test_attention_pages(dtype, page, order, q_lens):
    b = Batch([257, 500], q_lens, 6, 2, 128, page=page, dtype=dtype, order=order, seed=page)
    check_attention(*run_attention(b), b.reference())


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("kv_lens,q_lens", [([0], [3]), ([2], [5]), ([0, 5, 3, 40], [0, 0, 3, 50]), ([100, 0], [1, 1])],
                         ids=str)
@pytest.mark.parametrize("hq,hk,dim", [(6, 1, 256), (4, 4, 64), (128, 1, 128)])
def test_attention_rows_that_see_nothing(dtype, kv_lens, q_lens, hq, hk, dim):
    b = Batch(kv_lens, q_lens, hq, hk, dim, dtype=dtype, seed=3)
    check_attention(*run_attention(b), b.reference())


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("max_q", [1, 5, 500])
def test_attention_hint_does_not_change_the_result(dtype, max_q):
    """max_q_len chooses the kernel only."""
    b = Batch([90, 300], [33, 4], 12, 2, 256, dtype=dtype, seed=5)
    b.args = b.args[:-1] + (max_q,)
    check_attention(*run_attention(b), b.reference())


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens", [[2, 1], [40, 30]], ids=str)
def test_attention_strided_heads_and_output(dtype, q_lens):
    b = Batch([150, 260], q_lens, 6, 2, 128, dtype=dtype, seed=9)
    t = sum(q_lens)
    wide = torch.full((t, 10, 136), float("nan"), dtype=BF16, device=DEV)
    wide[:, 2:8, :128] = b.q.to(DEV)
    out = torch.full((6, t + 1, 128), 5.0, dtype=BF16, device=DEV)
    view = out[:, :t].permute(1, 0, 2)
    got, lse = run_attention(b, q=wide[:, 2:8, :128], out=view)
    assert got.data_ptr() == out.data_ptr()
    check_attention(view, lse, b.reference())
    assert (out[:, t] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens", [[3], [70]], ids=str)
def test_attention_extreme_scores(dtype, q_lens):
    """Scores far apart (weights that underflow) and far from zero."""
    b = Batch([400], q_lens, 4, 2, 128, dtype=dtype, seed=11)
    b.q = (b.q.float() * 40).to(BF16)
    check_attention(*run_attention(b), b.reference())
    b.q = torch.zeros_like(b.q)
    check_attention(*run_attention(b), b.reference())
    b.q = (torch.randn(b.q.shape, generator=torch.Generator().manual_seed(1)) * 1e-20).to(BF16)
    check_attention(*run_attention(b), b.reference())


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [2, 9, 100])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_attention_non_finite_rows_reach_only_the_tokens_that_see_them(dtype, q_len, what):
    """A new token whose key and value rows hold NaN (or, bf16, infinity): the
    tokens before it do not see them."""
    if dtype == E4M3 and what == float("inf"):
        pytest.skip("e4m3 has no infinity")
    n, at = 150, 150 - q_len // 2 - 1
    b = Batch([n], [q_len], 6, 2, 128, dtype=dtype, seed=13)
    page = int(b.table[0, at // 16])
    want = b.reference()
    k, v = to_dev(b.k), to_dev(b.v)
    for x in (k, v):
        raw = x.view(torch.uint8) if dtype == E4M3 else x
        raw[page, at % 16, :, 3] = 0x7F if dtype == E4M3 else what
    b.cache = att.KVCache(k, v, b.cache.k_scale, b.cache.v_scale)
    b.args = (b.cache,) + b.args[1:]
    out, lse = run_attention(b)
    clean = at - (n - q_len)                       # tokens 0 .. clean - 1 come before the bad row
    check_attention(out[:clean], lse[:clean], [x[:clean] for x in want])
    if math.isnan(what):
        assert torch.isnan(out[clean:]).all()


def test_attention_long_context_many_parts():
    b = Batch([20011], [2], 6, 1, 256, page=64, seed=17)
    check_attention(*run_attention(b), b.reference())
    b = Batch([20011], [1], 4, 4, 128, page=64, dtype=E4M3, seed=18)
    check_attention(*run_attention(b), b.reference())


def test_attention_many_sequences():
    g = torch.Generator().manual_seed(1)
    n = 700
    kv = torch.randint(1, 60, (n,), generator=g).tolist()
    ql = [min(int(x), k) for x, k in zip(torch.randint(0, 4, (n,), generator=g), kv)]
    b = Batch(kv, ql, 2, 1, 64, seed=19)
    check_attention(*run_attention(b), b.reference())


def test_attention_offsets_past_32_bits():
    """Pages beyond 2^32 elements from the start of the cache."""
    pages, page, hk, dim = (1 << 18) + 8, 16, 4, 256
    big = torch.empty(pages, page, hk, dim, dtype=BF16, device=DEV)
    b = Batch([70], [2], 8, 4, 256, page=page, seed=21, poison=False)
    n = b.k.shape[0]
    big[pages - n:] = b.k.to(DEV)
    v = torch.as_strided(big, (pages, page, hk, dim), big.stride())
    b.args = (att.KVCache(big, v), (b.table + (pages - n)).to(DEV)) + b.args[2:]
    b.v = b.k
    for q_hint in (2, 200):
        b.args = b.args[:-1] + (q_hint,)
        check_attention(*run_attention(b), b.reference())


def test_attention_on_another_stream_and_in_a_graph():
    b = Batch([500, 90], [1, 20], 12, 2, 256, seed=23)
    want = b.reference()
    s = torch.cuda.Stream()
    q = torch.zeros(b.q.shape, dtype=BF16, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        q.copy_(b.q.pin_memory(), non_blocking=True)
        lse = torch.empty(q.shape[:2], device=DEV)
        out = att.paged_attention(q, *b.args, lse=lse)
    s.synchronize()
    check_attention(out, lse, want)
    w = att.attention_workspace(b.cache)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        att.paged_attention(q, *b.args, out=out, lse=lse, workspace=w)
    w.fill_(0xFF)                                  # the workspace needs no set-up
    g.replay()
    torch.cuda.synchronize()
    check_attention(out, lse, want)


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens", [[1, 3], [200, 90]], ids=str)
def test_attention_repeats_bit_for_bit(dtype, q_lens):
    b = Batch([3000, 260], q_lens, 24, 4, 256, page=64, dtype=dtype, seed=25)
    q = b.q.to(DEV)
    a, la = run_attention(b, q)
    for _ in range(5):
        c, lc = run_attention(b, q)
        assert torch.equal(a, c) and torch.equal(la, lc)


def test_attention_tokens_outside_the_sequences_are_left_alone():
    b = Batch([50], [3], 4, 2, 128, seed=27)
    q = torch.cat([b.q, b.q]).to(DEV)
    out = torch.full(q.shape, 3.0, dtype=BF16, device=DEV)
    _, lse = run_attention(b, q, out=out)
    check_attention(out[:3], lse[:3], b.reference())
    assert (out[3:] == 3.0).all() and (lse[3:] == 7.0).all()


@pytest.mark.parametrize("what", ["table", "kv_len", "starts"])
@pytest.mark.parametrize("hint", [1, 300])
def test_attention_reports_indexes_out_of_range(what, hint):
    """A bad index of one sequence sets the error bit, makes no access, and
    leaves the other sequence's result right."""
    b = Batch([90, 64], [2, 3], 4, 2, 128, seed=29)
    cache, table, kv, starts, _ = b.args
    if what == "table":
        table[1, 2] = 1 << 20
    elif what == "kv_len":
        kv[1] = 1 << 20
    else:
        starts[2] = 9                              # past the token dimension
    lse = torch.zeros(b.q.shape[:2], device=DEV)
    out = att.paged_attention(b.q.to(DEV), cache, table, kv, starts, hint, lse=lse)
    torch.cuda.synchronize()
    assert att.attention_error() == att.ATTENTION_BAD_INDEX
    check_attention(out[:2], lse[:2], [x[:2] for x in b.reference()])


# ------------------------------------------------------------------- mass
@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("kv_lens,q_lens", [
    ([1], [1]), ([15, 16, 17], [1, 1, 1]), ([700], [7]), ([333, 77], [5, 9]), ([130], [130]), ([0, 5, 3], [0, 0, 6]),
    ([200, 31], [64, 31])], ids=str)
def test_mass(dtype, hq, hk, dim, kv_lens, q_lens):
    b = Batch(kv_lens, q_lens, hq, hk, dim, dtype=dtype, seed=sum(kv_lens) + dim + 1)
    _, lse, _, _ = b.reference()
    lse = lse.float()
    room = b.table.shape[1] * 16
    g = torch.Generator().manual_seed(2)
    before = torch.rand(len(kv_lens), hk, room, generator=g)
    for start in (None, before):
        want, tol = ref.mass(b.q, b.k, b.ks, b.table, kv_lens, q_lens, b.scale, lse, start, room)
        out = torch.full((len(kv_lens), hk, room), 9.0, device=DEV)
        got = att.attention_mass(b.q.to(DEV), *b.args, lse.to(DEV), None if start is None else start.to(DEV), out=out)
        torch.cuda.synchronize()
        off = (got.double().cpu() - want).abs()
        assert (off <= tol).all(), float((off - tol).max())
        for s, n in enumerate(kv_lens):
            assert (got[s, :, n:] == 0).all()
    acc = before.to(DEV)
    att.attention_mass(b.q.to(DEV), *b.args, lse.to(DEV), acc, out=acc)          # in place
    assert torch.equal(acc, got)


@pytest.mark.parametrize("page,order", [(48, "tokens"), (64, "heads"), (256, "tokens")])
@pytest.mark.parametrize("hint", [1, 400])
def test_mass_pages_rooms_and_hints(page, order, hint):
    b = Batch([257, 500], [3, 40], 6, 2, 128, page=page, order=order, seed=page)
    _, lse, _, _ = b.reference()
    room = 531
    want, tol = ref.mass(b.q, b.k, b.ks, b.table, b.kv_lens, b.q_lens, b.scale, lse.float(), None, room)
    b.args = b.args[:-1] + (hint,)
    out = torch.empty(2, 2, room, device=DEV)
    got = att.attention_mass(b.q.to(DEV), *b.args, lse.float().to(DEV), out=out)
    assert ((got.double().cpu() - want).abs() <= tol).all()
    again = att.attention_mass(b.q.to(DEV), *b.args, lse.float().to(DEV))
    assert again.shape == (2, 2, b.table.shape[1] * page)
    for s, n in enumerate(b.kv_lens):
        assert torch.equal(again[s, :, :n], got[s, :, :n])


def test_mass_of_every_query_sums_to_its_weight():
    """Each query head's weights sum to one."""
    b = Batch([1000], [300], 12, 2, 256, page=64, seed=31)
    q = b.q.to(DEV)
    _, lse = run_attention(b, q)
    got = att.attention_mass(q, *b.args, lse)
    total = got.double().sum(-1)
    assert torch.allclose(total, torch.full_like(total, 300 * 6.0), rtol=1e-5, atol=0)


# ------------------------------------------------------------------ norm_rope
@pytest.mark.parametrize("tokens", [1, 7, 130])
@pytest.mark.parametrize("hq,hk,dim,rot", [(24, 4, 256, 64), (24, 4, 256, 256), (8, 2, 128, 128), (5, 1, 128, 32),
                                           (3, 3, 64, 16), (2, 1, 64, 0)])
def test_norm_rope(tokens, hq, hk, dim, rot):
    g = torch.Generator().manual_seed(tokens + dim)
    qkv = (torch.randn((tokens, (hq + 2 * hk) * dim), generator=g) * 3).to(BF16)
    q, k = qkv[:, :hq * dim].view(tokens, hq, dim), qkv[:, hq * dim:(hq + hk) * dim].view(tokens, hk, dim)
    wq, wk = ((1 + torch.randn(dim, generator=g)).to(BF16) for _ in range(2))
    table = torch.randn((500, rot), generator=g) if rot else None
    pos = torch.randint(0, 500, (tokens,), generator=g)
    dq = qkv.to(DEV)
    v1 = dq[:, :hq * dim].view(tokens, hq, dim)
    v2 = dq[:, hq * dim:(hq + hk) * dim].view(tokens, hk, dim)
    dev = [x.to(DEV) if x is not None else None for x in (wq, wk, table, pos)]
    for place in ("new", "same"):
        o = att.qk_norm_rope(v1, v2, *dev, eps=1e-5, **({} if place == "new" else dict(q_out=v1, k_out=v2)))
        torch.cuda.synchronize()
        for got, x, w in ((o[0], q, wq), (o[1], k, wk)):
            want = ref.norm_rope(x, w, table, pos, 1e-5)
            size = want.abs().amax(-1, keepdim=True)
            tol = 2.0 ** -8 * want.abs() + 2.0 ** -18 * size
            off = (got.float().double().cpu() - want).abs()
            assert (off <= tol).all(), float((off - tol).max())
    assert torch.equal(dq[:, (hq + hk) * dim:].cpu(), qkv[:, (hq + hk) * dim:])      # v untouched


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim,rot,page,order", [(24, 4, 256, 64, 16, "heads"), (8, 2, 128, 128, 48, "tokens"),
                                                      (3, 1, 64, 32, 64, "heads")])
@pytest.mark.parametrize("tokens", [1, 75])
def test_norm_rope_store(dtype, hq, hk, dim, rot, page, order, tokens):
    g = torch.Generator().manual_seed(tokens + dim)
    q, k, v = (torch.randn((tokens, h, dim), generator=g).to(BF16) for h in (hq, hk, hk))
    v[0, 0, 0], v[-1, 0, 1] = 1e6, -1e6              # beyond e4m3's largest value
    wq, wk = ((1 + torch.randn(dim, generator=g)).to(BF16) for _ in range(2))
    table = torch.randn((500, rot), generator=g)
    pos = torch.randint(0, 500, (tokens,), generator=g)
    n = -(-tokens // page) + 2
    slots = torch.randperm(n * page, generator=g)[:tokens]
    if tokens > 2:
        slots[2] = -1
    shape = (n, hk, page, dim) if order == "heads" else (n, page, hk, dim)
    kc, vc = (torch.full(shape, 9, dtype=torch.uint8, device=DEV).view(E4M3) if dtype == E4M3
              else torch.full(shape, 9.0, dtype=BF16, device=DEV) for _ in range(2))
    if order == "heads":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    ks, vs = ((0.5 + torch.rand(hk, generator=g)) / 32 for _ in range(2)) if dtype == E4M3 else (None, None)
    cache = att.KVCache(kc, vc, *(x if x is None else x.to(DEV) for x in (ks, vs)))
    before = [x.contiguous().view(torch.uint8).clone() for x in (kc, vc)]
    out = att.qk_norm_rope_store(q.to(DEV), k.to(DEV), v.to(DEV), wq.to(DEV), wk.to(DEV), table.to(DEV), pos.to(DEV),
                                 cache, slots.to(DEV), eps=1e-6)
    torch.cuda.synchronize()
    want = ref.norm_rope(q, wq, table, pos, 1e-6)
    assert ((out.float().double().cpu() - want).abs()
            <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * want.abs().amax(-1, keepdim=True)).all()
    held = slots >= 0
    at = (slots[held] // page, slots[held] % page)
    for got, x, scale in ((kc, ref.norm_rope(k, wk, table, pos, 1e-6), ks), (vc, v.float().double(), vs)):
        x = x[held]
        got = got.float().cpu()[at].double()
        if dtype == E4M3:
            size = x.abs().amax(-1, keepdim=True) / scale.double()[:, None]
            x = (x / scale.double()[:, None]).clamp(-448, 448)
            tol = torch.maximum(2.0 ** -4 * x.abs(), torch.full_like(x, 2.0 ** -10)) + 2.0 ** -18 * size.clamp(max=448)
        else:
            tol = 2.0 ** -8 * x.abs() + 2.0 ** -18 * x.abs().amax(-1, keepdim=True)
        assert ((got - x).abs() <= tol).all()
    free = torch.ones(n, page, dtype=torch.bool)
    free[at] = False
    for got, b in zip((kc, vc), before):
        assert torch.equal(got.contiguous().view(torch.uint8).cpu()[free], b.cpu()[free])


def test_norm_rope_values_at_the_edges():
    """Rows of zeros, of one large value, and non-finite rows stay to themselves."""
    x = torch.zeros(4, 2, 128, dtype=BF16)
    x[1, 0, 5] = 1e30
    x[2, 1, 7] = float("nan")
    x[3, 0, 9] = 1e-30
    w = torch.ones(128, dtype=BF16)
    q, k = att.qk_norm_rope(x.to(DEV), x.to(DEV), w.to(DEV), w.to(DEV), None, None)
    q = q.float().cpu()
    assert (q[0] == 0).all() and torch.isnan(q[2, 1]).all() and (q[2, 0] == 0).all()
    assert torch.isfinite(q[3]).all()
    assert torch.equal(q, k.float().cpu()) or torch.isnan(q[2, 1]).all()


def test_norm_rope_reports_indexes_out_of_range():
    cache = att.new_kv_cache(2, 16, 2, 64)
    x = torch.ones(3, 2, 64, dtype=BF16, device=DEV)
    w = torch.ones(64, dtype=BF16, device=DEV)
    cs = torch.ones(10, 32, device=DEV)
    pos = torch.tensor([1, 2, 3], device=DEV)
    for bad_pos, bad_slot in ((10, 1), (-1, 1), (3, 32), (3, -2)):
        pos[1] = bad_pos
        att.qk_norm_rope_store(x, x, x, w, w, cs, pos, cache, torch.tensor([0, bad_slot, 2], device=DEV))
        torch.cuda.synchronize()
        assert att.attention_error() == att.ATTENTION_BAD_INDEX


# ------------------------------------------------------------------ evict
def run_evict(mass, kv_lens, keep, recent, dim=64, hk=2, page=16, to_page=16, dtype=BF16, order="heads", seed=0):
    g = torch.Generator().manual_seed(seed)
    table, n = ref.table_for(kv_lens, page, g)
    k, v = (ref.pages(n, page, hk, dim, dtype, order, g, 16.0) for _ in range(2))
    w = -(-keep // to_page)
    to_n = w * len(kv_lens) + 1
    to = att.new_kv_cache(to_n, to_page, hk, dim, dtype=dtype)
    to_table = torch.randperm(to_n, generator=g)[:w * len(kv_lens)].to(torch.int32).view(len(kv_lens), w)
    cache = att.KVCache(to_dev(k), to_dev(v))
    lens, index, new = att.evict(cache, table.to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV),
                                 mass.to(DEV), keep, recent, to, to_table.to(DEV))
    torch.cuda.synchronize()
    lens, index, new = lens.cpu(), index.cpu(), new.cpu()
    assert lens.tolist() == [min(x, keep) for x in kv_lens]
    for s, n in enumerate(kv_lens):
        for h in range(hk):
            want = ref.kept(mass[s, h], n, keep, recent)
            m = len(want)
            assert index[s, h, :m].tolist() == want and (index[s, h, m:] == -1).all()
            assert torch.equal(new[s, h, :m].view(torch.int32), mass[s, h, want].view(torch.int32))
            assert (new[s, h, m:] == 0).all()
            at, r = torch.tensor(want, dtype=torch.long), torch.arange(m)
            for src, dst in ((k, to.k), (v, to.v)):
                raw = torch.uint8 if dtype == E4M3 else torch.int16
                a = src.view(raw)[table[s].long()[at // page], at % page, h]
                b = dst.view(raw).cpu()[to_table[s].long()[r // to_page], r % to_page, h]
                assert torch.equal(a, b)
    return to


@pytest.mark.parametrize("kv_lens,keep,recent", [
    ([1], 1, 0), ([0, 3], 5, 2), ([100, 17, 64], 16, 4), ([100, 17, 64], 16, 16), ([100, 17, 64], 50, 0),
    ([3000, 1025, 1024], 1000, 31), ([5000], 4999, 1), ([40, 30], 1, 1)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_evict(kv_lens, keep, recent, dtype):
    g = torch.Generator().manual_seed(keep)
    room = max(kv_lens + [1]) + 3
    run_evict(torch.rand(len(kv_lens), 2, room, generator=g), kv_lens, keep, recent, dtype=dtype)


@pytest.mark.parametrize("kind", ["equal", "few", "signed", "special"])
def test_evict_ties_and_special_values(kind):
    g = torch.Generator().manual_seed(5)
    m = torch.randn(2, 2, 2500, generator=g)
    if kind == "equal":
        m = torch.full_like(m, 0.25)
    elif kind == "few":
        m = (m * 2).round() / 2
    elif kind == "special":
        at = torch.randint(0, 6, m.shape, generator=g)
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0)):
            m[at == i] = x
    run_evict(m, [2500, 1900], 700, 13)


@pytest.mark.parametrize("dim,page,to_page,order", [(256, 64, 16, "tokens"), (128, 48, 64, "heads"), (64, 16, 112, "tokens")])
@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_evict_pages_and_types(dim, page, to_page, order, dtype):
    g = torch.Generator().manual_seed(7)
    run_evict(torch.rand(3, 3, 400, generator=g), [400, 33, 250], 100, 10, dim=dim, hk=3, page=page, to_page=to_page,
              order=order, dtype=dtype)


def test_evict_a_context_longer_than_one_block_can_hold():
    g = torch.Generator().manual_seed(8)
    n = 300000
    m = torch.rand(1, 1, n, generator=g)
    m[0, 0, ::3] = 0.5
    run_evict(m, [n], 150000, 100, hk=1, page=64, to_page=64)


def test_evict_reports_indexes_out_of_range():
    cache, to = att.new_kv_cache(4, 16, 1, 64), att.new_kv_cache(4, 16, 1, 64)
    mass = torch.ones(1, 1, 64, device=DEV)
    t = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device=DEV)
    for kv, table, to_table in ((65, t, t), (-1, t, t), (64, t + 1, t), (64, t, t - 1)):
        att.evict(cache, table, torch.tensor([kv], dtype=torch.int32, device=DEV), mass, 64, 64, to, to_table)
        torch.cuda.synchronize()
        assert att.attention_error() == att.ATTENTION_BAD_INDEX


# ------------------------------------------------------------------ refusals
def test_the_binding_refuses():
    c = att.new_kv_cache(4, 16, 2, 64)
    q = torch.zeros(3, 4, 64, dtype=BF16, device=DEV)
    t = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    kv = torch.tensor([3], dtype=torch.int32, device=DEV)
    st = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    lse = torch.zeros(3, 4, device=DEV)
    fresh = att.new_kv_cache(4, 16, 2, 64)
    mass = torch.zeros(1, 2, 32, device=DEV)
    att.paged_attention(q, c, t, kv, st, 3)
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q.cpu()), dict(q=torch.zeros(3, 4, 128, dtype=BF16, device=DEV)),
                dict(t=t.long()), dict(t=t.expand(2, 2)), dict(kv=kv.long()), dict(kv=kv.cpu()), dict(st=st[:1]),
                dict(lse=lse.double()), dict(lse=lse[:2]), dict(out=q[:2]), dict(out=lse),
                dict(workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        a = dict(q=q, t=t, kv=kv, st=st, lse=lse, out=None, workspace=None)
        a.update(bad)
        with pytest.raises((TypeError, ValueError, att.Nvfp4Error)):
            att.paged_attention(a["q"], c, a["t"], a["kv"], a["st"], 3, out=a["out"], lse=a["lse"], workspace=a["workspace"])
    with pytest.raises(ValueError):
        att.attention_mass(q, c, t, kv, st, 3, lse, mass[:, :1])
    with pytest.raises((ValueError, att.Nvfp4Error)):
        att.evict(c, t, kv, mass, 100, 1, fresh, t)                   # to_table too narrow
    with pytest.raises(att.Nvfp4Error):
        att.evict(c, t, kv, mass, 4, 5, fresh, t)                     # recent > keep
    with pytest.raises(att.Nvfp4Error):
        att.evict(c, t, kv, mass, 4, 1, att.new_kv_cache(4, 16, 2, 64, dtype=E4M3), t)
    w = torch.ones(64, dtype=BF16, device=DEV)
    cs, pos = torch.zeros(8, 32, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError):
        att.qk_norm_rope(q, q, w, w, cs, pos.int())
    with pytest.raises(ValueError):
        att.qk_norm_rope(q, q, w[:32], w, cs, pos)
    with pytest.raises(att.Nvfp4Error):
        att.qk_norm_rope(q, q, w, w, torch.zeros(8, 24, device=DEV), pos)
    for shape, kw in (((4, 8, 2, 64), {}), ((4, 16, 2, 96), {})):
        x = torch.zeros(shape, dtype=BF16, device=DEV)
        with pytest.raises(att.Nvfp4Error):
            att.paged_attention(torch.zeros(3, 4, shape[3], dtype=BF16, device=DEV), att.KVCache(x, x), t, kv, st, 3,
                                workspace=torch.empty(1 << 26, dtype=torch.uint8, device=DEV))
    x = torch.zeros(4, 16, 2, 64, dtype=BF16, device=DEV)
    for bad in ((x, x[:, :, :1], None, None), (x, x.half(), None, None), (x.half(), x.half(), None, None), (x, x.cpu(), None, None),
                (x[..., ::2], x[..., ::2], None, None), (x, x, torch.ones(2, device=DEV), None)):
        with pytest.raises((TypeError, ValueError)):
            att.KVCache(*bad)
    torch.cuda.synchronize()
