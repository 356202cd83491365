"""Calls with `stream=` while another stream is current: what a call makes itself
belongs to the stream that it runs on, so that memory which kernels of the
current stream still write is not handed to it."""
import pytest
import torch

from test_attention_gpu import BF16, DEV, E4M3, Batch, att, check_attention, no_device_error  # noqa: F401

pytestmark = pytest.mark.gpu


def _given(s, kind):
    return s if kind == "stream" else s.cuda_stream


@pytest.mark.parametrize("kind", ["stream", "raw"])
@pytest.mark.parametrize("q_lens", [[1, 2], [100, 30]], ids=str)
def test_workspace_beside_a_stream_that_still_writes_what_it_freed(kind, q_lens):
    b = Batch([3000, 900], q_lens, 24, 4, 256, page=64, seed=51)
    want = b.reference()
    q, s = b.q.to(DEV), torch.cuda.Stream()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        big = att.attention_workspace(b.cache)
        for _ in range(40):                            # some milliseconds of writes, all queued
            big.fill_(0x7F)
        del big
        for _ in range(10):
            att.paged_attention(q, *b.args, out=out, lse=lse, stream=_given(s, kind))
        s.synchronize()
        check_attention(out, lse, want)
        torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["stream", "raw"])
def test_results_beside_a_stream_that_still_writes_what_it_freed(kind):
    """Every result that a call makes itself, by its size and its value after both streams have ended."""
    b = Batch([300, 90], [5, 7], 8, 2, 128, seed=52)
    q, s = b.q.to(DEV), torch.cuda.Stream()
    w = torch.ones(128, dtype=BF16, device=DEV)
    lse = torch.zeros(q.shape[:2], device=DEV)
    att.paged_attention(q, *b.args, lse=lse)
    mass = att.attention_mass(q, *b.args, lse)
    to = att.new_kv_cache(8, 16, 2, 128)
    to_table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    k = torch.randn(12, 2, 128, device=DEV).to(BF16)
    slots = torch.full((12,), -1, dtype=torch.int64, device=DEV)
    calls = [lambda **kw: [att.paged_attention(q, *b.args, **kw)],
             lambda **kw: [att.attention_mass(q, *b.args, lse, **kw)],
             lambda **kw: list(att.qk_norm_rope(q, k, w, w, None, None, **kw)),
             lambda **kw: [att.qk_norm_rope_store(q, k, k, w, w, None, None, b.cache, slots, **kw)],
             lambda **kw: list(att.evict(b.cache, b.args[1], b.args[2], mass, 60, 3, to, to_table, **kw))]
    for call in calls:
        want = [x.clone() for x in call()]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        freed = [torch.empty_like(x) for x in want for _ in range(20)]
        torch.cuda._sleep(20_000_000)                  # about 10 ms
        for x in freed:
            x.view(torch.uint8).fill_(0x7F)
        del freed, x
        got = call(stream=_given(s, kind))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_capturing_stream_that_is_not_current():
    """The graph keeps no workspace that eager calls on its stream use."""
    b = Batch([500, 90], [1, 20], 12, 2, 256, dtype=E4M3, seed=53)
    want = b.reference()
    q, s = b.q.to(DEV), torch.cuda.Stream()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    att.paged_attention(q, *b.args, out=out, lse=lse, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with torch.cuda.stream(torch.cuda.Stream()):
            att.paged_attention(q, *b.args, out=out, lse=lse, stream=s)
    other = torch.zeros_like(q)
    for _ in range(5):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        att.paged_attention(q, *b.args, out=other, stream=s)
        torch.cuda.synchronize()
        check_attention(out, lse, want)
        assert torch.equal(out, other)


def test_kept_workspaces_are_bounded_and_given_back():
    b = Batch([300], [3], 8, 2, 128, seed=54)
    want = b.reference()
    q = b.q.to(DEV)
    att.release_workspaces()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    size = att.attention_workspace(b.cache).numel()
    for _ in range(40):
        with torch.cuda.stream(torch.cuda.Stream()):
            lse = torch.empty(q.shape[:2], device=DEV)
            out = att.paged_attention(q, *b.args, lse=lse)
        torch.cuda.synchronize()
        check_attention(out, lse, want)
    assert torch.cuda.memory_allocated() < before + 17 * size
    att.release_workspaces()
    assert torch.cuda.memory_allocated() < before + size
    out = att.paged_attention(q, *b.args, lse=lse)
    check_attention(out, lse, want)
