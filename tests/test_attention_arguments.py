"""Arguments of the attention block's entry points that are refused on the
host: scales that are not positive and finite, batches of more sequences than
the schedule counts, a workspace out of alignment; on the GPU a workspace that
is too small, with the output left as it was."""
import ctypes

import pytest
import torch

from nvfp4_block_scaled_linear_gb300 import _lib
from nvfp4_block_scaled_linear_gb300 import attention as att
from nvfp4_block_scaled_linear_gb300 import build as cuda_build

A = 0x10000           # fake, aligned, never dereferenced
INVALID, MISALIGNED, SHAPE, TOO_LARGE = -1, -2, -3, -6


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    _lib.load_library()
    return att._library()


def _args(count=1):
    heads = att._pack_heads(A, 1024, 256)
    cache = att._pack_cache(A, A, 8, 16384, 256, 4096, 16384, 256, 4096, 0, 0, 0, 16, 4, 256)
    return heads, cache, att._pack_seqs(A, A, A, count, 4, 4)


def _attend(lib, scale=1.0, count=1, workspace=A):
    heads, cache, seqs = _args(count)
    return lib.nvfp4_paged_attention(heads, 4, 8, cache, seqs, scale, heads, None, workspace, 1 << 30, None)


def _mass(lib, scale=1.0, count=1):
    heads, cache, seqs = _args(count)
    return lib.nvfp4_attention_mass(heads, 4, 8, cache, seqs, scale, A, None, A, 64, None)


@pytest.mark.parametrize("call", [_attend, _mass])
@pytest.mark.parametrize("scale", [0.0, -0.0, -1.0, float("nan"), float("inf"), float("-inf")])
def test_scale_has_to_be_positive_and_finite(lib, call, scale):
    assert call(lib, scale=scale) == INVALID


@pytest.mark.parametrize("call", [_attend, _mass])
def test_more_sequences_than_are_counted(lib, call):
    text = open(att.ATTENTION_HEADER).read()
    assert "NVFP4_ATTENTION_MAX_SEQUENCES 8192" in text
    assert call(lib, count=8193) == SHAPE
    assert call(lib, count=-1) == INVALID


@pytest.mark.parametrize("offset", [4, 8, 16])
def test_workspace_alignment(lib, offset):
    assert _attend(lib, workspace=A + offset) == MISALIGNED


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 40])
def test_workspace_that_is_too_small(lib, tokens):
    dev = torch.device("cuda:0")
    cache = att.new_kv_cache(4, 16, 4, 64, torch.bfloat16, device=dev)
    q = torch.zeros((tokens, 8, 64), dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, 3.0)
    ws = att.attention_workspace(cache)
    need = ws.numel()
    table = torch.arange(4, dtype=torch.int32, device=dev).view(1, 4)
    lens = torch.tensor([64], dtype=torch.int32, device=dev)
    starts = torch.tensor([0, tokens], dtype=torch.int32, device=dev)
    heads = [att._pack_heads(t.data_ptr(), 8 * 64, 64) for t in (q, out)]
    s = att._pack_seqs(table.data_ptr(), lens.data_ptr(), starts.data_ptr(), 1, 4, tokens)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def call(size):
        return lib.nvfp4_paged_attention(heads[0], tokens, 8, cache._c, s, 0.125, heads[1], None, ws.data_ptr(), size, stream)
    assert call(need - 1) == TOO_LARGE
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    assert call(need) == 0
    torch.cuda.synchronize()
    assert bool((out == 0.0).all())                     # over the cache's zeros
    assert att.attention_error() == 0
