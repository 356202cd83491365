"""The attention block's C ABI on the host: every declared function is
exported, and bad arguments are rejected before a device is touched (no call
here gets past validation)."""
import ctypes

import pytest

from nvfp4_block_scaled_linear_gb300 import _lib
from nvfp4_block_scaled_linear_gb300 import attention as att
from nvfp4_block_scaled_linear_gb300 import build as cuda_build

A = 0x10000           # fake, 16-byte aligned, never dereferenced
INVALID, MISALIGNED, SHAPE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    _lib.load_library()
    return att._library()


def test_exports_and_constants(lib):
    names = att.attention_header_functions()
    assert len(names) == 6, names
    for n in names:
        assert hasattr(lib, n)
    text = open(att.ATTENTION_HEADER).read()
    for name, value in (("CACHE_BF16", 0), ("CACHE_E4M3", 1)):
        assert "#define NVFP4_%s %d" % (name, value) in text and getattr(att, name) == value
    for name, value in (("TIMEOUT", 1), ("BAD_INDEX", 2)):
        assert "#define NVFP4_ATTENTION_%s %du" % (name, value) in text
        assert getattr(att, "ATTENTION_" + name) == value


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("type", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Seqs(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("q_starts", ctypes.c_void_p),
                ("count", ctypes.c_int32), ("table_width", ctypes.c_int32), ("max_q_len", ctypes.c_int32)]


def heads(data=A, ts=1024, hs=256):
    return _Heads(data, ts, hs)


def cache(**kw):
    c = _Cache(A, A, 8, (ctypes.c_int64 * 3)(16384, 256, 4096), (ctypes.c_int64 * 3)(16384, 256, 4096), None, None, 0, 16,
               4, 256)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def seqs(**kw):
    s = _Seqs(A, A, A, 2, 4, 1)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_packed_structures_have_the_c_layout():
    assert len(att._pack_heads(A, 8, 16)) == ctypes.sizeof(_Heads)
    assert att._pack_heads(A, 8, 16) == bytes(_Heads(A, 8, 16))
    a = att._pack_cache(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15)
    assert a == bytes(_Cache(1, 2, 3, (ctypes.c_int64 * 3)(4, 5, 6), (ctypes.c_int64 * 3)(7, 8, 9), 10, 11, 12, 13, 14, 15))
    assert att._pack_seqs(1, 2, 3, 4, 5, 6) == bytes(_Seqs(1, 2, 3, 4, 5, 6))


BAD_CACHES = [(None, INVALID), (cache(k=None), INVALID), (cache(type=2), INVALID), (cache(num_pages=0), INVALID),
              (cache(page_size=24), SHAPE), (cache(page_size=0), INVALID), (cache(head_dim=96), SHAPE),
              (cache(kv_heads=0), INVALID), (cache(k=A + 8), MISALIGNED), (cache(k_scale=A), INVALID),
              (cache(v_stride=(ctypes.c_int64 * 3)(16384, 260, 4096)), MISALIGNED),
              (cache(k_stride=(ctypes.c_int64 * 3)(0, 256, 4096)), INVALID),
              (cache(k_stride=(ctypes.c_int64 * 3)(1 << 40, 256, 4096)), SHAPE)]


def test_paged_attention_rejects(lib):
    def call(q=heads(), t=4, hq=8, c=cache(), s=seqs(), out=heads(), ws=A):
        return lib.nvfp4_paged_attention(ref(q), t, hq, ref(c), ref(s), 1.0, ref(out), None, ws, 1 << 30, None)
    for c, st in BAD_CACHES:
        assert call(c=c) == st
    assert call(q=None) == INVALID and call(out=None) == INVALID and call(s=None) == INVALID
    assert call(q=heads(data=None)) == INVALID and call(ws=None) == INVALID
    assert call(q=heads(data=A + 2)) == MISALIGNED and call(out=heads(hs=12)) == MISALIGNED and call(ws=A + 4) == MISALIGNED
    assert call(q=heads(ts=-8)) == INVALID
    assert call(t=-1) == INVALID and call(hq=0) == INVALID and call(hq=6) == SHAPE and call(hq=4 * 129) == SHAPE
    assert call(t=1 << 31) == SHAPE
    assert call(s=seqs(count=-1)) == INVALID and call(s=seqs(table_width=0)) == INVALID
    assert call(s=seqs(kv_lens=None)) == INVALID and call(s=seqs(q_starts=None)) == INVALID
    assert call(s=seqs(max_q_len=-1)) == INVALID
    assert call(t=0, q=None) == 0 and call(s=seqs(count=0, block_table=None)) == 0           # nothing to do


def test_attention_mass_rejects(lib):
    def call(q=heads(), t=4, hq=8, c=cache(), s=seqs(), lse=A, out=A, room=64):
        return lib.nvfp4_attention_mass(ref(q), t, hq, ref(c), ref(s), 1.0, lse, None, out, room, None)
    for c, st in BAD_CACHES:
        assert call(c=c) == st
    assert call(q=None) == INVALID and call(lse=None) == INVALID and call(out=None) == INVALID
    assert call(room=0) == INVALID and call(room=1 << 31) == SHAPE and call(hq=9) == SHAPE
    assert call(s=seqs(count=0)) == 0


def test_qk_norm_rope_rejects(lib):
    def call(q=heads(), k=heads(), v=heads(), t=2, hq=8, hk=4, d=256, qw=A, kw=A, eps=1e-6, cs=A, rows=10, rot=64, pos=A,
             qo=heads(), ko=None, c=cache(), slots=A):
        return lib.nvfp4_qk_norm_rope(ref(q), ref(k), ref(v), t, hq, hk, d, qw, kw, eps, cs, rows, rot, pos, ref(qo),
                                      ref(ko), ref(c), slots, None)
    for c, st in BAD_CACHES[1:]:
        assert call(c=c) == st
    assert call(c=None) == INVALID                                  # neither a cache nor k_out
    assert call(ko=heads()) == INVALID                              # both
    assert call(c=None, ko=heads()) == INVALID                      # v and slots without a cache
    assert call(q=None) == INVALID and call(v=None) == INVALID and call(qo=None) == INVALID and call(slots=None) == INVALID
    assert call(qw=None) == INVALID and call(kw=A + 2) == MISALIGNED and call(k=heads(ts=4)) == MISALIGNED
    assert call(t=-1) == INVALID and call(hq=0) == INVALID and call(hk=0) == INVALID and call(eps=-1.0) == INVALID
    assert call(eps=float("nan")) == INVALID
    assert call(d=100) == SHAPE and call(d=128) == SHAPE and call(rot=24) == SHAPE and call(rot=272) == SHAPE
    assert call(cs=None) == INVALID and call(pos=None) == INVALID and call(rows=0) == INVALID and call(rot=-16) == INVALID
    assert call(t=0, q=None, k=None, v=None, qo=None, slots=None, pos=None) == 0


def test_cache_evict_rejects(lib):
    def call(c=cache(), s=seqs(), mass=A, room=64, keep=32, recent=4, to=cache(), tt=A, tw=2, index=A, nm=A, nl=A):
        return lib.nvfp4_cache_evict(ref(c), ref(s), mass, room, keep, recent, ref(to), tt, tw, index, nm, nl, None)
    for c, st in BAD_CACHES:
        assert call(c=c) == st and call(to=c) == st
    assert call(to=cache(type=1)) == INVALID and call(to=cache(head_dim=128)) == SHAPE and call(to=cache(kv_heads=2)) == SHAPE
    assert call(mass=None) == INVALID and call(tt=None) == INVALID and call(index=None) == INVALID
    assert call(nm=None) == INVALID and call(nl=None) == INVALID
    assert call(keep=0) == INVALID and call(recent=33) == INVALID and call(recent=-1) == INVALID and call(room=0) == INVALID
    assert call(keep=33) == SHAPE and call(tw=0) == INVALID
    assert call(s=seqs(count=0, block_table=None, kv_lens=None)) == 0
