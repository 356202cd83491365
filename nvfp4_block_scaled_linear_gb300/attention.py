"""ctypes binding of the attention block's operators (include/nvfp4_attention.h).

Between a full-attention layer's stacked q/k/v projection and its output
projection:

    cache = new_kv_cache(num_pages, page_size, kv_heads, head_dim)
    q = qk_norm_rope_store(q, k, v, q_weight, k_weight, cos_sin, positions, cache, slots)
    y = paged_attention(q, cache, block_table, kv_lens, q_starts, max_q_len)

and, to bound a long context's cache,

    mass = attention_mass(q, cache, block_table, kv_lens, q_starts, max_q_len, lse, mass)
    lens, index, mass = evict(cache, block_table, kv_lens, mass, keep, recent, to, to_table)

Argument marshalling only, as in ``_lib``: every step runs in the library's
kernels, on the current CUDA stream unless one is given (a ``torch.cuda.Stream``
or a raw handle).  What a call makes itself, results and workspaces, belongs to
the stream that it runs on, as under ``torch.cuda.stream(stream)``.
"""
import ctypes
import os
import re
import struct

import torch

from . import _lib
from ._lib import OK, Nvfp4Error

ATTENTION_HEADER = os.path.join(os.path.dirname(_lib.HEADER), "nvfp4_attention.h")

CACHE_BF16, CACHE_E4M3 = 0, 1
ATTENTION_TIMEOUT, ATTENTION_BAD_INDEX = 1, 2


# The C structures, packed into bytes (which a pointer argument takes as they
# are: a ctypes.Structure costs several times as much to fill).
_pack_heads = struct.Struct("@Pqq").pack                   # nvfp4_heads
_pack_cache = struct.Struct("@PPqqqqqqqPPiiii").pack       # nvfp4_kv_cache
_pack_seqs = struct.Struct("@PPPiii4x").pack               # nvfp4_sequences

_ready = None


def _library():
    global _ready
    if _ready is None:
        lib = _lib.load_library()
        P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        signatures = {
            "nvfp4_qk_norm_rope": [P, P, P, i64, i32, i32, i32, P, P, f32, P, i64, i32, P, P, P, P,
                                   P, P],
            "nvfp4_paged_attention": [P, i64, i32, P, P, f32, P, P, P, i64, P],
            "nvfp4_attention_mass": [P, i64, i32, P, P, f32, P, P, P, i64, P],
            "nvfp4_cache_evict": [P, P, P, i64, i32, i32, P, P, i32, P, P, P, P],
            "nvfp4_attention_status": [P, ctypes.c_int],
        }
        for name, args in signatures.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = ctypes.c_int, args
        lib.nvfp4_paged_attention_workspace.restype = i64
        lib.nvfp4_paged_attention_workspace.argtypes = [i32]
        _ready = lib
    return _ready


def attention_header_functions():
    """Names of the functions declared in include/nvfp4_attention.h."""
    text = open(ATTENTION_HEADER).read()
    return sorted(set(re.findall(r"^(?:int|int64_t) (nvfp4_\w+)\(", text, re.M)))


def attention_error(clear: bool = True) -> int:
    """The attention kernels' device error word (ATTENTION_TIMEOUT,
    ATTENTION_BAD_INDEX); synchronises."""
    bits = ctypes.c_uint(0)
    st = _library().nvfp4_attention_status(ctypes.byref(bits), 1 if clear else 0)
    if st != OK:
        raise Nvfp4Error(st, "nvfp4_attention_status")
    return bits.value


class KVCache:
    """A handle of a paged key/value cache, kept as long as its pages.

    k, v     CUDA tensors [num_pages, page_size, kv_heads, head_dim], bfloat16
             or float8_e4m3fn; any strides that are multiples of 16 bytes, the
             last dimension dense.  page_size a multiple of 16, head_dim 64,
             128 or 256.
    k_scale, v_scale   float32 [kv_heads], for float8_e4m3fn: a row stands for
             its codes times its head's scale (None: 1).
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be 4-D tensors of one shape and type, got %s %s and %s %s"
                             % (tuple(k.shape), k.dtype, tuple(v.shape), v.dtype))
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError("cache pages must be bfloat16 or float8_e4m3fn, got %s" % k.dtype)
        if not k.is_cuda or k.device != v.device:
            raise ValueError("cache pages must be CUDA tensors on one device")
        if k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("the last dimension of the cache pages must be dense")
        e4m3 = k.dtype == torch.float8_e4m3fn
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None:
                continue
            if not e4m3:
                raise ValueError("%s is for float8_e4m3fn pages" % name)
            if (t.dtype != torch.float32 or tuple(t.shape) != (k.shape[2],) or t.stride(0) != 1
                    or t.device != k.device):
                raise ValueError("%s must be float32 [%d] on %s" % (name, k.shape[2], k.device))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.device = k.device
        self._c = _pack_cache(
            k.data_ptr(), v.data_ptr(), self.num_pages, *k.stride()[:3], *v.stride()[:3],
            0 if k_scale is None else k_scale.data_ptr(),
            0 if v_scale is None else v_scale.data_ptr(),
            CACHE_E4M3 if e4m3 else CACHE_BF16, self.page_size, self.kv_heads, self.head_dim)


def new_kv_cache(num_pages, page_size, kv_heads, head_dim, dtype=torch.bfloat16, k_scale=None,
                 v_scale=None, device="cuda"):
    """A KVCache of fresh pages, each head's slots of a page side by side in
    memory (the order in which attention reads them).  The pages start at
    zero."""
    def pages():
        raw = torch.zeros((num_pages, kv_heads, page_size, head_dim),
                          dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype,
                          device=device)
        return raw.view(dtype).permute(0, 2, 1, 3)
    return KVCache(pages(), pages(), k_scale, v_scale)


def _heads(t, name, tokens, heads, dim, device):
    if t.dtype != torch.bfloat16:
        raise TypeError("%s must be bfloat16, got %s" % (name, t.dtype))
    if t.shape != (tokens, heads, dim) or t.device != device:
        raise ValueError("%s must have shape %s on %s, got %s on %s"
                         % (name, (tokens, heads, dim), device, tuple(t.shape), t.device))
    a, b, c = t.stride()
    if c != 1:
        raise ValueError("the last dimension of %s must be dense" % name)
    return _pack_heads(t.data_ptr(), a, b)


def _flat(t, name, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape %s on %s, got %s on %s"
                         % (name, tuple(shape), device, tuple(t.shape), t.device))
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """A tensor that belongs to `stream` (the device's current one by default):
    its memory is reused only in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(function, device, stream, *args):
    """One library call on `stream` (the device's current one by default)."""
    index = device.index
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    f = getattr(_ready or _library(), function)
    if index == torch._C._cuda_getDevice():
        st = f(*args, stream)
    else:
        with torch.cuda.device(device):
            st = f(*args, stream)
    if st != OK:
        raise Nvfp4Error(st, function)


def _norm_rope(q, k, v, q_weight, k_weight, cos_sin, positions, eps, q_out, k_out, cache, slots,
               stream):
    if not q.is_cuda or q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be CUDA tensors [tokens, heads, head_dim]")
    tokens, hq, dim = q.shape
    hk, dev = k.shape[1], q.device
    if cache is not None and (cache.kv_heads != hk or cache.head_dim != dim or cache.device != dev):
        raise ValueError("the cache holds %d heads of %d on %s, k has %d of %d on %s"
                         % (cache.kv_heads, cache.head_dim, cache.device, hk, dim, dev))
    rot = 0 if cos_sin is None else cos_sin.shape[1]
    rows = 0 if cos_sin is None else cos_sin.shape[0]
    qh, kh = _heads(q, "q", tokens, hq, dim, dev), _heads(k, "k", tokens, hk, dim, dev)
    qo = _heads(q_out, "q_out", tokens, hq, dim, dev)
    ko = None if k_out is None else _heads(k_out, "k_out", tokens, hk, dim, dev)
    vh = None if v is None else _heads(v, "v", tokens, hk, dim, dev)
    _call("nvfp4_qk_norm_rope", dev, stream, qh, kh, vh, tokens, hq, hk, dim,
          _flat(q_weight, "q_weight", torch.bfloat16, (dim,), dev),
          _flat(k_weight, "k_weight", torch.bfloat16, (dim,), dev), eps,
          None if cos_sin is None else _flat(cos_sin, "cos_sin", torch.float32, (rows, rot), dev),
          rows, rot,
          None if positions is None else _flat(positions, "positions", torch.int64, (tokens,), dev),
          qo, ko, None if cache is None else cache._c,
          None if slots is None else _flat(slots, "slots", torch.int64, (tokens,), dev))


def qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps=1e-6, q_out=None, k_out=None,
                 stream=None):
    """RMS norm of each head of q [T, Hq, D] and k [T, Hk, D] (bfloat16, may
    be strided views of one projection's output) with weights [D], and the
    rotation of the first cos_sin.shape[1] dimensions by the tokens'
    positions (int64 [T], rows of the float32 table cos_sin: cosines, then
    sines).  Without a table nothing is rotated.  Returns (q_out, k_out);
    they may be q and k themselves."""
    q_out = _empty(q.shape, q.dtype, q.device, stream) if q_out is None else q_out
    k_out = _empty(k.shape, k.dtype, k.device, stream) if k_out is None else k_out
    _norm_rope(q, k, None, q_weight, k_weight, cos_sin, positions, eps, q_out, k_out, None, None,
               stream)
    return q_out, k_out


def qk_norm_rope_store(q, k, v, q_weight, k_weight, cos_sin, positions, cache, slots, eps=1e-6,
                       out=None, stream=None):
    """As ``qk_norm_rope`` for q, with the key rows and the rows of v stored
    in the cache: token t's in slot slots[t] % page_size of page slots[t] //
    page_size (int64 [T]; -1 stores nothing).  Returns the queries."""
    out = _empty(q.shape, q.dtype, q.device, stream) if out is None else out
    _norm_rope(q, k, v, q_weight, k_weight, cos_sin, positions, eps, out, None, cache, slots,
               stream)
    return out


def _seqs(cache, block_table, kv_lens, q_starts, max_q_len):
    dev = cache.device
    n, width = block_table.shape
    return _pack_seqs(
        _flat(block_table, "block_table", torch.int32, (n, width), dev),
        _flat(kv_lens, "kv_lens", torch.int32, (n,), dev),
        0 if q_starts is None else _flat(q_starts, "q_starts", torch.int32, (n + 1,), dev),
        n, width, max_q_len)


_workspace_bytes = {}
_workspaces = {}                 # (device index, head_dim, raw current stream): workspace
_MAX_WORKSPACES = 16


def attention_workspace(cache, stream=None):
    """A workspace for ``paged_attention`` calls that run one after another."""
    key = (cache.device.index, cache.head_dim)
    if key not in _workspace_bytes:
        with torch.cuda.device(cache.device):
            _workspace_bytes[key] = _library().nvfp4_paged_attention_workspace(cache.head_dim)
    return _empty(_workspace_bytes[key], torch.uint8, cache.device, stream)


def release_workspaces():
    """Give the workspaces kept for the streams of earlier calls back to
    PyTorch's allocator."""
    _workspaces.clear()


def _call_workspace(cache, stream):
    """The workspace of a call on `stream`.  One is kept for each stream that is
    current when it is called on (asking the allocator for 80 MB costs some 8 us of
    host time), for the last few of them; a call on another stream than the
    current one, or that is being captured into a graph, gets one of its own."""
    index = cache.device.index
    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None and current != (stream if isinstance(stream, int) else stream.cuda_stream):
        return attention_workspace(cache, stream)
    # (the query is of the current device's stream)
    if index != torch._C._cuda_getDevice() or torch.cuda.is_current_stream_capturing():
        return attention_workspace(cache)
    key = (index, cache.head_dim, current)
    w = _workspaces.get(key)
    if w is None:
        while len(_workspaces) >= _MAX_WORKSPACES:
            _workspaces.pop(next(iter(_workspaces)), None)
        w = _workspaces[key] = attention_workspace(cache)
    return w


def paged_attention(q, cache, block_table, kv_lens, q_starts, max_q_len, scale=None, out=None,
                    lse=None, workspace=None, stream=None):
    """Attention of q [T, Hq, D] over the cache, causal from the end of each
    sequence: sequence s has tokens q_starts[s] .. q_starts[s + 1] - 1
    (int32 [S + 1]), which are the last of its kv_lens[s] cached keys (int32
    [S]), in the pages block_table[s] (int32 [S, width]).  max_q_len: the most
    tokens that any sequence has.  scale: of the scores (1 / sqrt(D)).  lse:
    float32 [T, Hq], written if given.  A token that sees no key gets 0 and
    -inf.  Returns out [T, Hq, D] bfloat16."""
    if q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [tokens, heads, head_dim]")
    tokens, hq, dim = q.shape
    dev = q.device
    if cache.head_dim != dim or cache.device != dev or hq % cache.kv_heads:
        raise ValueError("the cache holds %d heads of %d on %s, q has %d of %d on %s"
                         % (cache.kv_heads, cache.head_dim, cache.device, hq, dim, dev))
    if out is None:
        out = _empty((tokens, hq, dim), torch.bfloat16, dev, stream)
    if workspace is None:
        workspace = _call_workspace(cache, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s, got strides %s on %s"
                         % (dev, workspace.stride(), workspace.device))
    _call("nvfp4_paged_attention", dev, stream, _heads(q, "q", tokens, hq, dim, dev), tokens, hq,
          cache._c, _seqs(cache, block_table, kv_lens, q_starts, max_q_len),
          dim ** -0.5 if scale is None else scale, _heads(out, "out", tokens, hq, dim, dev),
          None if lse is None else _flat(lse, "lse", torch.float32, (tokens, hq), dev),
          workspace.data_ptr(), workspace.nbytes)
    return out


def attention_mass(q, cache, block_table, kv_lens, q_starts, max_q_len, lse, mass=None, scale=None,
                   out=None, stream=None):
    """mass[s, h, j] (float32 [S, Hk, room]; None: 0) plus the attention weight
    that key j of sequence s received from the query heads of group h in a
    ``paged_attention`` call with the same arguments that wrote ``lse``; 0 past
    the sequence's length.  Returns out, which may be mass itself."""
    if q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [tokens, heads, head_dim]")
    tokens, hq, dim = q.shape
    dev = q.device
    if cache.head_dim != dim or cache.device != dev or hq % cache.kv_heads:
        raise ValueError("the cache holds %d heads of %d on %s, q has %d of %d on %s"
                         % (cache.kv_heads, cache.head_dim, cache.device, hq, dim, dev))
    seqs = _seqs(cache, block_table, kv_lens, q_starts, max_q_len)
    n, width = block_table.shape
    if out is None:
        shape = (n, cache.kv_heads, width * cache.page_size) if mass is None else mass.shape
        out = _empty(shape, torch.float32, dev, stream)
    if out.dim() != 3:
        raise ValueError("out must be [sequences, kv_heads, room], got %s" % (tuple(out.shape),))
    room = out.shape[2]
    shape = (n, cache.kv_heads, room)
    _call("nvfp4_attention_mass", dev, stream, _heads(q, "q", tokens, hq, dim, dev), tokens, hq,
          cache._c, seqs, dim ** -0.5 if scale is None else scale,
          _flat(lse, "lse", torch.float32, (tokens, hq), dev),
          None if mass is None else _flat(mass, "mass", torch.float32, shape, dev),
          _flat(out, "out", torch.float32, shape, dev), room)
    return out


def evict(cache, block_table, kv_lens, mass, keep, recent, to, to_table, index=None, new_mass=None,
          new_lens=None, stream=None):
    """Cut every sequence to its newest min(recent, keep) keys and, head by
    head, the others with the most mass, ``keep`` in all at most, in their
    order; their rows move to the pages to_table (int32 [S, to_width]) of the
    cache ``to``, keeping their values (rounded once more where the caches' scales
    differ).  Returns (new_lens int32 [S], index int32 [S, Hk, keep]: the
    kept keys' old places, new_mass float32 [S, Hk, keep]); past a sequence's
    new length index is -1 and new_mass 0."""
    dev = cache.device
    seqs = _seqs(cache, block_table, kv_lens, None, 0)
    if mass.dim() != 3:
        raise ValueError("mass must be [sequences, kv_heads, room], got %s" % (tuple(mass.shape),))
    n, hk, room = block_table.shape[0], cache.kv_heads, mass.shape[2]
    if index is None:
        index = _empty((n, hk, keep), torch.int32, dev, stream)
    if new_mass is None:
        new_mass = _empty((n, hk, keep), torch.float32, dev, stream)
    if new_lens is None:
        new_lens = _empty(n, torch.int32, dev, stream)
    if to.device != dev or to_table.dim() != 2:
        raise ValueError("to must live on %s and to_table be 2-D" % dev)
    _call("nvfp4_cache_evict", dev, stream, cache._c, seqs,
          _flat(mass, "mass", torch.float32, (n, hk, room), dev), room, keep, recent, to._c,
          _flat(to_table, "to_table", torch.int32, (n, to_table.shape[1]), dev), to_table.shape[1],
          _flat(index, "index", torch.int32, (n, hk, keep), dev),
          _flat(new_mass, "new_mass", torch.float32, (n, hk, keep), dev),
          _flat(new_lens, "new_lens", torch.int32, (n,), dev))
    return new_lens, index, new_mass
