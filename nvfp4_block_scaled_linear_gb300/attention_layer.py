"""One full-attention layer over the library's operators, as a serving loop
runs it: prompt in chunks, single tokens, a cache cut when it has grown.

    python -m nvfp4_block_scaled_linear_gb300.attention_layer [prompt] [chunk] [tokens] [keep]

draws a seeded layer of the 5120-wide model (24 query and 4 key/value heads of
256, 64 of them rotated; q/k/v 8192 x 5120 and o 5120 x 6144 in NVFP4), runs a
prompt in chunks through an e4m3 cache, generates tokens, cuts the cache to
``keep`` keys by the attention weight they received, generates again, and
prints the times and the largest difference that the cut made.
"""
import sys

import torch

from . import _lib
from .attention import (attention_mass, evict, new_kv_cache, paged_attention, qk_norm_rope_store)
from .inputs import make_linear


class AttentionLayer:
    """The projections' weights and the norms of one layer.

    qkv      (w_packed, w_scale, [gs_q, gs_k, gs_v]) of the stacked projections
    o        (w_packed, w_scale, gs)
    q_weight, k_weight   bfloat16 [head_dim]
    cos_sin  float32 [positions, rotary_dim]
    """

    def __init__(self, qkv, o, q_weight, k_weight, cos_sin, q_heads, kv_heads, head_dim, eps=1e-6):
        self.qkv, self.o = qkv, o
        self.q_weight, self.k_weight, self.cos_sin = q_weight, k_weight, cos_sin
        self.q_heads, self.kv_heads, self.head_dim, self.eps = q_heads, kv_heads, head_dim, eps

    def __call__(self, x, cache, slots, positions, block_table, kv_lens, q_starts, max_q_len,
                 mass=None):
        """x [T, hidden] -> [T, hidden].  The tokens' keys and values go to
        ``slots`` of the cache first; kv_lens counts them.  With ``mass`` (float32
        [S, kv_heads, room]) the weight that every key received is added to it."""
        hq, hk, d = self.q_heads, self.kv_heads, self.head_dim
        w, s, gs = self.qkv
        rows = [hq * d, hk * d, hk * d]
        y = _lib.linear_segmented(x, w, s, gs, rows)
        q, k, v = (t.unflatten(1, (-1, d)) for t in y.split(rows, dim=1))
        q = qk_norm_rope_store(q, k, v, self.q_weight, self.k_weight, self.cos_sin, positions,
                               cache, slots, eps=self.eps)
        lse = None
        if mass is not None:
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        seqs = (block_table, kv_lens, q_starts, max_q_len)
        out = paged_attention(q, cache, *seqs, lse=lse)
        if mass is not None:
            attention_mass(q, cache, *seqs, lse, mass, out=mass)
        return _lib.linear(out.flatten(1), *self.o)


def seeded_layer(hidden=5120, q_heads=24, kv_heads=4, head_dim=256, rotary_dim=64,
                 positions=65536, theta=1e7, seed=5, device="cuda"):
    """A layer with random weights of the given sizes."""
    dev = torch.device(device)
    width = q_heads * head_dim

    def projection(n, k, seed):
        t = make_linear(1, n, k, seed)
        # scales that keep the outputs near one for inputs near one
        gs = float(t.global_scale) * 2.0 * k ** 0.5
        return torch.from_numpy(t.w_packed).to(dev), torch.from_numpy(t.w_scale).to(dev), gs

    w, s, gs = projection((q_heads + 2 * kv_heads) * head_dim, hidden, seed)
    g = torch.Generator().manual_seed(seed)
    norms = [(1 + 0.2 * torch.randn(head_dim, generator=g)).to(torch.bfloat16).to(dev) for _ in range(2)]
    angle = (torch.arange(positions, dtype=torch.float64)[:, None]
             * theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim))
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(dev)
    return AttentionLayer((w, s, [gs] * 3), projection(hidden, width, seed + 1), *norms, cos_sin,
                          q_heads, kv_heads, head_dim)


def serve(layer, prompt, chunk, tokens, keep, recent=64, page=64, dtype=torch.float8_e4m3fn,
          seed=7):
    """A prompt in chunks, ``tokens`` single tokens, the cut to ``keep`` keys, and
    the same tokens again over the whole and over the cut cache.  Returns the
    outputs of the last over both, and the lengths of the two caches."""
    dev = layer.cos_sin.device
    hk, d = layer.kv_heads, layer.head_dim
    hidden = layer.qkv[0].shape[1] * 2
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((prompt + 2 * tokens, hidden), generator=g, device=dev).to(torch.bfloat16)
    total = prompt + 2 * tokens
    n_pages = -(-total // page)
    scale = torch.full((hk,), 1 / 32, device=dev) if dtype == torch.float8_e4m3fn else None
    cache = new_kv_cache(n_pages, page, hk, d, dtype, scale, scale, dev)
    table = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).view(1, -1)
    mass = torch.zeros((1, hk, n_pages * page), device=dev)

    def step(cache, table, at, position, n, mass=None):
        """n tokens at cache places `at` and on."""
        place = torch.arange(at, at + n, device=dev)
        slots = table[0].long()[place // page] * page + place % page
        return layer(x[position:position + n], cache, slots,
                     torch.arange(position, position + n, device=dev), table,
                     torch.tensor([at + n], dtype=torch.int32, device=dev),
                     torch.tensor([0, n], dtype=torch.int32, device=dev), n, mass)

    for a in range(0, prompt, chunk):
        step(cache, table, a, a, min(chunk, prompt - a), mass)
    for t in range(prompt, prompt + tokens):
        step(cache, table, t, t, 1, mass)
    held = prompt + tokens
    # the cut: fresh pages for the kept keys and the tokens to come
    width = -(-(keep + tokens) // page)
    small = new_kv_cache(width, page, hk, d, dtype, scale, scale, dev)
    to = torch.arange(width, dtype=torch.int32, device=dev).view(1, -1)
    lens, _, _ = evict(cache, table, torch.tensor([held], dtype=torch.int32, device=dev), mass, keep,
                       min(recent, keep), small, to)
    cut = int(lens)
    whole = [step(cache, table, t, t, 1) for t in range(held, total)]
    short = [step(small, to, cut + i, held + i, 1) for i in range(tokens)]
    return torch.cat(whole), torch.cat(short), held, cut


def main(argv=None):
    argv = sys.argv[1:] if argv is None else argv
    prompt, chunk, tokens, keep = ([int(v) for v in argv] + [8192, 2048, 16, 4096][len(argv):])[:4]
    layer = seeded_layer(positions=max(prompt + 2 * tokens, 256 + 2 * 2))
    serve(layer, min(prompt, 256), 128, 2, 64)                       # warm-up
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    whole, short, held, cut = serve(layer, prompt, chunk, tokens, keep)
    end.record()
    torch.cuda.synchronize()
    diff = (whole.float() - short.float()).abs().max() / whole.float().abs().max()
    print("prompt %d in chunks of %d, %d + 2 x %d tokens, cache cut from %d to %d keys: %.2f ms, "
          "largest difference over the cut cache %.3f of the largest output"
          % (prompt, chunk, tokens, tokens, held, cut, start.elapsed_time(end), float(diff)))


if __name__ == "__main__":
    main()
