"""The attention block's operators next to the NVFP4 projections, as measured cases.

A full-attention layer's stacked q/k/v projection leaves one row of heads per
token.  Four operators take it from there:

    norm_rope  RMS norm of every query and key head, rotation of the first
               `rot` dimensions by the token's position, and the key and value
               rows stored in a paged cache (bf16, or e4m3 with a scale per head)
    attend     softmax attention of a chunk of new tokens (one token in decode)
               over the paged cache, causal from the end of the sequence
    mass       the weight that each cached key has received from the chunk's
               queries, added to what it had received before
    evict      the keys with the most weight (and the newest ones) kept, their
               rows moved together into fresh pages

Where `own` is false run() computes them with elementary torch operations in 32
bits; where it is true it calls the package's operators.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one generated token of the 24/4-head, 256-wide attention, partial rotation: launch latency
        dict(name="norm_rope_decode_1", op="norm_rope", tokens=1, hq=24, hk=4, d=256, rot=64, page=16, fp8=False, head_major=True),
        # a whole prefill chunk stored in an e4m3 cache: bandwidth
        dict(name="norm_rope_prompt_8192_e4m3", op="norm_rope", tokens=8192, hq=24, hk=4, d=256, rot=64, page=64, fp8=True, head_major=True),
        # an odd batch of narrower heads, fully rotated, token-major pages
        dict(name="norm_rope_odd_357_d128", op="norm_rope", tokens=357, hq=32, hk=8, d=128, rot=128, page=32, fp8=False, head_major=False),
        # one token of one client over a context of 4K: latency
        dict(name="attend_decode_4099", op="attend", seqs=1, q_len=1, ctx=4099, hq=24, hk=4, d=256, page=16, fp8=False, head_major=True),
        # speculative verify: 7 tokens over a long e4m3 context
        dict(name="attend_verify_7_e4m3", op="attend", seqs=1, q_len=7, ctx=32771, hq=24, hk=4, d=256, page=64, fp8=True, head_major=True),
        # continuous batch of 32 clients, ragged contexts up to 16K
        dict(name="attend_batch_32", op="attend", seqs=32, q_len=1, ctx=16384, hq=24, hk=4, d=256, page=64, fp8=False, head_major=True),
        # a cold 8192-token prefill chunk
        dict(name="attend_prompt_8192", op="attend", seqs=1, q_len=8192, ctx=8192, hq=24, hk=4, d=256, page=64, fp8=False, head_major=True),
        # ragged chunks of three clients over longer e4m3 contexts, narrower heads
        dict(name="attend_chunk_e4m3_d128", op="attend", seqs=3, q_len=1111, ctx=20011, hq=32, hk=8, d=128, page=32, fp8=True, head_major=False),
        # weights received during one decode step of eight clients
        dict(name="mass_decode_8", op="mass", seqs=8, q_len=1, ctx=8209, hq=24, hk=4, d=256, page=64, fp8=False, head_major=True),
        # weights received from a chunk of prompt over a longer context
        dict(name="mass_chunk_2048", op="mass", seqs=1, q_len=2048, ctx=16411, hq=24, hk=4, d=256, page=64, fp8=False, head_major=True),
        # one long context cut to an eighth
        dict(name="evict_long", op="evict", seqs=1, ctx=65543, keep=8192, recent=1024, hq=24, hk=4, d=256, page=64, fp8=False, head_major=True),
        # ragged e4m3 contexts of a batch cut to 1000 keys each; the shortest ones keep all they have
        dict(name="evict_batch_16_e4m3", op="evict", seqs=16, ctx=9001, keep=1000, recent=64, hq=32, hk=8, d=128, page=32, fp8=True, head_major=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "attend", "attend", "mass", "evict"])
    hq, hk, d = rng.choice([(24, 4, 256), (24, 4, 256), (32, 8, 128), (8, 8, 128), (12, 1, 64), (14, 2, 64)])
    c = dict(op=op, hq=hq, hk=hk, d=d, page=rng.choice([16, 32, 48, 64, 128]), fp8=rng.random() < 0.4,
             head_major=rng.random() < 0.5)
    if op == "norm_rope":
        c.update(tokens=_log_int(rng, 1, 8192), rot=rng.choice([r for r in (32, 64, 128, 256) if r <= d]))
    elif op in ("attend", "mass"):
        q = rng.choice([1, rng.randint(2, 9), _log_int(rng, 10, 4096)])
        ctx = q + _log_int(rng, 1, 32768)
        # as many sequences as keep the work below the largest listed case's
        room = min(3e10 / (q * ctx * hq * d / 256), 2.5e9 / (ctx * hk * d * 4))
        c.update(q_len=q, ctx=ctx, seqs=_log_int(rng, 1, max(1, min(64, int(room)))))
    else:
        ctx = _log_int(rng, 64, 65536)
        keep = _log_int(rng, 16, max(16, ctx // 2))
        c.update(ctx=ctx, keep=keep, recent=rng.randint(0, keep),
                 seqs=_log_int(rng, 1, max(1, min(32, int(1.5e9 / (ctx * hk * d * 4))))))
    return c


def lengths(c):
    """Each sequence's new tokens and its cached keys (the new ones among them): the case's own
    largest values first, the others spread below them."""
    r = random.Random("%(seqs)d %(ctx)d" % c)
    new, kv = [], []
    for i in range(c["seqs"]):
        q = c.get("q_len", 0)
        q = q if i == 0 or q <= 1 else r.randint(1, q)
        new.append(q)
        kv.append(c["ctx"] if i == 0 else max(q, int(c["ctx"] * math.exp(-r.random() * 4))))
    return new, kv


# ------------------------------------------------------------------ the inputs
def _pages(c, n, g, fill):
    """k and v pages [n, page, hk, d], in the case's type and order of memory."""
    dev = torch.device("cuda")
    out = []
    for _ in range(2):
        shape = (n, c["hk"], c["page"], c["d"]) if c["head_major"] else (n, c["page"], c["hk"], c["d"])
        if fill:
            t = torch.empty(shape, dtype=torch.float8_e4m3fn if c["fp8"] else torch.bfloat16, device=dev)
            for i in range(0, n, 256):
                x = torch.randn((min(256, n - i),) + shape[1:], generator=g, device=dev)
                t[i:i + 256] = (x * 16.0 if c["fp8"] else x).to(t.dtype)
        else:
            t = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
            t = t.to(torch.float8_e4m3fn) if c["fp8"] else t
        out.append(t.permute(0, 2, 1, 3) if c["head_major"] else t)
    return out


def _scales(c, g, base):
    if not c["fp8"]:
        return None
    return base * (1.0 + 0.25 * torch.rand(c["hk"], generator=g, device="cuda"))


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    hq, hk, d, page = c["hq"], c["hk"], c["d"], c["page"]
    s = dict(case=c)
    if c["op"] == "norm_rope":
        t = c["tokens"]
        qkv = torch.randn((t, (hq + 2 * hk) * d), generator=g, device=dev)
        qkv *= torch.exp(0.5 * torch.randn((t, 1), generator=g, device=dev))
        qkv = qkv.to(torch.bfloat16)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
        for n in ("q_weight", "k_weight"):
            s[n] = (1.0 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16)
        first = 1000
        pos = torch.arange(first + t + 1, dtype=torch.float64, device=dev)
        inv = 1e7 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        ang = pos[:, None] * inv[None, :]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["positions"] = first + torch.arange(t, device=dev)
        n_pages = -(-t // page) + 3
        table = torch.randperm(n_pages, generator=g, device=dev)
        at = torch.arange(t, device=dev) + 5                      # the chunk starts inside a page
        s["slots"] = table[at // page] * page + at % page
        s["k_pages"], s["v_pages"] = _pages(c, n_pages, g, False)
        s["k_scale"], s["v_scale"] = _scales(c, g, 1 / 64), _scales(c, g, 1 / 32)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
    else:
        new, kv = lengths(c)
        width = -(-max(kv) // page)
        n_pages = sum(-(-n // page) for n in kv)
        table = torch.zeros((len(kv), width), dtype=torch.int32)
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(int(seed))).to(torch.int32)
        at = 0
        for i, n in enumerate(kv):
            m = -(-n // page)
            table[i, :m] = order[at:at + m]
            at += m
        s["k_pages"], s["v_pages"] = _pages(c, n_pages, g, True)
        s["k_scale"], s["v_scale"] = _scales(c, g, 1 / 16), _scales(c, g, 1 / 16)
        s["block_table"] = table.to(dev)
        s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        s["new"], s["kv"] = new, kv                               # the scheduler's own record of the lengths
        if c["op"] in ("attend", "mass"):
            t = sum(new)
            s["q"] = (1.5 * torch.randn((t, hq, d), generator=g, device=dev)).to(torch.bfloat16)
            s["q_starts"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=dev)
            s["out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
            s["lse"] = torch.empty((t, hq), dtype=torch.float32, device=dev)
        if c["op"] in ("mass", "evict"):
            room = width * page
            m = torch.rand((len(kv), hk, room), generator=g, device=dev) ** 8 * 20.0
            s["mass"] = m * (torch.arange(room, device=dev) < s["kv_lens"][:, None, None])
        if c["op"] == "mass":
            s["lse"] = _attend(s)[1]                              # the attention call before it left these
            s["mass_out"] = torch.empty_like(s["mass"])
        if c["op"] == "evict":
            # as evicted caches are: some keys have exactly the same weight
            s["mass"] = torch.where(s["mass"] < 0.01, torch.zeros_like(s["mass"]), s["mass"])
            w = -(-c["keep"] // page)
            s["k_fresh"], s["v_fresh"] = _pages(c, w * len(kv), g, False)
            s["fresh_table"] = torch.randperm(w * len(kv), generator=g, device=dev).to(torch.int32).view(len(kv), w)
    if own:
        # a serving program keeps a handle of its cache for as long as the cache lives
        import nvfp4_block_scaled_linear_gb300 as nvfp4
        s["cache"] = nvfp4.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        if c["op"] == "evict":
            s["fresh"] = nvfp4.KVCache(s["k_fresh"], s["v_fresh"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------------ plain forms
def _norm_rope(x, w, cos, sin):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    h = cos.shape[-1]
    a, b = y[..., :h], y[..., h:2 * h]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * h:]], -1)


def _store(pages, slots, x, scale):
    page = pages.shape[1]
    if pages.dtype == torch.float8_e4m3fn:
        x = (x / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        pages = pages.view(torch.uint8)
    else:
        x = x.to(pages.dtype)
    pages[slots // page, slots % page] = x


def _rows(pages, scale, table, n):
    """The first n cached rows of a sequence, [hk, n, d] in 32 bits."""
    page = pages.shape[1]
    x = pages[table[:-(-n // page)].long()].reshape(-1, pages.shape[2], pages.shape[3])[:n].float()
    if scale is not None:
        x = x * scale[:, None]
    return x.permute(1, 0, 2).contiguous()


def _hidden(q_len, n, device):
    """True where the i-th new token may not look: keys after its own place at the sequence's end."""
    at = torch.arange(n - q_len, n, device=device)
    return torch.arange(n, device=device)[None, :] > at[:, None]


def _scores(s, i, a):
    """[hk, group, q_len, kv_len] scores of sequence i, whose first token is a, hidden keys at -inf."""
    c, q_len, n = s["case"], s["new"][i], s["kv"][i]
    k = _rows(s["k_pages"], s["k_scale"], s["block_table"][i], n)
    q = s["q"][a:a + q_len].float().view(q_len, c["hk"], -1, c["d"]).permute(1, 2, 0, 3)
    x = torch.matmul(q.reshape(c["hk"], -1, c["d"]), k.transpose(1, 2)) * (1.0 / math.sqrt(c["d"]))
    x = x.view(c["hk"], -1, q_len, n)
    return x.masked_fill_(_hidden(q_len, n, x.device), -math.inf) if q_len > 1 else x


def _attend(s):
    c = s["case"]
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    a = 0
    for i, (q_len, n) in enumerate(zip(s["new"], s["kv"])):
        x = _scores(s, i, a)
        top = x.max(-1, keepdim=True).values
        x = x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        v = _rows(s["v_pages"], s["v_scale"], s["block_table"][i], n)
        y = torch.matmul(x.view(c["hk"], -1, n), v).view(c["hk"], -1, q_len, c["d"]) / total
        out[a:a + q_len] = y.permute(2, 0, 1, 3).reshape(q_len, c["hq"], c["d"]).to(out.dtype)
        lse[a:a + q_len] = (top + total.log())[..., 0].permute(2, 0, 1).reshape(q_len, c["hq"])
        a += q_len
    return out, lse


def _mass(s):
    c = s["case"]
    out = torch.zeros_like(s["mass"])
    a = 0
    for i, (q_len, n) in enumerate(zip(s["new"], s["kv"])):
        x = _scores(s, i, a)
        l = s["lse"][a:a + q_len].view(q_len, c["hk"], -1).permute(1, 2, 0)
        out[i, :, :n] = s["mass"][i, :, :n] + x.sub_(l[..., None]).exp_().sum((1, 2))
        a += q_len
    return out


def _evict(s):
    c = s["case"]
    keep, page = c["keep"], c["page"]
    seqs, hk = len(s["kv"]), c["hk"]
    lens = torch.clamp(s["kv_lens"], max=keep)
    index = torch.full((seqs, hk, keep), -1, dtype=torch.int32, device="cuda")
    mass = torch.zeros((seqs, hk, keep), device="cuda")
    raw = torch.uint8 if c["fp8"] else torch.bfloat16
    heads = torch.arange(hk, device="cuda")[:, None]
    for i, n in enumerate(s["kv"]):
        m = min(n, keep)
        newest = min(c["recent"], m)
        w = s["mass"][i, :, :n]
        best = torch.sort(w[:, :n - newest], dim=-1, descending=True, stable=True).indices[:, :m - newest]
        last = torch.arange(n - newest, n, device="cuda").expand(hk, newest)
        at = torch.cat([best.sort(-1).values, last], 1)
        index[i, :, :m] = at.to(torch.int32)
        mass[i, :, :m] = w.gather(1, at)
        src = s["block_table"][i].long()[at // page]
        to = torch.arange(m, device="cuda")
        dst = s["fresh_table"][i].long()[to // page].expand(hk, m)
        for a, b in ((s["k_pages"], s["k_fresh"]), (s["v_pages"], s["v_fresh"])):
            b.view(raw)[dst, (to % page).expand(hk, m), heads] = a.view(raw)[src, at % page, heads]
    return lens, index, mass, s["k_fresh"], s["v_fresh"]


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "norm_rope":
            h = s["cos_sin"].shape[1] // 2
            t = s["cos_sin"][s["positions"]][:, None, :]
            cos, sin = t[..., :h], t[..., h:]
            q = _norm_rope(s["q"], s["q_weight"], cos, sin).to(torch.bfloat16)
            _store(s["k_pages"], s["slots"], _norm_rope(s["k"], s["k_weight"], cos, sin), s["k_scale"])
            _store(s["v_pages"], s["slots"], s["v"].float(), s["v_scale"])
            return q, s["k_pages"], s["v_pages"]
        return {"attend": _attend, "mass": _mass, "evict": _evict}[c["op"]](s)
    import nvfp4_block_scaled_linear_gb300 as nvfp4
    if c["op"] == "norm_rope":
        nvfp4.qk_norm_rope_store(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"],
                                 s["cache"], s["slots"], eps=EPS, out=s["q_out"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    if c["op"] == "attend":
        nvfp4.paged_attention(s["q"], s["cache"], s["block_table"], s["kv_lens"], s["q_starts"], c["q_len"],
                              out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if c["op"] == "mass":
        return nvfp4.attention_mass(s["q"], s["cache"], s["block_table"], s["kv_lens"], s["q_starts"], c["q_len"],
                                    s["lse"], s["mass"], out=s["mass_out"])
    lens, index, mass = nvfp4.evict(s["cache"], s["block_table"], s["kv_lens"], s["mass"], c["keep"], c["recent"],
                                    s["fresh"], s["fresh_table"])
    return lens, index, mass, s["k_fresh"], s["v_fresh"]


# ------------------------------------------------------------------ the work
def work(case):
    c = case
    hq, hk, d = c["hq"], c["hk"], c["d"]
    size = 1 if c["fp8"] else 2
    if c["op"] == "norm_rope":
        t = c["tokens"]
        return {"bytes": t * ((2 * hq + 2 * hk) * d * 2 + 2 * hk * d * size + 4 * c["rot"] + 16) + 4 * d,
                "flops": t * (hq + hk) * (4 * d + 3 * c["rot"])}
    new, kv = lengths(c)
    pairs = sum(q * n - q * (q - 1) // 2 for q, n in zip(new, kv))
    if c["op"] == "attend":
        return {"bytes": sum(kv) * hk * d * 2 * size + sum(new) * hq * (4 * d + 4), "flops": 4 * pairs * hq * d}
    if c["op"] == "mass":
        return {"bytes": sum(kv) * hk * (d * size + 8) + sum(new) * hq * (2 * d + 4), "flops": 2 * pairs * hq * d}
    kept = sum(min(n, c["keep"]) for n in kv)
    return {"bytes": hk * (4 * sum(kv) + 4 * kept * d * size + 8 * len(kv) * c["keep"]), "flops": hk * sum(kv)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    hk, d, page = c["hk"], c["d"], c["page"]
    grp = c["hq"] // hk

    def f64(x):
        return x.to(torch.float32).double()

    if c["op"] == "norm_rope":
        rot = c["rot"]
        tab = s["cos_sin"].double()[s["positions"]]
        turn = torch.complex(tab[:, :rot // 2], tab[:, rot // 2:])[:, None, :]

        def turned(x, w):
            x = f64(x)
            x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * f64(w)
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
            x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
            return x

        found = [turned(s["q"], s["q_weight"])]
        for pages, x, scale in ((s["k_pages"], turned(s["k"], s["k_weight"]), s["k_scale"]),
                                (s["v_pages"], f64(s["v"]), s["v_scale"])):
            y = torch.zeros(pages.shape, dtype=torch.float64, device="cuda")
            if scale is not None:
                x = (x / scale.double()[None, :, None]).clamp(-448.0, 448.0)
            y[s["slots"] // page, s["slots"] % page] = x
            found.append(y)
        return tuple(found)

    if c["op"] == "evict":
        lens, index, mass, k, v = _kept(s)
        return None, None, mass, k, v

    def gathered(pages, scale, i, n, h):
        at = torch.arange(n, device="cuda")
        x = f64(pages[s["block_table"][i].long()[at // page], at % page, h])
        return x if scale is None else x * scale[h].double()

    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    mass = s["mass"].double().clone() if c["op"] == "mass" else None
    a = 0
    for i, (m, n) in enumerate(zip(s["new"], s["kv"])):
        for h in range(hk):
            k = gathered(s["k_pages"], s["k_scale"], i, n, h)
            v = gathered(s["v_pages"], s["v_scale"], i, n, h) if mass is None else None
            for g in range(h * grp, h * grp + grp):
                for b in range(0, m, 2048):
                    e = min(m, b + 2048)
                    x = f64(s["q"][a + b:a + e, g]) @ k.T / math.sqrt(d)
                    seen = torch.ones_like(x, dtype=torch.bool).tril(n - m + b)
                    x = x.where(seen, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                    if mass is not None:
                        mass[i, h, :n] += torch.exp(x - s["lse"][a + b:a + e, g].double()[:, None]).sum(0)
                        continue
                    l = torch.logsumexp(x, 1)
                    out[a + b:a + e, g] = torch.exp(x - l[:, None]) @ v
                    lse[a + b:a + e, g] = l
        a += m
    return mass if mass is not None else (out, lse)


def _kept(s):
    """evict on the host: the kept keys by sorting (weight, place) pairs."""
    c = s["case"]
    keep, page, hk = c["keep"], c["page"], c["hk"]
    w = s["mass"].double().cpu().numpy()
    index = np.full((len(s["kv"]), hk, keep), -1, dtype=np.int32)
    mass = np.zeros((len(s["kv"]), hk, keep))
    k = torch.zeros(s["k_fresh"].shape, dtype=torch.float64, device="cuda")
    v = torch.zeros(s["v_fresh"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["kv"]):
        m = min(n, keep)
        newest = min(c["recent"], m)
        for h in range(hk):
            old = w[i, h, :n - newest]
            at = np.lexsort((np.arange(old.size), -old))[:m - newest]
            at = np.concatenate([np.sort(at), np.arange(n - newest, n)])
            index[i, h, :m], mass[i, h, :m] = at, w[i, h, at]
            src = torch.from_numpy(at).cuda()
            to = torch.arange(m, device="cuda")
            dst = s["fresh_table"][i].long()[to // page]
            for a, b in ((s["k_pages"], k), (s["v_pages"], v)):
                rows = a[s["block_table"][i].long()[src // page], src % page, h]
                b[dst, to % page, h] = rows.to(torch.float32).double()
    return np.minimum(np.array(s["kv"], dtype=np.int32), keep), index, mass, k, v
