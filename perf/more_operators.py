"""The operators of layers whose activations are NVFP4 as well as their weights, as measured cases.

The library's linear layer multiplies NVFP4 weights with bf16 activations.  These
operators bring the activations to the same format (blocks of 16 along k: an e2m1
code per element, an e4m3 scale per block, one fp32 scale per tensor) and multiply
the two directly:

    norm          the residual's addition and the root-mean-square norm of each row, in bf16
    norm_project  the same into NVFP4 rows, and their product with a projection stacked
                  from three (q, k and v, each with a scale of its own)
    project       rows of a bf16 tensor quantised, and their product with one weight
    feed_forward  addition and norm into NVFP4 rows, the gated pair of projections with
                  silu(gate) * up quantised again as it is produced, and the projection back

Where `own` is false run() computes them with elementary torch operations in 32
bits; where it is true it calls the package's operators.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one generated token's norm: launch latency
        dict(name="norm_decode_1", op="norm", m=1, k=5120),
        # a prefill chunk's norm: bandwidth
        dict(name="norm_prompt_8192", op="norm", m=8192, k=5120),
        # an odd batch of a narrower model
        dict(name="norm_odd_357", op="norm", m=357, k=2048),
        # one token's norm and q/k/v projection: the weights' bytes and two launches
        dict(name="norm_qkv_decode_1", op="norm_project", m=1, k=5120, parts="6144 1024 1024"),
        # the same for a ragged batch of prompt chunks
        dict(name="norm_qkv_batch_1111", op="norm_project", m=1111, k=5120, parts="6144 1024 1024"),
        # speculative verify of 7 tokens through the output projection
        dict(name="o_verify_7", op="project", m=7, k=6144, n=5120),
        # a batch of 100 clients through the down projection
        dict(name="down_batch_100", op="project", m=100, k=17408, n=5120),
        # a prefill chunk through the output projection
        dict(name="o_prompt_8192", op="project", m=8192, k=6144, n=5120),
        # the feed-forward block for one token: its 150 MB of weights
        dict(name="ffn_decode_1", op="feed_forward", m=1, k=5120, inner=17408),
        # for 32 clients' tokens
        dict(name="ffn_batch_32", op="feed_forward", m=32, k=5120, inner=17408),
        # an odd chunk of a narrower model
        dict(name="ffn_odd_515", op="feed_forward", m=515, k=2048, inner=6144),
        # a prefill chunk: products
        dict(name="ffn_prompt_8192", op="feed_forward", m=8192, k=5120, inner=17408),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_project", "project", "project", "feed_forward", "feed_forward"])
    m = rng.choice([rng.randint(1, 8), rng.randint(9, 128), _log_int(rng, 129, 8192)])
    k = 256 * _log_int(rng, 1, 24)
    if op == "norm":
        return dict(op=op, m=m, k=rng.choice([k, 16 * _log_int(rng, 1, 512)]))
    if op == "norm_project":
        kv = 128 * rng.randint(1, 8)
        return dict(op=op, m=m, k=k, parts="%d %d %d" % (128 * rng.randint(1, 48), kv, kv))
    if op == "project":
        return dict(op=op, m=m, k=256 * _log_int(rng, 1, 68), n=128 * _log_int(rng, 1, 112))
    return dict(op=op, m=m, k=k, inner=256 * _log_int(rng, 1, 56))


def _parts(c):
    if c["op"] == "norm_project":
        return [int(n) for n in c["parts"].split()]
    return [c["n"]] if c["op"] == "project" else []


# ------------------------------------------------------------------ the inputs
def _weight(n, k, g):
    """A weight's packed codes and block scales, and the scale that makes its outputs near one for inputs near one."""
    packed = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.randint(0x20, 0x51, (n, k // 16), generator=g, device="cuda", dtype=torch.uint8)
    return packed, scale, 8.1 * math.sqrt(k)


def _rows(m, k, g):
    """Hidden states: rows of different size, and a few columns that stand out as trained models' do."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((m, 1), generator=g, device="cuda"))
    x[:, torch.randint(0, k, (max(1, k // 256),), generator=g, device="cuda")] *= 6.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    m, k = c["m"], c["k"]
    s = dict(case=c, x=_rows(m, k, g), gs=336.0, inner_gs=96.0)
    if c["op"] != "project":
        s["residual"] = _rows(m, k, g)
        s["norm_weight"] = (1.0 + 0.2 * torch.randn(k, generator=g, device="cuda")).to(torch.bfloat16)
    if c["op"] in ("project", "norm_project"):
        parts = _parts(c)
        packed, scale, gs = _weight(sum(parts), k, g)
        s["weight"] = packed, scale, [gs * (1.0 + 0.25 * i) for i in range(len(parts))], parts
    if c["op"] == "feed_forward":
        packed, scale, gs = _weight(2 * c["inner"], k, g)
        s["gate_up"] = packed, scale, [gs, gs * 1.25], [c["inner"]] * 2
        packed, scale, gs = _weight(k, c["inner"], g)
        s["down"] = packed, scale, [gs], [k]
    if own:
        # a program lays its weights' scales out once, when it loads them
        import nvfp4_block_scaled_linear_gb300 as nvfp4
        for name in ("weight", "gate_up", "down"):
            if name in s:
                packed, scale, gs, parts = s[name]
                s[name] = nvfp4.Fp4Weight(packed, scale, gs, parts)
    return s


# ------------------------------------------------------------------ plain forms
def _e2m1(x):
    """The nearest e2m1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6), ties to the even code, 6 beyond."""
    a = x.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, x)


def _nvfp4(x, gs):
    """x (fp32 [m, k]) rounded to NVFP4 with the tensor scale gs, as the values it stands for times gs."""
    t = x.unflatten(1, (-1, 16))
    scale = (t.abs().amax(-1, keepdim=True) * gs / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    code = torch.where(scale > 0, _e2m1(t * gs / torch.where(scale > 0, scale, torch.ones_like(scale))), torch.zeros_like(t))
    return (code * scale).flatten(1)


def _values(packed, scale):
    """A weight's codes times its block scales, fp32 [n, k]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(1).int()
    s = scale.view(torch.float8_e4m3fn).float()
    return (table[code].unflatten(1, (-1, 16)) * s[:, :, None]).flatten(1)


def _product(values, gs, weight):
    """NVFP4 rows (values times gs) through a weight stacked from parts with scales of their own, fp32."""
    packed, scale, scales, parts = weight
    y = torch.matmul(values, _values(packed, scale).t())
    per = torch.tensor([1.0 / (gs * w) for w in scales], dtype=torch.float64).float().cuda()
    return y * per.repeat_interleave(torch.tensor(parts, device="cuda"), output_size=sum(parts))


def _add_norm(s):
    r = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    f = r.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["norm_weight"].float()
    return y, r


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "project":
            return _product(_nvfp4(s["x"].float(), s["gs"]), s["gs"], s["weight"]).to(torch.bfloat16)
        y, r = _add_norm(s)
        if op == "norm":
            return y.to(torch.bfloat16), r
        a = _nvfp4(y, s["gs"])
        if op == "norm_project":
            return _product(a, s["gs"], s["weight"]).to(torch.bfloat16), r
        g, u = _product(a, s["gs"], s["gate_up"]).chunk(2, 1)
        h = _nvfp4(g / (1.0 + torch.exp(-g)) * u, s["inner_gs"])
        return _product(h, s["inner_gs"], s["down"]).to(torch.bfloat16), r
    import nvfp4_block_scaled_linear_gb300 as nvfp4
    if op == "norm":
        return nvfp4.add_rms_norm(s["x"], s["residual"], s["norm_weight"], EPS)
    if op == "project":
        return nvfp4.linear_w4a4(nvfp4.quantize_rows(s["x"], s["gs"]), s["weight"])
    a, r = nvfp4.add_rms_norm_quantize(s["x"], s["residual"], s["norm_weight"], EPS, s["gs"])
    if op == "norm_project":
        return nvfp4.linear_w4a4(a, s["weight"]), r
    h = nvfp4.linear_w4a4_swiglu_quantize(a, s["gate_up"], s["inner_gs"])
    return nvfp4.linear_w4a4(h, s["down"]), r


# ------------------------------------------------------------------ the work
def work(case):
    c = case
    m, k = c["m"], c["k"]
    if c["op"] == "norm":
        return {"bytes": m * k * 8 + k * 2, "flops": 6 * m * k}
    if c["op"] == "feed_forward":
        return {"bytes": m * k * 8 + k * 2 + 3 * k * c["inner"] * 9 // 16, "flops": 6 * m * k * c["inner"]}
    n = sum(_parts(c))
    rows = 2 if c["op"] == "project" else 6
    return {"bytes": m * k * rows + n * k * 9 // 16 + m * n * 2, "flops": 2 * m * n * k}


# ------------------------------------------------------------------ 64 bits
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest(x, values):
    """The place in `values` (ascending, from 0) of the nearest one to each |x|, ties to the even place, by comparing with the middles."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    mid = (v[1:] + v[:-1]) / 2
    a = x.abs().contiguous()
    low, high = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
    return v[torch.where(low % 2 == 0, low, high)]


def exact(case, seed):
    c = case
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    e4m3 = [(8 + i % 8) * 2.0 ** (i // 8 - 10) if i >= 8 else i * 2.0 ** -9 for i in range(127)]

    def rounded(x, gs):
        t = x.reshape(x.shape[0], -1, 16) * gs
        scale = _nearest(t.abs().max(-1).values / 6, e4m3)[:, :, None]
        code = _nearest(t / scale.clamp(min=2.0 ** -9), _E2M1)
        return (code * scale * t.sign() * (scale > 0) / gs).reshape(x.shape)

    def through(x, weight):
        packed, scale, scales, parts = weight
        w = torch.empty((packed.shape[0], 2 * packed.shape[1]), dtype=torch.float64, device="cuda")
        values = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
        for half in (0, 1):
            code = (packed // 16 if half else packed % 16).long()
            w[:, half::2] = values[code % 8] * (1 - 2 * (code // 8))
        block = torch.tensor(e4m3 + [math.nan], dtype=torch.float64, device="cuda")[scale.long()]
        w = (w.view(w.shape[0], -1, 16) * block[:, :, None]).view(w.shape)
        at = 0
        for n, gs in zip(parts, scales):
            w[at:at + n] /= gs
            at += n
        return x @ w.T

    if c["op"] == "project":
        return through(rounded(s["x"].double(), s["gs"]), s["weight"])
    # the stream of residuals is bf16: the norm is of what it holds
    total = s["x"].double() + s["residual"].double()
    f = total.to(torch.bfloat16).double()
    y = f / (f.square().sum(-1, keepdim=True) / f.shape[1] + EPS).sqrt() * s["norm_weight"].double()
    if c["op"] == "norm":
        return y, total
    y = rounded(y, s["gs"])
    if c["op"] == "norm_project":
        return through(y, s["weight"]), total
    z = through(y, s["gate_up"])
    g, u = z[:, :c["inner"]], z[:, c["inner"]:]
    return through(rounded(g * torch.sigmoid(g) * u, s["inner_gs"]), s["down"]), total
