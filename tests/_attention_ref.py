"""Plain 64-bit forms of the attention block's operators, and random batches
for them.  Nothing here uses the package."""
import math

import torch


def pages(n, page, heads, dim, dtype, order, gen, amp=1.0):
    """[n, page, heads, dim] of normal values; `order` is the memory's order
    ("heads": a head's slots side by side; "tokens": a slot's heads)."""
    shape = (n, heads, page, dim) if order == "heads" else (n, page, heads, dim)
    x = (amp * torch.randn(shape, generator=gen)).to(dtype)
    return x.permute(0, 2, 1, 3) if order == "heads" else x


def table_for(kv_lens, page, gen, spare=2, width=0):
    """A block table of distinct pages in random order (unused entries -1)
    and the number of pages."""
    need = [-(-n // page) for n in kv_lens]
    width = max([width, 1] + need)
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen).to(torch.int32)
    t = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        t[i, :m] = order[at:at + m]
        at += m
    return t, total


def rows(pages_, scale, table, n, h):
    """The first n rows of head h, float64 [n, dim]."""
    page = pages_.shape[1]
    at = torch.arange(n)
    x = pages_.float().double()[table.long()[at // page], at % page, h]
    return x if scale is None else x * float(scale[h])


def attention(q, k, v, k_scale, v_scale, table, kv_lens, q_lens, scale):
    """(out, lse, mag, err): float64 [T, Hq, D], [T, Hq], the weighted sum of
    |v|, and the bound on a score's fp32 rounding errors: (D + 4) 2^-23 of the
    largest sum of |q||k|."""
    T, Hq, D = q.shape
    Hk = k.shape[2]
    out, mag = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    err = torch.zeros(T, Hq, dtype=torch.float64)
    a = 0
    for s, (n, m) in enumerate(zip(kv_lens, q_lens)):
        for h in range(Hq):
            g = h // (Hq // Hk)
            kk, vv = rows(k, k_scale, table[s], n, g), rows(v, v_scale, table[s], n, g)
            for i in range(m):
                seen = n - m + i + 1
                if seen <= 0:
                    continue
                x = q[a + i, h].float().double()
                sc = kk[:seen] @ x * scale
                err[a + i, h] = (D + 4) * 2.0 ** -23 * float((kk[:seen].abs() @ x.abs()).max()) * scale
                l = torch.logsumexp(sc, 0)
                p = torch.exp(sc - l)
                out[a + i, h], mag[a + i, h], lse[a + i, h] = p @ vv[:seen], p @ vv[:seen].abs(), l
        a += m
    return out, lse, mag, err


def mass(q, k, k_scale, table, kv_lens, q_lens, scale, lse, before, room):
    """(mass, count, score error bound): float64 [S, Hk, room] twice."""
    T, Hq, D = q.shape
    S, Hk = len(kv_lens), k.shape[2]
    out, tol = torch.zeros(S, Hk, room, dtype=torch.float64), torch.zeros(S, Hk, room, dtype=torch.float64)
    a = 0
    for s, (n, m) in enumerate(zip(kv_lens, q_lens)):
        for h in range(Hq):
            g = h // (Hq // Hk)
            kk = rows(k, k_scale, table[s], n, g)
            for i in range(m):
                seen = n - m + i + 1
                if seen <= 0:
                    continue
                x = q[a + i, h].float().double()
                w = torch.exp(kk[:seen] @ x * scale - lse[a + i, h].double())
                e = (D + 4) * 2.0 ** -23 * float((kk[:seen].abs() @ x.abs()).max()) * scale + 2.0 ** -18
                out[s, g, :seen] += w
                tol[s, g, :seen] += w * 2 * e
        if before is not None:
            out[s, :, :n] += before[s, :, :n].double()
        a += m
    return out, tol + out.abs() * 2.0 ** -18


def norm_rope(x, w, cos_sin, positions, eps):
    """float64 [T, H, D] of the normed and rotated heads."""
    x = x.float().double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.float().double()
    if cos_sin is None:
        return y
    r = cos_sin.shape[1] // 2
    c = cos_sin.double()[positions][:, None, :]
    a, b = y[..., :r].clone(), y[..., r:2 * r].clone()
    y[..., :r] = a * c[..., :r] - b * c[..., r:]
    y[..., r:2 * r] = b * c[..., :r] + a * c[..., r:]
    return y


def kept(mass_row, n, keep, recent):
    """The kept places of one sequence and head, ascending."""
    m = min(n, keep)
    newest = min(recent, m)
    old = [(float("inf") if math.isnan(x) else x, math.isnan(x)) for x in mass_row[:n - newest].tolist()]
    best = sorted(range(n - newest), key=lambda j: (not old[j][1], -old[j][0], j))[:m - newest]
    return sorted(best) + list(range(n - newest, n))
