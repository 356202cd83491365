"""The persistent pairs' kernel of the NVFP4 x NVFP4 products, plain and gated: sizes that give it more tiles of 128
rows by 128 outputs than the device has SMs, which is what chooses it, derived from the device."""
import os
import subprocess
import sys

import pytest
import torch

import _w4a4_ref as ref
from test_w4a4_gpu import BF16, DEV, FP32, gated64, hidden, no_device_error, pkg, product64, weight  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_for_pairs(outputs, extra):
    """The fewest rows, ending `extra` rows into a tile of 128, with more tiles than SMs for `outputs` outputs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 128 * (sms // (outputs // 128)) + extra


# outputs, k and rows into the last 128: single rows behind a tile, halves of a pair's tile without a row, one
# stage and more than the ring has, several tiles for a pair
SHAPES = [(1024, 512, 1), (2048, 256, 127), (4096, 512, 128), (1792, 1280, 70), (768, 1536, 5), (256, 768, 33)]


@pytest.mark.parametrize("outputs, k, extra", SHAPES, ids=str)
def test_gated(outputs, k, extra):
    m, n = rows_for_pairs(outputs, extra), 2 * outputs
    rows = pkg.quantize_rows(hidden(m, k, m + n + k).to(DEV), 30.0)
    w, w64, per_row = weight(n, k, n + 1, gs=[3.0 * k ** 0.5, 5.0 * k ** 0.5], rows=[n // 2, n // 2])
    want, err = gated64(rows, w64, per_row, 30.0, k)
    y = pkg.linear_w4a4_swiglu(rows, w)
    assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + err * (1 + 2.0 ** -8)).all())
    out_gs = 40.0
    h = pkg.linear_w4a4_swiglu_quantize(rows, w, out_gs)
    assert h.shape == (m, n // 2) and h.global_scale == out_gs
    want, err = (want * out_gs).cpu().unflatten(1, (-1, 16)), (err * out_gs).cpu().unflatten(1, (-1, 16))
    s = ref.e4m3(ref.plain_scales(h))
    top, slack = (want.abs().amax(-1) / 6).clamp(max=448.0), err.amax(-1) / 6
    assert bool(((s - top).abs() <= ((top + slack) * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + FP32) + slack).all())
    code = ref.E2M1[ref.unpack(h.codes)].unflatten(1, (-1, 16))
    v = code * s[:, :, None]
    q = want.abs() + err
    # half a code's step, what exceeds the largest code, and the product's own error
    half = torch.where(q <= 2 * s[:, :, None], 0.25, torch.where(q <= 4 * s[:, :, None], 0.5, 1.0)) * s[:, :, None]
    over = (q - 6 * s[:, :, None]).clamp(min=0.0)
    some = (s > 0)[:, :, None].expand_as(v)
    assert bool(((v - want).abs() <= half * (1 + FP32) + over + err)[some].all())


def test_gated_segments():
    """Segments of their own scales that end inside a tile, in either half."""
    outputs, k = 1024, 512
    m = rows_for_pairs(outputs, 9)
    parts, gs = [400, 624, 16, 752, 256], [60.0, 90.0, 40.0, 75.0, 120.0]
    rows = pkg.quantize_rows(hidden(m, k, 3).to(DEV), 30.0)
    w, w64, per_row = weight(2 * outputs, k, 4, gs=gs, rows=parts)
    want, err = gated64(rows, w64, per_row, 30.0, k)
    y = pkg.linear_w4a4_swiglu(rows, w)
    assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + err * (1 + 2.0 ** -8)).all())


def test_plain_and_gated_of_one_weight():
    """silu(gate) * up from the plain product's outputs, over tiles of 256 and of 192 weight rows."""
    for outputs, k, extra in ((4096, 256, 40), (1024, 2048, 130)):
        m = rows_for_pairs(outputs, extra)
        rows = pkg.quantize_rows(hidden(m, k, m).to(DEV), 30.0)
        w, w64, per_row = weight(2 * outputs, k, 6, gs=[30.0 * k ** 0.5] * 2, rows=[outputs] * 2)
        y = pkg.linear_w4a4(rows, w)
        want, total = product64(rows, w64, per_row, 30.0)
        assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + total * ref.product_bound(k)).all())
        z = pkg.linear_w4a4_swiglu(rows, w).double()
        g, u = y.double().chunk(2, 1)
        # each factor off by half a step of bf16, and either call's by its sum's error; |silu'| < 1.1
        silu = g * torch.sigmoid(g)
        eg, eu = (2 * total * ref.product_bound(k)).chunk(2, 1)
        eg, eu = eg + g.abs() * 2.0 ** -8, eu + u.abs() * 2.0 ** -8
        off = (z - silu * u).abs()
        bound = (1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (silu * u).abs() * 2.0 ** -8) * (1 + 2.0 ** -6) + 1e-30
        assert bool((off <= bound).all())


def layer(m, k=512, inner=1024, seed=51):
    """A feed-forward block whose three products are the pairs' for m rows, and one pass over it."""
    x, res = hidden(m, k, seed).to(DEV), hidden(m, k, seed + 1).to(DEV)
    nw = torch.ones(k, dtype=BF16, device=DEV)
    gu, dn = weight(2 * inner, k, seed + 2)[0], weight(1024, inner, seed + 3)[0]

    def run(stream=None):
        a, r = pkg.add_rms_norm_quantize(x, res, nw, 1e-6, 200.0, stream=stream)
        h = pkg.linear_w4a4_swiglu_quantize(a, gu, 90.0, stream=stream)
        return (pkg.linear_w4a4(h, dn, stream=stream), r, pkg.linear_w4a4_swiglu(a, gu, stream=stream), h.codes,
                ref.plain_scales(h) if stream is None and not torch.cuda.is_current_stream_capturing() else None)
    return run, (x, res)


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))


def test_repeated_calls_give_the_same_bits():
    run, _ = layer(rows_for_pairs(1024, 77))
    want = run()
    for _ in range(20):
        got = run()
        assert same(got, want) and torch.equal(got[4], want[4])


@pytest.mark.parametrize("kind", ["stream", "raw"])
def test_on_another_stream(kind):
    """Results on a stream that is not current, beside memory that the current one has freed and still writes."""
    run, _ = layer(rows_for_pairs(1024, 20))
    want = [t.clone() for t in run()[:4]]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        freed = [torch.empty_like(t) for t in want for _ in range(8)]
        torch.cuda._sleep(20_000_000)
        for t in freed:
            t.fill_(7)
        del freed, t
        got = run(s if kind == "stream" else s.cuda_stream)
        s.synchronize()
        torch.cuda.synchronize()
        assert same(got, want)


def test_two_streams_at_once():
    runs = [layer(rows_for_pairs(1024, e), seed=60 + e)[0] for e in (1, 100)]
    want = [run() for run in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    got = [[] for _ in runs]
    for _ in range(6):
        for run, s, g in zip(runs, streams, got):
            with torch.cuda.stream(s):
                g.append(run(s.cuda_stream))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(same(outs, w) for outs in g)


def test_captured_and_replayed():
    m = rows_for_pairs(1024, 64)
    run, (x, res) = layer(m)
    other = layer(m, seed=87)[0]
    graphs, outs = [], []
    for f in (run, other):
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for seed in (1, 2):
        x.copy_(hidden(m, x.shape[1], seed).to(DEV))
        res.copy_(hidden(m, x.shape[1], seed + 5).to(DEV))
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, (run(), other())):
            assert same(got, want)


_FIRST = """
import torch, nvfp4_block_scaled_linear_gb300 as pkg
dev = torch.device("cuda:0")
sms = torch.cuda.get_device_properties(0).multi_processor_count
m = 128 * (sms // 4) + 3                                           # 512 outputs: more tiles than SMs
w = pkg.Fp4Weight(torch.full((1024, 512), 0x22, dtype=torch.uint8, device=dev),
                  torch.full((1024, 64), 0x38, dtype=torch.uint8, device=dev), [1.0, 1024.0], [512, 512])
x = torch.ones((m, 1024), dtype=torch.bfloat16, device=dev)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    # (ones with the global scale 6: block scales of one, codes of 6, without a rounding; gate 1024, up 1)
    a = pkg.quantize_rows(x, 6.0)
    z, y, h = pkg.linear_w4a4_swiglu(a, w), pkg.linear_w4a4(a, w), pkg.linear_w4a4_swiglu_quantize(a, w, 6.0 / 1024)
g.replay()
torch.cuda.synchronize()
assert bool((z == 1024.0).all()), z
assert bool((y[:, :512] == 1024.0).all()) and bool((y[:, 512:] == 1.0).all()), y
assert bool((h.codes == 0x77).all())
at = torch.arange(m, device=dev)
at = (at // 128) * (512 // 64) * 512 + at % 32 * 16 + at // 32 % 4 * 4
for b in range(512 // 16):
    assert bool((h.scales.view(-1)[at + b // 4 * 512 + b % 4] == 0x38).all())
assert pkg.w4a4_error() == 0
"""


def test_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-1500:]


def test_padding_is_left_and_does_not_matter():
    m = rows_for_pairs(1024, 7)
    w = weight(2048, 512, 5)[0]
    a = pkg.quantize_rows(hidden(m, 512, 5).to(DEV))
    want = pkg.linear_w4a4_swiglu_quantize(a, w, 20.0)
    plain, gate = pkg.linear_w4a4(a, w), pkg.linear_w4a4_swiglu(a, w)
    left = torch.ones(a.scales.numel(), dtype=torch.bool)
    left[ref.scale_index(m, 512).flatten()] = False
    a.scales.view(-1)[left.to(DEV)] = 0x7F
    out = pkg.new_fp4_rows(m, 1024, 20.0)
    out.scales.fill_(0xAB)
    pkg.linear_w4a4_swiglu_quantize(a, w, 20.0, out=out)
    left = torch.ones(out.scales.numel(), dtype=torch.bool)
    left[ref.scale_index(m, 1024).flatten()] = False
    assert bool((out.scales.cpu().flatten()[left] == 0xAB).all())
    assert torch.equal(ref.plain_scales(out), ref.plain_scales(want)) and torch.equal(out.codes, want.codes)
    assert torch.equal(pkg.linear_w4a4(a, w), plain) and torch.equal(pkg.linear_w4a4_swiglu(a, w), gate)


def test_a_row_does_not_depend_on_the_others():
    m = rows_for_pairs(1024, 50)
    w = weight(2048, 512, 7)[0]
    x = hidden(m, 512, 7)
    a = pkg.quantize_rows(x.to(DEV))
    want, gate, h = pkg.linear_w4a4(a, w), pkg.linear_w4a4_swiglu(a, w), pkg.linear_w4a4_swiglu_quantize(a, w, 9.0)
    x[1::2] = float("nan")
    a = pkg.quantize_rows(x.to(DEV))
    y, z, q = pkg.linear_w4a4(a, w), pkg.linear_w4a4_swiglu(a, w), pkg.linear_w4a4_swiglu_quantize(a, w, 9.0)
    assert torch.equal(y[::2], want[::2]) and torch.equal(z[::2], gate[::2]) and torch.equal(q.codes[::2], h.codes[::2])
    assert bool(torch.isnan(y[1::2]).all()) and bool(torch.isnan(z[1::2]).all())
    byte = ref.plain_scales(q)
    assert bool((byte[1::2] == 0x7F).all()) and torch.equal(byte[::2], ref.plain_scales(h)[::2])
