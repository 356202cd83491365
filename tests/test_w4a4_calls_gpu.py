"""How the NVFP4 x NVFP4 operators are called: refusals of the binding, streams, captured graphs, repeated and
concurrent calls, offsets beyond 32 bits, padding left as it was."""
import pytest
import torch

import _w4a4_ref as ref
from test_w4a4_gpu import BF16, DEV, hidden, no_device_error, pkg, product64, weight  # noqa: F401

pytestmark = pytest.mark.gpu


def test_binding_refuses():
    x = hidden(4, 512, 1).to(DEV)
    w, _, _ = weight(512, 512, 1)
    nw = torch.ones(512, dtype=BF16, device=DEV)
    rows = pkg.quantize_rows(x)
    for bad in (x.float(), x.half()):
        with pytest.raises(TypeError):
            pkg.quantize_rows(bad)
        with pytest.raises(TypeError):
            pkg.add_rms_norm(bad, None, nw)
        with pytest.raises(TypeError):
            pkg.add_rms_norm(x, bad, nw)
        with pytest.raises(TypeError):
            pkg.add_rms_norm(x, None, bad[0])
    for bad in (x.cpu(), x[0], x[:, :500].contiguous(), x[:, :500], x[:, ::2]):
        with pytest.raises((ValueError, RuntimeError)):
            pkg.quantize_rows(bad)
    for bad in (x.cpu(), x[:2], x[:, :256], x.t().contiguous().t()):
        with pytest.raises((ValueError, RuntimeError)):
            pkg.add_rms_norm(x, bad, nw)
    with pytest.raises(ValueError):
        pkg.add_rms_norm(x, None, nw[:256])
    with pytest.raises(ValueError):
        pkg.add_rms_norm(x, None, nw.cpu())
    with pytest.raises(ValueError):
        pkg.add_rms_norm(x, None, nw, out=x[:2])
    with pytest.raises(RuntimeError):
        pkg.add_rms_norm(x, None, nw, eps=-1.0)
    for gs in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            pkg.quantize_rows(x, gs)
        with pytest.raises(ValueError):
            pkg.add_rms_norm_quantize(x, None, nw, 1e-6, gs)
        with pytest.raises(ValueError):
            pkg.linear_w4a4_swiglu_quantize(rows, w, gs)
        with pytest.raises(ValueError):
            pkg.Fp4Weight(w.codes, torch.zeros((512, 32), dtype=torch.uint8, device=DEV), gs)
        with pytest.raises(ValueError):
            pkg.new_fp4_rows(1, 256, gs)
    with pytest.raises(ValueError):
        pkg.quantize_rows(x, 2.0, out=pkg.new_fp4_rows(4, 512, 1.0))
    with pytest.raises(ValueError):
        pkg.quantize_rows(x, out=pkg.new_fp4_rows(5, 512))
    for bad in ((x, w), (rows, w.codes), (w, w), (rows, rows)):
        for call in (pkg.linear_w4a4, pkg.linear_w4a4_swiglu, pkg.linear_w4a4_swiglu_quantize):
            with pytest.raises(TypeError):
                call(*bad)
    with pytest.raises(ValueError):
        pkg.linear_w4a4(pkg.quantize_rows(x[:, :256]), w)
    with pytest.raises(ValueError):
        pkg.linear_w4a4(rows, w, out=torch.empty((4, 512), device=DEV))
    with pytest.raises(ValueError):
        pkg.linear_w4a4(rows, w, out=torch.empty((4, 1024), dtype=BF16, device=DEV)[:, :512])
    with pytest.raises(ValueError):
        pkg.linear_w4a4_swiglu_quantize(rows, weight(768, 512, 1)[0])
    with pytest.raises(RuntimeError):
        pkg.linear_w4a4_swiglu(rows, weight(384, 512, 1)[0])
    for m, k in ((-1, 256), (1, 0), (1, 128)):
        with pytest.raises(ValueError):
            pkg.new_fp4_rows(m, k)


def test_weights_refused():
    packed = torch.zeros((256, 256), dtype=torch.uint8, device=DEV)
    scale = torch.full((256, 32), 0x38, dtype=torch.uint8, device=DEV)
    pkg.Fp4Weight(packed, scale, 1.0)
    pkg.Fp4Weight(packed, scale.view(torch.float8_e4m3fn), [1.0, 2.0], [16, 240])
    for args in ((packed.cpu(), scale, 1.0), (packed, scale[:, :16], 1.0), (packed[:100], scale[:100], 1.0),
                 (packed[:, :64], scale[:, :8], 1.0), (packed, scale, [1.0, 2.0]), (packed, scale, [1.0, 2.0], [256]),
                 (packed, scale, [1.0, 2.0], [250, 6]), (packed, scale, [1.0, 2.0], [128, 64]), (packed, scale, [], []),
                 (packed, scale, [1.0] * 9, [16] * 8 + [128]), (packed.t(), scale, 1.0)):
        with pytest.raises(ValueError):
            pkg.Fp4Weight(*args)
    with pytest.raises(TypeError):
        pkg.Fp4Weight(packed.float(), scale, 1.0)
    for byte in (0x7F, 0xFF, 0x81, 0xB8, 0xFE):
        bad = scale.clone()
        bad[131, 17] = byte
        with pytest.raises(ValueError):
            pkg.Fp4Weight(packed, bad, 1.0)
    zero = scale.clone()
    zero[131, 17] = 0x80                                            # -0
    w = pkg.Fp4Weight(packed, zero, 1.0)
    want = scale.cpu().clone()
    want[131, 17] = 0
    assert torch.equal(ref.plain_scales(w), want)


def layer(m, k=512, inner=768, seed=31):
    """A feed-forward block's inputs and one pass over it."""
    x, res = hidden(m, k, seed).to(DEV), hidden(m, k, seed + 1).to(DEV)
    nw = torch.ones(k, dtype=BF16, device=DEV)
    gu, dn = weight(2 * inner, k, seed + 2)[0], weight(k, inner, seed + 3)[0]

    def run(stream=None):
        a, r = pkg.add_rms_norm_quantize(x, res, nw, 1e-6, 200.0, stream=stream)
        h = pkg.linear_w4a4_swiglu_quantize(a, gu, 90.0, stream=stream)
        z = pkg.linear_w4a4_swiglu(a, gu, stream=stream)
        n, _ = pkg.add_rms_norm(x, res, nw, stream=stream)
        q = pkg.quantize_rows(n, 50.0, stream=stream)
        return pkg.linear_w4a4(h, dn, stream=stream), r, z, n, pkg.linear_w4a4_swiglu(q, gu, stream=stream)
    return run, (x, res)


@pytest.mark.parametrize("m", [1, 33, 300, 900])
def test_repeated_calls_give_the_same_bits(m):
    run, _ = layer(m)
    want = run()
    for _ in range(20):
        for a, b in zip(run(), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("m", [1, 40, 600])
@pytest.mark.parametrize("kind", ["stream", "raw"])
def test_on_another_stream(m, kind):
    """Results on a stream that is not current, beside memory that the current one has freed and still writes."""
    run, _ = layer(m)
    want = [t.clone() for t in run()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        freed = [torch.empty_like(t) for t in want for _ in range(8)]
        torch.cuda._sleep(20_000_000)                               # about 10 ms
        for t in freed:
            t.fill_(7.0)
        del freed, t
        got = run(s if kind == "stream" else s.cuda_stream)
        s.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    runs = [layer(m, seed=40 + m)[0] for m in (5, 200, 700)]
    want = [run() for run in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    got = [[] for _ in runs]
    for _ in range(10):
        for run, s, g in zip(runs, streams, got):
            with torch.cuda.stream(s):
                g.append(run())
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for outs in g:
            for a, b in zip(outs, w):
                assert torch.equal(a, b)


@pytest.mark.parametrize("m", [1, 64, 400])
def test_captured_and_replayed(m):
    run, (x, res) = layer(m)
    other = layer(m, seed=77)[0]
    run()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in (run, other):
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
            for a, b in zip(got, want):
                assert torch.equal(a, b)


_FIRST = """
import torch, nvfp4_block_scaled_linear_gb300 as pkg
dev = torch.device("cuda:0")
w = pkg.Fp4Weight(torch.full((512, 512), 0x22, dtype=torch.uint8, device=dev),
                  torch.full((512, 64), 0x38, dtype=torch.uint8, device=dev), 1.0)
xs = [torch.ones((m, 1024), dtype=torch.bfloat16, device=dev) for m in (1, 100, 1000)]
nw = torch.ones(1024, dtype=torch.bfloat16, device=dev)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    # (ones with the global scale 6: block scales of one, codes of 6, without a rounding)
    ys = [pkg.linear_w4a4(pkg.quantize_rows(x, 6.0), w) for x in xs]
    zs = [pkg.linear_w4a4_swiglu_quantize(pkg.add_rms_norm_quantize(x, x, nw)[0], w) for x in xs]
g.replay()
torch.cuda.synchronize()
assert all(bool((y == 1024.0).all()) for y in ys), ys
assert pkg.w4a4_error() == 0
"""


def test_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-1500:]


def test_back_to_back_over_the_same_buffers():
    """A chain of products whose rows and results live in the same memory, with nothing between them: each reads
    what the one before wrote."""
    m, k = 48, 1024
    w = [weight(k, k, 60 + i)[0] for i in range(4)]
    x = hidden(m, k, 6, 0.2).to(DEV)
    rows, y = pkg.new_fp4_rows(m, k, 100.0), torch.empty((m, k), dtype=BF16, device=DEV)

    def chain(wait):
        y.copy_(x)
        for i in range(24):
            pkg.quantize_rows(y, 100.0, out=rows)
            if wait:
                torch.cuda.synchronize()
            pkg.linear_w4a4(rows, w[i % 4], out=y)
            if wait:
                torch.cuda.synchronize()
        return y.clone()
    want = chain(True)
    for _ in range(10):
        assert torch.equal(chain(False), want)


@pytest.mark.parametrize("m", [3, 130, 600])
def test_padding_of_gated_rows_is_left(m):
    w = weight(1024, 512, 5)[0]
    a = pkg.quantize_rows(hidden(m, 512, 5).to(DEV))
    out = pkg.new_fp4_rows(m, 512, 20.0)
    out.scales.fill_(0xAB)
    guard = out.codes.clone().fill_(0xCD)
    out.codes.copy_(guard)
    pkg.linear_w4a4_swiglu_quantize(a, w, 20.0, out=out)
    want = pkg.linear_w4a4_swiglu_quantize(a, w, 20.0)
    left = torch.ones(out.scales.numel(), dtype=torch.bool)
    left[ref.scale_index(m, 512).flatten()] = False
    assert bool((out.scales.cpu().flatten()[left] == 0xAB).all())
    assert torch.equal(ref.plain_scales(out), ref.plain_scales(want)) and torch.equal(out.codes, want.codes)


@pytest.mark.parametrize("m", [1, 100, 129, 700])
def test_padding_rows_do_not_matter(m):
    """Scales behind the last row may be anything, NaN included."""
    w = weight(512, 512, 6)[0]
    a = pkg.quantize_rows(hidden(m, 512, 6).to(DEV))
    want = [pkg.linear_w4a4(a, w), pkg.linear_w4a4_swiglu(a, w)]
    left = torch.ones(a.scales.numel(), dtype=torch.bool)
    left[ref.scale_index(m, 512).flatten()] = False
    a.scales.view(-1)[left.to(DEV)] = 0x7F
    assert torch.equal(pkg.linear_w4a4(a, w), want[0]) and torch.equal(pkg.linear_w4a4_swiglu(a, w), want[1])


@pytest.mark.parametrize("m", [2, 140, 600])
def test_a_row_does_not_depend_on_the_others(m):
    """Rows of NaN beside a row leave its bits; the same row at the largest M of a kernel and alone is within the
    sums' order."""
    w, w64, per_row = weight(512, 1024, 7)
    x = hidden(m, 1024, 7)
    want = pkg.linear_w4a4(pkg.quantize_rows(x.to(DEV)), w)
    gate = pkg.linear_w4a4_swiglu(pkg.quantize_rows(x.to(DEV)), w)
    x[1::2] = float("nan")
    rows = pkg.quantize_rows(x.to(DEV))
    y, z = pkg.linear_w4a4(rows, w), pkg.linear_w4a4_swiglu(rows, w)
    assert torch.equal(y[::2], want[::2]) and torch.equal(z[::2], gate[::2])
    assert bool(torch.isnan(y[1::2]).all()) and bool(torch.isnan(z[1::2]).all())
    h = pkg.linear_w4a4_swiglu_quantize(rows, w, 9.0)
    byte = ref.plain_scales(h)
    assert bool((byte[1::2] == 0x7F).all()) and bool((byte[::2] < 0x7F).all())


def test_tokens_verified_together_are_those_decoded_alone():
    """Up to 8 rows share one schedule: a row's bits are the same alone and among them."""
    for n, k in ((5120, 6144), (1024, 17408), (640, 512)):
        w, _, _ = weight(n, k, 12)
        x = hidden(8, k, 13).to(DEV)
        y = pkg.linear_w4a4(pkg.quantize_rows(x, 30.0), w)
        for m in (1, 3, 7):
            assert torch.equal(pkg.linear_w4a4(pkg.quantize_rows(x[:m], 30.0), w), y[:m])


def test_offsets_beyond_32_bits():
    """Inputs, codes and results whose last rows lie more than 2^32 bytes behind their first."""
    m, k = 70_000, 32768                                            # bf16: 4.6 GB
    x = torch.zeros((m, k), dtype=BF16, device=DEV)
    tail = hidden(3, k, 8)
    x[-3:] = tail.to(DEV)
    rows = pkg.quantize_rows(x, 40.0)
    want, byte = ref.quantize(tail.float(), 40.0)
    r = torch.arange(m - 3, m)[:, None]
    b = torch.arange(k // 16)[None, :]
    at = ((r // 128) * (k // 64) + b // 4) * 512 + (r % 32) * 16 + (r // 32) % 4 * 4 + b % 4
    assert torch.equal(rows.scales.view(-1)[at.to(DEV)].cpu(), byte)
    assert torch.equal(ref.E2M1[ref.unpack(rows.codes[-3:])], want)
    nw = torch.ones(k, dtype=BF16, device=DEV)
    y, _ = pkg.add_rms_norm(x, None, nw)
    short, _ = pkg.add_rms_norm(x[-3:].contiguous(), None, nw)
    assert torch.equal(y[-3:], short) and bool((y[:3] == 0).all())
    del x, y
    a = pkg.quantize_rows(tail[:, :256].to(DEV).contiguous().repeat(50_000, 1), 40.0)
    w = weight(16640, 256, 9)[0]
    z = pkg.linear_w4a4(a, w)                                       # 150000 x 16640 bf16: 5 GB
    first = pkg.linear_w4a4(pkg.quantize_rows(tail[:, :256].to(DEV).contiguous(), 40.0), w)
    assert torch.equal(z[:3], z[-3:])
    # (another kernel: another order of the sums)
    assert float((z[-3:].double() - first.double()).abs().max()) <= float(first.double().abs().max()) * 2.0 ** -7


def test_many_tiles_turn_the_ring_many_times():
    for m, n, k in ((1500, 16384, 256), (3000, 256, 16384), (777, 4224, 4352), (1111, 8192, 4096), (2048, 5120, 2048)):
        rows = pkg.quantize_rows(hidden(m, k, 10).to(DEV), 64.0)
        w, w64, per_row = weight(n, k, 11)
        y = pkg.linear_w4a4(rows, w)
        want, total = product64(rows, w64, per_row, 64.0)
        assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + total * ref.product_bound(k)).all()), (m, n, k)
