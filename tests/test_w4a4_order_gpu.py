"""A weight's scales laid out in the stream of the products that read them: the C ABI's calls, with nothing between
them that waits."""
import threading

import pytest
import torch

from test_w4a4_gpu import BF16, DEV, hidden, no_device_error, pkg, weight  # noqa: F401
from nvfp4_block_scaled_linear_gb300 import w4a4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m, n, k", [(1, 34816, 5120), (100, 5120, 17408), (2048, 34816, 1024)])
@pytest.mark.parametrize("between", [0, 1, 3])
def test_scales_laid_out_ahead_of_products(m, n, k, between):
    """Scales of two contents in turn, laid out anew and then read by a product, directly or with products of another
    weight between: each has the scales that were laid out last."""
    lib = w4a4._library()
    g = torch.Generator(device=DEV).manual_seed(m)
    packed = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    plain = [torch.randint(0x20, 0x51, (n, k // 16), generator=g, device=DEV, dtype=torch.uint8) for _ in range(2)]
    weights = [pkg.Fp4Weight(packed, s, 8.0 * k ** 0.5) for s in plain]
    other = pkg.Fp4Weight(packed[:512], plain[0][:512], 1.0)
    a = pkg.quantize_rows(hidden(m, k, 1).to(DEV), 64.0)
    want = [pkg.linear_w4a4(a, w) for w in weights]
    blocked, refused = weights[0].scales.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
    c = w4a4._pack_weight(packed.data_ptr(), blocked.data_ptr(), n, k, 1, 8.0 * k ** 0.5, *[0.0] * 7, n, *[0] * 7)
    out = [torch.empty((m, n), dtype=BF16, device=DEV) for _ in range(2)]
    small = torch.empty((m, 512), dtype=BF16, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    for _ in range(5):
        for i in (1, 0):
            st = lib.nvfp4_w4a4_scale_layout(plain[i].data_ptr(), n, k, blocked.data_ptr(), refused.data_ptr(), stream)
            for _ in range(between):
                st |= lib.nvfp4_linear_w4a4(a._c, m, other._c, 0, small.data_ptr(), None, stream)
            st |= lib.nvfp4_linear_w4a4(a._c, m, c, 0, out[i].data_ptr(), None, stream)
            assert st == 0
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert int(refused) == 0


@pytest.mark.parametrize("m", [1, 100, 2048])
def test_scales_laid_out_in_a_graph(m):
    """The same captured: layout, a product of another weight and one of this, replayed over scales of two contents."""
    n, k = 34816, 1024
    lib = w4a4._library()
    g = torch.Generator(device=DEV).manual_seed(m)
    packed = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    plain = [torch.randint(0x20, 0x51, (n, k // 16), generator=g, device=DEV, dtype=torch.uint8) for _ in range(2)]
    weights = [pkg.Fp4Weight(packed, s, 8.0 * k ** 0.5) for s in plain]
    a = pkg.quantize_rows(hidden(m, k, 1).to(DEV), 64.0)
    want = [pkg.linear_w4a4(a, w) for w in weights]
    given, blocked = plain[0].clone(), weights[0].scales.clone()
    refused = torch.zeros(1, dtype=torch.int32, device=DEV)
    c = w4a4._pack_weight(packed.data_ptr(), blocked.data_ptr(), n, k, 1, 8.0 * k ** 0.5, *[0.0] * 7, n, *[0] * 7)
    first, second = (torch.empty((m, n), dtype=BF16, device=DEV) for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stream = torch.cuda.current_stream().cuda_stream
        st = lib.nvfp4_w4a4_scale_layout(given.data_ptr(), n, k, blocked.data_ptr(), refused.data_ptr(), stream)
        st |= lib.nvfp4_linear_w4a4(a._c, m, c, 0, first.data_ptr(), None, stream)
        st |= lib.nvfp4_w4a4_scale_layout(given.data_ptr(), n, k, blocked.data_ptr(), refused.data_ptr(), stream)
        st |= lib.nvfp4_linear_w4a4(a._c, m, weights[0]._c, 0, second.data_ptr(), None, stream)
        st |= lib.nvfp4_linear_w4a4(a._c, m, c, 0, second.data_ptr(), None, stream)
    assert st == 0
    for i in (1, 0, 1, 1, 0):
        given.copy_(plain[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, want[i]) and torch.equal(second, want[i])


def test_calls_of_several_threads():
    """Host threads with a stream each, through every kernel."""
    def pass_of(m, seed):
        x, w = hidden(m, 512, seed).to(DEV), weight(1024, 512, seed)[0]
        nw = torch.ones(512, dtype=BF16, device=DEV)

        def run():
            a, r = pkg.add_rms_norm_quantize(x, x, nw, 1e-6, 30.0)
            h = pkg.linear_w4a4_swiglu_quantize(a, w, 20.0)
            return pkg.linear_w4a4(a, w), r, h.codes, pkg.linear_w4a4_swiglu(pkg.quantize_rows(x, 30.0), w)
        return run
    runs = [pass_of(m, m) for m in (1, 20, 100, 128 * 40)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    wrong = []

    def work(run, expected):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got = [run() for _ in range(30)]
                stream.synchronize()
            wrong.extend(1 for outs in got for a, b in zip(outs, expected) if not torch.equal(a, b))
        except Exception as e:
            wrong.append(e)
    threads = [threading.Thread(target=work, args=pair) for pair in zip(runs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
