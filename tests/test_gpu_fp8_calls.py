"""GPU: calls of the products with 8-bit weights that overlap or lie far apart: streams, threads, captured graphs, offsets past 32 bits."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import fp8_oracle as FO
from test_gpu_fp8 import HALF, _bytes, _input, _np, _off, _reach, _weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _block(x, w, stream=None):
    c, s = binding.fp8_quantise(x, gain=w["gain"], residual=x, total=torch.empty_like(x), stream=stream)
    c, s = binding.fp8_gated(c, s, *w["g"], *w["u"], stream=stream)
    return binding.fp8_linear(c, s, *w["d"], stream=stream)


def _weights(K, F):
    return dict(gain=_input(1, 1, K, "bf16", 1)[0, 0], g=_weight(F, K, 2), u=_weight(F, K, 3), d=_weight(K, F, 4))


def test_streams_at_once():
    """Blocks of one row, of a few and of many on streams of their own, over and over, against the same calls alone."""
    K, F = 512, 1100
    w = _weights(K, F)
    xs = [_input(1, rows, K, "bf16", rows) for rows in (1, 40, 300, 700)]
    want = [_block(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=DEV) for _ in xs]
    got = [[] for _ in xs]
    for _ in range(30):
        for x, s, g in zip(xs, streams, got):
            g.append(_block(x, w, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(y, a) for a, g in zip(want, got) for y in g)


def test_two_graphs_of_one_layer():
    K, F = 384, 640
    w = _weights(K, F)
    xs = [_input(1, rows, K, "bf16", rows) for rows in (8, 600)]
    want = [_block(x, w) for x in xs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(device=DEV) for _ in xs]
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(_block(x, w, stream=s))
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_weights_written_just_before_their_product():
    """A product begins while the kernel before it ends, but not to read what that one writes: weights copied in place, then multiplied."""
    K, N = 2048, 1024
    c, s = binding.fp8_quantise(_input(1, 8, K, "bf16", 1))
    ws = [_weight(N, K, i) for i in range(3)]
    want = [binding.fp8_linear(c, s, *w) for w in ws]
    buf = [torch.empty_like(t) for t in ws[0]]
    stream, outs = torch.cuda.Stream(device=DEV), []
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for i in range(60):
            for d, src in zip(buf, ws[i % 3]):
                d.copy_(src)
            outs.append(binding.fp8_linear(c, s, *buf))
    stream.synchronize()
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(outs))


def test_threads():
    """Calls of several host threads at once, each on its own stream."""
    lib, calls, rows = binding.load(), 1500, (1, 33, 260, 900)
    K, N = 512, 700
    w, ws = _weight(N, K, 1)
    ins = [binding.fp8_quantise(_input(1, r, K, "bf16", r)) for r in rows]
    want = [binding.fp8_linear(c, s, w, ws) for c, s in ins]
    got = [torch.zeros_like(y) for y in want]
    torch.cuda.synchronize()
    start, codes = threading.Barrier(len(rows)), [set() for _ in rows]

    def loop(i):
        stream, (c, s) = torch.cuda.Stream(device=DEV), ins[i]
        a = binding.Fp8LinearArgs(1, rows[i], K, N, binding.DLITE_BF16, c.data_ptr(), K, s.data_ptr(), w.data_ptr(), w.stride(0), ws.data_ptr(),
                                  got[i].data_ptr(), N, None, None)
        ref, ptr = ctypes.byref(a), stream.cuda_stream
        start.wait()
        for _ in range(calls):
            codes[i].add(lib.dlite_fp8_linear(ref, ptr))
        stream.synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(rows))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert codes == [{0}] * len(rows), codes
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("rows", [5, 300])
def test_offsets_past_32_bits(rows):
    """Rows so far apart that the last begins past 2^32 bytes: x and codes of a quantisation, codes and results of the products."""
    K, N = 272, 150
    far = (1 << 32) // (rows - 1) // 16 * 16 + 16
    free = torch.cuda.mem_get_info()[0]
    if free < 5 * (5 << 30):
        pytest.skip("needs 25 GB")
    xw = torch.zeros(rows * far // 2, dtype=torch.bfloat16, device=DEV).view(1, rows, far // 2)[..., :K]
    cw = torch.zeros(rows * far, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).view(1, rows, far)[..., :K]
    x = _input(1, rows, K, "bf16", 2)
    xw.copy_(x)
    c0, s0 = binding.fp8_quantise(x)
    c, s = binding.fp8_quantise(xw, codes=cw)
    assert torch.equal(c.contiguous().view(torch.uint8), c0.view(torch.uint8)) and torch.equal(s, s0)
    w, ws = _weight(N, K, 3)
    ow = torch.zeros(rows * far // 4, dtype=torch.float32, device=DEV).view(1, rows, far // 4)[..., :N]
    y0 = binding.fp8_linear(c0, s0, w, ws, dtype=torch.float32)
    assert torch.equal(binding.fp8_linear(c, s, w, ws, out=ow).contiguous(), y0)
    oc = torch.zeros(rows * far, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).view(1, rows, far)[..., :N]
    g0, gs0 = binding.fp8_gated(c0, s0, w, ws, w, ws)
    g, gs = binding.fp8_gated(c, s, w, ws, w, ws, out=oc)
    assert torch.equal(g.contiguous().view(torch.uint8), g0.contiguous().view(torch.uint8)) and torch.equal(gs, gs0)


@pytest.mark.parametrize("rows", [3, 300])
def test_a_weight_whose_offsets_pass_32_bits(rows):
    """A weight of 2^32 bytes and more: the last rows of it."""
    K, N = 1 << 14, (1 << 18) + 70
    c, s = binding.fp8_quantise(_input(1, rows, K, "bf16", 6))
    w = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    scale = torch.full((-(-N // 128), K // 128), 0.5, device=DEV)
    g = torch.Generator().manual_seed(7)
    some = torch.randn(100, K, generator=g).mul(30).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    w[-100:] = some
    y = binding.fp8_linear(c, s, w.view(torch.float8_e4m3fn), scale, dtype=torch.float32)
    x, wv = FO.values(_bytes(c), _np(s))[0], FO.VALUES[_bytes(some)] * 0.5
    want = x @ wv.T
    tol = _off(K // 128) * _reach(x, wv) + HALF["f32"] * np.abs(want)
    assert np.all(np.abs(_np(y[0, :, -100:]) - want) <= tol) and not bool(y[..., :-100].any())


def test_status_of_a_stream_of_its_own_and_new_outputs():
    """Tensors made for a call on another stream than the current one belong to that stream."""
    x = _input(1, 4, 256, "f32", 1)
    x[0, 2, 5] = float("inf")
    st, s = torch.zeros(1, dtype=torch.int32, device=DEV), torch.cuda.Stream(device=DEV)
    torch.cuda.synchronize()
    c, sc = binding.fp8_quantise(x, status=st, stream=s)
    s.synchronize()
    assert int(st.item()) == binding.DEV_NONFINITE
    c0, sc0 = binding.fp8_quantise(x)
    assert torch.equal(c.view(torch.uint8), c0.view(torch.uint8)) and torch.equal(sc, sc0)
