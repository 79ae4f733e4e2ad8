"""GPU: the products with 8-bit weights through the binding, against the CPU oracle in 64 bits. Codes and scales of given
numbers are compared bit for bit; sums within what float32 sums may be off."""
import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import fp8_oracle as FO

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}     # a rounding's share of the value (bf16: eps / 2 = 2^-8)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _bytes(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def _input(B, T, K, dtype, seed, pad=0, offset=0):
    """[B, T, K] of columns of different sizes, on the device: dense, or rows K + pad apart, or `offset` elements into its memory."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, T, K, generator=g) * torch.exp(torch.randn(K, generator=g))).to(DT[dtype])
    buf = torch.zeros(offset + B * T * (K + pad), dtype=x.dtype, device=DEV)
    y = buf[offset:].view(B, T, K + pad)[..., :K]
    y.copy_(x)
    return y


def _weight(N, K, seed, pad=0):
    """Random codes (no NaN) and scales of any sign and size; rows on 16 bytes, `pad` bytes between them."""
    g = torch.Generator().manual_seed(seed)
    pitch = -(-K // 16) * 16 + pad
    c = torch.randn(N, pitch, generator=g).mul(30).to(torch.float8_e4m3fn).to(DEV)[:, :K]
    s = (torch.randn(-(-N // 128), -(-K // 128), generator=g).exp() * 1e-2).to(DEV)
    return c, s


def _reach(x, w):
    """Sum of the products' magnitudes: what a float32 sum's error is relative to."""
    return np.abs(x) @ np.abs(w).T


def _off(kblocks):
    """What a product may be off, relative to its reach: 128 products of a block (exact) added in the tensor cores, an add cut off at one
    step of 2^-23; the scales' product and one rounding add a block, up to 8 runs joined: half steps of 2^-24."""
    return 128 * 2.0 ** -23 + (kblocks + 8 + 2) * 2.0 ** -24


def _quantised(c, s, want, err):
    """Codes and scales as a rounding of numbers within err of `want`: the scale is the rule's for one of them, the values are within half a
    step."""
    y, e = FO.blocked(want), FO.blocked(err)
    hi, lo = np.max(np.abs(y) + e, -1), np.max(np.maximum(np.abs(y) - e, 0), -1)
    assert np.all(s >= FO.block_scale(lo)) and np.all(s <= FO.block_scale(hi))
    got = FO.blocked(FO.values(c, s))
    size = np.maximum((np.abs(y) + e) / s[..., None], 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(size)) - 3) * s[..., None]
    assert np.all(np.abs(got - y) <= step / 2 + e)


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,K,pad,offset", [(1, 1, 1, 0, 0), (1, 1, 4096, 0, 0), (2, 3, 128, 0, 0), (1, 5, 129, 0, 0), (3, 2, 1000, 0, 0), (2, 4, 777, 3, 0),
                                              (1, 3, 2560, 64, 0), (2, 2, 512, 0, 1), (1, 2, 12288, 0, 0), (4, 1, 16, 8, 0), (1, 2, 20000, 0, 0)])
def test_quantise(dtype, B, T, K, pad, offset):
    x = _input(B, T, K, dtype, K + T, pad, offset)
    x[0, 0] *= 1e-3
    c, s = binding.fp8_quantise(x)
    want, ws = FO.quantise(_np(x))
    assert np.array_equal(_np(s), ws)
    assert np.array_equal(_bytes(c), want)


def test_quantise_borders():
    """The scale's borders, zeros, subnormal numbers, the largest ones, ties of the codes."""
    f = torch.finfo(torch.float32)
    tops = [0.0, 448.0, float(np.nextafter(np.float32(448), np.float32(1e9))), 447.9, 224.0, 1e-45, f.tiny, 448 * 2.0 ** -126, 449 * 2.0 ** -126, f.max, 1.0, 2.0 ** -120]
    grid = torch.from_numpy((FO.E4M3[:-1] + FO.E4M3[1:]) / 2).float()      # 126 ties
    x = torch.zeros(1, len(tops), 128)
    for i, t in enumerate(tops):
        x[0, i, 1:127] = grid * (t / 448 if t > 1e-30 else 0.0)
        x[0, i, 3::2] *= -1
        x[0, i, 0] = t
    c, s = binding.fp8_quantise(x.to(DEV))
    want, ws = FO.quantise(x.double().numpy())
    assert np.array_equal(_np(s), ws) and np.array_equal(_bytes(c), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [256, 1000, 9000])
def test_quantise_of_what_is_not_finite(dtype, K):
    x = _input(1, 3, K, dtype, 5)
    x[0, 1, 3], x[0, 1, 130], x[0, 1, 131] = float("nan"), float("inf"), float("-inf")
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c, s = binding.fp8_quantise(x, status=st)
    want, ws = FO.quantise(_np(x))
    assert np.array_equal(_np(s), ws) and np.array_equal(_bytes(c) & 0x7F, want & 0x7F)
    assert int(st.item()) == binding.DEV_NONFINITE
    fin = np.isfinite(_np(x))
    assert np.array_equal(_bytes(c)[fin], want[fin])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,K,pad", [(1, 1, 4096, 0), (2, 3, 1000, 0), (1, 4, 130, 6), (1, 2, 9728, 0), (1, 2, 8200, 8), (2, 1, 8, 0), (1, 1, 1, 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_and_quantise(dtype, B, T, K, pad, residual):
    x, gain = _input(B, T, K, dtype, 1, pad), _input(1, 1, K, dtype, 2)[0, 0]
    res = _input(B, T, K, dtype, 3, 2 * pad) if residual else None
    total = torch.full((B, T, K), 7.0, dtype=DT[dtype], device=DEV) if residual else None
    c, s = binding.fp8_quantise(x, gain=gain, eps=1e-5, residual=res, total=total)
    v = _np(x)
    if residual:
        v = FO.total(v, _np(res), dtype)
        assert np.array_equal(_np(total), v)
    y = FO.norm(v, _np(gain), 1e-5)
    # the sum of squares: 16 a thread (two rounds of them at most), ten joins; its root halves that and the mean's and the eps' steps; rsqrt 2 steps of 2^-23; two products
    err = ((32 + 10 + 3) / 2 + 4 + 2) * 2.0 ** -24 * np.abs(y)
    _quantised(_bytes(c), _np(s), y, err)
    if residual:      # in place, and without the norm
        keep = res.clone()
        binding.fp8_quantise(x, gain=gain, eps=1e-5, residual=res)
        assert torch.equal(res.contiguous(), total)
        res.copy_(keep)
        c, s = binding.fp8_quantise(x, residual=res, total=total)
        want, ws = FO.quantise(v)
        assert np.array_equal(_np(total), v) and np.array_equal(_np(s), ws) and np.array_equal(_bytes(c), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,pad", [(3, 8193, 0), (2, 20001, 2), (5, 511, 0), (5, 514, 1), (2, 16385, 0)])
def test_rows_off_16_bytes(dtype, T, K, pad):
    """Widths and starts of every parity, sums over several rounds of a row; the stream in place."""
    B = 2
    x, gain = _input(B, T, K, dtype, 1, pad), _input(1, 1, K + 1, dtype, 2)[0, 0][1:]
    res = torch.full((B, T, K + 5), 7.0, dtype=DT[dtype], device=DEV)
    res[..., 3:3 + K] = _input(B, T, K, dtype, 3)
    inner = res[..., 3:3 + K]
    v = FO.total(_np(x), _np(inner), dtype)
    n_rows = torch.tensor([T, T - 1], dtype=torch.int32, device=DEV)
    m = (torch.arange(T, device=DEV)[None] < n_rows[:, None]).cpu().numpy()
    old = _np(inner)
    c, s = binding.fp8_quantise(x, gain=gain, eps=1e-5, residual=inner, n_rows=n_rows)
    assert np.array_equal(_np(inner)[m], v[m]) and np.array_equal(_np(inner)[~m], old[~m])
    assert bool((res[..., :3] == 7).all()) and bool((res[..., 3 + K:] == 7).all())
    y = FO.norm(v, _np(gain), 1e-5)
    # as in test_norm_and_quantise, with 16 numbers a thread and round of 8,192
    err = ((16 * -(-K // 8192) + 10 + 3) / 2 + 4 + 2) * 2.0 ** -24 * np.abs(y)
    _quantised(_bytes(c)[m][None], _np(s)[m][None], y[m][None], err[m][None])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,pad", [(128, 128, 0), (1, 1, 0), (130, 300, 0), (257, 1000, 5), (64, 129, 0)])
def test_weight(dtype, N, K, pad):
    w = _input(1, N, K, dtype, 9, pad)[0]
    c, s = binding.fp8_weight(w)
    want, ws = FO.quantise_weight(_np(w))
    assert np.array_equal(_np(s), ws) and np.array_equal(_bytes(c), want)
    assert c.stride(0) % 16 == 0


def test_weight_that_is_not_finite():
    w = _input(1, 140, 300, "f32", 9)[0]
    w[3, 4], w[130, 299] = float("nan"), float("-inf")
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c, s = binding.fp8_weight(w, status=st)
    want, ws = FO.quantise_weight(_np(w))
    assert np.array_equal(_np(s), ws) and np.array_equal(_bytes(c), want) and int(st.item()) == binding.DEV_NONFINITE


@pytest.mark.parametrize("dtype,K", [("bf16", 300), ("bf16", 304), ("f32", 304)])
def test_weight_blocks_without_a_finite_element(dtype, K):
    w = _input(1, 260, K, dtype, 19)[0]
    w[:128, :128] = float("inf")
    w[128:256, 128:256] = float("nan")
    w[259, K - 1] = -float("inf")
    w[5, 200] = torch.finfo(w.dtype).max  # the largest magnitude that counts
    w[6, 201] = float("inf")
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c, s = binding.fp8_weight(w, status=st)
    want, ws = FO.quantise_weight(_np(w))
    assert np.array_equal(_np(s), ws) and np.array_equal(_bytes(c), want) and int(st.item()) == binding.DEV_NONFINITE


# ---------------------------------------------------------------- products

SHAPES = [(1, 1, 128, 128), (1, 1, 1, 1), (1, 1, 4096, 4096), (1, 8, 2560, 1000), (1, 7, 100, 129), (3, 3, 129, 64), (1, 33, 384, 200), (2, 64, 1000, 777),
          (1, 129, 256, 130), (4, 75, 640, 384), (1, 65, 4100, 65), (16, 8, 9728, 256), (1, 200, 16, 5),
          (1, 513, 1000, 777), (3, 171, 4100, 300), (1, 260, 16, 5), (1, 1025, 384, 2600)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,K,N", SHAPES)
def test_linear(B, T, K, N, out):
    c, s = binding.fp8_quantise(_input(B, T, K, "f32", K + N))
    w, ws = _weight(N, K, N)
    y = binding.fp8_linear(c, s, w, ws, dtype=DT[out])
    x, wv = FO.values(_bytes(c), _np(s)).reshape(B * T, K), FO.weight_values(_bytes(w), _np(ws))
    want = x @ wv.T
    tol = _off(-(-K // 128)) * _reach(x, wv) + HALF[out] * np.abs(want)
    assert np.all(np.abs(_np(y).reshape(B * T, N) - want) <= tol * 1.0000001)
    assert torch.equal(binding.fp8_linear(c, s, w, ws, dtype=DT[out]), y)


@pytest.mark.parametrize("B,T,K,F", SHAPES)
def test_gated(B, T, K, F):
    c, s = binding.fp8_quantise(_input(B, T, K, "bf16", K + F))
    (g, gs), (u, us) = _weight(F, K, F), _weight(F, K, F + 1, pad=16)
    gs, us = gs * K ** -0.5, us * K ** -0.5
    oc, os_ = binding.fp8_gated(c, s, g, gs, u, us)
    x = FO.values(_bytes(c), _np(s)).reshape(B * T, K)
    gv, uv = FO.weight_values(_bytes(g), _np(gs)), FO.weight_values(_bytes(u), _np(us))
    gw, uw, off = x @ gv.T, x @ uv.T, _off(-(-K // 128))
    ge, ue = off * _reach(x, gv), off * _reach(x, uv)
    want = FO.silu(gw) * uw
    # |silu'| < 1.1; in steps of 2^-24: exp2 4, its argument's factor and product 2 |g|, the sum 1, the reciprocal 2, two products 2;
    # a result below 2^-120 may be 0 (the reciprocal's)
    err = 1.1 * ge * (np.abs(uw) + ue) + np.abs(FO.silu(gw)) * ue + (9 + 2 * np.abs(gw)) * 2.0 ** -24 * np.abs(want) + 2.0 ** -110 * np.abs(uw)
    _quantised(_bytes(oc).reshape(B * T, F), _np(os_).reshape(B * T, -1), want, err)


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("size", [1e2, 1e5, 1e30])
def test_gated_far(rows, size):
    """Gates far from 0: exp(-g) from nothing to infinity. Results past float32 become NaN codes and flag the status."""
    K, F = 256, 130
    c, s = binding.fp8_quantise(_input(1, rows, K, "bf16", 8))
    (g, gs), (u, us) = _weight(F, K, 9), _weight(F, K, 10)
    gs = gs * size
    us = us * (1e15 if size == 1e30 else 1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    oc, os_ = binding.fp8_gated(c, s, g, gs, u, us, status=st)
    x = FO.values(_bytes(c), _np(s))[0]
    gv, uv = FO.weight_values(_bytes(g), _np(gs)), FO.weight_values(_bytes(u), _np(us))
    gw, uw, off = x @ gv.T, x @ uv.T, _off(2)
    ge, ue = off * _reach(x, gv), off * _reach(x, uv)
    want, big = FO.silu(gw) * uw, 3.4e38
    # as in test_gated; above 128 exp(-g) is nothing to 1, below -128 the result is less than 2^-110 of u
    err = 1.1 * ge * (np.abs(uw) + ue) + np.abs(FO.silu(gw)) * ue + (9 + 2 * np.minimum(np.abs(gw), 128)) * 2.0 ** -24 * np.abs(want) + 2.0 ** -110 * np.abs(uw)
    got, sure = _bytes(oc)[0], np.abs(want) - err > big
    nan = (got & 0x7F) == 0x7F
    assert np.all(nan[sure]) and not nan[np.abs(want) + err < big].any() and int(st.item()) == (binding.DEV_NONFINITE if nan.any() else 0)
    assert nan.any() == (size == 1e30)
    ok = ~FO.blocked(nan.astype(float)).any(-1)[..., None] & (FO.blocked(np.ones_like(want)) > 0)      # blocks without one
    y, e, v = FO.blocked(want), FO.blocked(err), FO.blocked(FO.values(np.where(nan, 0, got), _np(os_)[0]))
    sc = _np(os_)[0][..., None]
    step = 2.0 ** (np.floor(np.log2(np.maximum((np.abs(y) + e) / sc, 2.0 ** -6))) - 3) * sc
    assert np.all((np.abs(v - y) <= step / 2 + e)[ok])


# ---------------------------------------------------------------- the largest sizes

@pytest.mark.parametrize("B,T,K,N", [(1, 2, 1 << 20, 130), (1, 2, 16, 1 << 22), (1 << 11, 1 << 11, 16, 8), (1, 300, 1 << 18, 20)])
@pytest.mark.parametrize("ragged", [False, True])
def test_largest_sizes(B, T, K, N, ragged):
    """The ends of K, N and rows, against products in 64 bits on the device."""
    x = torch.randn(B, T, K, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    n = torch.arange(B, dtype=torch.int32, device=DEV) * 7 % (T + 1) if ragged else None
    c, s = binding.fp8_quantise(x, n_rows=n)
    c0, s0 = binding.fp8_quantise(x)
    m = torch.arange(T, device=DEV)[None] < n[:, None] if ragged else torch.ones(B, T, dtype=torch.bool, device=DEV)
    assert torch.equal(c.view(torch.uint8)[m], c0.view(torch.uint8)[m]) and torch.equal(s[m], s0[m])
    w, ws = _weight(N, K, 2)
    y = binding.fp8_linear(c, s, w, ws, dtype=torch.float32, n_rows=n)
    oc, os_ = binding.fp8_gated(c, s, w, ws * K ** -0.5, w, ws * K ** -0.5, n_rows=n)
    assert not bool(y[~m].any())
    xv = (c0.double() * s0.double().repeat_interleave(128, -1)[..., :K]).view(B * T, K)
    wv = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    want, reach = (xv @ wv.T).view(B, T, N), (xv.abs() @ wv.abs().T).view(B, T, N)
    tol = _off(-(-K // 128)) * reach + HALF["f32"] * want.abs()
    assert bool(((y.double() - want).abs() <= tol)[m].all())
    g = want * K ** -0.5
    a = g / (1 + torch.exp(-g)) * g
    v = oc.double() * os_.double().repeat_interleave(128, -1)[..., :N]
    # half a step of the value, of the least step where it is small, and the sums' error through the product: |d(silu(g) g)| < 2.2 |g| + 1 times it
    e = tol * K ** -0.5
    err = a.abs() / 16 + os_.double().repeat_interleave(128, -1)[..., :N] * 2.0 ** -10 + e * (2.2 * g.abs() + 1 + e) + (9 + 2 * g.abs()) * 2.0 ** -24 * a.abs()
    assert bool(((v - a).abs() <= err * 1.07)[m].all())      # the step is that of the value with its error


# ---------------------------------------------------------------- rows of a ragged batch

@pytest.mark.parametrize("B,T,K,N", [(3, 7, 300, 200), (5, 40, 1000, 130), (6, 90, 640, 520), (2, 700, 256, 256), (4, 1, 128, 64)])
def test_rows_behind_a_requests_last(B, T, K, N):
    """Rows t >= n_rows[b] hold anything, NaN codes and scales too: neither do they reach a result nor is one of theirs written."""
    n = torch.tensor([(b * 5 * T // 7 + (b == 1) * 3) % (T + 1) if b else -4 for b in range(B)], dtype=torch.int32)
    n[-1] = T + 9                                  # values outside [0, T] are taken to its ends
    x = _input(B, T, K, "bf16", 1)
    ok = torch.arange(T)[None] < n[:, None]
    x[~ok.to(DEV)] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(n_rows=n.to(DEV), status=st)
    codes = torch.full((B, T, -(-K // 16) * 16), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[..., :K]
    scale = binding.fp8_scale(B, T, K).fill_(float("nan"))
    res, total = torch.ones_like(x), torch.full_like(x, 5.0)
    binding.fp8_quantise(x, residual=res, total=total, codes=codes, scale=scale, **kw)
    v = FO.total(np.where(ok.numpy()[..., None], _np(x), 0), _np(res), "bf16")
    want, ws = FO.quantise(v)
    m = ok.numpy()
    assert np.array_equal(_bytes(codes)[m], want[m]) and np.array_equal(_np(scale)[m], ws[m]) and np.array_equal(_np(total)[m], v[m])
    assert np.all(_bytes(codes)[~m] == 0x7F) and np.all(np.isnan(_np(scale)[~m])) and np.all(_np(total)[~m] == 5)
    w, wsc = _weight(N, K, 3)
    out = torch.full((B, T, N + 8), 3.0, device=DEV)[..., :N]
    binding.fp8_linear(codes, scale, w, wsc, out=out, **kw)
    xv, wv = np.where(m[..., None], FO.values(np.where(m[..., None], want, 0), ws), 0), FO.weight_values(_bytes(w), _np(wsc))
    y = xv @ wv.T
    tol = _off(-(-K // 128)) * (np.abs(xv) @ np.abs(wv).T) + HALF["f32"] * np.abs(y)
    got = _np(out)
    assert np.all(np.abs(got - y)[m] <= tol[m]) and np.all(got[~m] == 3) and bool((out.as_strided((B, T, 8), (T * (N + 8), N + 8, 1), N) == 3).all())
    F = N
    oc = torch.full((B, T, -(-F // 16) * 16 + 16), 0x55, dtype=torch.uint8, device=DEV)
    os_ = binding.fp8_scale(B, T, F).fill_(9.0)
    binding.fp8_gated(codes, scale, w, wsc, w, wsc, out=oc.view(torch.float8_e4m3fn)[..., :F], out_scale=os_, **kw)
    full, fs = binding.fp8_gated(*binding.fp8_quantise(torch.from_numpy(v).float().to(DEV)), w, wsc, w, wsc)
    assert np.array_equal(_bytes(oc)[..., :F][m], _bytes(full)[m]) and np.array_equal(_np(os_)[m], _np(fs)[m])
    assert np.all(_bytes(oc)[~m] == 0x55) and np.all(_bytes(oc)[..., F:] == 0x55) and np.all(_np(os_)[~m] == 9)
    assert int(st.item()) == 0
    assert bool((binding.fp8_linear(codes, scale, w, wsc, n_rows=kw["n_rows"])[~ok.to(DEV)] == 0).all())


# ---------------------------------------------------------------- strides, alignment, what is not finite

@pytest.mark.parametrize("rows,K,N", [(5, 200, 70), (300, 200, 333)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_strides_of_products(rows, K, N, out):
    """Codes as a slice of wider rows, weights as a slice of wider ones, outputs off 16 bytes and as a slice: the results of dense ones."""
    c, s = binding.fp8_quantise(_input(1, rows, K, "bf16", 4))
    w, ws = _weight(N, K, 5, pad=48)
    want = binding.fp8_linear(c, s, w, ws, dtype=DT[out])
    wide = torch.zeros(1, rows, 400, dtype=torch.uint8, device=DEV).fill_(0x7F).view(torch.float8_e4m3fn)
    cw = wide[..., 16:16 + K]
    cw.view(torch.uint8).copy_(c.view(torch.uint8))
    for off, pad in ((0, 0), (1, 0), (0, 3), (8, 16)):
        buf = torch.full((off + rows * (N + pad),), 2.0, dtype=DT[out], device=DEV)
        y = buf[off:].view(1, rows, N + pad)[..., :N]
        assert binding.fp8_linear(cw, s, w, ws, out=y) is y and torch.equal(y, want)
        assert bool((buf[:off] == 2).all()) and bool((buf[off:].view(rows, N + pad)[:, N:] == 2).all())


@pytest.mark.parametrize("rows", [9, 300, 513])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 2, 3, 63, 65, 66, 127, 193, 258, 450])
def test_outputs_of_odd_widths(rows, out, N):
    """Rows of any width, begun anywhere: the bits of rows on 16 bytes, and nothing beside them."""
    B, T, K = 3, rows // 3, 200
    c, s = binding.fp8_quantise(_input(B, T, K, "bf16", 4))
    w, ws = _weight(N, K, 5)
    n_rows = torch.tensor([T, T - 1, 1], dtype=torch.int32, device=DEV)
    m = torch.arange(T, device=DEV)[None] < n_rows[:, None]
    want = torch.full((B, T, -(-N // 8) * 8), 2.0, dtype=DT[out], device=DEV)[..., :N]
    binding.fp8_linear(c, s, w, ws, n_rows=n_rows, out=want)
    for off, pad in ((0, 0), (1, 0), (0, 1), (1, 1), (2, 2), (3, 5)):
        buf = torch.full((off + rows * (N + pad) + 8,), 2.0, dtype=DT[out], device=DEV)
        y = buf[off:off + rows * (N + pad)].view(B, T, N + pad)[..., :N]
        binding.fp8_linear(c, s, w, ws, n_rows=n_rows, out=y)
        assert torch.equal(y, want) and bool((y[~m] == 2).all())
        assert bool((buf[:off] == 2).all()) and bool((buf[-8:] == 2).all())
        assert bool((buf[off:-8].view(rows, N + pad)[:, N:] == 2).all())


@pytest.mark.parametrize("rows", [3, 300])
def test_nan_codes_stay_in_their_row(rows):
    K, N = 300, 260
    c, s = binding.fp8_quantise(_input(1, rows, K, "bf16", 4))
    w, ws = _weight(N, K, 5)
    y0 = binding.fp8_linear(c, s, w, ws)
    g0, gs0 = binding.fp8_gated(c, s, w, ws * 0.1, w, ws * 0.1)
    c.view(torch.uint8)[0, 1, 290] = 0xFF
    w.view(torch.uint8)[200, 7] = 0x7F
    y = binding.fp8_linear(c, s, w, ws)
    hit = torch.zeros(rows, N, dtype=torch.bool, device=DEV)
    hit[1], hit[:, 200] = True, True
    assert torch.equal(torch.isnan(y[0]), hit) and torch.equal(y[0][~hit], y0[0][~hit])
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    g, gs = binding.fp8_gated(c, s, w, ws * 0.1, w, ws * 0.1, status=st)
    assert int(st.item()) == binding.DEV_NONFINITE
    assert torch.equal((g.view(torch.uint8)[0] & 0x7F) == 0x7F, hit)
    same = ~hit & (torch.arange(N, device=DEV) // 128 != 1)      # the block of column 200 may have lost its largest
    assert torch.equal(g.view(torch.uint8)[0][same], g0.view(torch.uint8)[0][same])


@pytest.mark.parametrize("rows", [2, 300])
@pytest.mark.parametrize("size", [-100, -60, 60, 100])
def test_far_scales(rows, size):
    """Rows and weights of far sizes whose products are float32 numbers."""
    K, N = 384, 140
    x = _input(1, rows, K, "f32", 4)
    c, s = binding.fp8_quantise(x * 2.0 ** size)
    c0, s0 = binding.fp8_quantise(x)
    w, ws = _weight(N, K, 5)
    assert torch.equal(c.view(torch.uint8), c0.view(torch.uint8)) and torch.equal(s, s0 * 2.0 ** size)
    y, y0 = (binding.fp8_linear(c, a, w, b, dtype=torch.float32) for a, b in ((s, ws * 2.0 ** -size), (s0, ws)))
    assert torch.equal(y, y0)
