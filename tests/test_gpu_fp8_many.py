"""GPU: the products with 8-bit weights where the many-row kernel serves them, against the CPU oracle in 64 bits: runs of k blocks past the ring of a
row's scales, more tiles than pairs of CTAs, tiles left out in the middle of a walk."""
import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import fp8_oracle as FO
from test_gpu_fp8 import DT, HALF, _bytes, _input, _np, _off, _quantised, _reach, _weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _up(a, b):
    return -(-a // b)


def _served_by_pairs(rows, K, N, gated):
    """The binding's choice between both kernels, by its two estimates: a case that drifts to the other kernel fails here."""
    sms, kb = torch.cuda.get_device_properties(0).multi_processor_count, _up(K, 128)
    halves, best, splits = 2 if gated else 1, None, 1
    tiles = _up(N, 128) * halves * _up(rows, 128)
    for s in (1, 2, 3, 4, 6, 8):
        ctas, run = tiles * s, _up(kb, s)
        if s > 1 and (halves * s > 8 or run < 4 or ctas > (2 * sms * 7 // 8 if halves * s >= 4 else 2 * sms)):
            break
        t = _up(ctas, 2 * sms) * run * (5 if ctas <= sms else 8)
        if best is None or t < best:
            best, splits = t, s
    few = 4.5 + best * (0.5 / 5 if tiles * splits <= sms else 0.6 / 8)
    pairs = max(1, sms // 2)
    tiles = _up(rows, 256) * (_up(N, 128) if gated else _up(N, 256))
    assert tiles > pairs, "one tile a pair"
    return rows > 128 and 3.0 + 0.43 * _up(tiles, pairs) * kb < few


def _n_rows(B, T, kind):
    """kind 'hole': no valid row among rows 256..511, the second tile of rows; the others' blocks ragged."""
    if kind == "all":
        return None, np.ones((B, T), dtype=bool)
    first = np.arange(B) * T
    n = np.where((first + T > 256) & (first < 512), np.maximum(256 - first, 0), 1 + first % 7 % T).astype(np.int32)
    m = np.arange(T)[None] < n[:, None]
    assert not m.reshape(-1)[256:512].any() and m.reshape(-1)[512:].any()
    return torch.from_numpy(n).to(DEV), m


@pytest.mark.parametrize("B,T,K,F,kind", [(1, 520, 2200, 6272, "all"), (130, 4, 2200, 6250, "hole"), (1, 520, 5003, 6260, "all")])
def test_gated_of_many_blocks_and_tiles(B, T, K, F, kind):
    assert _served_by_pairs(B * T, K, F, True)
    n_rows, m = _n_rows(B, T, kind)
    c, s = binding.fp8_quantise(_input(B, T, K, "bf16", K + F))
    (g, gs), (u, us) = _weight(F, K, F), _weight(F, K, F + 1, pad=16)
    gs, us = gs * K ** -0.5, us * K ** -0.5
    out = torch.full((B, T, _up(F, 16) * 16), 0x55, dtype=torch.uint8, device=DEV)
    osc = binding.fp8_scale(B, T, F).fill_(9.0)
    binding.fp8_gated(c, s, g, gs, u, us, n_rows=n_rows, out=out.view(torch.float8_e4m3fn)[..., :F], out_scale=osc)
    x = FO.values(_bytes(c), _np(s))[m]
    gv, uv = FO.weight_values(_bytes(g), _np(gs)), FO.weight_values(_bytes(u), _np(us))
    gw, uw, off = x @ gv.T, x @ uv.T, _off(_up(K, 128))
    ge, ue = off * _reach(x, gv), off * _reach(x, uv)
    want = FO.silu(gw) * uw
    # as in test_gpu_fp8.test_gated: |silu'| < 1.1, nine half steps and those of the exponential's argument
    err = 1.1 * ge * (np.abs(uw) + ue) + np.abs(FO.silu(gw)) * ue + (9 + 2 * np.abs(gw)) * 2.0 ** -24 * np.abs(want) + 2.0 ** -110 * np.abs(uw)
    _quantised(_bytes(out)[..., :F][m], _np(osc)[m], want, err)
    assert np.all(_bytes(out)[~m] == 0x55) and np.all(_bytes(out)[..., F:] == 0x55) and np.all(_np(osc)[~m] == 9)
    for _ in range(20):      # the same bits, whichever warp is ahead
        oc, os_ = binding.fp8_gated(c, s, g, gs, u, us, n_rows=n_rows)
        same = oc.view(torch.uint8) == out[..., :F]
        assert bool(same[torch.from_numpy(m).to(DEV)].all()) and np.array_equal(_np(os_)[m], _np(osc)[m])


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,K,N,kind", [(1, 777, 2200, 9440, "all"), (1, 777, 2200, 9445, "all"), (259, 3, 2183, 9448, "hole")])
def test_linear_of_many_blocks_and_tiles(B, T, K, N, kind, out):
    assert _served_by_pairs(B * T, K, N, False)
    n_rows, m = _n_rows(B, T, kind)
    c, s = binding.fp8_quantise(_input(B, T, K, "f32", K + N))
    w, ws = _weight(N, K, N)
    y = torch.full((B, T, N + 3), 2.0, dtype=DT[out], device=DEV) if N % 8 else torch.full((B, T, N), 2.0, dtype=DT[out], device=DEV)
    binding.fp8_linear(c, s, w, ws, n_rows=n_rows, out=y[..., :N])
    x, wv = FO.values(_bytes(c), _np(s))[m], FO.weight_values(_bytes(w), _np(ws))
    want = x @ wv.T
    tol = _off(_up(K, 128)) * _reach(x, wv) + HALF[out] * np.abs(want)
    got = _np(y)
    assert np.all(np.abs(got[..., :N][m] - want) <= tol * 1.0000001) and np.all(got[~m] == 2) and np.all(got[..., N:] == 2)
