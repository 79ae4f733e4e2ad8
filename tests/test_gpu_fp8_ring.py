"""GPU: rows into codes behind a norm, where a CTA takes its rows out of a ring of copies: its bounded waits, and its results against the CPU oracle in 64
bits with every CTA's ring in several turns."""
import time

import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import fp8_oracle as FO
from test_gpu_fp8 import DT, _bytes, _input, _np, _quantised

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_ring_gives_up_as_a_whole():
    """Rows that do not come: every thread leaves behind the same row, in two limits (the wait's, the copies' in flight), not in one a row."""
    limit = 20_000_000
    st, res = torch.zeros(1, dtype=torch.int32, device=DEV), torch.full((3, 4), -1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    binding.selftest_ring(limit, st, res)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5
    got = res.tolist()
    assert [g[:3] for g in got] == [[0, 1, 0], [5, 1, 0], [7, 1, 0]]
    assert 1 <= got[0][3] <= 3 and 1 <= got[1][3] <= 3 and got[2][3] == 0
    assert int(st.item()) == binding.DEV_TIMEOUT
    for bad in (0, 1_000_000_001):
        with pytest.raises(binding.DliteError):
            binding.selftest_ring(bad, st, res)


def _ring(rows, K, dtype, residual):
    """(slots, turns of the busiest CTA) of the launch, restated: a case that drifts to the other kernel fails."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    t = min(1024, -(-(-(-K // 16)) // 32) * 32)
    assert K % 8 == 0 and K <= 16 * t and rows > 4 * sms
    ctas = min(16, max(1, 1536 // t))
    slots = max(1, min(4, 200 * 1024 // ctas // (K * DT[dtype].itemsize * (2 if residual else 1))))
    return slots, -(-rows // min(rows, sms * ctas))


# (type, B, T, K, elements between rows, where the sum goes (None: no residual), slots of the ring)
RING = [("f32", 100, 7, 16384, 0, "residual", 1), ("bf16", 100, 7, 16384, 0, "x", 3), ("bf16", 58, 50, 4096, 0, "residual", 2),
        ("f32", 1, 1900, 4096, 16, None, 2), ("bf16", 875, 8, 1000, 24, "new", 3), ("bf16", 3000, 5, 1000, 0, None, 4),
        ("f32", 20000, 1, 8, 8, "x", 4), ("f32", 500, 10, 2048, 0, "new", 1)]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dtype,B,T,K,pad,total,slots", RING)
def test_norm_over_a_ring_of_rows(dtype, B, T, K, pad, total, slots, ragged):
    got_slots, turns = _ring(B * T, K, dtype, total is not None)
    assert got_slots == slots and turns >= 3
    x, gain = _input(B, T, K, dtype, 1, pad), _input(1, 1, K, dtype, 2)[0, 0]
    res = _input(B, T, K, dtype, 3, 2 * pad) if total else None
    b = np.arange(B)
    n = np.where(b % 5 == 3, -(b % 2), (b * 7 + 3) % (T + 2)) if ragged else np.full(B, T)      # outside [0, T] too
    m = np.arange(T)[None] < n[:, None]
    dm = torch.from_numpy(m).to(DEV)
    v = _np(x)
    if total:
        v = FO.total(v, _np(res), dtype)
        x[~dm], res[~dm] = float("nan"), float("inf")
    to = {None: None, "x": x, "residual": res, "new": torch.full_like(x, 7.0)}[total]
    behind = None if to is None else to[~dm].clone()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    codes = torch.full((B, T, -(-K // 16) * 16), 0x55, dtype=torch.uint8, device=DEV)
    scale = binding.fp8_scale(B, T, K).fill_(9.0)
    binding.fp8_quantise(x, gain=gain, eps=1e-5, residual=res, total=to, codes=codes.view(torch.float8_e4m3fn)[..., :K], scale=scale, status=st,
                         n_rows=torch.from_numpy(n).to(torch.int32).to(DEV) if ragged else None)
    assert int(st.item()) == 0
    if total:
        assert np.array_equal(_np(to)[m], v[m]) and torch.equal(to[~dm].view(torch.uint8), behind.view(torch.uint8))
    assert np.all(_bytes(codes)[~m] == 0x55) and np.all(_bytes(codes)[..., K:] == 0x55) and np.all(_np(scale)[~m] == 9)
    y = FO.norm(v[m], _np(gain), 1e-5)
    # the sum of squares: 16 a thread, ten joins; its root halves that and the mean's and the eps' steps; rsqrt 2 steps of 2^-23; two products
    err = ((16 + 10 + 3) / 2 + 4 + 2) * 2.0 ** -24 * np.abs(y)
    _quantised(_bytes(codes)[..., :K][m], _np(scale)[m], y, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(3, 512), (3, 513), (2500, 512)])      # read twice, off 16 bytes, over the ring
def test_rows_of_zeros(dtype, rows, K):
    """With eps a row of zeros has codes of 0; without, it is 0 / 0: NaN, flagged, in its row."""
    x = _input(1, rows, K, dtype, 4)
    x[0, 1] = 0
    gain, st = _input(1, 1, K, dtype, 5)[0, 0], torch.zeros(1, dtype=torch.int32, device=DEV)
    c, s = binding.fp8_quantise(x, gain=gain, eps=1e-6, status=st)
    assert int(st.item()) == 0 and np.all(_bytes(c)[0, 1] & 0x7F == 0) and np.all(_np(s)[0, 1] == 2.0 ** -126)
    c, s = binding.fp8_quantise(x, gain=gain, eps=0.0, status=st)
    nan = (_bytes(c)[0] & 0x7F) == 0x7F
    assert int(st.item()) == binding.DEV_NONFINITE and nan[1].all() and not nan[0].any() and not nan[2:].any()
