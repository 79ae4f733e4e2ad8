"""GPU: long contexts in the kernel of float32 queries and of heads of 64: warps with many pages of a piece (rescales from page to
page, a ring in many turns), segments cut among all CTAs, joins of more pieces than lanes, tiles of 16 and 32 rows. Tolerances as
derived in test_gpu_kv_attention.py."""
import math

import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import target_oracle as TO
from test_gpu_kv_attention import DEV, DT, _cache, _gen, _tolerance, _within

pytestmark = pytest.mark.gpu
KINDS = [("f32", 64), ("f32", 128), ("bf16", 64)]


def _plain(q, pages, bt, pos, window=0, n_rows=None):
    """(out, lse, reach, eps) of the rows in 64 bits on the device; q [B, T, nq, d], holes are negative ids."""
    B, T, nq, d = q.shape
    nkv, keys = pages.shape[1], 64 * bt.shape[1]
    k, v = binding.kv_read(pages, bt, torch.zeros_like(pos), keys, dtype=torch.float32)     # zeros in holes
    j = torch.arange(keys, device=DEV)
    there = (bt >= 0).repeat_interleave(64, 1)[:, None]                                     # [B, 1, keys]
    at = pos[:, None] + torch.arange(T, device=DEV)
    see = (j <= at[..., None]) & there
    if window:
        see &= j > at[..., None] - window
    res = [torch.zeros(B, T, nq, d, dtype=torch.float64, device=DEV), torch.full((B, T, nq), -math.inf, dtype=torch.float64, device=DEV),
           torch.zeros(B, T, nq, d, dtype=torch.float64, device=DEV), torch.zeros(B, T, nq, dtype=torch.float64, device=DEV)]
    for b in range(B):
        for h in range(nq):
            kd, vd, qd = (x.double() for x in (k[b, :, h // (nq // nkv)], v[b, :, h // (nq // nkv)], q[b, :, h]))
            s = (qd @ kd.T * d ** -0.5).masked_fill(~see[b], -math.inf)
            some = see[b].any(-1)
            p = torch.softmax(s[some], -1)
            res[0][b, some, h], res[1][b, :, h], res[2][b, some, h] = p @ vd, torch.logsumexp(s, -1), p @ vd.abs()
            res[3][b, :, h] = (qd.abs() @ kd.abs().T * d ** -0.5).amax(-1)
    return [x.cpu().numpy() for x in res]


@pytest.mark.parametrize("T", [1, 8])
@pytest.mark.parametrize("dtype,d", KINDS)
def test_one_request_over_all_ctas(dtype, d, T):
    """Four pages and holes named over and over: the softmax over all of them is the one over four with counted keys. A CTA
    has more than 100 pages, a warp fills its ring four times and more; the join has one piece per CTA."""
    nq, n_pages = 4, 4
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * 112
    pages, _ = _cache(n_pages, 1, d, 1, n_pages, 51)
    ids = torch.randint(0, 10, (n,), generator=_gen(52))
    ids = torch.where(ids == 9, -1, ids % n_pages).to(torch.int32)     # a tenth of them holes
    ids[-1] = 2
    keys = 64 * n
    q = torch.randn(1, T, nq, d, generator=_gen(53)).to(DT[dtype])
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (q.to(DEV), pages.to(DEV), ids.view(1, -1).to(DEV), torch.tensor([keys - T], device=DEV))
    out, lse = binding.kv_attention(*args, lse=True, status=st)
    assert st.item() == 0
    kv = [TO.read_record(pages.numpy()[p, 0], 0, 0) for p in range(n_pages)]
    k, v = (np.concatenate([x[i] for x in kv]) for i in (0, 1))
    qd = q[0].double().numpy()
    s = qd @ k.T * d ** -0.5                                            # [T, nq, 256]
    count = np.repeat([(ids == p).sum().item() for p in range(n_pages)], 64)[None, None].repeat(T, 0).astype(np.float64)
    for t in range(T - 1):
        count[t, 0, 64 * 3 - (T - 1 - t):64 * 3] -= 1                   # keys of the last page (id 2) that row t does not see
    m = s.max(-1, keepdims=True)
    p = count * np.exp(s - m)
    total = p.sum(-1, keepdims=True)
    want, wl = p @ v / total, (m + np.log(total))[..., 0]
    eps = (np.abs(qd) @ np.abs(k).T * d ** -0.5).max(-1)
    # a lane adds one weight in four of a warp's pages, 1,216 warps share the pages and their sums are added in order
    tol, ltol = _tolerance(want, p @ np.abs(v) / total, eps, keys // sms // 8 + 16 * 8 * sms, d, dtype)
    _within(out[0], want, tol + keys * 2.0 ** -39 * 6 * 0.6875)
    _within(lse[0], wl, ltol + 2.0 ** -24 * np.abs(wl))
    again, lse2 = binding.kv_attention(*args, lse=True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("T,window", [(1, 0), (8, 0), (8, 700)])
@pytest.mark.parametrize("dtype,d", KINDS)
def test_ragged_batch(dtype, d, T, window):
    """Requests from no key to 12,000, holes among their pages, blocks of ragged lengths."""
    B, nq, nkv, mp, n_pages = 9, 8, 2, 190, 64
    pages, _ = _cache(n_pages, nkv, d, 1, 1, 54)
    g = _gen(55)
    bt = torch.randint(-4, n_pages, (B, mp), generator=g)
    bt = torch.where(bt < 0, -1, bt).to(torch.int32).to(DEV)
    pos = torch.tensor([12000, 0, 11900, 63, 700, 6000, 64, 9001, 3333], device=DEV)
    n_rows = [T, 1, max(1, T - 3), T, 0, 1, T, T, max(1, T - 1)]
    q = torch.randn(B, T, nq, d, generator=g).to(DT[dtype]).to(DEV)
    pages = pages.to(DEV)
    out, lse = torch.full((B, T, nq, d), 5.0, dtype=DT[dtype], device=DEV), torch.full((B, T, nq), 5.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.kv_attention(q, pages, bt, pos, window=window, n_rows=torch.tensor(n_rows, dtype=torch.int32, device=DEV), out=out, lse=lse,
                         status=st)
    want, wl, reach, eps = _plain(q, pages, bt, pos, window)
    tol, ltol = _tolerance(want, reach, eps, 12000 + T, d, dtype)
    for b in range(B):
        for t in range(T):
            if t >= n_rows[b]:
                assert bool((out[b, t] == 5).all()) and bool((lse[b, t] == 5).all())
            else:
                _within(out[b, t], want[b, t], tol[b, t])
                _within(lse[b, t], wl[b, t], ltol[b, t])
    assert st.item() == 0


@pytest.mark.parametrize("dtype,d", KINDS + [("bf16", 128)])
def test_prompts_in_whole_segments(dtype, d):
    """More row tiles than the cut's list holds: tiles of whole segments, causal, of prompts behind cached rows, some of them
    with a window."""
    T, nq, nkv = 530, 8, 2
    B = 2048 // (T * (nq // nkv) // 32) + 1
    mp = (T + 100 + 63) // 64
    pages, _ = _cache(40, nkv, d, 1, 1, 56)
    g = _gen(57)
    bt = torch.randint(0, 40, (B, mp), generator=g).to(torch.int32).to(DEV)
    pos = torch.randint(0, 100, (B,), generator=g).to(DEV)
    q = torch.randn(B, T, nq, d, generator=g).to(DT[dtype]).to(DEV)
    pages = pages.to(DEV)
    assert binding.kv_attention_workspace(B, T, nq, nkv, d, mp, DT[dtype]) == 0
    for window in (0, 75):
        out, lse = binding.kv_attention(q, pages, bt, pos, window=window, lse=True)
        for b in (0, 7, B - 1):
            want, wl, reach, eps = _plain(q[b:b + 1], pages, bt[b:b + 1], pos[b:b + 1], window)
            tol, ltol = _tolerance(want, reach, eps, T + 100, d, dtype)
            _within(out[b:b + 1], want, tol)
            _within(lse[b:b + 1], wl, ltol)


@pytest.mark.parametrize("dtype,d", KINDS + [("bf16", 128)])
def test_prompts_in_a_cut(dtype, d):
    """Two prompts behind cached rows whose causal tiles are cut among the CTAs, one of them padded."""
    B, T, nq, nkv, mp = 2, 1500, 8, 2, 36
    pages, _ = _cache(60, nkv, d, 1, 1, 58)
    g = _gen(59)
    bt = torch.randint(0, 60, (B, mp), generator=g).to(torch.int32).to(DEV)
    pos, n_rows = torch.tensor([777, 30], device=DEV), [T, 1111]
    q = torch.randn(B, T, nq, d, generator=g).to(DT[dtype]).to(DEV)
    pages = pages.to(DEV)
    assert binding.kv_attention_workspace(B, T, nq, nkv, d, mp, DT[dtype]) > 0
    for window in (0, 300):
        out, lse = binding.kv_attention(q, pages, bt, pos, window=window, n_rows=torch.tensor(n_rows, dtype=torch.int32, device=DEV), lse=True)
        want, wl, reach, eps = _plain(q, pages, bt, pos, window)
        tol, ltol = _tolerance(want, reach, eps, 64 * mp, d, dtype)
        for b, n in enumerate(n_rows):
            _within(out[b, :n], want[b, :n], tol[b, :n])
            _within(lse[b, :n], wl[b, :n], ltol[b, :n])
            assert not out[b, n:].any() and not lse[b, n:].any()
