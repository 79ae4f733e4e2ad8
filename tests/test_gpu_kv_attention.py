"""GPU: attention over the paged 4-bit cache against the float64 oracle.

Tolerance of one output, derived: the weights are f16 (half a step 2^-11 relative; float32 calls keep hi + lo planes,
2^-21), a score is an fp32 sum of d exact products plus two roundings, taken as off by at most (d / 8 + 8) 2^-23 of
sum |q k| scale (the accumulator may truncate), exp2 adds 2^-22, and the sums over the keys of a lane and the joins
(n / 16 + 64) 2^-24. Each relative error of a weight moves the output by at most twice
reach = sum p |v| / sum p (numerator and denominator); the result is rounded once (bf16: 2^-8 relative).
Far weights add an absolute term: f16's smallest step is 2^-24 and the largest weight is kept as 2^14 (bf16 queries with heads of
128: as at least 2^6, since a row's reference is passed by at most 2^8), so each is off by at most 2^-25 / 2^14 = 2^-39
(2^-31) of the largest, which is at most their sum: `keys` of them move an output by at most keys 2^-39 (2^-31) max |v|, and no
scale of these tests' caches is above 0.6875 (byte 0x33), no code above 6."""
import math

import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import target_oracle as TO

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cache(n_pages, H, d, B, max_pages, seed, k_exp=0, v_exp=0):
    """Cache bytes with scales around 2^-exp / 4 (values of order one) and a table of distinct pages."""
    g = _gen(seed)
    pages = torch.randint(0, 256, (n_pages, H, 72 * d), generator=g, dtype=torch.uint8)
    pages[..., 64 * d:68 * d] = 0x24 + pages[..., 64 * d:68 * d] % 8
    pages[..., 68 * d:] = 0x24 + pages[..., 68 * d:] % 16
    return pages, torch.randperm(n_pages, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32)


def _tolerance(want, reach, eps, keys, d, dtype, v_exp=0):
    far = keys * 2.0 ** (-31 if dtype == "bf16" and d == 128 else -39) * 6 * 0.6875 * 2.0 ** v_exp
    s = (d / 8 + 8) * 2.0 ** -23 * eps                       # nats
    w = (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) + 2.0 ** -22 + (keys / 16 + 64) * 2.0 ** -24 + s
    return (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(want) + 2 * w[..., None] * reach + far, 2 * w + 2.0 ** -22 * 20


def _within(got, want, tol):
    """The largest share of the tolerance that an element takes (equal infinities take none)."""
    got = got.double().cpu().numpy()
    off = np.where(got == want, 0.0, np.abs(got - np.where(np.isinf(want), 0.0, want)))
    worst = float((off / tol).max())
    assert worst <= 1, worst
    return worst


CASES = [
    # B, T, nq, nkv, d, dtype, pos, n_rows, window, exps, extra pages in the table
    (1, 1, 1, 1, 64, "bf16", [0], None, 0, (0, 0), 0),            # one token, one key
    (1, 1, 4, 2, 64, "f32", [0], None, 0, (0, 0), 3),
    (1, 1, 8, 8, 128, "bf16", [63], None, 0, (0, 0), 0),          # exactly one page
    (1, 1, 8, 2, 128, "bf16", [64], None, 0, (0, 0), 0),
    (2, 1, 32, 8, 128, "bf16", [700, 5], None, 0, (0, 0), 9),     # a split tile beside a short one
    (1, 8, 32, 8, 128, "bf16", [1500], None, 0, (-3, 2), 0),      # 32-row tiles, many splits
    (3, 8, 8, 2, 128, "bf16", [61, 128, 0], [8, 3, 8], 0, (0, 0), 0),
    (3, 5, 6, 2, 64, "bf16", [61, 200, 31], [5, 0, 9], 0, (1, -2), 2),   # 15 rows; none; more than T
    (3, 5, 6, 2, 128, "f32", [61, 200, 31], [5, -1, 2], 0, (1, -2), 2),
    (2, 32, 5, 1, 64, "bf16", [40, 333], None, 0, (0, 0), 0),     # 160 rows: five tiles
    (2, 32, 5, 1, 64, "f32", [40, 333], [32, 17], 0, (0, 0), 0),
    (1, 32, 16, 2, 128, "bf16", [100], None, 0, (0, 0), 0),
    (2, 8, 8, 2, 128, "bf16", [1000, 90], None, 128, (0, 0), 0),  # windows: inside, at and across pages
    (2, 8, 8, 2, 64, "f32", [1000, 90], None, 1, (0, 0), 0),
    (2, 3, 3, 3, 128, "bf16", [640, 639], None, 64, (0, 0), 0),
    (2, 3, 3, 3, 64, "bf16", [640, 639], None, 65, (0, 0), 0),
    (1, 100, 3, 1, 128, "bf16", [0], None, 0, (0, 0), 0),         # a prompt over its own rows
    (1, 130, 2, 1, 64, "f32", [70], None, 33, (0, 0), 0),
    (40, 1, 4, 4, 64, "bf16", None, None, 0, (0, 0), 0),          # more tiles than SMs
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(case):
    B, T, nq, nkv, d, dtype, pos, n_rows, window, (ke, ve), extra = case
    pos = pos or [(37 * b) % 200 for b in range(B)]
    mp = (max(pos) + T + 63) // 64 + extra
    pages, bt = _cache(B * mp + 2, nkv, d, B, mp, 5, ke, ve)
    for b in range(B):                        # bytes of rows not yet appended hold anything: NaN scales
        for p in range(pos[b] + (T if n_rows is None else min(max(n_rows[b], 0), T)), mp * 64):
            rec = pages[bt[b, p // 64]]
            rec[:, 64 * d + p % 64 * (d // 16):64 * d + (p % 64 + 1) * (d // 16)] = 0x7F
            rec[:, 68 * d + p % 64::64] = 0x7F
    q = (torch.randn(B, T, nq, d, generator=_gen(6)) * 2.0 ** -ke).to(DT[dtype])
    scale = d ** -0.5
    qn = q.float().numpy()
    dev = [t.to(DEV) for t in (q, pages, bt)] + [torch.tensor(pos, dtype=torch.int64, device=DEV)]
    nr = torch.tensor(n_rows, dtype=torch.int32, device=DEV) if n_rows else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = torch.full((B, T, nq, d), 5.0, dtype=DT[dtype], device=DEV), torch.full((B, T, nq), 5.0, device=DEV)
    want, wlse, reach, eps = TO.attention(qn, pages.numpy(), bt.numpy(), pos, scale, window, n_rows, ke, ve,
                                          np.full((B, T, nq, d), 5.0), np.full((B, T, nq), 5.0))
    o2, l2 = binding.kv_attention(*dev, window=window, n_rows=nr, k_exp=ke, v_exp=ve, out=out, lse=lse, status=st)
    assert o2 is out and l2 is lse
    tol, ltol = _tolerance(want, reach, eps, max(pos) + T, d, dtype, ve)
    assert bool(torch.isfinite(out).all())
    _within(out, want, tol)
    _within(lse, wlse, ltol)
    assert int(st.item()) == 0
    # again, and without the lse, with a new output: the same bits
    o3, l3 = binding.kv_attention(*dev, window=window, n_rows=nr, k_exp=ke, v_exp=ve)
    keep = torch.ones(B, T, dtype=torch.bool) if n_rows is None else torch.arange(T) < torch.tensor(n_rows)[:, None]
    assert l3 is None and torch.equal(o3.cpu()[keep], out.cpu()[keep]) and not o3.cpu()[~keep].any()


def test_long_context_in_splits_and_in_a_graph():
    """20,000 keys over 152 SMs' worth of splits; captured, replayed with other queries and positions."""
    B, T, nq, nkv, d = 1, 8, 8, 2, 128
    mp = 320
    pages, bt = _cache(mp, nkv, d, B, mp, 8)
    q = torch.randn(2, B, T, nq, d, generator=_gen(9)).bfloat16()
    pos = [20000, 13]
    dq, dp = q[0].to(DEV), torch.tensor([pos[0]], device=DEV)
    args = (dq, pages.to(DEV), bt.to(DEV), dp)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out, lse = binding.kv_attention(*args, lse=True, stream=s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            gout, glse = binding.kv_attention(*args, lse=True, stream=s)
        for i in (0, 1):
            dq.copy_(q[i])
            dp.fill_(pos[i])
            graph.replay()
            s.synchronize()
            want, wl, reach, eps = TO.attention(q[i].float().numpy(), pages.numpy(), bt.numpy(), [pos[i]], d ** -0.5)
            tol, ltol = _tolerance(want, reach, eps, pos[i] + T, d, "bf16")
            _within(gout, want, tol)
            _within(glse, wl, ltol)
            if i == 0:
                assert torch.equal(out, gout) and torch.equal(lse, glse)


def test_holes_bad_ids_and_rows_without_keys():
    B, T, nq, nkv, d = 5, 2, 2, 1, 64
    pages, _ = _cache(3, nkv, d, 1, 1, 3)
    bt = np.array([[0, 1], [-1, 1], [-1, 7], [2, -3], [0, 1]], dtype=np.int32)
    pos = [80, 63, 100, 90, 127]            # the last block runs past the cache's end
    q = torch.randn(B, T, nq, d, generator=_gen(4))
    want, wl, reach, eps = TO.attention(q.numpy(), pages.numpy(), bt, pos, 0.125)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = binding.kv_attention(q.to(DEV), pages.to(DEV), torch.from_numpy(bt).to(DEV), torch.tensor(pos, device=DEV), lse=True, status=st)
    tol, ltol = _tolerance(want, reach, eps, 128, d, "f32")
    _within(out, want, tol)
    _within(lse, wl, ltol)
    assert not out[2].any() and not out[1, 0].any() and int(st.item()) == binding.DEV_BOUNDS
    # positions before 0 and far past the end: no keys, or the whole cache
    st.zero_()
    out, lse = binding.kv_attention(q[:2].to(DEV), pages.to(DEV), torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device=DEV),
                                    torch.tensor([-2, 1 << 41], device=DEV), lse=True, status=st)
    assert not out[0].any() and bool((lse[0] == -math.inf).all()) and bool(torch.isfinite(lse[1]).all()) and int(st.item()) == binding.DEV_BOUNDS


def test_queries_of_any_size_and_not_finite():
    """Queries far outside f16's range (their scores stay moderate through the scale), zero queries, NaN and infinity."""
    nkv, d = 1, 64
    pages, bt = _cache(2, nkv, d, 1, 2, 13)
    dev = (pages.to(DEV), bt.to(DEV), torch.tensor([100], device=DEV))
    base = torch.randn(1, 1, 4, d, generator=_gen(14))
    for dtype, size, scale in (("bf16", 2.0 ** 60, 2.0 ** -63), ("f32", 2.0 ** -70, 2.0 ** 67), ("f32", 2.0 ** 90, 2.0 ** -93),
                               ("bf16", 0.0, 1.0), ("f32", 1.0, 0.125)):
        q = (base * size).to(DT[dtype])
        want, wl, reach, eps = TO.attention(q.float().numpy(), pages.numpy(), bt.numpy(), [100], scale)
        out, lse = binding.kv_attention(q.to(DEV), *dev, scale=scale, lse=True)
        tol, ltol = _tolerance(want, reach, eps, 101, d, dtype)
        _within(out, want, tol)
        _within(lse, wl, ltol)
    q = base.clone()
    q[0, 0, 0, 5], q[0, 0, 2, 6], q[0, 0, 3, 7] = math.nan, math.inf, -math.inf
    for dtype in DT:
        out, lse = binding.kv_attention(q.to(DT[dtype]).to(DEV), *dev, lse=True)
        assert [bool(out[0, 0, i].isnan().all()) for i in range(4)] == [True, False, True, True]
        assert bool(torch.isfinite(out[0, 0, 1]).all()) and bool(lse[0, 0, 0].isnan())


def test_peaked_rows():
    """One key far above the rest, and all scores equal: weights at both ends of their range."""
    nkv, d = 1, 64
    pages, bt = _cache(4, nkv, d, 1, 4, 17)
    k, _ = TO.read_record(pages.numpy()[bt[0, 1], 0], 0, 0)
    q = torch.stack([torch.from_numpy(k[9]) * 40, torch.from_numpy(k[9]) * 3, torch.zeros(d), torch.from_numpy(-k[9])]).float()[None, None]
    dev = (pages.to(DEV), bt.to(DEV), torch.tensor([250], device=DEV))
    for dtype in DT:
        qd = q.to(DT[dtype])
        want, wl, reach, eps = TO.attention(qd.float().numpy(), pages.numpy(), bt.numpy(), [250], 0.125)
        out, lse = binding.kv_attention(qd.to(DEV), *dev, scale=0.125, lse=True)
        tol, ltol = _tolerance(want, reach, eps, 251, d, dtype)
        _within(out, want, tol)
        _within(lse, wl, ltol + 2.0 ** -22 * np.abs(wl))


def test_strided_rows_other_streams_and_workspaces():
    B, T, nq, nkv, d = 2, 4, 8, 2, 128
    mp = 40
    pages, bt = _cache(B * mp, nkv, d, B, mp, 19)
    pos = torch.tensor([2400, 1111], device=DEV)
    qkv = torch.randn(B, T, nq + 2 * nkv, d, generator=_gen(20)).bfloat16().to(DEV)
    q, dp, db = qkv[:, :, :nq], pages.to(DEV), bt.to(DEV)
    want, _ = binding.kv_attention(q.contiguous(), dp, db, pos)
    wide = torch.full((B, T, nq + 3, d), 2.0, dtype=torch.bfloat16, device=DEV)
    got, _ = binding.kv_attention(q, dp, db, pos, out=wide[:, :, :nq])
    assert torch.equal(got, want) and bool((wide[:, :, nq:] == 2).all())
    odd = torch.empty(q.numel() + 1, dtype=torch.bfloat16, device=DEV)[1:].view(q.shape)      # rows off 16 bytes
    odd.copy_(q)
    out = torch.empty(q.numel() + 3, dtype=torch.bfloat16, device=DEV)[3:].view(q.shape)
    assert torch.equal(binding.kv_attention(odd, dp, db, pos, out=out)[0], want)
    need = binding.kv_attention_workspace(B, T, nq, nkv, d, mp)
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)     # NaN bytes beforehand do not matter
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = [binding.kv_attention(q, dp, db, pos, stream=s, workspace=ws if i else None)[0] for i, s in enumerate(streams * 1)]
    torch.cuda.synchronize()
    assert all(torch.equal(r, want) for r in res) and bool((ws[need:] == 0xFF).all())
    with pytest.raises(binding.DliteError):
        binding.kv_attention(q, dp, db, pos, workspace=ws[:need - 16])
