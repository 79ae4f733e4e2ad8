"""GPU: rotary positions and the paged 4-bit cache (append, read back) through the C ABI,
against the CPU oracle. The rotation's float32 steps and the quantisation are part of the
operators' definition, so rotated values and cache bytes are compared bit for bit."""
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


def _rows(shape, dtype, seed, packed=0, offset=0, scale=1.0):
    """A device tensor [B, T, H, d]: dense, or `packed` heads wide rows with the heads at a head offset
    (as a slice of fused projections), or starting `offset` elements into its storage."""
    B, T, H, d = shape
    x = (torch.randn(B, T, max(packed, H), d, generator=_gen(seed)) * scale).to(DT[dtype])
    if offset:
        buf = torch.empty(x.numel() + offset, dtype=x.dtype, device=DEV)
        y = buf[offset:].view(x.shape)
        y.copy_(x)
        x = y
    x = x.to(DEV)
    return x[:, :, packed - H:] if packed else x


def _np(x):
    return x.detach().float().cpu().numpy()


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("kw", [
    dict(rot=128), dict(rot=64, theta=1e4), dict(rot=48, scaling="linear", factor=8.0), dict(rot=2), dict(rot=256),
    dict(rot=128, scaling="ntk", factor=4.0), dict(rot=128, scaling="yarn", factor=4.0, orig_len=32768.0),
    dict(rot=64, scaling="yarn", factor=32.0, orig_len=4096.0, beta_fast=16.0, beta_slow=2.0, attn_factor=1.25),
], ids=str)
def test_rope_table(kw):
    n = 3001
    got = binding.rope_table(n, **kw).cpu().numpy()
    want = TO.rope_table(n, **kw)
    assert got.shape == want.shape
    # cos and sin in float64 (errors far below 2^-24) rounded once: one float32 step apart at a border, else equal
    assert np.all(np.abs(got.astype(np.float64) - want) <= np.spacing(np.abs(want)) + 1e-12)
    assert (got != want).mean() < 1e-3


def test_rope_table_far_positions():
    """A million positions: the angle of the fastest pair is a million radians; float32 would hold it to 0.03."""
    n = 1 << 20
    got = binding.rope_table(n, rot=8, theta=1e6)
    p = np.array([n - 1, n - 2, 999_983, 524_287])
    a = p[:, None] * TO.rope_freqs(8)
    assert np.abs(got[torch.from_numpy(p).to(DEV)].cpu().numpy() - np.stack([np.cos(a), np.sin(a)], -1)).max() < 2.0 ** -24 + 1e-9


ROPE_CASES = [
    # B, T, H, d, rot, layout, dtype, packed, offset, ragged
    (1, 1, 32, 128, 128, "half", "bf16", 0, 0, False),
    (3, 8, 5, 128, 128, "half", "bf16", 11, 0, True),
    (3, 8, 5, 128, 128, "interleaved", "f32", 11, 0, True),
    (2, 5, 4, 64, 48, "half", "f32", 0, 0, False),       # part of the head
    (2, 5, 4, 64, 48, "half", "bf16", 0, 0, False),
    (2, 3, 3, 64, 24, "interleaved", "bf16", 0, 0, False),
    (2, 3, 3, 64, 20, "interleaved", "bf16", 0, 0, False),   # 20: no whole 16-byte pieces
    (2, 3, 3, 64, 20, "half", "f32", 0, 0, False),
    (2, 3, 2, 33, 2, "half", "bf16", 0, 0, False),       # odd head
    (2, 3, 2, 33, 32, "interleaved", "f32", 5, 0, False),
    (2, 9, 2, 128, 128, "half", "bf16", 0, 1, False),    # rows off 16 bytes
    (2, 9, 2, 128, 64, "interleaved", "f32", 0, 3, True),
    (1, 300, 2, 256, 256, "half", "f32", 0, 0, False),
    (65, 1, 1, 96, 96, "half", "bf16", 0, 0, False),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=str)
def test_rope(case):
    B, T, H, d, rot, layout, dtype, packed, offset, ragged = case
    x = _rows((B, T, H, d), dtype, 11, packed, offset)
    table = binding.rope_table(900, rot)
    pos = torch.randint(0, 900 - T, (B,), generator=_gen(2))
    n_rows = [(3 * b + 1) % (T + 2) - (1 if b == 2 else 0) for b in range(B)] if ragged else None   # past T, and below 0
    if ragged:
        n_rows[0] = 0
    nr = torch.tensor(n_rows, dtype=torch.int32, device=DEV) if ragged else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((B, T, H, d), 7.0, dtype=x.dtype, device=DEV)
    want = TO.rope(_np(x), pos, table.cpu().numpy(), layout, n_rows, np.full((B, T, H, d), 7.0), dtype)
    assert binding.rope(x, pos.to(DEV), table, layout, n_rows=nr, out=out, status=st) is out
    assert np.array_equal(_np(out), want.astype(np.float32))
    if not ragged:
        assert torch.equal(binding.rope(x, pos.to(DEV), table, layout), out)
        binding.rope(x, pos.to(DEV), table, layout, out=x)     # in place, neighbours of a slice untouched
        assert torch.equal(x, out)
    assert int(st.item()) == 0


def test_rope_in_place_leaves_the_other_heads():
    qkv = torch.randn(2, 3, 6, 128, generator=_gen(3)).to(DEV)
    want = qkv.clone()
    table, pos = binding.rope_table(50, 64), torch.tensor([4, 40], device=DEV)
    want[:, :, 1:4] = binding.rope(qkv[:, :, 1:4], pos, table, "interleaved")
    binding.rope(qkv[:, :, 1:4], pos, table, "interleaved", out=qkv[:, :, 1:4])
    assert torch.equal(qkv, want)


def test_rope_positions_outside_the_table():
    x = _rows((3, 2, 1, 64), "f32", 5)
    table = binding.rope_table(10, 64)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos = torch.tensor([-5, 9, 1 << 40], device=DEV)
    got = binding.rope(x, pos, table, status=st)
    assert np.array_equal(_np(got), TO.rope(_np(x), [-5, 9, 1 << 40], table.cpu().numpy(), "half"))
    assert int(st.item()) == binding.DEV_BOUNDS


def test_rope_propagates_non_finite_values():
    x = torch.zeros(1, 1, 2, 64, device=DEV)
    x[0, 0, 0, 3], x[0, 0, 1, 40] = math.nan, math.inf
    got = binding.rope(x, torch.tensor([3], device=DEV), binding.rope_table(8, 32))
    assert bool(got[0, 0, 0, [3, 19]].isnan().all()) and int(got.isnan().sum()) == 2 and float(got[0, 0, 1, 40]) == math.inf


# ---------------------------------------------------------------- cache

def _cache(n_pages, H, d, B, max_pages, seed):
    """Random (finite) cache contents and a table of distinct pages."""
    g = _gen(seed)
    pages = torch.randint(0, 256, (n_pages, H, 72 * d), generator=g, dtype=torch.uint8)
    pages[..., 64 * d:] %= 0x7F
    bt = torch.randperm(n_pages, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32)
    return pages, bt


APPEND_CASES = [
    # B, T, H, d, dtype, rot, layout, packed, offset, pos, n_rows, exps
    (1, 1, 8, 128, "bf16", 128, "half", 0, 0, [1000], None, (0, 0)),
    (1, 1, 1, 64, "f32", 0, "half", 0, 0, [0], None, (0, 0)),
    (3, 2, 2, 64, "f32", 64, "half", 0, 0, [63, 64, 127], None, (0, 0)),       # across a page's end
    (3, 8, 3, 128, "bf16", 128, "half", 9, 0, [5, 60, 122], [8, 0, 5], (-3, 2)),
    (3, 8, 1, 128, "f32", 64, "interleaved", 0, 0, [5, 61, 120], [9, -2, 1], (1, 1)),
    (2, 7, 2, 64, "bf16", 24, "interleaved", 0, 0, [1, 62], None, (0, 0)),
    (2, 7, 2, 64, "bf16", 24, "half", 0, 0, [1, 62], None, (0, 0)),              # halves of 12 columns
    (2, 7, 2, 64, "f32", 62, "interleaved", 3, 0, [3, 58], None, (0, 0)),
    (2, 5, 2, 128, "bf16", 128, "half", 0, 1, [3, 59], None, (0, 0)),            # rows off 16 bytes
    (1, 64, 1, 128, "bf16", 128, "half", 0, 0, [64], None, (0, 0)),              # exactly one page
    (1, 64, 2, 64, "f32", 32, "interleaved", 0, 0, [17], None, (0, 0)),
    (2, 200, 1, 64, "bf16", 64, "half", 0, 0, [1, 63], [200, 131], (0, -4)),     # a prompt, whole and cut pages
    (1, 129, 2, 128, "f32", 128, "half", 0, 0, [63], None, (0, 0)),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=str)
def test_append_bytes_and_read_back(case):
    B, T, H, d, dtype, rot, layout, packed, offset, pos, n_rows, (ke, ve) = case
    max_pages = max(pos) // 64 + (T + 126) // 64
    pages, bt = _cache(B * max_pages + 3, H, d, B, max_pages, 21)
    k = _rows((B, T, H, d), dtype, 31, packed, offset, scale=2.0 ** ke)
    v = _rows((B, T, H, d), dtype, 32, packed, offset, scale=3.0 * 2.0 ** ve)
    table = binding.rope_table(max(pos) + T, rot) if rot else None
    want = pages.numpy().copy()
    flags = TO.append(want, bt.numpy(), _np(k), _np(v), pos, None if table is None else table.cpu().numpy(), layout, n_rows, ke, ve)
    assert not flags
    dp, dbt = pages.to(DEV), bt.to(DEV)
    dpos = torch.tensor(pos, dtype=torch.int64, device=DEV)
    nr = torch.tensor(n_rows, dtype=torch.int32, device=DEV) if n_rows else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.kv_append(dp, dbt, k, v, dpos, table, layout, n_rows=nr, k_exp=ke, v_exp=ve, status=st)
    got = dp.cpu().numpy()
    bad = np.argwhere(got != want)
    assert not len(bad), (len(bad), bad[:4], [(got[tuple(i)], want[tuple(i)]) for i in bad[:4]])
    for odt in (torch.bfloat16, torch.float32):
        ko, vo = (torch.full((B, T, H, d), 9.0, dtype=odt, device=DEV) for _ in range(2))
        binding.kv_read(dp, dbt, dpos, T, n_rows=nr, k_exp=ke, v_exp=ve, k_out=ko, v_out=vo, status=st)
        for b in range(B):
            n = T if n_rows is None else min(max(n_rows[b], 0), T)
            assert float((ko[b, n:] - 9).abs().sum() + (vo[b, n:] - 9).abs().sum()) == 0
            for t in range(n):
                for h in range(H):
                    p = pos[b] + t
                    kk, vv = TO.read_row(want[bt[b, p // 64], h], p % 64, ke, ve)
                    assert np.array_equal(_np(ko[b, t, h]), kk) and np.array_equal(_np(vo[b, t, h]), vv)
    assert int(st.item()) == 0


def test_append_special_values():
    """Ties, zeros, saturation, subnormal scales, NaN and infinities: the same bytes as the definition's."""
    d = 64
    rng = np.random.default_rng(9)
    rows = [np.full(d, 1e-30), np.zeros(d), -np.zeros(d), np.full(d, 3e38), np.full(d, 5e3), rng.normal(size=d) * 1e-3,
            rng.normal(size=d) * 0.01, np.arange(d) / 8.0, np.where(np.arange(d) % 5 == 0, np.nan, 1.0 + np.arange(d)),
            np.where(np.arange(d) % 7 == 0, -np.inf, 0.25 * np.arange(d)), np.where(np.arange(d) == 20, np.inf, 0.0),
            np.tile([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25], 4)]
    k = np.stack(rows).astype(np.float32)[None, :, None]
    v = np.ascontiguousarray(k[:, ::-1])
    T = len(rows)
    want = np.zeros((1, 1, 72 * d), dtype=np.uint8)
    flags = TO.append(want, np.array([[0]]), k, v, [3])
    assert flags == {"nonfinite"}
    pages = binding.kv_pages(1, 1, d)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.kv_append(pages, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV),
                      torch.tensor([3], device=DEV), status=st)
    assert np.array_equal(pages.cpu().numpy(), want)
    assert int(st.item()) == binding.DEV_NONFINITE
    assert bool(torch.isfinite(binding.kv_read(pages, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([3], device=DEV),
                                               T, dtype=torch.float32)[0]).all())


def test_append_outside_the_cache():
    """Rows before position 0, past the table, in holes or in pages that do not exist: not stored, flagged; the rest is."""
    B, T, H, d = 5, 4, 1, 64
    pages, _ = _cache(4, H, d, 1, 1, 2)
    bt = np.array([[0, 1], [2, -1], [3, 4], [-7, 99], [-1, -1]], dtype=np.int32)
    pos = [-2, 62, 62, 63, 1 << 40]
    k, v = _rows((B, T, H, d), "f32", 1), _rows((B, T, H, d), "f32", 2)
    want = pages.numpy().copy()
    assert TO.append(want, bt, _np(k), _np(v), pos) == {"bounds"}
    dp, st = pages.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    dpos = torch.tensor(pos, dtype=torch.int64, device=DEV)
    binding.kv_append(dp, torch.from_numpy(bt).to(DEV), k, v, dpos, status=st)
    assert np.array_equal(dp.cpu().numpy(), want)
    assert int(st.item()) == binding.DEV_BOUNDS
    st.zero_()
    ko, _ = binding.kv_read(dp, torch.from_numpy(bt).to(DEV), dpos, T, dtype=torch.float32, status=st)
    assert int(st.item()) == binding.DEV_BOUNDS
    assert [[bool(ko[b, t].any()) for t in range(T)] for b in range(B)] == [
        [False, False, True, True], [True, True, False, False], [True, True, False, False], [False] * 4, [False] * 4]


def test_append_position_past_the_rope_table():
    pages = binding.kv_pages(2, 1, 64)
    bt = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    k, v = _rows((1, 3, 1, 64), "f32", 1), _rows((1, 3, 1, 64), "f32", 2)
    table, st = binding.rope_table(41, 64), torch.zeros(1, dtype=torch.int32, device=DEV)
    want = pages.cpu().numpy()
    assert TO.append(want, bt.cpu().numpy(), _np(k), _np(v), [40], table.cpu().numpy()) == {"bounds"}
    binding.kv_append(pages, bt, k, v, torch.tensor([40], device=DEV), table, status=st)
    assert np.array_equal(pages.cpu().numpy(), want) and int(st.item()) == binding.DEV_BOUNDS


def test_append_token_by_token_equals_a_prompt():
    """Neighbouring tokens share bytes: one at a time, in a captured and replayed call too, the cache is the prompt's."""
    H, d, N = 2, 128, 70
    k, v = _rows((1, N, H, d), "bf16", 4), _rows((1, N, H, d), "bf16", 5)
    table = binding.rope_table(200, d)
    bt = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    whole, single = binding.kv_pages(3, H, d), binding.kv_pages(3, H, d)
    binding.kv_append(whole, bt, k, v, torch.tensor([33], device=DEV), table)
    pos = torch.tensor([33], device=DEV)
    kb, vb, one = torch.empty_like(k[:, :1]), torch.empty_like(v[:, :1]), torch.ones(1, dtype=torch.int64, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            binding.kv_append(single, bt, kb, vb, pos, table, stream=s)
            pos += one
        for i in range(N):
            kb.copy_(k[:, i:i + 1])
            vb.copy_(v[:, i:i + 1])
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(whole, single)


def test_the_binding_refuses_what_it_does_not_take():
    x, pos, table = _rows((2, 3, 2, 64), "f32", 1), torch.zeros(2, dtype=torch.int64, device=DEV), binding.rope_table(8, 64)
    pages, bt = binding.kv_pages(4, 2, 64), torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    V = ValueError
    for err, call in [
            (V, lambda: binding.rope(x, pos.int(), table)), (V, lambda: binding.rope(x, pos[:1], table)),
            (V, lambda: binding.rope(x.half(), pos, table)), (V, lambda: binding.rope(x, pos, table, layout="pairs")),
            (V, lambda: binding.rope(x, pos, table.double())), (V, lambda: binding.rope(x, pos, table, out=x[:1])),
            (V, lambda: binding.rope(x, pos, table, n_rows=pos)), (V, lambda: binding.rope(x.transpose(1, 2), pos, table)),
            (V, lambda: binding.rope(x, pos, table, status=torch.zeros(2, dtype=torch.int32, device=DEV))),
            (V, lambda: binding.rope_table(8, 64, scaling="other")), (binding.DliteError, lambda: binding.rope_table(0, 64)),
            (binding.DliteError, lambda: binding.rope(x[..., :32].contiguous(), pos, table)),
            (V, lambda: binding.kv_append(pages, bt, x, x[:, :, :1], pos)), (V, lambda: binding.kv_append(pages, bt.long(), x, x, pos)),
            (V, lambda: binding.kv_append(pages[:, :1], bt, x, x, pos)), (V, lambda: binding.kv_append(pages, bt[:1], x, x, pos)),
            (V, lambda: binding.kv_append(pages, bt, x, x.bfloat16(), pos)), (V, lambda: binding.kv_append(pages.int(), bt, x, x, pos)),
            (V, lambda: binding.kv_read(pages, bt, pos, 1, k_out=x)), (V, lambda: binding.kv_read(pages, bt, pos, 2, k_out=x, v_out=x)),
            (V, lambda: binding.kv_attention(x[..., :32], pages, bt, pos)), (V, lambda: binding.kv_attention(x, pages, bt, pos, lse=pos)),
            (V, lambda: binding.kv_attention(x, pages, bt, pos, out=x.bfloat16())),
            (binding.DliteError, lambda: binding.kv_attention(x[:, :, :1], pages, bt, pos)),
            (binding.DliteError, lambda: binding.kv_attention(x, pages, bt, pos, scale=-1.0)),
            (V, lambda: binding.token_logprobs(x, bt)), (V, lambda: binding.token_logprobs(x[0, 0], pos)),
            (V, lambda: binding.token_logprobs(x[0, 0].half(), bt[0])), (V, lambda: binding.token_logprobs(x[0, 0].t().contiguous().t(), bt[0])),
            (binding.DliteError, lambda: binding.token_logprobs(x[0, 0], bt[0], temperature=0.0)),
            (binding.DliteError, lambda: binding.token_logprobs(x[0, 0], bt[0], n_top=33))]:
        with pytest.raises(err):
            call()
