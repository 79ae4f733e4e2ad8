"""GPU: attention over the paged 4-bit cache at the ends of what a call takes: query rows of very different sizes side by side,
queries, scales and scores at the ends of float32. Tolerances as derived in test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import target_oracle as TO
from test_gpu_kv_attention import DEV, DT, _cache, _gen, _tolerance, _within

pytestmark = pytest.mark.gpu
KINDS = [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)]


def _check(q, pages, bt, pos, scale, dtype, k_exp=0):
    """One call against the oracle; returns (out, lse)."""
    want, wl, reach, eps = TO.attention(q.float().numpy(), pages.numpy(), bt.numpy(), [pos], scale, k_exp=k_exp)
    out, lse = binding.kv_attention(q.to(DEV), pages.to(DEV), bt.to(DEV), torch.tensor([pos], device=DEV), scale=scale, k_exp=k_exp,
                                    lse=True)
    tol, ltol = _tolerance(want, reach, eps, pos + q.shape[1], q.shape[3], dtype)
    _within(out, want, tol)
    _within(lse, wl, ltol + 2.0 ** -22 * np.abs(wl))
    return out, lse


@pytest.mark.parametrize("size,scale,k_exp", [(1.0, 1e-42, 0), (2.0 ** -87, 0.125, -46), (2.0 ** -130, 2.0 ** 64, 64)])
@pytest.mark.parametrize("dtype,d", KINDS)
def test_factors_of_the_scores_at_the_ends_of_float32(dtype, d, size, scale, k_exp):
    """scale 2^k_exp and the queries' own factor, whose product is below or one of which is above what float32 holds: nearly
    equal weights, and scores of order one."""
    pages, bt = _cache(5, 1, d, 1, 5, 45)
    q = (torch.randn(1, 2, 4, d, generator=_gen(46)) * size).to(DT[dtype])
    _check(q, pages, bt, 270, scale, dtype, k_exp)


@pytest.mark.parametrize("T", [1, 8])
@pytest.mark.parametrize("dtype,d", KINDS)
def test_scores_below_minus_10_to_the_30(dtype, d, T):
    """Keys of 2 and then of 1 in every column, queries of -2^100: scores of -2 d 2^100 and -d 2^100, exact in any order. The keys of
    1 share the weight alike; before the first of them a row has the others'."""
    nq = 4
    pages, _ = _cache(5, 1, d, 1, 5, 47)
    pages[..., :32 * d] = 0x22            # codes of 1
    pages[..., 64 * d:68 * d] = 0x38      # scales of 1
    pages[:3, :, 64 * d:68 * d] = 0x40    # of 2
    bt = torch.arange(5, dtype=torch.int32)[None]
    q = torch.full((1, T, nq, d), -2.0 ** 100).to(DT[dtype])
    for pos in (100, 300):
        first, n, key = (0, pos, -2.0) if pos < 192 else (192, pos, -1.0)
        out, lse = binding.kv_attention(q.to(DEV), pages.to(DEV), bt.to(DEV), torch.tensor([pos], device=DEV), scale=1.0, lse=True)
        v = np.concatenate([TO.read_record(pages.numpy()[p, 0], 0, 0)[1] for p in range(5)])
        want = np.stack([v[first:n + t + 1].mean(0) for t in range(T)])[None, :, None].repeat(nq, 2)
        reach = np.stack([np.abs(v[first:n + t + 1]).mean(0) for t in range(T)])[None, :, None].repeat(nq, 2)
        tol, _ = _tolerance(want, reach, np.zeros((1, T, nq)), pos + T, d, dtype)
        _within(out, want, tol)
        wl = np.full((1, T, nq), key * d * 2.0 ** 100)
        _within(lse, wl, 2.0 ** -21 * np.abs(wl))


@pytest.mark.parametrize("pos", [300, 4000])       # one piece, and pieces of several CTAs
@pytest.mark.parametrize("scale", [1.1 * 2.0 ** 18, 1.1 * 2.0 ** 40, 1.1 * 2.0 ** 100])
@pytest.mark.parametrize("dtype,d", KINDS)
def test_scores_far_above_their_rounding(dtype, d, scale, pos):
    """Sharp rows, as with a scale that makes attention take the best key alone. q . k are multiples of a half below 2^13, exact in
    float32, so a row's weights are those of its largest keys, equal among equals."""
    T, nq, mp = 8, 4, pos // 64 + 2
    pages, bt = _cache(mp, 1, d, 1, mp, 48)
    pages[..., 64 * d:68 * d] = 0x38      # key scales of 1
    q = torch.randint(-3, 4, (1, T, nq, d), generator=_gen(49)).to(DT[dtype])
    want, wl, reach, eps = TO.attention(q.float().numpy(), pages.numpy(), bt.numpy(), [pos], scale)
    out, lse = binding.kv_attention(q.to(DEV), pages.to(DEV), bt.to(DEV), torch.tensor([pos], device=DEV), scale=scale, lse=True)
    tol, _ = _tolerance(want, reach, np.zeros_like(eps), pos + T, d, dtype)
    _within(out, want, tol)
    _within(lse, wl, 2.0 ** -21 * np.abs(wl))


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("T", [1, 8])
@pytest.mark.parametrize("dtype,d", KINDS)
def test_rows_of_different_sizes_in_one_tile(dtype, d, T, near):
    """A row's result does not depend on the rows beside it: rows of 1, 2^40 and 2^-40 (near: 2^4 and 2^-4), each with scores of order one at
    one of the scales (the others: a row of nearly equal weights, or one key alone, whose tolerance is wide)."""
    nq = 8
    pages, bt = _cache(6, 1, d, 1, 6, 41)
    size = torch.tensor([0, 4, -4, 0, -3, 0, 4, -4, 0, 3, 0] if near else [0, 40, -40, 0, -33, 0, 40, -40, 0, 33, 0])
    size = size.repeat((T * nq + 10) // 11)[:T * nq].view(1, T, nq, 1)
    q = (torch.randn(1, T, nq, d, generator=_gen(42)) * torch.exp2(size.float())).to(DT[dtype])
    for e in (0, 4, -4) if near else (0, 40, -40):
        _check(q, pages, bt, 300, d ** -0.5 * 2.0 ** -e, dtype)


@pytest.mark.parametrize("size,scale", [(2.0 ** 125, 2.0 ** -128), (2.0 ** 116, 2.0 ** -119), (2.0 ** -125, 2.0 ** 122)])
@pytest.mark.parametrize("dtype,d", KINDS)
def test_queries_at_the_ends_of_float32(dtype, d, size, scale):
    pages, bt = _cache(5, 1, d, 1, 5, 43)
    q = (torch.randn(1, 2, 4, d, generator=_gen(44)) * size).to(DT[dtype])
    assert bool(torch.isfinite(q).all()) and bool((q != 0).any(-1).all())
    _check(q, pages, bt, 270, scale, dtype)
