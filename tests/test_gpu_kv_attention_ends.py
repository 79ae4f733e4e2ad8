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


@pytest.mark.parametrize("size,scale,k_exp", [(1.0, 1e-42, 0), (2.0 ** -87, 0.125, -46)])
@pytest.mark.parametrize("dtype,d", KINDS)
def test_factors_of_the_scores_at_the_ends_of_float32(dtype, d, size, scale, k_exp):
    """scale 2^k_exp and the queries' own factor, whose product is below what float32 holds: nearly equal weights."""
    pages, bt = _cache(5, 1, d, 1, 5, 45)
    q = (torch.randn(1, 2, 4, d, generator=_gen(46)) * size).to(DT[dtype])
    _check(q, pages, bt, 270, scale, dtype, k_exp)
