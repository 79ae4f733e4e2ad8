"""GPU: target-side calls on tensors whose offsets pass 32 bits: the far end gives what the same rows give in a small tensor."""
import math

import pytest
import torch

from history_free_speculative_gb300 import binding
from test_gpu_kv_attention import DEV, DT, _gen
from test_gpu_token_logprobs import _rel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_pages_behind_4_gib(dtype, d):
    nkv, nq, T, few = 8, 16, 5, 3
    n_pages = (1 << 32) // (nkv * 72 * d) + 100
    pages = torch.empty(n_pages, nkv, 72 * d, dtype=torch.uint8, device=DEV)
    pages[-few:] = 0
    small = binding.kv_pages(few, nkv, d)
    k, v, q = (torch.randn(1, T, h, d, generator=_gen(81 + h)).to(DEV, DT[dtype]) for h in (nkv, nkv, nq))
    past = [torch.randn(1, 130, nkv, d, generator=_gen(90 + i)).to(DEV, DT[dtype]) for i in range(2)]
    pos, table = torch.tensor([130], device=DEV), binding.rope_table(200, d)
    got = []
    for cache, first in ((pages, n_pages - few), (small, 0)):
        bt = torch.arange(first, first + few, dtype=torch.int32, device=DEV)[None]
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        binding.kv_append(cache, bt, *past, torch.zeros_like(pos), table, status=st)
        binding.kv_append(cache, bt, k, v, pos, table, status=st)
        got.append((cache[first:].clone(), *binding.kv_read(cache, bt, pos, T, status=st), *binding.kv_attention(q, cache, bt, pos, lse=True, status=st)))
        assert st.item() == 0
    assert all(torch.equal(a, b) for a, b in zip(*got)) and bool(got[0][3].any())


def test_rows_behind_2_to_the_31_elements():
    H, d = 32, 128
    n = (1 << 31) // (H * d) + 50
    x = torch.empty(n, 1, H, d, dtype=torch.bfloat16, device=DEV)
    x[-7:] = torch.randn(7, 1, H, d, generator=_gen(95)).to(DEV, torch.bfloat16)
    rows = torch.zeros(n, dtype=torch.int32, device=DEV)
    rows[-7:] = 1
    pos, table = torch.full((n,), 11, dtype=torch.int64, device=DEV), binding.rope_table(20, d)
    want = binding.rope(x[-7:].clone(), pos[-7:].clone(), table)
    assert torch.equal(binding.rope(x, pos, table, n_rows=rows, out=x)[-7:], want)
    del x
    V = 151936
    n = (1 << 31) // V + 20
    x = torch.empty(n, V, dtype=torch.bfloat16, device=DEV)
    x[-7:] = torch.randn(7, V, generator=_gen(96)).to(DEV, torch.bfloat16)
    tok = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    tok[-7:] = torch.arange(7, dtype=torch.int32, device=DEV)
    got = {k: t[-7:] for k, t in binding.token_logprobs(x, tok, n_top=3).items()}
    want = binding.token_logprobs(x[-7:].clone(), tok[-7:].clone(), n_top=3)
    assert torch.equal(got["top_ids"], want["top_ids"])
    # other slices of a row, so sums in another order: both calls lie within the tolerance of test_gpu_token_logprobs.py (logits of this size
    # give entropies and log S below ln V, log probabilities above -30)
    tol = 2 * (2 * _rel(V) * math.log(V) + 4 * 2.0 ** -24 * 30)
    for k in ("logprob", "entropy", "top_logprobs"):
        assert bool((want[k].abs() < 30).all()) and (got[k] - want[k]).abs().max().item() <= tol
