"""GPU: token log probabilities of more rows than four CTAs an SM, every row of many stages of the shortest ring. Tolerances as
derived in test_gpu_token_logprobs.py."""
import pytest
import torch

from history_free_speculative_gb300 import binding
from test_gpu_token_logprobs import DEV, DT, _check, _gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_at_the_shortest_ring(dtype):
    rows, V, n_top = 4 * torch.cuda.get_device_properties(0).multi_processor_count + 9, 50257, 7
    g = _gen(61)
    x = (torch.randn(rows, V, generator=g) * 2.5).to(DT[dtype])
    x[::3].copy_(x[::3].sort(1).values)      # rising rows: their alternatives come last
    tok = torch.randint(0, V, (rows,), generator=g).to(torch.int32)
    tok[5::11] = -1
    got = binding.token_logprobs(x.to(DEV), tok.to(DEV), n_top=n_top)
    sel = torch.cat([torch.arange(0, rows, 23), torch.arange(rows - 4, rows)])
    _check(x[sel].double().numpy(), tok[sel], 1.0, n_top, {k: v.cpu()[sel] for k, v in got.items()})
    left = tok.to(DEV) < 0
    assert not got["logprob"][left].any() and not got["entropy"][left].any() and bool((got["top_ids"][left] == -1).all())
