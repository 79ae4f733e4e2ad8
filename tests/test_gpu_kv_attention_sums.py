"""GPU: float32 outputs of the attention over the paged 4-bit cache do not drift with the number of keys."""
import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import target_oracle as TO
from test_gpu_kv_attention import DEV, _gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_means_of_100_000_values(d):
    """Queries of 0: every weight is the same power of two, their sum is exact, and a row is the mean of its positive values, whose sum
    is not. One whole segment a CTA, so that a warp adds 200 pages in 400 halves. Derived: a half's products are two
    sums of 16 that may be cut off (2^-23 each, at most); each of the 400 adds, 8 joins of warps and 3 last steps rounds by at
    most 2^-24 of the sum, to either side: they stay within 7 sqrt(411) 2^-24 but for one case in 10^10 (Hoeffding). Sums that
    are cut off 800 times would be off by about 800 2^-25 = 400 2^-24 on the average."""
    sms, pool, n = torch.cuda.get_device_properties(0).multi_processor_count, 64, 1600
    g = _gen(71)
    pages = torch.randint(0, 256, (pool, 1, 72 * d), generator=g, dtype=torch.uint8)
    pages[..., 32 * d:64 * d] &= 0x77                                                    # positive codes
    pages[..., 64 * d:68 * d] = 0x38
    pages[..., 68 * d:] = torch.randint(0x08, 0x60, (pool, 1, 4 * d), generator=g).to(torch.uint8)   # scales from 2^-6 to 30
    bt = torch.randint(0, pool, (sms, n), generator=g).to(torch.int32)
    q = torch.zeros(sms, 1, 1, d, device=DEV)
    out, _ = binding.kv_attention(q, pages.to(DEV), bt.to(DEV), torch.full((sms,), 64 * n - 1, device=DEV))
    sums = np.stack([TO.read_record(pages.numpy()[p, 0], 0, 0)[1].sum(0) for p in range(pool)])
    count = np.stack([np.bincount(row, minlength=pool) for row in bt.numpy()])
    want = count @ sums / (64 * n)
    off = np.abs(out[:, 0, 0].double().cpu().numpy() / want - 1)
    assert off.max() <= 2 * 2.0 ** -23 + 7 * 411 ** 0.5 * 2.0 ** -24, off.max() * 2.0 ** 24
