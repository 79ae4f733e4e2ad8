"""GPU: attention over the paged 4-bit cache, bf16 queries with heads of 128 (keys and values as operands in tensor memory):
holes in a tile, odd queries, references that move, lists of pieces longer than one batch. Tolerances as derived in
test_gpu_kv_attention.py."""
import math

import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import target_oracle as TO
from test_gpu_kv_attention import DEV, _cache, _gen, _tolerance, _within

pytestmark = pytest.mark.gpu
D = 128


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("T", [1, 8])       # tiles of 16 and of 32 query rows
def test_holes_and_bad_ids(T):
    nq, nkv = 8, 2
    pages, _ = _cache(6, nkv, D, 1, 6, 31)
    bt = np.array([[0, 1, 2, 3, 4, 5], [-1, 1, 2, 3, 4, 5], [0, -1, 2, -7, 4, 5], [-1, -1, 2, 3, -1, -1], [-1] * 6,
                   [0, 1, 2, 9, 4, 5], [0, 1, 2, 3, 4, -1]], dtype=np.int32)
    pos = [300, 300, 320, 200, 383 - T, 250, 383 - T]
    q = torch.randn(len(pos), T, nq, D, generator=_gen(32)).bfloat16()
    for window in (0, 130):
        st = _status()
        want, wl, reach, eps = TO.attention(q.float().numpy(), pages.numpy(), bt, pos, D ** -0.5, window)
        out, lse = binding.kv_attention(q.to(DEV), pages.to(DEV), torch.from_numpy(bt).to(DEV), torch.tensor(pos, device=DEV),
                                        window=window, lse=True, status=st)
        tol, ltol = _tolerance(want, reach, eps, 384, D, "bf16")
        _within(out, want, tol)
        _within(lse, wl, ltol)
        assert not out[4].any() and int(st.item()) == binding.DEV_BOUNDS      # the id 9


def test_queries_of_any_size_and_not_finite():
    nkv = 1
    pages, bt = _cache(5, nkv, D, 1, 5, 33)
    dev = (pages.to(DEV), bt.to(DEV), torch.tensor([300], device=DEV))
    base = torch.randn(1, 1, 4, D, generator=_gen(34))
    for size, scale in ((2.0 ** 60, 2.0 ** -63), (2.0 ** -70, 2.0 ** 67), (2.0 ** 90, 2.0 ** -93), (0.0, 1.0)):
        q = (base * size).bfloat16()
        want, wl, reach, eps = TO.attention(q.float().numpy(), pages.numpy(), bt.numpy(), [300], scale)
        out, lse = binding.kv_attention(q.to(DEV), *dev, scale=scale, lse=True)
        tol, ltol = _tolerance(want, reach, eps, 301, D, "bf16")
        _within(out, want, tol)
        _within(lse, wl, ltol)
    q = base.bfloat16()
    want, wl, reach, eps = TO.attention(q.float().numpy(), pages.numpy(), bt.numpy(), [300], D ** -0.5)
    q[0, 0, 0, 5], q[0, 0, 2, 6], q[0, 0, 3, 7] = math.nan, math.inf, -math.inf
    out, lse = binding.kv_attention(q.to(DEV), *dev, lse=True)
    assert [bool(out[0, 0, i].isnan().all()) for i in range(4)] == [True, False, True, True]
    assert [bool(lse[0, 0, i].isnan()) for i in range(4)] == [True, False, True, True]
    tol, ltol = _tolerance(want, reach, eps, 301, D, "bf16")
    _within(out[:, :, 1], want[:, :, 1], tol[:, :, 1])
    _within(lse[:, :, 1], wl[:, :, 1], ltol[:, :, 1])


@pytest.mark.parametrize("T", [1, 8])
def test_references_that_move(T):
    """Scores with a wide spread, so that a later key passes the reference by more than 2^8 time and again, and rows whose
    scores rise, or fall, from page to page."""
    nq, nkv, mp = 4, 1, 40
    pages, bt = _cache(mp, nkv, D, 1, mp, 35)
    q = torch.randn(1, T, nq, D, generator=_gen(36)).bfloat16()
    k = np.concatenate([TO.read_record(pages.numpy()[p, 0], 0, 0)[0] for p in range(mp)])      # [64 mp, D] in page order
    top = (k @ q[0, 0, 0].float().numpy()).reshape(mp, 64).max(1)
    assert (top.max() - top.min()) / math.log(2) > 2 * 8      # rising pages pass a reference twice at least
    for order in (bt[0].numpy(), np.argsort(top), np.argsort(-top)):
        tab = order.astype(np.int32)[None]
        pos = [64 * mp - T - 5]
        want, wl, reach, eps = TO.attention(q.float().numpy(), pages.numpy(), tab, pos, 1.0)
        out, lse = binding.kv_attention(q.to(DEV), pages.to(DEV), torch.from_numpy(tab).to(DEV), torch.tensor(pos, device=DEV),
                                        scale=1.0, lse=True)
        tol, ltol = _tolerance(want, reach, eps, 64 * mp, D, "bf16")
        _within(out, want, tol)
        _within(lse, wl, ltol + 2.0 ** -22 * np.abs(wl))


@pytest.mark.parametrize("mp", [2, 10], ids=["whole segments", "cut"])
def test_more_pieces_a_cta_than_a_list_holds(mp):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    nkv, n_pages = 8, 64
    B = (36 * sms + nkv - 1) // nkv
    pages, _ = _cache(n_pages, nkv, D, 1, 1, 37)
    g = _gen(38)
    bt = torch.randint(0, n_pages, (B, mp), generator=g).to(torch.int32).to(DEV)
    pos = torch.randint(0, 64 * mp, (B,), generator=g).to(DEV)
    q = torch.randn(B, 1, nkv, D, generator=g).bfloat16().to(DEV)
    pages = pages.to(DEV)
    st = _status()
    out, lse = binding.kv_attention(q, pages, bt, pos, lse=True, status=st)
    assert int(st.item()) == 0
    k, v = binding.kv_read(pages, bt, torch.zeros_like(pos), 64 * mp, dtype=torch.float32)     # [B, keys, nkv, D]
    k, v, qd = k.double(), v.double(), q[:, 0].double()
    s = torch.einsum("bhd,bjhd->bhj", qd, k) * D ** -0.5
    eps = torch.einsum("bhd,bjhd->bhj", qd.abs(), k.abs()).amax(-1) * D ** -0.5
    s = s.masked_fill(torch.arange(64 * mp, device=DEV)[None, None] > pos[:, None, None], -math.inf)
    p = torch.softmax(s, -1)
    want, reach = torch.einsum("bhj,bjhd->bhd", p, v), torch.einsum("bhj,bjhd->bhd", p, v.abs())
    wl = torch.logsumexp(s, -1)
    want, reach, eps, wl = (x.cpu().numpy() for x in (want, reach, eps, wl))
    tol, ltol = _tolerance(want, reach, eps, 64 * mp, D, "bf16")
    _within(out[:, 0], want, tol)
    _within(lse[:, 0], wl, ltol)
