"""GPU: the ends of what the target-side calls take: positions at the ends of 64 bits, one CTA with many tiles,
workspaces that only look large enough. Tolerances as derived in test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from test_gpu_kv_attention import DEV, DT, _cache, _gen, _tolerance, _within

pytestmark = pytest.mark.gpu
MOST, LEAST = 2 ** 63 - 1, -2 ** 63
BOUNDS = 2


def _pos(*p):
    return torch.tensor(p, dtype=torch.int64, device=DEV)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype, d", [("bf16", 128), ("f32", 64)])
def test_positions_at_the_ends_of_64_bits(dtype, d):
    H, nq, T, n_pages = 2, 4, 2, 3
    pages, bt = _cache(n_pages, H, d, 1, n_pages, 5)
    pages, bt = pages.to(DEV), bt.to(DEV)
    g = _gen(6)
    q, k, v = (torch.randn(1, T, h, d, generator=g).to(DEV, DT[dtype]) for h in (nq, H, H))
    table = binding.rope_table(50, d)

    # rope: the nearest end of the table
    for p, end in ((MOST, 49), (LEAST, 0)):
        st = _status()
        got = binding.rope(q, _pos(p), table, status=st)
        want = torch.cat([binding.rope(q[:, t:t + 1].contiguous(), _pos(end), table) for t in range(T)], 1)
        assert torch.equal(got, want) and st.item() == BOUNDS

    # append and read: nothing is stored, nothing is read
    for p in (MOST, LEAST):
        st, copy = _status(), pages.clone()
        binding.kv_append(copy, bt, k, v, _pos(p), table=table, status=st)
        assert torch.equal(copy, pages) and st.item() & BOUNDS
        st, out = _status(), [torch.full_like(k, 7.0) for _ in range(2)]
        binding.kv_read(pages, bt, _pos(p), T, k_out=out[0], v_out=out[1], status=st)
        assert all(bool((o == 7).all()) for o in out) and st.item() & BOUNDS

    # attention: behind the cache's end a row sees all of it, before its beginning nothing
    st = _status()
    out, lse = binding.kv_attention(q, pages, bt, _pos(MOST), lse=True, status=st)
    for t in range(T):
        want, want_lse = binding.kv_attention(q[:, t:t + 1].contiguous(), pages, bt, _pos(64 * n_pages - 1), lse=True)
        n = 64 * n_pages
        tol = 2 * (2.0 ** -8 + 2.0 ** -10) if dtype == "bf16" else 2.0 ** -16   # both calls round weights and outputs
        scale = 6 * 0.6875
        assert (out[:, t:t + 1].double() - want.double()).abs().max().item() <= tol * scale
        assert (lse[:, t:t + 1] - want_lse).abs().max().item() <= 2 * (2.0 ** -11 + 2.0 ** -22 * 20 + (n / 16 + 64) * 2.0 ** -24)
    assert st.item() & BOUNDS
    for window in (0, 5):
        st = _status()
        out, lse = binding.kv_attention(q, pages, bt, _pos(LEAST), window=window, lse=True, status=st)
        assert not out.any() and bool((lse == -float("inf")).all()) and st.item() & BOUNDS


@pytest.mark.parametrize("T", [1, 8])
def test_many_tiles_a_cta(T):
    """Four pages named over and over: the softmax over all of them is the one over four with counted keys."""
    nq, d, n_pages = 4, 128, 4
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    repeats = (sms * 45 * 2 + n_pages - 1) // n_pages       # 45 tiles of two pages for every CTA
    pages, _ = _cache(n_pages, 1, d, 1, n_pages, 9)
    pages = pages.to(DEV)
    bt = torch.arange(n_pages, dtype=torch.int32, device=DEV).repeat(repeats).view(1, -1)
    keys = 64 * n_pages * repeats
    q = torch.randn(1, T, nq, d, generator=_gen(10)).to(DEV, torch.bfloat16)
    st = _status()
    out, lse = binding.kv_attention(q, pages, bt, _pos(keys - T), lse=True, status=st)
    assert st.item() == 0
    k, v = (x[0, :, 0].double().cpu().numpy() for x in binding.kv_read(pages, bt[:, :n_pages].contiguous(), _pos(0), 64 * n_pages,
                                                                      dtype=torch.float32))
    qd = q[0].double().cpu().numpy()
    s = qd @ k.T * d ** -0.5                                # [T, nq, 256]
    count = np.full((T, 1, 64 * n_pages), float(repeats))
    for t in range(T):
        if T - 1 - t:
            count[t, 0, -(T - 1 - t):] -= 1                 # the last keys that row t does not see
    m = s.max(-1, keepdims=True)
    p = count * np.exp(s - m)
    total = p.sum(-1, keepdims=True)
    want, want_lse = p @ v / total, (m + np.log(total))[..., 0]
    reach = p @ np.abs(v) / total
    eps = (np.abs(qd) @ np.abs(k).T * d ** -0.5).max(-1)
    tol, tol_lse = _tolerance(want, reach, eps, keys, d, "bf16")
    _within(out[0], want, tol)
    _within(lse[0], want_lse, tol_lse + 2.0 ** -24 * np.abs(want_lse))


def test_workspaces_that_are_not_dense():
    pages, bt = _cache(40, 1, 128, 1, 40, 11)
    q = torch.zeros(1, 1, 2, 128, device=DEV, dtype=torch.bfloat16)
    need = binding.kv_attention_workspace(1, 1, 2, 1, 128, 40)
    assert need > 0
    for bad in (torch.empty(1, dtype=torch.uint8, device=DEV).expand(need), torch.empty(need, device=DEV)):
        with pytest.raises(ValueError):
            binding.kv_attention(q, pages.to(DEV), bt.to(DEV), _pos(100), workspace=bad)
    with pytest.raises(binding.DliteError):
        binding.kv_attention(q, pages.to(DEV), bt.to(DEV), _pos(100), workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
