"""GPU: the gated product's activation where exp(-g) is near float32's largest number: no gate above -88.72 makes a result 0."""
import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import fp8_oracle as FO
from test_gpu_fp8 import _bytes, _np, _quantised

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("rows", [3, 300])      # the few-row kernel and the many-row one
def test_gates_far_below_zero(rows):
    g = np.concatenate([np.linspace(-88.72, -87.3, 60), np.linspace(-87, -1, 30), [-89.0, -100.0, -1e30, 0.0, 1e-30, 1.0, 90.0, 3e4]]).astype(np.float32)
    u = np.where(np.arange(len(g)) % 2, 1e30, -3e33).astype(np.float32)
    F = 128 * len(g)
    one = torch.zeros(max(F, rows), 128, device=DEV)
    one[:, 0] = 1
    one = one.to(torch.float8_e4m3fn)
    c, s = one[:rows].view(1, rows, 128), binding.fp8_scale(1, rows, 128).fill_(1.0)
    w = one[:F]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    oc, os_ = binding.fp8_gated(c, s, w, torch.from_numpy(g[:, None]).to(DEV), w, torch.from_numpy(u[:, None]).to(DEV), status=st)
    assert int(st.item()) == 0
    gd, ud = g.astype(np.float64), u.astype(np.float64)
    with np.errstate(over="ignore"):
        want = np.where(gd < -88.723, 0.0, gd / (1 + np.exp(-gd)) * ud)
    # steps of 2^-24: exp2 4, its argument's factor and product 2 |g|, the sum 1, the reciprocal 2, three products 3; the quarter of the reciprocal
    # is 2^-128 or more, its half step of 2^-149 a share of 2^-22, four steps
    err = (4 + 2 * np.clip(-gd, 0, 128) + 1 + 2 + 3 + 4) * 2.0 ** -24 * np.abs(want)
    _quantised(_bytes(oc)[0], _np(os_)[0], np.tile(want.repeat(128), (rows, 1)), np.tile(err.repeat(128), (rows, 1)))
    assert np.all((_bytes(oc)[0, :, ::128] & 0x7F == 0) == (want == 0)[None])
