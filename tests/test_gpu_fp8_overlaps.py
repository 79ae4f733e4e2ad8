"""GPU: inputs and outputs of the calls with 8-bit weights side by side in the rows of one memory: taken, with the results of separate ones; over one
another: refused."""
import pytest
import torch

from history_free_speculative_gb300 import binding
from test_gpu_fp8 import _bytes, _input, _np, _weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("rows", [1, 6, 300])
def test_operands_in_the_same_rows(rows):
    K = 256
    x = _input(1, rows, K, "bf16", 1)
    w, ws = _weight(K, K, 2)
    c0, s0 = binding.fp8_quantise(x)
    y0 = binding.fp8_linear(c0, s0, w, ws)
    g0, gs0 = binding.fp8_gated(c0, s0, w, ws, w, ws)
    # [codes | codes of the activation | result, 16 bits]
    wide = torch.zeros(1, rows, 4 * K, dtype=torch.uint8, device=DEV)
    c, g, y = wide[..., :K].view(torch.float8_e4m3fn), wide[..., K:2 * K].view(torch.float8_e4m3fn), wide[..., 2 * K:].view(torch.bfloat16)
    _, s = binding.fp8_quantise(x, codes=c)
    binding.fp8_gated(c, s, w, ws, w, ws, out=g)
    binding.fp8_linear(c, s, w, ws, out=y)
    for a, b in ((c, c0), (g, g0)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert torch.equal(y, y0) and torch.equal(s, s0)
    # x, residual and sum likewise, and the sum in place of either
    both = torch.cat([x, 3 * x, torch.zeros_like(x)], -1)
    a, r, t = both[..., :K], both[..., K:2 * K], both[..., 2 * K:]
    binding.fp8_quantise(a, residual=r, total=t)
    want = t.clone()
    for to in (a, r):
        keep = to.clone()
        binding.fp8_quantise(a, residual=r, total=to)
        assert torch.equal(to, want)
        to.copy_(keep)
    binding.fp8_quantise(x, residual=x, total=x)
    assert torch.equal(x, (2 * a.float()).bfloat16())


@pytest.mark.parametrize("rows", [1, 6, 300])
def test_operands_over_one_another(rows):
    K = 256
    w, ws = _weight(K, K, 2)
    c, s = binding.fp8_quantise(_input(1, rows, K, "bf16", 1))
    before, scale = _bytes(c).copy(), _np(s)
    wide = torch.zeros(1, rows, 2 * K, dtype=torch.bfloat16, device=DEV)
    for call in (lambda: binding.fp8_gated(c, s, w, ws, w, ws, out=c), lambda: binding.fp8_gated(c, s, w, ws, w, ws, out_scale=s),
                 lambda: binding.fp8_quantise(wide[..., :K], residual=wide[..., 16:K + 16], total=wide[..., 32:K + 32])):
        with pytest.raises(binding.DliteError):
            call()
    torch.cuda.synchronize()
    assert (before == _bytes(c)).all() and (scale == _np(s)).all() and not bool(wide.any())
