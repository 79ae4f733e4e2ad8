"""Outputs of the calls with 8-bit weights that lie over an input or another output are refused, before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from history_free_speculative_gb300 import binding, build

INVALID = -1
A = 1 << 30      # addresses that nothing reads, a gigabyte apart


def _args(cls, **kw):
    """Every pointer at an address of its own."""
    names = [n for n, t in cls._fields_ if t is ctypes.c_void_p and n not in ("n_rows", "status")]
    return dict({n: A * (i + 1) for i, n in enumerate(names)}, **kw)


X = dict(B=2, T=3, K=200, codes_stride=208)
QUANTISE = _args(binding.Fp8QuantiseArgs, B=2, T=3, K=200, dtype=1, x_stride=200, residual_stride=200, total_stride=200, eps=1e-6, codes_stride=208)
WEIGHT = _args(binding.Fp8WeightArgs, N=300, K=200, dtype=0, w_stride=200, codes_stride=208)
LINEAR = _args(binding.Fp8LinearArgs, **X, N=300, dtype=1, w_stride=208, out_stride=304)
GATED = _args(binding.Fp8GatedArgs, **X, F=200, gate_stride=208, up_stride=208, out_stride=208)
CASES = [("dlite_fp8_quantise", binding.Fp8QuantiseArgs, QUANTISE, out, to, d)
         # the first byte, the last byte of what is there, the last byte of the output on its first
         for out, last in (("codes", 5 * 208 + 200), ("scale", 6 * 2 * 4))
         for to, size in (("x", 2 * 1200), ("residual", 2 * 1200), ("total", 2 * 1200), ("gain", 400), ("scale", 48), ("codes", 1240)) if to != out
         for d in (0, (size - 1) // 16 * 16, -((last - 1) // 16 * 16))]
CASES += [("dlite_fp8_quantise", binding.Fp8QuantiseArgs, QUANTISE, "total", to, d) for to, size in (("x", 2400), ("residual", 2400), ("gain", 400))
          for d in (size - 2, -2 * 1199, 2 * 200, 16) if d < size]
CASES += [("dlite_fp8_quantise", binding.Fp8QuantiseArgs, QUANTISE, "total", "gain", 0)]
CASES += [("dlite_fp8_weight", binding.Fp8WeightArgs, WEIGHT, out, to, d) for out, to in (("codes", "w"), ("scale", "w"), ("codes", "scale")) for d in (0, 16, -16)]
CASES += [("dlite_fp8_linear", binding.Fp8LinearArgs, LINEAR, "out", to, d) for to in ("codes", "scale", "w", "w_scale") for d in (0, 16, -16, -2 * 6 * 300)]
CASES += [("dlite_fp8_gated", binding.Fp8GatedArgs, GATED, out, to, d) for out in ("out_codes", "out_scale")
          for to in ("codes", "scale", "gate", "gate_scale", "up", "up_scale", "out_scale", "out_codes") if to != out for d in (0, 16, -16)
          if not (d == 16 and to in ("gate_scale", "up_scale"))]      # 2 x 2 blocks: 16 bytes
# rows of one stride: the columns of one reach into the other's
CASES += [("dlite_fp8_gated", binding.Fp8GatedArgs, dict(GATED, codes_stride=416, out_stride=416), "out_codes", "codes", d) for d in (192, -192, 416 + 192, 240)]
# of other strides: the whole ranges
CASES += [("dlite_fp8_gated", binding.Fp8GatedArgs, dict(GATED, codes_stride=416, out_stride=432), "out_codes", "codes", 208)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("name,cls,good,out,to,d", CASES, ids=[f"{c[0][10:]}-{c[3]}-{c[4]}{c[5]:+d}-{i}" for i, c in enumerate(CASES)])
def test_outputs_over_other_operands(lib, name, cls, good, out, to, d):
    assert good[to] + d > 0
    a = cls(**dict(good, **{out: good[to] + d}))
    assert getattr(lib, name)(ctypes.byref(a), None) == INVALID
