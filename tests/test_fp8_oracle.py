"""Pins of the 8-bit products' oracle against facts fixed outside itself: torch's float8, closed forms."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as FO


def test_values_are_torchs():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(FO.VALUES, want, equal_nan=True)


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (224.5, 1.0), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7), (0.0, 2.0 ** -126),
                                        (448 * 2.0 ** -126, 2.0 ** -126), (449 * 2.0 ** -126, 2.0 ** -125), (3.4e38, 2.0 ** 120)])
def test_scales(amax, scale):
    assert FO.block_scale(amax) == scale


def test_scales_are_the_least_powers():
    a = np.exp2(np.random.default_rng(0).uniform(-100, 120, 20000))
    s = FO.block_scale(a)
    assert np.all(a <= 448 * s) and np.all(a > 224 * s) and np.all(np.log2(s) == np.floor(np.log2(s)))


def test_codes_are_torchs():
    x = torch.randn(40, 300, generator=torch.Generator().manual_seed(1)) * torch.logspace(-3, 3, 300)
    c, s = FO.quantise(x.double().numpy())
    y = x / torch.from_numpy(s.repeat(128, -1)[:, :300]).float()
    assert np.array_equal(c, y.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    # a value is off by at most a sixteenth of itself, or half of the least step, 2^-9 of the scale
    v = FO.values(c, s)
    assert np.all(np.abs(v - x.double().numpy()) <= np.maximum(np.abs(x.double().numpy()) / 16, s.repeat(128, -1)[:, :300] * 2.0 ** -10))


def test_blocks_of_a_weight():
    w = torch.randn(200, 260, generator=torch.Generator().manual_seed(2))
    w[130:, :128] *= 100
    c, s = FO.quantise_weight(w.double().numpy())
    assert s.shape == (2, 3)
    for i in range(2):
        for j in range(3):
            b = w[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            assert s[i, j] == FO.block_scale(float(b.abs().max()))
    assert np.abs(FO.weight_values(c, s) - w.double().numpy()).max() <= 448 * s.max() / 16


def test_what_is_not_finite():
    x = np.ones((1, 130))
    x[0, 3], x[0, 4], x[0, 129] = np.nan, np.inf, -np.inf
    c, s = FO.quantise(x)
    assert np.array_equal(s, [[2.0 ** -8, 2.0 ** -8]]) and c[0, 3] == c[0, 4] == c[0, 129] == 0x7F and FO.VALUES[c[0, 0]] * s[0, 0] == 1


def test_norm_and_silu():
    x = np.array([[3.0, -4.0]])
    assert np.allclose(FO.norm(x, np.array([2.0, 1.0]), 0.0), [[6 / 12.5 ** 0.5, -4 / 12.5 ** 0.5]])
    assert np.allclose(FO.silu(np.array([0.0, 50.0, -800.0])), [0, 50, 0])
    assert np.array_equal(FO.total(np.array([[1.0]]), np.array([[2.0 ** -9]]), "bf16"), [[1.0]])
