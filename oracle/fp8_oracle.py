"""Plain CPU oracle of the products with 8-bit weights (numpy, float64).

TEST INFRASTRUCTURE ONLY, like target_oracle. Codes are bytes: sign, four exponent bits (bias 7), three of mantissa;
0x7f and 0xff are NaN. A block is 128 columns of a row (activations) or 128 x 128 elements (weights).
"""
import numpy as np

from .dlite_oracle import bf16_round
from .target_oracle import E4M3, _nearest_even

BLOCK = 128
VALUES = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])    # by byte


def block_scale(amax):
    """The least 2^e, e >= -126, with amax <= 448 2^e."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.ceil(np.log2(np.maximum(amax, 2.0 ** -140) / 448))
    e = np.where(amax > 448 * 2.0 ** e, e + 1, np.where(amax <= 448 * 2.0 ** (e - 1), e - 1, e))    # log2 rounds
    return 2.0 ** np.maximum(e, -126)


def blocked(x):
    """x [..., K] with its columns in blocks [..., ceil(K / 128), 128], zeros behind the last."""
    pad = -x.shape[-1] % BLOCK
    x = np.concatenate([x, np.zeros(x.shape[:-1] + (pad,))], axis=-1)
    return x.reshape(x.shape[:-1] + (-1, BLOCK))


def codes(y, scale):
    """Nearest code of y / scale (a power of two), ties to even; NaN where y is not finite."""
    fin = np.isfinite(y)
    q = np.where(fin, y, 0) / scale
    c = _nearest_even(np.abs(q), E4M3).astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 7)
    return np.where(fin, c, 0x7F).astype(np.uint8)


def quantise(x):
    """Codes [..., K] and scales [..., ceil(K / 128)] of x."""
    K = x.shape[-1]
    y = blocked(np.asarray(x, dtype=np.float64))
    s = block_scale(np.max(np.where(np.isfinite(y), np.abs(y), 0), axis=-1))
    return codes(y, s[..., None]).reshape(x.shape[:-1] + (-1,))[..., :K], s


def quantise_weight(w):
    N, K = w.shape
    w = np.asarray(w, dtype=np.float64)
    s = np.array([[block_scale(np.max(np.abs(b)[np.isfinite(b)], initial=0.0)) for b in np.split(r, range(BLOCK, K, BLOCK), axis=1)]
                  for r in np.split(w, range(BLOCK, N, BLOCK), axis=0)])
    return codes(w, widened(s, N, K)), s


def widened(s, N, K):
    """A weight's scales, one per element."""
    return s.repeat(BLOCK, 0)[:N].repeat(BLOCK, 1)[:, :K]


def values(c, s):
    """What codes [..., K] with scales [..., ceil(K / 128)] stand for."""
    return VALUES[c] * np.asarray(s, dtype=np.float64).repeat(BLOCK, -1)[..., :c.shape[-1]]


def weight_values(c, s):
    return VALUES[c] * widened(np.asarray(s, dtype=np.float64), *c.shape)


def total(x, residual, dtype):
    """x + residual, rounded once to the stream's type."""
    y = (x.astype(np.float32) + residual.astype(np.float32)).astype(np.float32)
    return (bf16_round(y) if dtype == "bf16" else y).astype(np.float64)


def norm(x, gain, eps):
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * gain


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))
