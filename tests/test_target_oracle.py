"""Pins of the target-side oracle against facts fixed outside itself: closed forms,
torch's float8 and attention on the CPU, exhaustive small formats."""
import math

import numpy as np
import pytest
import torch

from oracle import target_oracle as TO


def test_e4m3_values_are_torchs():
    want = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(TO.E4M3, want)


def test_e4m3_rounding_is_torchs():
    x = torch.cat([torch.rand(4000, generator=torch.Generator().manual_seed(1)) * s for s in (448.0, 1.0, 0.02, 0.002)])
    x = torch.cat([x, (torch.from_numpy(TO.E4M3[1:]).float() + torch.from_numpy(TO.E4M3[:-1]).float()) / 2])   # and the ties
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(TO._nearest_even(x.double().numpy(), TO.E4M3), want)


@pytest.mark.parametrize("x,code", [(0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
                                    (5.0001, 7), (6.0, 7), (6.9, 7), (0.0, 0), (0.7499, 1), (3.4, 5)])
def test_e2m1_rounding(x, code):
    assert int(TO._nearest_even(x, TO.E2M1)) == code


def test_quantise_closed_forms():
    y = np.array([6, -6, 4, 3, 2, 1.5, 1, 0.5, -0.5, -1, -1.5, -2, -3, -4, 0, 5.0], dtype=np.float32)   # 5.0: a tie, to 4
    c, s, bad = TO.quantise16(y * 8, 2)     # y 8 = 2^2 (2 y): scale 2
    assert s == 0x40 and TO.E4M3[s] == 2.0 and not bad
    assert np.array_equal(TO.dequantise16(c, s, 2), np.where(y == 5, 4, y) * 8)
    c, s, bad = TO.quantise16(np.full(16, 1e-6, np.float32), 0)   # a scale that rounds to zero
    assert s == 0 and not c.any() and not bad
    z = np.zeros(16, np.float32)
    z[3], z[4], z[5], z[6] = np.nan, np.inf, -np.inf, 12.0
    c, s, bad = TO.quantise16(z, 0)
    v = TO.dequantise16(c, s, 0)
    assert bad and v[3] == 0 and v[4] == 12 and v[5] == -12 and v[6] == 12
    c, s, bad = TO.quantise16(np.full(16, 1e9, np.float32), 0)    # saturates at 448 * 6
    assert (TO.dequantise16(c, s, 0) == 2688).all()


def test_quantise_error_bound():
    """A value is off by at most half a code step (1 of 6) of the block's scale, itself rounded by 2^-4."""
    rng = np.random.default_rng(0)
    for _ in range(200):
        x = (rng.normal(0, 1, 16) * 2.0 ** rng.integers(-4, 5)).astype(np.float32)
        c, s, _ = TO.quantise16(x, 0)
        amax = np.abs(x).max()
        # codes below 4 sit at most 1/2 apart from x / s, above at most 1; a scale rounded down by 2^-4 clips 6 (1 + 2^-4)
        assert np.abs(TO.dequantise16(c, s, 0) - x).max() <= (1.0 / 6) * (1 + 2.0 ** -4) * amax + 1e-7


def test_record_layout_and_round_trip():
    rng = np.random.default_rng(3)
    for d in (64, 128):
        rec = rng.integers(0, 256, 72 * d, dtype=np.uint8)
        rec[64 * d:] %= 0x7F
        before = rec.copy()
        k, v = rng.normal(size=(2, d)).astype(np.float32)
        TO.write_row(rec, 21, k, v, 0, -2)
        # the bytes a row may change: its key codes and scales, the high nibbles of byte 10 of every value column, its value scales
        touched = np.zeros(72 * d, dtype=bool)
        touched[21 * d // 2:22 * d // 2] = True
        touched[32 * d + 10:64 * d:32] = True
        touched[64 * d + 21 * d // 16:64 * d + 22 * d // 16] = True
        touched[68 * d + 21::64] = True
        assert np.array_equal(rec[~touched], before[~touched])
        assert np.array_equal(rec[32 * d + 10:64 * d:32] & 15, before[32 * d + 10:64 * d:32] & 15)
        kk, vv = TO.read_row(rec, 21, 0, -2)
        for j in range(d // 16):
            c, s, _ = TO.quantise16(k[16 * j:16 * j + 16], 0)
            assert np.array_equal(kk[16 * j:16 * j + 16], TO.dequantise16(c, s, 0))
            c, s, _ = TO.quantise16(v[16 * j:16 * j + 16], -2)
            assert np.array_equal(vv[16 * j:16 * j + 16], TO.dequantise16(c, s, -2))
        TO.write_row(rec, 20, v, k, 0, 0)       # the byte's other token
        assert np.array_equal(TO.read_row(rec, 21, 0, -2)[1], vv)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_a_complex_product(layout):
    rng = np.random.default_rng(5)
    d, rot, p = 64, 48, 777
    x = rng.normal(size=d).astype(np.float32)
    tab = TO.rope_table(p + 1, rot, theta=1e4)
    y = TO.rotate(x, tab[p], layout)
    n = rot // 2
    a = np.exp(1j * p * 1e4 ** (-2 * np.arange(n) / rot))
    i = np.arange(n)
    u, w = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    z = (x[u].astype(np.float64) + 1j * x[w]) * a
    # table entries and two products and a sum, each rounded by 2^-24
    assert np.abs(y[u] - z.real).max() < 8 * 2.0 ** -24 * np.abs(z).max() * 2
    assert np.abs(y[w] - z.imag).max() < 8 * 2.0 ** -24 * np.abs(z).max() * 2
    assert np.array_equal(y[rot:], x[rot:])
    assert np.array_equal(TO.rotate(x, tab[0], layout), x)


def test_frequency_scalings():
    plain = TO.rope_freqs(128)
    assert plain[0] == 1.0 and math.isclose(plain[-1], 1e6 ** (-126 / 128))
    assert np.allclose(TO.rope_freqs(128, scaling="linear", factor=4.0), plain / 4)
    ntk = TO.rope_freqs(128, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 4)        # the slowest pair is stretched by the whole factor
    y = TO.rope_freqs(128, scaling="yarn", factor=4.0, orig_len=32768.0)
    assert y[0] == plain[0] and math.isclose(y[-1], plain[-1] / 4)        # fast pairs as they are, slow ones stretched
    assert np.all(np.diff(y / plain) <= 1e-15)
    turns = 32768.0 * plain / (2 * math.pi)
    assert np.allclose(y[turns > 40], plain[turns > 40]) and np.allclose(y[turns < 0.8], plain[turns < 0.8] / 4)
    assert np.allclose(TO.rope_freqs(128, scaling="yarn", factor=1.0, orig_len=32768.0), plain)
    assert math.isclose(TO.rope_table(1, 8, scaling="yarn", factor=4.0, orig_len=64.0)[0, 0, 0], 0.1 * math.log(4.0) + 1, rel_tol=1e-6)


def test_append_places_rows_by_the_table():
    rng = np.random.default_rng(7)
    pages = np.zeros((6, 2, 72 * 64), dtype=np.uint8)
    bt = np.array([[4, 1], [0, -1]])
    k, v = rng.normal(size=(2, 2, 3, 2, 64)).astype(np.float32)
    flags = TO.append(pages, bt, k, v, [62, 63], n_rows=[3, 2])
    assert flags == {"bounds"}           # request 1's second row falls into a hole
    for b, t, page, row in ((0, 0, 4, 62), (0, 1, 4, 63), (0, 2, 1, 0), (1, 0, 0, 63)):
        kk, vv = TO.read_row(pages[page, 1], row, 0, 0)
        assert np.abs(kk - k[b, t, 1]).max() < 0.18 * np.abs(k[b, t, 1]).max() and np.abs(vv - v[b, t, 1]).max() < 0.18 * np.abs(v[b, t, 1]).max()
    assert not pages[2].any() and not pages[3].any() and not pages[5].any()


def test_attention_is_torchs_on_the_decoded_cache():
    rng = np.random.default_rng(11)
    B, T, nq, nkv, d = 2, 3, 4, 2, 64
    pages = rng.integers(0, 256, (7, nkv, 72 * d), dtype=np.uint8)
    pages[..., 64 * d:] = 0x28 + pages[..., 64 * d:] % 24
    bt = np.array([[3, 0, 5], [1, 6, 2]])
    pos, q = [100, 130], rng.normal(size=(B, T, nq, d)) * 0.2
    out, lse, reach, eps = TO.attention(q, pages, bt, pos, 0.125, k_exp=1, v_exp=-1)
    win = TO.attention(q, pages, bt, pos, 0.125, window=40, k_exp=1, v_exp=-1)[0]
    for b in range(B):
        for h in range(nkv):
            kk, vv = (np.concatenate([TO.read_record(pages[i, h], 1, -1)[w] for i in bt[b]]) for w in (0, 1))
            r, rv = TO.read_row(pages[bt[b, 1], h], 9, 1, -1)
            assert np.array_equal(kk[73], r) and np.array_equal(vv[73], rv)
            key, row = torch.arange(192), pos[b] + torch.arange(T)[:, None]
            for mask, got in ((key <= row, out), ((key <= row) & (key > row - 40), win)):
                want = torch.nn.functional.scaled_dot_product_attention(
                    torch.from_numpy(q[b, :, 2 * h:2 * h + 2]).transpose(0, 1), torch.from_numpy(kk).expand(2, -1, -1),
                    torch.from_numpy(vv).expand(2, -1, -1), attn_mask=mask, scale=0.125)
                assert np.abs(got[b, :, 2 * h:2 * h + 2] - want.transpose(0, 1).numpy()).max() < 1e-10
            s = 0.125 * torch.from_numpy(q[b, 1, 2 * h] @ kk.T)
            assert math.isclose(float(torch.logsumexp(s[:pos[b] + 2], 0)), lse[b, 1, 2 * h], rel_tol=1e-12)
    assert (reach >= np.abs(out) - 1e-12).all() and (eps > 0).all()


def test_attention_holes_and_empty_rows():
    rng = np.random.default_rng(12)
    pages = rng.integers(0, 0x70, (3, 1, 72 * 64), dtype=np.uint8)
    q = rng.normal(size=(3, 2, 1, 64)) * 0.05
    bt = np.array([[0, 1], [-1, 1], [-1, 7]])
    out, lse, _, _ = TO.attention(q, pages, bt, [80, 63, 100], 0.1, n_rows=[1, 2, 2], out=np.full(q.shape, 5.0), lse=np.full((3, 2, 1), 5.0))
    assert (out[0, 1] == 5).all() and lse[0, 1] == 5                 # a row behind the last valid one
    assert not out[1, 0].any() and lse[1, 0] == -np.inf               # keys 0..63 lie in a hole
    assert np.allclose(out[1, 1], TO.read_row(pages[1, 0], 0, 0, 0)[1])   # one key left
    assert not out[2].any() and (lse[2] == -np.inf).all()


def test_logprobs_are_torchs():
    rng = np.random.default_rng(15)
    x = rng.normal(size=500) * 3
    x[7], x[100:110] = x[3], -np.inf
    for T in (1.0, 0.7):
        lp = torch.log_softmax(torch.from_numpy(x) / T, 0)
        got, h, ids, top = TO.token_logprobs(x, 42, T, 6)
        assert math.isclose(got, float(lp[42]), rel_tol=1e-13)
        assert math.isclose(h, float(torch.distributions.Categorical(logits=torch.from_numpy(x[np.isfinite(x)]) / T).entropy()), rel_tol=1e-12)
        want = torch.from_numpy(x).sort(descending=True, stable=True).indices[:6]
        assert np.array_equal(ids, want.numpy()) and np.allclose(top, lp[want].numpy())
    assert TO.token_logprobs(x, 100)[0] == -np.inf and np.isnan(TO.token_logprobs(x, 500)[0])
    # a near-certain row: H = sum q (1 + ln 1/q ...) for one other token of probability q
    q = 1e-9
    h = TO.token_logprobs(np.array([0.0, math.log(q)]), 0)[1]
    assert math.isclose(h, q * (1 - math.log(q)), rel_tol=1e-6)
    lp, h, ids, top = TO.token_logprobs(np.full(4, -np.inf), 1, 1.0, 2)
    assert lp == -np.inf and h == 0 and list(ids) == [0, 1] and (top == -np.inf).all()
