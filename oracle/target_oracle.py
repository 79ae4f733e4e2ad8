"""Plain CPU oracle of the target-side operators (numpy): rotary positions, the paged 4-bit
cache, attention over it, and token log probabilities.

TEST INFRASTRUCTURE ONLY, like dlite_oracle. Float64 throughout, except where the
operator's own definition fixes float32 steps (the rotation's products and the
quantisation, whose codes are compared bit for bit).
"""
import math

import numpy as np

from .dlite_oracle import bf16_round

PAGE = 64
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """Value of every scale byte 0x00..0x7e: exponent 4 bits (bias 7), mantissa 3 bits."""
    out = []
    for b in range(0x7F):
        e, m = b >> 3, b & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


E4M3 = e4m3_values()


def _nearest_even(x, grid):
    """Index of the grid value nearest to each x >= 0 (grid ascending); ties to the even index; saturating."""
    x = np.minimum(np.asarray(x, dtype=np.float64), grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


# ---------------------------------------------------------------- rotary positions

def rope_freqs(rot, theta=1e6, scaling="plain", factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        c = lambda b: rot * math.log(orig_len / (2 * math.pi * b)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(c(beta_fast)), 0), min(math.ceil(c(beta_slow)), rot - 1)
        r = np.clip((i - lo) / (hi - lo), 0, 1) if hi > lo else (i > lo).astype(np.float64)
        f = f * (1 - r) + f / factor * r
    return f


def rope_table(n_pos, rot, attn_factor=0.0, scaling="plain", factor=1.0, **kw):
    """float32 [n_pos, rot / 2, 2] of (m cos, m sin)(p f_i), rounded once from float64."""
    a = np.arange(n_pos, dtype=np.float64)[:, None] * rope_freqs(rot, scaling=scaling, factor=factor, **kw)
    m = attn_factor if attn_factor > 0 else (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)
    return np.stack([m * np.cos(a), m * np.sin(a)], axis=-1).astype(np.float32)


def rotate(x, table_row, layout):
    """One head's float32 columns x [d] rotated by table_row [rot / 2, 2]; the products rounded to float32."""
    x = np.array(x, dtype=np.float32)
    half = table_row.shape[0]
    c, s = table_row[:, 0], table_row[:, 1]
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    x0, x1 = x[..., a].copy(), x[..., b].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        x[..., a] = (x0 * c).astype(np.float32) - (x1 * s).astype(np.float32)
        x[..., b] = (x1 * c).astype(np.float32) + (x0 * s).astype(np.float32)
    return x


def rope(x, pos, table, layout, n_rows=None, out=None, dtype="f32"):
    """x [B, T, H, d] float32 values; rows past n_rows keep out's values. bf16: rounded once at the end."""
    out = np.zeros_like(x, dtype=np.float32) if out is None else np.array(out, dtype=np.float32)
    B, T = x.shape[:2]
    for b in range(B):
        for t in range(T if n_rows is None else min(max(int(n_rows[b]), 0), T)):
            p = min(max(int(pos[b]) + t, 0), len(table) - 1)
            y = rotate(x[b, t], table[p], layout)
            out[b, t] = bf16_round(y) if dtype == "bf16" else y
    return out


# ---------------------------------------------------------------- the 4-bit format

def quantise16(x, exp):
    """Codes (16 of 0..15) and scale byte of 16 float32 values, by the format's float32 steps."""
    with np.errstate(over="ignore", under="ignore"):
        y = np.asarray(x, dtype=np.float32) * np.float32(2.0 ** -exp)
    fin = np.isfinite(y)
    amax = np.float32(np.max(np.abs(y[fin]), initial=0.0))
    sb = int(_nearest_even(np.minimum(amax / np.float32(6.0), np.float32(448.0)), E4M3))
    s = np.float32(E4M3[sb])
    if s == 0:
        return np.zeros(16, dtype=np.uint8), 0, not fin.all()
    y = np.where(np.isnan(y), np.float32(0), y)
    with np.errstate(over="ignore"):
        q = (y / s).astype(np.float32)
    code = _nearest_even(np.abs(q), E2M1).astype(np.uint8)
    return code | (np.signbit(q).astype(np.uint8) << 3), sb, not fin.all()


def dequantise16(code, sb, exp):
    code = np.asarray(code)
    return np.where(code & 8, -1.0, 1.0) * E2M1[code & 7] * E4M3[sb] * 2.0 ** exp


def rec_parts(rec):
    """Views of one record (uint8 [72 d]): key codes [64, d/2], value codes [d, 32], scales [64, d/16], [d/16, 64]."""
    d = rec.shape[0] // 72
    k, v, ks, vs = rec[:32 * d], rec[32 * d:64 * d], rec[64 * d:68 * d], rec[68 * d:]
    return k.reshape(64, d // 2), v.reshape(d, 32), ks.reshape(64, d // 16), vs.reshape(d // 16, 64)


def write_row(rec, row, k, v, k_exp, v_exp):
    """Quantise one token's key and value (float32 [d]) into row `row` of a record; whether one was not finite."""
    kd, vd, ks, vs = rec_parts(rec)
    bad = False
    for j in range(len(k) // 16):
        c, s, nf = quantise16(k[16 * j:16 * j + 16], k_exp)
        kd[row, 8 * j:8 * j + 8] = c[0::2] | c[1::2] << 4
        ks[row, j] = s
        bad |= nf
        c, s, nf = quantise16(v[16 * j:16 * j + 16], v_exp)
        byte = vd[16 * j:16 * j + 16, row // 2]
        vd[16 * j:16 * j + 16, row // 2] = byte & 0x0F | c << 4 if row % 2 else byte & 0xF0 | c
        vs[j, row] = s
        bad |= nf
    return bad


def read_row(rec, row, k_exp, v_exp):
    """(key, value) float64 [d] of one row of a record."""
    kd, vd, ks, vs = rec_parts(rec)
    d = vd.shape[0]
    k, v = np.empty(d), np.empty(d)
    for j in range(d // 16):
        c = np.empty(16, dtype=np.uint8)
        c[0::2], c[1::2] = kd[row, 8 * j:8 * j + 8] & 15, kd[row, 8 * j:8 * j + 8] >> 4
        k[16 * j:16 * j + 16] = dequantise16(c, ks[row, j], k_exp)
        c = vd[16 * j:16 * j + 16, row // 2] >> (4 * (row % 2)) & 15
        v[16 * j:16 * j + 16] = dequantise16(c, vs[j, row], v_exp)
    return k, v


def append(pages, block_table, k, v, pos, table=None, layout="half", n_rows=None, k_exp=0, v_exp=0):
    """Rows into pages (uint8 [n_pages, n_kv, 72 d], in place). Returns the set of status names flagged."""
    flags = set()
    B, T, H = k.shape[:3]
    for b in range(B):
        for t in range(T if n_rows is None else min(max(int(n_rows[b]), 0), T)):
            p = int(pos[b]) + t
            if not 0 <= p < block_table.shape[1] * PAGE or not 0 <= block_table[b, p // PAGE] < len(pages):
                flags.add("bounds")
                continue
            for h in range(H):
                kr = np.asarray(k[b, t, h], dtype=np.float32)
                if table is not None:
                    if p >= len(table):
                        flags.add("bounds")
                    kr = rotate(kr, table[min(p, len(table) - 1)], layout)
                if write_row(pages[block_table[b, p // PAGE], h], p % PAGE, kr, np.asarray(v[b, t, h], dtype=np.float32),
                             k_exp, v_exp):
                    flags.add("nonfinite")
    return flags


# ---------------------------------------------------------------- attention

def read_record(rec, k_exp, v_exp):
    """(keys, values) float64 [64, d] of a record."""
    kd, vd, ks, vs = rec_parts(rec)
    d = vd.shape[0]
    kc, vc = np.empty((64, d), dtype=np.uint8), np.empty((64, d), dtype=np.uint8)
    kc[:, 0::2], kc[:, 1::2] = kd & 15, kd >> 4
    vc[0::2], vc[1::2] = vd.T & 15, vd.T >> 4
    sc = np.append(E4M3, np.nan)      # 0x7f, and every byte with the sign bit, is not a scale
    pick = lambda b: sc[np.minimum(b, 0x7F)]  # noqa: E731
    val = lambda c, s: np.where(c & 8, -1.0, 1.0) * E2M1[c & 7] * np.repeat(s, 16, axis=1)  # noqa: E731
    return val(kc, pick(ks)) * 2.0 ** k_exp, val(vc, pick(vs.T)) * 2.0 ** v_exp


def attention(q, pages, block_table, pos, scale, window=0, n_rows=None, k_exp=0, v_exp=0, out=None, lse=None):
    """q [B, T, n_q, d]. Returns (out, lse, reach, eps): reach = sum p |v| / sum p bounds how far weights off by a
    relative amount move an output; eps = the largest scale sum |q| |k| of a row, the size of a score's terms."""
    B, T, nq, d = q.shape
    nkv = pages.shape[1]
    out = np.zeros((B, T, nq, d)) if out is None else np.array(out, dtype=np.float64)
    lse = np.zeros((B, T, nq)) if lse is None else np.array(lse, dtype=np.float64)
    reach, eps = np.zeros((B, T, nq, d)), np.zeros((B, T, nq))
    for b in range(B):
        n = T if n_rows is None else min(max(int(n_rows[b]), 0), T)
        last = min(max(int(pos[b]) + n, 0), block_table.shape[1] * PAGE)
        ids = block_table[b, :(last + PAGE - 1) // PAGE]
        for h in range(nkv if n else 0):
            ks, vs, js = [np.zeros((0, d))], [np.zeros((0, d))], [np.zeros(0, dtype=np.int64)]
            for i, pid in enumerate(ids):
                if 0 <= pid < len(pages):
                    k, v = read_record(pages[pid, h], k_exp, v_exp)
                    ks.append(k), vs.append(v), js.append(i * PAGE + np.arange(PAGE))
            k, v, j = np.concatenate(ks), np.concatenate(vs), np.concatenate(js)
            for t in range(n):
                p = int(pos[b]) + t
                see = (j <= p) & (j < block_table.shape[1] * PAGE)
                if window:
                    see &= j > p - window
                for i in range(h * (nq // nkv), (h + 1) * (nq // nkv)):
                    qq = q[b, t, i].astype(np.float64)
                    if not see.any():
                        out[b, t, i], lse[b, t, i] = 0, -np.inf
                        continue
                    s = scale * (k[see] @ qq)
                    m = s.max()
                    w = np.exp(s - m)
                    lse[b, t, i] = m + np.log(w.sum())
                    out[b, t, i] = (w[:, None] * v[see]).sum(0) / w.sum()
                    reach[b, t, i] = (w[:, None] * np.abs(v[see])).sum(0) / w.sum()
                    eps[b, t, i] = scale * (np.abs(k[see]) @ np.abs(qq)).max()
    return out, lse, reach, eps


# ---------------------------------------------------------------- token log probabilities

def token_logprobs(x, token, temperature=1.0, n_top=0):
    """(ln p(token), entropy, top ids, their ln p) of one row of logits."""
    x = np.asarray(x, dtype=np.float64)
    order = np.lexsort((np.arange(len(x)), -np.where(np.isnan(x), -np.inf, x)))[:n_top]
    if np.isnan(x).any() or (x == np.inf).any():
        return np.nan, np.nan, order, np.full(n_top, np.nan)
    m = x.max()
    if m == -np.inf:
        return -np.inf if token < len(x) else np.nan, 0.0, order, np.full(n_top, -np.inf)
    d = (m - x) / temperature
    e = np.exp(-d)
    others = np.sort(np.delete(e, x.argmax()))     # S - 1, small terms first
    lp = -d - np.log1p(others.sum())
    p = np.exp(lp)
    h = -np.sum(np.where(p > 0, p * np.where(p > 0, lp, 0), 0))
    return lp[token] if token < len(x) else np.nan, h, order, lp[order]
