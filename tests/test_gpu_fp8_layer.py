"""GPU: the products with 8-bit weights as a target's layer uses them beside the paged cache. The rows [a, d_1..d_K] of a
ragged batch: norm and codes, the fused projection, rotary positions, append, attention, the output projection, sum and norm, the gated block and its
down projection, the logits. The layer is captured once and replayed with other rows, lengths and positions; every stage is checked
against the oracle on its own inputs."""
import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import fp8_oracle as FO
from oracle import target_oracle as TO
from test_gpu_fp8 import HALF, _bytes, _np, _off, _quantised
from test_gpu_kv_attention import _tolerance, _within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, T, D, NQ, NKV, DH, F, V, MP, EPS = 5, 4, 256, 4, 2, 64, 600, 1000, 3, 1e-6


def _product(got, codes, scale, w, m, name):
    x, wv = FO.values(_bytes(codes), _np(scale)), FO.weight_values(_bytes(w[0]), _np(w[1]))
    want = np.where(m[..., None], x, 0) @ wv.T
    tol = _off(-(-x.shape[-1] // 128)) * (np.abs(np.where(m[..., None], x, 0)) @ np.abs(wv).T) + HALF[name] * np.abs(want)
    assert np.all(np.abs(_np(got) - want)[m] <= tol[m] * 1.0000001)


def _normed(codes, scale, total, x, res, gain, m):
    v = FO.total(_np(x), _np(res), "bf16")
    assert np.array_equal(_np(total)[m], v[m])
    y = FO.norm(v, _np(gain), EPS)[m]
    _quantised(_bytes(codes)[m], _np(scale)[m], y, ((32 + 10 + 3) / 2 + 4 + 2) * 2.0 ** -24 * np.abs(y))


def test_a_layer_over_a_paged_cache():
    g = torch.Generator(device=DEV).manual_seed(3)
    weight = lambda n, k: binding.fp8_weight(torch.randn(n, k, generator=g, device=DEV) * k ** -0.5)  # noqa: E731
    wqkv, wo, wg, wu, wd, wl = (weight(*s) for s in (((NQ + 2 * NKV) * DH, D), (D, NQ * DH), (F, D), (F, D), (D, F), (V, D)))
    g1, g2, g3 = ((1 + 0.2 * torch.randn(D, generator=g, device=DEV)).bfloat16() for _ in range(3))
    table = binding.rope_table(64 * MP, DH, theta=1e4)
    pages = binding.kv_pages(B * MP, NKV, DH)
    bt = torch.randperm(B * MP, generator=torch.Generator().manual_seed(4)).view(B, MP).to(torch.int32).to(DEV)
    x, h = (torch.zeros(B, T, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pos, n = torch.zeros(B, dtype=torch.int64, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    past = [torch.randn(B, 130, NKV, DH, generator=g, device=DEV).bfloat16() for _ in range(2)]
    binding.kv_append(pages, bt, *past, torch.zeros_like(pos), table)
    s = torch.cuda.Stream(device=DEV)

    def layer():
        kw = dict(n_rows=n, status=st, stream=s)
        r1, r2, r3 = (torch.zeros_like(h) for _ in range(3))
        c1, s1 = binding.fp8_quantise(x, gain=g1, eps=EPS, residual=h, total=r1, **kw)
        qkv = binding.fp8_linear(c1, s1, *wqkv, **kw)
        q, k, v = qkv.view(B, T, NQ + 2 * NKV, DH).split((NQ, NKV, NKV), dim=2)
        rq = binding.rope(q, pos, table, **kw)
        binding.kv_append(pages, bt, k, v, pos, table, **kw)
        o, _ = binding.kv_attention(rq, pages, bt, pos, **kw)
        c2, s2 = binding.fp8_quantise(o.view(B, T, NQ * DH), **kw)
        y = binding.fp8_linear(c2, s2, *wo, **kw)
        c3, s3 = binding.fp8_quantise(y, gain=g2, eps=EPS, residual=r1, total=r2, **kw)
        c4, s4 = binding.fp8_gated(c3, s3, *wg, *wu, **kw)
        z = binding.fp8_linear(c4, s4, *wd, **kw)
        c5, s5 = binding.fp8_quantise(z, gain=g3, eps=EPS, residual=r2, total=r3, **kw)
        logits = binding.fp8_linear(c5, s5, *wl, dtype=torch.float32, **kw)
        return dict(r1=r1, r2=r2, r3=r3, c1=c1, s1=s1, qkv=qkv, rq=rq, o=o, c2=c2, s2=s2, y=y, c3=c3, s3=s3, c4=c4, s4=s4, z=z, c5=c5, s5=s5, logits=logits)

    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        layer()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            r = layer()
    for turn in range(3):
        x.copy_(torch.randn(B, T, D, generator=g, device=DEV))
        h.copy_(torch.randn(B, T, D, generator=g, device=DEV))
        lens = [T, turn, 0, T, (2 * turn) % (T + 1)]
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        pos.copy_(torch.tensor([0, 60 + turn, 63, 126, 30 * turn]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        m = np.arange(T)[None] < np.array(lens)[:, None]
        _normed(r["c1"], r["s1"], r["r1"], x, h, g1, m)
        _product(r["qkv"], r["c1"], r["s1"], wqkv, m, "bf16")
        want, _, reach, eps = TO.attention(r["rq"].float().cpu().numpy(), pages.cpu().numpy(), bt.cpu().numpy(), pos.tolist(), DH ** -0.5, n_rows=lens)
        tol, _ = _tolerance(want, reach, eps, 64 * MP, DH, "bf16", v_exp=2)
        _within(r["o"][torch.from_numpy(m)], want[m], tol[m])
        o = _np(r["o"]).reshape(B, T, NQ * DH)
        wc, ws = FO.quantise(o)
        assert np.array_equal(_bytes(r["c2"])[m], wc[m]) and np.array_equal(_np(r["s2"])[m], ws[m])
        _product(r["y"], r["c2"], r["s2"], wo, m, "bf16")
        _normed(r["c3"], r["s3"], r["r2"], r["y"], r["r1"], g2, m)
        xv = FO.values(_bytes(r["c3"]), _np(r["s3"]))[m]
        gv, uv, off = FO.weight_values(_bytes(wg[0]), _np(wg[1])), FO.weight_values(_bytes(wu[0]), _np(wu[1])), _off(2)
        gw, uw = xv @ gv.T, xv @ uv.T
        ge, ue = off * (np.abs(xv) @ np.abs(gv).T), off * (np.abs(xv) @ np.abs(uv).T)
        a = FO.silu(gw) * uw
        err = 1.1 * ge * (np.abs(uw) + ue) + np.abs(FO.silu(gw)) * ue + (9 + 2 * np.abs(gw)) * 2.0 ** -24 * np.abs(a) + 2.0 ** -110 * np.abs(uw)
        _quantised(_bytes(r["c4"])[m], _np(r["s4"])[m], a, err)
        _product(r["z"], r["c4"], r["s4"], wd, m, "bf16")
        _normed(r["c5"], r["s5"], r["r3"], r["z"], r["r2"], g3, m)
        _product(r["logits"], r["c5"], r["s5"], wl, m, "f32")
        for k in ("qkv", "y", "z", "logits", "r1", "r2", "r3"):
            assert not _np(r[k])[~m].any()
