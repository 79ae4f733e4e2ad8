"""Refusals of the target-side calls: argument errors come back before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from history_free_speculative_gb300 import binding, build

INVALID, SHAPE = -1, -2
P = 4096      # an aligned address nothing reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _cache(**kw):
    d = dict(pages=P, block_table=P, n_pages=4, n_kv=2, d_h=128, max_pages=3, k_exp=0, v_exp=0)
    d.update(kw)
    return binding.KvCacheDesc(**d)


CALLS = {
    "dlite_rope": (binding.RopeArgs, dict(B=2, T=3, heads=4, d_h=128, rot=128, layout=0, dtype=1, n_pos=10, x=P, x_stride=512, out=P,
                                          out_stride=512, pos=P, table=P)),
    "dlite_kv_append": (binding.KvAppendArgs, dict(B=2, T=3, dtype=1, rot=128, layout=0, n_pos=10, k=P, k_stride=256, v=P,
                                                   v_stride=256, pos=P, table=P)),
    "dlite_kv_read": (binding.KvReadArgs, dict(B=2, T=3, dtype=1, k_out=P, k_stride=256, v_out=P, v_stride=256, pos=P)),
    "dlite_kv_attention": (binding.KvAttentionArgs, dict(B=2, T=3, n_q=8, dtype=1, window=0, scale=0.1, q=P, q_stride=1024, out=P,
                                                         out_stride=1024, pos=P, workspace=P, workspace_bytes=1 << 40)),
    "dlite_token_logprobs": (binding.LogprobsArgs, dict(rows=2, V=1000, n_top=5, dtype=0, temperature=1.0, logits=P, stride=1000,
                                                        tokens=P, top_ids=P, top_logprobs=P)),
}
NAN, INF = float("nan"), float("inf")
CACHE = [({"cache": _cache(pages=None)}, INVALID), ({"cache": _cache(pages=P + 8)}, INVALID), ({"cache": _cache(block_table=None)}, INVALID),
         ({"cache": _cache(block_table=P + 2)}, INVALID), ({"cache": _cache(n_pages=0)}, INVALID), ({"cache": _cache(n_kv=0)}, INVALID),
         ({"cache": _cache(max_pages=0)}, INVALID), ({"cache": _cache(k_exp=65)}, INVALID), ({"cache": _cache(v_exp=-65)}, INVALID),
         ({"cache": _cache(d_h=96)}, SHAPE), ({"cache": _cache(max_pages=1 << 25)}, SHAPE), ({"pos": None}, INVALID),
         ({"pos": P + 4}, INVALID), ({"B": 0}, INVALID), ({"T": 0}, INVALID), ({"B": 70000}, SHAPE), ({"dtype": 2}, INVALID)]
BAD = {
    "dlite_rope": [({"x": None}, INVALID), ({"out": None}, INVALID), ({"pos": None}, INVALID), ({"table": None}, INVALID), ({"B": 0}, INVALID),
                   ({"T": -1}, INVALID), ({"heads": 0}, INVALID), ({"n_pos": 0}, INVALID), ({"dtype": 3}, INVALID), ({"layout": 2}, INVALID),
                   ({"rot": 3}, SHAPE), ({"rot": 130}, SHAPE), ({"rot": 0}, SHAPE), ({"d_h": 1}, SHAPE), ({"x_stride": 511}, INVALID),
                   ({"out_stride": 100}, INVALID), ({"out_stride": 1024}, INVALID), ({"x": P + 1}, INVALID), ({"table": P + 4}, INVALID),
                   ({"B": 1 << 30}, SHAPE)],
    "dlite_kv_append": CACHE + [({"k": None}, INVALID), ({"v": None}, INVALID), ({"k_stride": 255}, INVALID), ({"v_stride": 0}, INVALID),
                                ({"v": P + 1}, INVALID), ({"layout": -1}, INVALID), ({"n_pos": 0}, INVALID), ({"rot": 130}, SHAPE),
                                ({"rot": 63}, SHAPE)],
    "dlite_kv_read": CACHE + [({"k_out": None}, INVALID), ({"v_out": None}, INVALID), ({"k_stride": 255}, INVALID), ({"v_stride": -1}, INVALID),
                              ({"k_out": P + 1}, INVALID)],
    "dlite_kv_attention": CACHE + [({"q": None}, INVALID), ({"out": None}, INVALID), ({"n_q": 7}, INVALID), ({"n_q": 0}, INVALID),
                                   ({"window": -1}, INVALID), ({"scale": 0.0}, INVALID), ({"scale": -1.0}, INVALID), ({"scale": NAN}, INVALID),
                                   ({"scale": INF}, INVALID), ({"q_stride": 1000}, INVALID), ({"out_stride": 8}, INVALID), ({"lse": P + 2}, INVALID),
                                   ({"q": P + 1}, INVALID), ({"T": 1 << 19}, SHAPE)],
    "dlite_token_logprobs": [({"logits": None}, INVALID), ({"tokens": None}, INVALID), ({"rows": 0}, INVALID), ({"V": 0}, INVALID),
                             ({"stride": 999}, INVALID), ({"n_top": -1}, INVALID), ({"n_top": 33}, SHAPE), ({"V": 3, "n_top": 4}, INVALID),
                             ({"dtype": 2}, INVALID), ({"temperature": 0.0}, INVALID), ({"temperature": -1.0}, INVALID),
                             ({"temperature": NAN}, INVALID), ({"temperature": INF}, INVALID), ({"top_ids": None}, INVALID),
                             ({"top_logprobs": None}, INVALID), ({"logits": P + 2}, INVALID)],
}


@pytest.mark.parametrize("name,change,code", [(n, c, k) for n, l in BAD.items() for c, k in l], ids=str)
def test_bad_arguments(lib, name, change, code):
    cls, good = CALLS[name]
    kw = dict(good, **change)
    if "cache" in dict(cls._fields_):
        kw.setdefault("cache", _cache())
    a = cls(**kw)
    assert getattr(lib, name)(ctypes.byref(a), None) == code
    if name == "dlite_kv_attention":
        assert lib.dlite_kv_attention_workspace(ctypes.byref(a)) == 0


def test_null_arguments(lib):
    for name in CALLS:
        assert getattr(lib, name)(None, None) == INVALID
    assert lib.dlite_kv_attention_workspace(None) == 0


@pytest.mark.parametrize("change,code", [({"rot": 3}, SHAPE), ({"rot": 258}, SHAPE), ({"rot": 0}, SHAPE), ({"theta": 1.0}, INVALID),
                                         ({"theta": NAN}, INVALID), ({"theta": INF}, INVALID), ({"scaling": 4}, INVALID),
                                         ({"scaling": 1, "factor": 0.5}, INVALID), ({"scaling": 2, "factor": 2.0, "rot": 2}, SHAPE),
                                         ({"scaling": 3, "factor": 2.0, "orig_len": 0.0}, INVALID),
                                         ({"scaling": 3, "factor": 2.0, "beta_slow": 40.0}, INVALID), ({"attn_factor": -1.0}, INVALID)], ids=str)
def test_bad_rope_tables(lib, change, code):
    c = binding.RopeConfig(**dict(dict(rot=128, scaling=0, theta=1e6, factor=1.0, orig_len=32768.0, beta_fast=32.0, beta_slow=1.0), **change))
    assert lib.dlite_rope_table(ctypes.byref(c), 10, P, None) == code
    good = binding.RopeConfig(rot=128, theta=1e6)
    assert lib.dlite_rope_table(ctypes.byref(good), 0, P, None) == INVALID
    assert lib.dlite_rope_table(ctypes.byref(good), 10, None, None) == INVALID
    assert lib.dlite_rope_table(None, 10, P, None) == INVALID


def test_the_binding_wants_device_tensors():
    x, pos = torch.zeros(1, 1, 2, 64), torch.zeros(1, dtype=torch.int64)
    pages, bt = torch.zeros(1, 2, 72 * 64, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: binding.rope(x, pos, torch.zeros(4, 32, 2)), lambda: binding.kv_append(pages, bt, x, x, pos),
                 lambda: binding.kv_read(pages, bt, pos, 1), lambda: binding.kv_attention(x, pages, bt, pos),
                 lambda: binding.token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


def test_the_bindings_row_strides():
    x = torch.zeros(3, 4, 6, 64)
    assert binding._row_stride(x, "x") == 384 and binding._row_stride(x[:, :, 2:4], "x") == 384
    assert binding._row_stride(x[:1, :, :2], "x") == 384 and binding._row_stride(x[:, :1, :2], "x") == 4 * 384
    assert binding._row_stride(x[:, ::2], "x") == 768 and binding._row_stride(x[:1, :1, 1:3], "x") == 128
    for bad in (x[:, :3], x[:, :, ::2], x[..., ::2], x.transpose(1, 2), x[:, :1].expand(3, 4, 6, 64), x[0]):
        with pytest.raises(ValueError):
            binding._row_stride(bad, "x")
