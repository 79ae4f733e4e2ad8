"""Refusals of the target-side calls: every pointer off its element type, the optional ones among them, comes back before any CUDA call
(no GPU needed)."""
import ctypes

import pytest

from test_target_refusals import CALLS, INVALID, P, _cache, lib  # noqa: F401

POINTERS = {      # pointer fields and the bytes of their elements (dtype 1: bf16, 0: float32)
    "dlite_rope": dict(x=2, out=2, pos=8, n_rows=4, table=8, status=4),
    "dlite_kv_append": dict(k=2, v=2, pos=8, n_rows=4, table=8, status=4),
    "dlite_kv_read": dict(k_out=2, v_out=2, pos=8, n_rows=4, status=4),
    "dlite_kv_attention": dict(q=2, out=2, lse=4, pos=8, n_rows=4, status=4, workspace=16),
    "dlite_token_logprobs": dict(logits=4, tokens=4, logprob=4, entropy=4, top_ids=4, top_logprobs=4, status=4),
}


def test_every_pointer_is_named():
    for name, fields in POINTERS.items():
        cls = CALLS[name][0]
        assert set(fields) == {n for n, t in cls._fields_ if t is ctypes.c_void_p}, name


@pytest.mark.parametrize("name,field,size", [(n, f, s) for n, d in POINTERS.items() for f, s in d.items()])
def test_misaligned_pointers(lib, name, field, size):  # noqa: F811
    cls, good = CALLS[name]
    kw = dict(good, **{field: P + size // 2})
    if "cache" in dict(cls._fields_):
        kw["cache"] = _cache(max_pages=100)      # a cache whose attention needs its workspace
    assert getattr(lib, name)(ctypes.byref(cls(**kw)), None) == INVALID
