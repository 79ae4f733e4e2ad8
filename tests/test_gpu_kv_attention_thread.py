"""GPU: attention over the paged cache as the first CUDA call of a host thread."""
import ctypes
import threading

import pytest
import torch

from history_free_speculative_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype,d_h", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128)])
def test_a_threads_first_call(dtype, d_h, monkeypatch):
    """The device's context is not current in a thread that has made no call of the runtime yet."""
    g = torch.Generator(device=DEV).manual_seed(1)
    B, T, nq, nkv, mp = 2, 3, 4, 2, 3
    q, past = (torch.randn(B, n, h, d_h, generator=g, device=DEV).to(dtype) for n, h in ((T, nq), (130, nkv)))
    pages, bt = binding.kv_pages(B * mp, nkv, d_h), torch.arange(B * mp, dtype=torch.int32, device=DEV).view(B, mp)
    pos = torch.tensor([100, 7], device=DEV)
    binding.kv_append(pages, bt, past, past, torch.zeros_like(pos), None)
    calls, lib = [], binding.load()

    class Kept:      # the call's arguments, to be made again by another thread
        def __getattr__(self, name):
            fn = getattr(lib, name)
            if name != "dlite_kv_attention":
                return fn
            return lambda ref, stream: calls.append((ref, stream)) or fn(ref, stream)

    monkeypatch.setattr(binding, "load", lambda: Kept())
    ws = torch.zeros(max(16, binding.kv_attention_workspace(B, T, nq, nkv, d_h, mp, dtype)), dtype=torch.uint8, device=DEV)
    want, _ = binding.kv_attention(q, pages, bt, pos, workspace=ws)
    torch.cuda.synchronize()
    first, codes = want.clone(), []
    want.zero_()
    torch.cuda.synchronize()
    (ref, stream), = calls
    t = threading.Thread(target=lambda: codes.append(lib.dlite_kv_attention(ref, stream)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert codes == [0] and torch.equal(want, first)
