"""GPU: target-side calls of several host threads at once, each on its own stream."""
import ctypes
import threading

import pytest
import torch

from history_free_speculative_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_token_logprobs_of_threads_with_different_row_counts():
    """The launches of one kernel take shared memory by their row counts (here one to five CTAs an SM); the calls of one thread do
    not disturb another's."""
    V, n_top, calls, lib = 2000, 4, 4000, binding.load()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    sizes = (2 * sms, 3 * sms, 4 * sms, 5 * sms)
    rows = [torch.randn(n, V, generator=torch.Generator().manual_seed(n)).bfloat16().to(DEV) for n in sizes]
    tok = [torch.arange(n, dtype=torch.int32, device=DEV) for n in sizes]
    want = [binding.token_logprobs(x, t, n_top=n_top) for x, t in zip(rows, tok)]
    got = [{k: torch.zeros_like(v) for k, v in w.items()} for w in want]
    torch.cuda.synchronize()
    start, codes = threading.Barrier(len(sizes)), [set() for _ in sizes]

    def loop(i):
        s, o = torch.cuda.Stream(device=DEV), got[i]
        a = binding.LogprobsArgs(sizes[i], V, n_top, binding.DLITE_BF16, 1.0, rows[i].data_ptr(), V, tok[i].data_ptr(),
                                 *(o[k].data_ptr() for k in ("logprob", "entropy", "top_ids", "top_logprobs")), None)
        ref, stream = ctypes.byref(a), s.cuda_stream
        start.wait()
        for _ in range(calls):
            codes[i].add(lib.dlite_token_logprobs(ref, stream))
        s.synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert codes == [{0}] * len(sizes), codes
    for w, g in zip(want, got):
        assert all(torch.equal(w[k], g[k]) for k in w)
