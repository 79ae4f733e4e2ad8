"""GPU: token log probabilities, entropy and alternatives against the float64 oracle.

Tolerances, derived: d = (m - x) k is off by three roundings, 3 2^-24 relative, e^-d by that times d (below 104 for a weight that
counts in float32) times ln 2 plus 2^-22 from exp2, so by at most 2^-16; typical weights sit at d < 30. A thread's sum of at most
n / 512 + 32 terms adds that many 2^-24. S and the entropy's sum share these relative errors: log S moves by the
relative error of S (times S1 / S <= 1) and the entropy by twice its own size times it; logprob = -d - log S is rounded
at the size of its two terms. The alternatives' ids are compared exactly."""
import math

import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from oracle import target_oracle as TO

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rel(V):
    """Relative error of S and of the entropy's sum: weights that matter lie at d < 30 (below 2^-30 of the largest, V < 2^19 of
    them change the sums by less than 2^-11 of their own 2^-16)."""
    return 30 * 3 * 2.0 ** -24 * math.log(2) + 2.0 ** -22 + (V / 512 + 32) * 2.0 ** -24 + 2.0 ** -27


def _check(x, tokens, T, n_top, got):
    """x: logits as the device holds them [rows, V] float64."""
    V = x.shape[1]
    r = _rel(V)
    g = {k: v.cpu().numpy().reshape((len(x),) + tuple(v.shape[tokens.dim():])) for k, v in got.items()}
    for i, tok in enumerate(tokens.flatten().tolist()):
        if tok < 0:
            continue
        lp, h, ids, top = TO.token_logprobs(x[i], tok, T, n_top)
        assert list(g["top_ids"][i]) == list(ids), i
        for a, b in [(g["logprob"][i], lp)] + list(zip(g["top_logprobs"][i], top)):
            if np.isfinite(b):
                # log S moves by r S1 / S at most, and S1 / S <= -ln p for the row's likeliest token: log1p(S1) >= S1 / S
                logS = -TO.token_logprobs(x[i], 0, T, 1)[3][0]
                assert abs(a - b) <= 4 * 2.0 ** -24 * abs(b) + r * logS + 1e-30, (i, a, b)
            else:
                assert (np.isnan(a) and np.isnan(b)) or a == b, (i, a, b)
        if np.isfinite(h):
            assert abs(g["entropy"][i] - h) <= 2 * r * h + 1e-30, (i, g["entropy"][i], h)
        else:
            assert np.isnan(g["entropy"][i])


CASES = [
    # shape, V, dtype, T, n_top
    ((1,), 1, "f32", 1.0, 1), ((3,), 2, "bf16", 0.7, 2), ((2, 3), 7, "f32", 1.3, 0), ((4,), 33, "bf16", 1.0, 32),
    ((5,), 1000, "f32", 0.7, 20), ((3,), 4097, "bf16", 1.0, 5), ((2,), 50257, "bf16", 1.0, 20), ((3,), 50257, "f32", 0.7, 32),
    ((1,), 151936, "f32", 1.0, 20), ((1, 8), 151936, "bf16", 0.7, 5), ((160,), 8191, "bf16", 1.0, 3), ((320,), 2049, "f32", 1.0, 1),
    ((1,), 262144, "bf16", 2.0, 32), ((0,), 100, "f32", 1.0, 1),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_logprobs(case):
    shape, V, dtype, T, n_top = case
    rows = math.prod(shape)
    if rows == 0:
        with pytest.raises(binding.DliteError):
            binding.token_logprobs(torch.zeros(0, V, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV))
        return
    g = _gen(V + rows)
    x = torch.randn(*shape, V, generator=g) * 3
    x.view(rows, V)[::2, torch.randint(0, V, (4,), generator=g)] += 9.0
    x = x.to(DT[dtype])
    tok = torch.randint(0, V, shape, generator=g).to(torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = binding.token_logprobs(x.to(DEV), tok.to(DEV), T, n_top, status=st)
    assert got["logprob"].shape == shape and got["top_ids"].shape == shape + (n_top,)
    _check(x.view(rows, V).double().numpy(), tok, T, n_top, got)
    again = binding.token_logprobs(x.to(DEV), tok.to(DEV), T, n_top)
    assert all(torch.equal(again[k], got[k]) for k in got) and int(st.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,rows", [(5000, 1), (5003, 400)])
def test_ties_excluded_ids_and_special_rows(dtype, V, rows):
    """Equal logits everywhere, few distinct values, banned ids, the type's lowest value, -0, NaN, +inf, near certainty."""
    low = torch.finfo(DT[dtype]).min
    base = torch.randn(V, generator=_gen(1)) * 2
    kinds = [torch.zeros(V), torch.randint(-2, 3, (V,), generator=_gen(2)).float(), base.clone(), base.clone(), base.clone(),
             torch.full((V,), -math.inf), torch.full((V,), low), base.clone(), base.clone(), torch.full((V,), -30.0), base * 1e4,
             torch.where(torch.arange(V) % 3 == 0, torch.tensor(-0.0), torch.tensor(0.0)), torch.arange(V, 0, -1).float(),
             torch.arange(V).float()]
    kinds[2][torch.rand(V, generator=_gen(3)) < 0.9] = -math.inf
    kinds[3][torch.rand(V, generator=_gen(4)) < 0.9] = low
    kinds[4][:] = -math.inf
    kinds[4][[9, V - 1, 3]] = torch.tensor([1.0, 1.0, -40.0])
    kinds[7][V // 2] = math.nan
    kinds[8][V // 3] = math.inf
    kinds[9][1234] = 5.0
    for n_top in (0, 1, 20, 32):
        for lo in range(0, len(kinds), rows):
            x = torch.stack([kinds[(lo + i) % len(kinds)] for i in range(rows)]).to(DT[dtype])
            tok = torch.tensor([(1234 + 7 * i) % V for i in range(rows)], dtype=torch.int32)
            _check(x[:28].double().numpy(), tok[:28], 1.0, n_top,
                   {k: v[:28] for k, v in binding.token_logprobs(x.to(DEV), tok.to(DEV), 1.0, n_top).items()})


def test_strides_alignment_skipped_rows_and_bad_ids():
    V = 1003
    buf = torch.randn(40 * 1100, generator=_gen(5))
    for dtype in DT:
        d = buf.to(DT[dtype]).to(DEV)
        for off, stride in ((0, 1003), (1, 1003), (3, 1011), (5, 1008), (8, 1024)):
            x = torch.as_strided(d, (3, 4, V), (4 * stride, stride, 1), off)
            tok = torch.tensor([[5, -1, 1002, 0], [-7, 8, 1003, 9], [1, 2, 3, 1 << 30]], dtype=torch.int32)
            st = torch.zeros(1, dtype=torch.int32, device=DEV)
            keep = dict(logprob=torch.full((3, 4), 5.0, device=DEV), entropy=torch.full((3, 4), 5.0, device=DEV),
                        top_ids=torch.full((3, 4, 3), 77, dtype=torch.int32, device=DEV), top_logprobs=torch.full((3, 4, 3), 5.0, device=DEV))
            got = binding.token_logprobs(x, tok.to(DEV), 0.9, 3, status=st, **keep)
            assert got["logprob"] is keep["logprob"]
            _check(x.double().cpu().numpy().reshape(12, V), tok, 0.9, 3, got)
            skipped = (tok < 0).to(DEV)
            assert not got["logprob"][skipped].any() and not got["entropy"][skipped].any() and not got["top_logprobs"][skipped].any()
            assert bool((got["top_ids"][skipped] == -1).all())
            assert bool(got["logprob"][1, 2].isnan()) and bool(got["logprob"][2, 3].isnan()) and int(st.item()) == binding.DEV_BOUNDS


def test_graph_replay_and_streams():
    x = torch.randn(2, 6, 151936, generator=_gen(6))
    tok = torch.randint(0, 151936, (2, 6), generator=_gen(7)).to(torch.int32)
    dx, dt = x[0].to(DEV), tok[0].to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        binding.token_logprobs(dx, dt, 0.8, 10, stream=s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = binding.token_logprobs(dx, dt, 0.8, 10, stream=s)
        for i in (1, 0):
            dx.copy_(x[i])
            dt.copy_(tok[i])
            graph.replay()
            s.synchronize()
            _check(x[i].double().numpy(), tok[i], 0.8, 10, got)


@pytest.mark.parametrize("V,rows", [(262144, 1), (65536, 200)])
def test_large_elements_in_the_same_threads(V, rows):
    """Thousands of large logits at ids a multiple of 4096 (+ 0..7) apart: a few threads own them all."""
    x = torch.randn(rows, V, generator=_gen(8)) * 0.1
    i = torch.arange(V)
    for mod, width in ((4096, 8), (4096, 64), (2048, 1500)):
        y = x + torch.where(i % mod < width, 20.0 + (i * 7919 % 100003).float() / 1e4, torch.tensor(0.0))
        tok = torch.full((rows,), 5, dtype=torch.int32)
        got = binding.token_logprobs(y.to(DEV), tok.to(DEV), 1.0, 32)
        _check(y[:2].double().numpy(), tok[:2], 1.0, 32, {k: v[:2] for k, v in got.items()})
