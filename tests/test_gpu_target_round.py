"""GPU: the target-side operators as a round uses them. A draft of K tokens, then one layer of a
stand-in target over [a, d_1..d_K] (torch products for its projections): queries rotated, keys and
values appended at pos[b] + t, attention over the paged 4-bit cache, logits, greedy verification, the commits' log
probabilities, pos += n_commit (the crop: rejected rows are overwritten by the next round's append). The whole
round is captured once and replayed; every stage is checked against the oracle on its own inputs."""
import numpy as np
import pytest
import torch

from history_free_speculative_gb300 import binding
from history_free_speculative_gb300 import workload as wk
from oracle import dlite_oracle as O
from oracle import target_oracle as TO
from test_gpu_kv_attention import _tolerance, _within
from test_gpu_token_logprobs import _check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_rounds_over_a_paged_cache(dtype):
    wl = wk.WORKLOADS["tiny"]
    cfg, B, R, MP = wl.cfg, wl.B, 4, 4
    T, nq, nkv, d, V = cfg.K + 1, cfg.n_q, cfg.n_kv, cfg.d_h, cfg.V
    g = torch.Generator(device=DEV).manual_seed(3)
    mat = lambda *s: (torch.randn(*s, generator=g, device=DEV) * s[-1] ** -0.5).to(dtype)  # noqa: E731
    Wqkv, Wo = mat((nq + 2 * nkv) * d, cfg.D), mat(V, nq * d)
    Emb = torch.randn(V, cfg.D, generator=g, device=DEV).to(dtype)
    W = wk.make_weights(cfg, wl.weight_seed)
    dr = binding.Drafter(cfg, wk.weights_to(W, DEV), B_max=B)
    try:
        hidden, anchor, _ = wk.make_round_inputs(wl, round_index=1)
        hd, ad = hidden.to(DEV), anchor.to(DEV)
        pos = torch.tensor([0, 60, 63, 130], dtype=torch.int64, device=DEV)
        pages = binding.kv_pages(B * MP + 1, nkv, d)
        bt = torch.randperm(B * MP + 1, generator=torch.Generator().manual_seed(4))[:B * MP].view(B, MP).to(torch.int32).to(DEV)
        table = binding.rope_table(64 * MP, d, theta=1e4)
        # the requests' past: random rows, appended as prompts of ragged lengths
        past = [torch.randn(B, 130, nkv, d, generator=g, device=DEV).to(dtype) for _ in range(2)]
        binding.kv_append(pages, bt, *past, torch.zeros_like(pos), table, n_rows=pos.to(torch.int32))
        out = dr.new_outputs(B, DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        s = torch.cuda.Stream(device=DEV)

        def round_():
            dr.draft_round(hd, ad, 0.0, wl.rng_seed, pos, out["cand"], out["qstats"], stream=s)
            tokens = torch.cat([ad.view(B, 1), out["cand"]], dim=1)
            qkv = (Emb[tokens.long()] @ Wqkv.T).view(B, T, nq + 2 * nkv, d)
            q, k, v = qkv.split((nq, nkv, nkv), dim=2)
            rq = binding.rope(q, pos, table, status=st, stream=s)
            binding.kv_append(pages, bt, k, v, pos, table, status=st, stream=s)
            o, lse = binding.kv_attention(rq, pages, bt, pos, lse=True, status=st, stream=s)
            logits = o.view(B, T, nq * d) @ Wo.T
            tgt = logits.argmax(-1).to(torch.int32)
            tgt[:, 0] = out["cand"][:, 0]          # an agreement, so that rounds accept something
            tgt[1::2, 1] = out["cand"][1::2, 1]
            dr.verify(out["cand"], tgt, out["accepted"], out["commits"], out["n_commit"], ad, stream=s)
            lp = binding.token_logprobs(logits, out["commits"], n_top=3, status=st, stream=s)
            before = pos.clone()
            dr.advance(out["n_commit"], pos, stream=s)
            return dict(tokens=tokens, q=q, k=k, v=v, rq=rq, o=o, lse=lse, logits=logits, tgt=tgt, lp=lp, before=before)

        keep = [t.clone() for t in (ad, pos, pages)]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            round_()
            s.synchronize()
            for t, k in zip((ad, pos, pages), keep):
                t.copy_(k)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                r = round_()
        np_pages, tab, want_pos = pages.cpu().numpy().copy(), table.cpu().numpy(), pos.tolist()
        name = "bf16" if dtype == torch.bfloat16 else "f32"
        f = lambda t: t.float().cpu().numpy()  # noqa: E731
        for _ in range(R):
            graph.replay()
            torch.cuda.synchronize()
            p = r["before"].tolist()
            assert p == want_pos and int(st.item()) == 0
            assert np.array_equal(f(r["rq"]), TO.rope(f(r["q"]), p, tab, "half", dtype=name).astype(np.float32))
            assert TO.append(np_pages, bt.cpu().numpy(), f(r["k"]), f(r["v"]), p, tab) == set()
            assert np.array_equal(pages.cpu().numpy(), np_pages)
            want, wl_, reach, eps = TO.attention(f(r["rq"]), np_pages, bt.cpu().numpy(), p, d ** -0.5)
            tol, ltol = _tolerance(want, reach, eps, 64 * MP, d, name, v_exp=2)
            _within(r["o"], want, tol)
            _within(r["lse"], wl_, ltol)
            commits = out["commits"].cpu()
            for b in range(B):
                v = O.verify_greedy(r["tokens"][b, 1:].cpu().numpy(), r["tgt"][b].cpu().numpy())
                assert commits[b, :v["n_commit"]].tolist() == v["commits"] and bool((commits[b, v["n_commit"]:] == -1).all())
                want_pos[b] += v["n_commit"]
            assert int(out["n_commit"].sum()) > B and int(out["n_commit"].min()) < T     # both acceptance and a crop
            _check(r["logits"].double().cpu().numpy().reshape(B * T, V), commits, 1.0, 3, r["lp"])
        assert pos.tolist() == want_pos
    finally:
        dr.close()
