"""The target-side operators of a draft-and-verify round, as measured cases.

A round's target forward runs T = K + 1 rows per request ([anchor, d_1..d_K]) at positions pos[b] + t:
their queries and keys are rotated, keys and values go into a paged 4-bit cache, the rows attend over
that cache, and the committed tokens are scored against the target's logits. `run` makes one pass of one
of these operators; with `own` false it computes the plain form with elementary torch operations.

Cache format: pages [n_pages, n_kv, 72 d_h] bytes; one record holds 64 tokens of one key/value head:
key codes [64][d_h / 2] (byte: column 2j in the low nibble, 2j + 1 in the high one), value codes
[d_h][32] (byte: token 2i low, 2i + 1 high), key scales [64][d_h / 16] and value scales [d_h / 16][64].
A code is an e2m1 number, a scale an e4m3 one shared by 16 columns of a token; the value it stands for
is code * scale * 2^exp. Token p of request b is row p % 64 of page block_table[b, p / 64].
"""
import math

import torch

own = False

PAGE = 64
HALF, INTERLEAVED = "half", "interleaved"
THETA = 1e6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    head = dict(nq=32, nkv=8, d=128)
    return [
        # one request decoding one token: the queries of one row (latency)
        dict(name="rope-one-token", op="rope", B=1, T=1, ctx=1000, rot=128, layout=HALF, dtype="bf16", packed=False, **head),
        # the verification block of 32 requests, queries taken out of the fused QKV rows
        dict(name="rope-verify-block", op="rope", B=32, T=8, ctx=8192, rot=128, layout=HALF, dtype="bf16", packed=True, **head),
        # a prompt's queries, half of each head rotated, neighbouring columns paired, float32
        dict(name="rope-prompt-f32", op="rope", B=1, T=8192, ctx=0, rot=64, layout=INTERLEAVED, dtype="f32", packed=False, **head),
        # one request decoding one token: its key / value row into the cache, and read back
        dict(name="append-one-token", op="append", B=1, T=1, ctx=1000, rot=128, layout=HALF, dtype="bf16", packed=False, ragged=False, exp=0, **head),
        # the verification block of 32 requests at ragged positions
        dict(name="append-verify-block", op="append", B=32, T=8, ctx=40960, rot=128, layout=HALF, dtype="bf16", packed=True, ragged=True, exp=-3, **head),
        # a prompt going into the cache
        dict(name="append-prompt", op="append", B=1, T=8192, ctx=37, rot=128, layout=HALF, dtype="bf16", packed=True, ragged=False, exp=0, **head),
        # one request, one token, a short context (latency), float32 queries, heads of 64
        dict(name="attend-short-f32", op="attend", B=1, T=1, ctx=500, window=0, dtype="f32", ragged=False, exp=0, nq=4, nkv=2, d=64),
        # plain decoding of eight requests, one token each
        dict(name="attend-decode", op="attend", B=8, T=1, ctx=8192, window=0, dtype="bf16", ragged=False, exp=0, **head),
        # one agentic request with a long history, its verification block
        dict(name="attend-verify-long", op="attend", B=1, T=8, ctx=118000, window=0, dtype="bf16", ragged=False, exp=0, **head),
        # 32 requests of ragged lengths and ragged blocks
        dict(name="attend-verify-batch", op="attend", B=32, T=8, ctx=40960, window=0, dtype="bf16", ragged=True, exp=-3, **head),
        # the committed tokens of one request scored against float32 logits
        dict(name="logprobs-one-block", op="logprobs", rows=8, V=151936, n_top=5, dtype="f32", T=0.7, banned=False),
        # the verification rows of 64 requests, bf16 logits with banned ids
        dict(name="logprobs-batch", op="logprobs", rows=512, V=151936, n_top=20, dtype="bf16", T=1.0, banned=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "logprobs"))
    if op == "logprobs":
        V = _log_int(rng, 1000, 262144)
        return dict(op=op, rows=_log_int(rng, 1, max(1, min(2048, (512 * 151936) // (2 * V)))), V=V, n_top=rng.randint(0, 20),
                    dtype=rng.choice(("bf16", "f32")), T=rng.choice((0.7, 1.0, 1.3)), banned=rng.random() < 0.5)
    d = rng.choice((64, 128))
    nkv = rng.choice((1, 2, 3, 4, 8))
    c = dict(op=op, nq=nkv * rng.choice((1, 2, 3, 4, 5, 8)), nkv=nkv, d=d, dtype=rng.choice(("bf16", "bf16", "f32")))
    if op == "attend":
        B, T = _log_int(rng, 1, 64), rng.choice((1, 1, 2, 5, 8, 8, 17, 32))
        most = max(2, 400000 // (B * max(1, T * c["nq"] // (nkv * 32))))
        c.update(B=B, T=T, ctx=_log_int(rng, 1, min(118000, most)), window=rng.choice((0, 0, 0, 128, 512)),
                 ragged=rng.random() < 0.5, exp=rng.choice((0, -3, 2)))
        return c
    B = _log_int(rng, 1, 64)
    c.update(B=B, T=_log_int(rng, 1, max(1, 4096 // B)), ctx=_log_int(rng, 1, 40960), rot=rng.choice((d, d, d // 2, 48)),
             layout=rng.choice((HALF, INTERLEAVED)), packed=rng.random() < 0.5)
    if op == "append":
        c.update(ragged=rng.random() < 0.5, exp=rng.choice((0, -3, 2)))
    return c


def _positions(case):
    """Rows already cached, per request: the longest first, the others spread over the range."""
    return [int(case["ctx"] * (1.0 if b == 0 else 0.02 + 0.98 * ((b * 0.6180339887) % 1.0))) for b in range(case["B"])]


def _n_rows(case):
    """Valid rows of each request's block (ragged: from none to all T)."""
    T = case["T"]
    return [T if b == 0 or not case.get("ragged") else (b * 5) % (T + 1) for b in range(case["B"])]


# ------------------------------------------------------------------ the format, in torch

def _quantise(x, exp):
    """Codes (uint8, one per value) and scale bytes (one per 16) of float32 x [..., d]."""
    y = (x * 2.0 ** -exp).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()
    a = torch.where(sf > 0, y.abs() / sf, torch.zeros_like(y))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * (torch.signbit(y) & (sf > 0)).to(torch.uint8)
    return code.flatten(-2), s.view(torch.uint8).squeeze(-1)


def _pack(kc, ks, vc, vs):
    """Records [..., n_kv, 72 d] of codes kc, vc [..., 64, n_kv, d] and scales ks, vs [..., 64, n_kv, d / 16]."""
    kc, ks = kc.transpose(-3, -2), ks.transpose(-3, -2)
    vc, vs = vc.movedim(-3, -1), vs.movedim(-3, -1)
    return torch.cat([(kc[..., 0::2] | kc[..., 1::2] << 4).flatten(-2), (vc[..., 0::2] | vc[..., 1::2] << 4).flatten(-2),
                      ks.flatten(-2), vs.flatten(-2)], dim=-1)


def _codes(rec):
    """The inverse of _pack."""
    d = rec.shape[-1] // 72
    k, v, ks, vs = rec.split((32 * d, 32 * d, 4 * d, 4 * d), dim=-1)
    k, v = k.unflatten(-1, (PAGE, d // 2)), v.unflatten(-1, (d, PAGE // 2))
    kc = torch.stack([k & 15, k >> 4], dim=-1).flatten(-2)
    vc = torch.stack([v & 15, v >> 4], dim=-1).flatten(-2)
    return (kc.transpose(-3, -2), ks.unflatten(-1, (PAGE, d // 16)).transpose(-3, -2),
            vc.movedim(-1, -3), vs.unflatten(-1, (d // 16, PAGE)).movedim(-1, -3))


def _values(code, scale, exp):
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    val = torch.cat([e2m1, -e2m1])[code.int()].unflatten(-1, (-1, 16))
    return (val * scale.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2) * 2.0 ** exp


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    if case["op"] == "logprobs":
        rows, V = case["rows"], case["V"]
        x = torch.randn(rows, V, generator=g, device=dev) * 2.5
        peak = torch.randint(0, V, (rows, 12), generator=g, device=dev)
        x.scatter_add_(1, peak, 6.0 + 8.0 * torch.rand(rows, 12, generator=g, device=dev))
        if case["banned"]:
            x[:, torch.randint(0, V, (max(1, V // 50),), generator=g, device=dev)] = -math.inf
        x = x.to(dt)
        tok = torch.where(torch.rand(rows, generator=g, device=dev) < 0.7, x.float().argmax(1),
                          torch.randint(0, V, (rows,), generator=g, device=dev)).to(torch.int32)
        return dict(case=case, logits=x, tokens=tok)

    B, T, nq, nkv, d = (case[k] for k in ("B", "T", "nq", "nkv", "d"))
    pos = _positions(case)
    st = dict(case=case, pos=torch.tensor(pos, dtype=torch.int64, device=dev),
              n_rows=torch.tensor(_n_rows(case), dtype=torch.int32, device=dev) if case.get("ragged") else None)
    if case["op"] in ("rope", "append"):
        f = THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
        a = torch.arange(max(pos) + T, dtype=torch.float64, device=dev)[:, None] * f
        st["table"] = torch.stack([a.cos(), a.sin()], dim=-1).float()   # [positions, rot / 2, 2]
        qkv = torch.randn(B, T, nq + 2 * nkv, d, generator=g, device=dev)
        qkv = (qkv * torch.exp(0.5 * torch.randn(nq + 2 * nkv, d, generator=g, device=dev))).to(dt)
        st["q"], st["k"], st["v"] = qkv.split((nq, nkv, nkv), dim=2)
        if not case["packed"]:
            st["q"], st["k"], st["v"] = (t.contiguous() for t in (st["q"], st["k"], st["v"]))
        if case["op"] == "rope":
            return st
    max_pages = case["ctx"] // PAGE + (T + 2 * PAGE - 2) // PAGE
    n_pages = B * max_pages + 5
    st["block_table"] = torch.randperm(n_pages, generator=g, device=dev)[:B * max_pages].view(B, max_pages).to(torch.int32)
    if case["op"] == "append":
        # what the pages held before: other tokens of the same kind
        kv = torch.randint(0, 256, (n_pages, nkv, 72 * d), generator=g, device=dev, dtype=torch.uint8)
        kv[..., 64 * d:] = 0x30 + kv[..., 64 * d:] % 16
        st.update(pages=kv, k_out=torch.zeros(B, T, nkv, d, dtype=torch.bfloat16, device=dev),
                  v_out=torch.zeros(B, T, nkv, d, dtype=torch.bfloat16, device=dev))
        return st
    chan = torch.exp(0.5 * torch.randn(2, nkv, d, generator=g, device=dev))
    st["pages"] = torch.empty(n_pages, nkv, 72 * d, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // (PAGE * nkv * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        k, v = (torch.randn(n, PAGE, nkv, d, generator=g, device=dev) * chan[j] * 2.0 ** case["exp"] for j in (0, 1))
        st["pages"][i:i + n] = _pack(*_quantise(k, case["exp"]), *_quantise(v, case["exp"]))
    st["q"] = (2.0 * torch.randn(B, T, nq, d, generator=g, device=dev) * 2.0 ** -case["exp"]).to(dt)
    st["out"] = torch.zeros(B, T, nq, d, dtype=dt, device=dev)
    st["lse"] = torch.zeros(B, T, nq, dtype=torch.float32, device=dev)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return globals()["_%s_%s" % ("own" if own else "plain", st["case"]["op"])](st)


def _own_rope(st):
    from history_free_speculative_gb300 import binding
    return binding.rope(st["q"], st["pos"], st["table"], layout=st["case"]["layout"])


def _own_append(st):
    from history_free_speculative_gb300 import binding
    c = st["case"]
    binding.kv_append(st["pages"], st["block_table"], st["k"], st["v"], st["pos"], table=st["table"], layout=c["layout"],
                      n_rows=st["n_rows"], k_exp=c["exp"], v_exp=c["exp"])
    return binding.kv_read(st["pages"], st["block_table"], st["pos"], c["T"], n_rows=st["n_rows"], k_exp=c["exp"], v_exp=c["exp"],
                           k_out=st["k_out"], v_out=st["v_out"])


def _own_attend(st):
    from history_free_speculative_gb300 import binding
    c = st["case"]
    return binding.kv_attention(st["q"], st["pages"], st["block_table"], st["pos"], window=c["window"], n_rows=st["n_rows"],
                                k_exp=c["exp"], v_exp=c["exp"], out=st["out"], lse=st["lse"])


def _own_logprobs(st):
    from history_free_speculative_gb300 import binding
    return binding.token_logprobs(st["logits"], st["tokens"], temperature=st["case"]["T"], n_top=st["case"]["n_top"])


def _rotated(x, pos, table, layout):
    """x [B, T, H, d] in float32 with its first columns rotated by the angles of position pos[b] + t."""
    x = x.float()
    half = table.shape[1]
    cs = table[pos[:, None] + torch.arange(x.shape[1], device=x.device)][:, :, None]
    c, s = cs[..., 0], cs[..., 1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    x0, x1 = (r[..., :half], r[..., half:]) if layout == HALF else (r[..., 0::2], r[..., 1::2])
    y0, y1 = x0 * c - x1 * s, x1 * c + x0 * s
    r = torch.cat([y0, y1], dim=-1) if layout == HALF else torch.stack([y0, y1], dim=-1).flatten(-2)
    return torch.cat([r, rest], dim=-1)


def _plain_rope(st):
    return _rotated(st["q"], st["pos"], st["table"], st["case"]["layout"]).to(st["q"].dtype)


def _touched(st):
    """Page ids [B, P] covering the block's rows, and each row's place [B, T] in them."""
    c, pos = st["case"], st["pos"]
    t = torch.arange(c["T"], device=pos.device)
    first = pos // PAGE
    P = (c["T"] + 2 * PAGE - 2) // PAGE
    col = first[:, None] + torch.arange(P, device=pos.device)
    return st["block_table"].gather(1, col).long(), (pos % PAGE)[:, None] + t


def _valid(st):
    c = st["case"]
    t = torch.arange(c["T"], device=st["pos"].device).expand(c["B"], -1)
    return t >= 0 if st["n_rows"] is None else t < st["n_rows"][:, None]


def _plain_append(st):
    c, B = st["case"], st["case"]["B"]
    new = (*_quantise(_rotated(st["k"], st["pos"], st["table"], c["layout"]), c["exp"]), *_quantise(st["v"].float(), c["exp"]))
    ids, place = _touched(st)
    b = torch.arange(B, device=ids.device)[:, None].expand_as(place)
    m = _valid(st)[..., None, None]
    parts = [p.flatten(1, 2).contiguous() for p in _codes(st["pages"][ids])]   # [B, P 64, n_kv, ...]
    for p, n in zip(parts, new):
        p[b, place] = torch.where(m, n, p[b, place])
    st["pages"][ids] = _pack(*(p.unflatten(1, (-1, PAGE)) for p in parts))
    # and read back
    kc, ks, vc, vs = (p.flatten(1, 2)[b, place] for p in _codes(st["pages"][ids]))
    st["k_out"].copy_(torch.where(m, _values(kc, ks, c["exp"]), st["k_out"].float()))
    st["v_out"].copy_(torch.where(m, _values(vc, vs, c["exp"]), st["v_out"].float()))
    return st["k_out"], st["v_out"]


def _plain_attend(st):
    c = st["case"]
    B, T, nq, nkv, d = (c[k] for k in ("B", "T", "nq", "nkv", "d"))
    kc, ks, vc, vs = (p.flatten(1, 2) for p in _codes(st["pages"][st["block_table"].long()]))
    k = _values(kc, ks, c["exp"])
    q = st["q"].float().unflatten(2, (nkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [B, n_kv, g T, d]
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).unflatten(2, (-1, T)) / math.sqrt(d)      # [B, n_kv, g, T, keys]
    del k
    hi = st["pos"][:, None] + torch.arange(T, device=q.device)
    j = torch.arange(s.shape[-1], device=q.device)
    see = j <= hi[..., None]
    if c["window"]:
        see &= j > hi[..., None] - c["window"]
    s = s.masked_fill(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    v = _values(vc, vs, c["exp"]).permute(0, 2, 1, 3)
    o = torch.matmul((p / z).flatten(2, 3), v).unflatten(2, (-1, T)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    lse = (m + z.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)
    ok = _valid(st)[..., None]
    st["out"].copy_(torch.where(ok[..., None], o, st["out"].float()))
    st["lse"].copy_(torch.where(ok, lse, st["lse"]))
    return st["out"], st["lse"]


def _plain_logprobs(st):
    c, x = st["case"], st["logits"].float() + 0.0
    far = (x.amax(1, keepdim=True) - x) / c["T"]      # >= 0, inf where banned
    e = torch.exp(-far)
    S = e.sum(1)
    logS = S.log()
    out = dict(logprob=-far.gather(1, st["tokens"].long()[:, None]).squeeze(1) - logS,
               entropy=logS + torch.where(e > 0, e * far, torch.zeros_like(e)).sum(1) / S)
    # alternatives by logit, the lower id first among equals: one 64-bit key per id
    bits = x.view(torch.int32).long()
    key = (torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF) << 32) + (c["V"] - 1 - torch.arange(c["V"], device=x.device))
    top = c["V"] - 1 - (key.topk(c["n_top"], dim=1).values & 0xFFFFFFFF)
    out.update(top_ids=top.to(torch.int32), top_logprobs=-far.gather(1, top) - logS[:, None])
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprobs":
        n = case["rows"] * case["V"]
        return dict(bytes=n * b + case["rows"] * (12 + 8 * case["n_top"]), flops=5 * n)
    B, T, nq, nkv, d = (case[k] for k in ("B", "T", "nq", "nkv", "d"))
    n, pos = _n_rows(case), _positions(case)
    if case["op"] == "rope":
        return dict(bytes=2 * B * T * nq * d * b + B * T * case["rot"] * 4, flops=3 * B * T * nq * case["rot"])
    if case["op"] == "append":   # k and v in, their codes and scales out and in again, the values out
        return dict(bytes=sum(n) * (nkv * d * (2 * b + 2 * 9 / 8 + 4) + case["rot"] * 4), flops=sum(n) * nkv * d * 12)
    by, fl = 0, 0
    for p, r in zip(pos, n):
        if r:
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            by += (p + r - lo) * nkv * d * 9 / 8
            seen = sum((min(p + t + 1, case["window"]) if case["window"] else p + t + 1) for t in range(r))
            fl += 4 * seen * nq * d
        by += r * nq * (2 * d * b + 4)
    return dict(bytes=by, flops=fl)


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return globals()["_exact_" + case["op"]](st, case)


def _exact_rotate(x, st, case):
    x = x.double().clone()
    n = case["rot"] // 2
    p = st["pos"][:, None] + torch.arange(case["T"], device=x.device)
    z = torch.view_as_complex(st["table"].double())[p][:, :, None]
    i = torch.arange(n, device=x.device)
    a, b = (i, i + n) if case["layout"] == HALF else (2 * i, 2 * i + 1)
    y = torch.complex(x[..., a], x[..., b]) * z
    x[..., a], x[..., b] = y.real, y.imag
    return x


def _exact_rope(st, case):
    return _exact_rotate(st["q"], st, case)


def _exact_fp4(x, exp):
    """The nearest value the format holds, by its grid: steps of 2^(e - 1) between powers of two, of 1/2 below one."""
    def grid(v, bits, least):
        step = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** least))).clamp(min=least) - bits)
        return torch.round(v / step) * step
    y = x.unflatten(-1, (-1, 16)) / 2.0 ** exp
    s = grid(y.abs().amax(-1, keepdim=True) / 6, 3, -6).clamp(max=448)
    q = grid(y.abs() / s.clamp(min=2.0 ** -9), 1, 0).clamp(max=6) * s
    return (torch.sign(y) * q).flatten(-2) * 2.0 ** exp


def _exact_append(st, case):
    ok = torch.tensor(_n_rows(case), device=st["pos"].device)[:, None] > torch.arange(case["T"], device=st["pos"].device)
    ok = ok[..., None, None].double()
    return _exact_fp4(_exact_rotate(st["k"], st, case), case["exp"]) * ok, _exact_fp4(st["v"].double(), case["exp"]) * ok


def _exact_decode(b, ebits, mbits, bias):
    e, m = (b.int() >> mbits) & (2 ** ebits - 1), (b.int() & (2 ** mbits - 1)).double() / 2 ** mbits
    return torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * torch.exp2((e - bias).double()))


def _exact_attend(st, case):
    B, T, nq, nkv, d = (case[k] for k in ("B", "T", "nq", "nkv", "d"))
    out = torch.zeros(B, T, nq, d, dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros(B, T, nq, dtype=torch.float64, device=st["q"].device)
    for b, (p, n) in enumerate(zip(_positions(case), _n_rows(case))):
        if not n:
            continue
        lo = max(0, p - case["window"] + 1) // PAGE if case["window"] else 0
        rec = st["pages"][st["block_table"][b, lo:(p + n + PAGE - 1) // PAGE].long()]
        key = lo * PAGE + torch.arange(rec.shape[0] * PAGE, device=rec.device)
        t = p + torch.arange(n, device=rec.device)[:, None]
        see = (key <= t) & ((key > t - case["window"]) if case["window"] else (key >= 0))
        for h in range(nkv):
            kd, vd, ks, vs = rec[:, h].split((32 * d, 32 * d, 4 * d, 4 * d), dim=1)
            kd, vd = kd.reshape(-1, d // 2), vd.reshape(-1, d, 32).transpose(1, 2).reshape(-1, d)
            k = torch.empty(len(key), d, dtype=torch.float64, device=rec.device)
            v = torch.empty_like(k)
            for odd in (0, 1):
                cut = lambda c: torch.where((c >> 4 * odd) & 8 != 0, -1.0, 1.0).double() * _exact_decode((c >> 4 * odd) & 7, 2, 1, 1)  # noqa: E731
                k[:, odd::2], v[odd::2] = cut(kd), cut(vd)
            k *= _exact_decode(ks.reshape(-1, d // 16), 4, 3, 7).repeat_interleave(16, 1) * 2.0 ** case["exp"]
            v *= _exact_decode(vs.reshape(-1, d // 16, PAGE).transpose(1, 2).reshape(-1, d // 16), 4, 3, 7).repeat_interleave(16, 1) * 2.0 ** case["exp"]
            for i in range(h * (nq // nkv), (h + 1) * (nq // nkv)):
                s = (st["q"][b, :n, i].double() @ k.T) * d ** -0.5
                s[~see] = -math.inf
                lse[b, :n, i] = torch.logsumexp(s, 1)
                out[b, :n, i] = torch.exp(s - lse[b, :n, i, None]) @ v
    return out, lse


def _exact_logprobs(st, case):
    x = st["logits"].double() / case["T"]
    lp = torch.cat([torch.log_softmax(r, 1) for r in x.split(64)])
    ent = torch.cat([-torch.where(r > -math.inf, r.exp() * r, torch.zeros_like(r)).sum(1) for r in lp.split(64)])
    top = st["logits"].float().sort(dim=1, descending=True, stable=True).indices[:, :case["n_top"]]
    return dict(logprob=lp.gather(1, st["tokens"].long()[:, None]).squeeze(1), entropy=ent, top_ids=None,
                top_logprobs=lp.gather(1, top))
