"""The target's products with 8-bit weights, as measured cases.

Between draft and verification the target runs T = K + 1 rows per request through its layers. `linear` is one
projection of such a layer and `feed_forward` its gated feed-forward half, both with the residual sum and the norm in
front of them where the layer has them there. `run` makes one pass of one of them; with `own` false it computes
the plain form with elementary torch operations.

Numbers in 8 bits: e4m3 codes, 128 columns of a row sharing a scale for activations, 128 x 128 elements for
weights. A weight's scale is any float32. An activation block's is the least 2^e (e >= -126) with max |x| <= 448 2^e, so a code is one
rounding of x 2^-e, to nearest even. Products of codes are summed and scaled in 32 bits.
"""
import math

import torch
import torch.nn.functional as F

own = False

BLOCK = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request decoding one token: the attention's output projection (latency)
        dict(name="linear-one-token", op="linear", B=1, T=1, K=4096, N=4096, dtype="bf16", out="bf16", norm=False, ragged=False),
        # the verification block of 32 requests: sum, norm and the fused query / key / value projection
        dict(name="linear-verify-block", op="linear", B=32, T=8, K=4096, N=6144, dtype="bf16", out="bf16", norm=True, ragged=False),
        # ragged blocks of 16 requests through the smaller target's down projection
        dict(name="linear-ragged", op="linear", B=16, T=8, K=9728, N=2560, dtype="bf16", out="bf16", norm=False, ragged=True),
        # odd sizes, float32 in and out, ragged
        dict(name="linear-odd-f32", op="linear", B=7, T=11, K=1000, N=777, dtype="f32", out="f32", norm=False, ragged=True),
        # one verification block (normed before) against the vocabulary, float32 logits
        dict(name="linear-logits", op="linear", B=1, T=8, K=4096, N=151936, dtype="bf16", out="f32", norm=False, ragged=False),
        # a prompt through the fused query / key / value projection
        dict(name="linear-prompt", op="linear", B=1, T=8192, K=4096, N=6144, dtype="bf16", out="bf16", norm=True, ragged=False),
        # one request decoding one token (latency)
        dict(name="ffn-one-token", op="feed_forward", B=1, T=1, K=4096, F=12288, dtype="bf16", out="bf16", ragged=False),
        # one request's verification block, the smaller target
        dict(name="ffn-one-block", op="feed_forward", B=1, T=8, K=2560, F=9728, dtype="bf16", out="bf16", ragged=False),
        # the verification block of 32 requests
        dict(name="ffn-verify-block", op="feed_forward", B=32, T=8, K=4096, F=12288, dtype="bf16", out="bf16", ragged=False),
        # odd sizes, float32 stream, ragged blocks
        dict(name="ffn-odd-f32", op="feed_forward", B=20, T=17, K=1000, F=2222, dtype="f32", out="bf16", ragged=True),
        # a prompt
        dict(name="ffn-prompt", op="feed_forward", B=1, T=8192, K=4096, F=12288, dtype="bf16", out="bf16", ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "feed_forward"))
    c = dict(op=op, K=_log_int(rng, 64, 8192), dtype=rng.choice(("bf16", "bf16", "f32")), ragged=rng.random() < 0.4)
    # float32 results where the codes are a function of the inputs bit for bit: behind a norm or another product a last bit of 32
    # may move a code, by up to a sixteenth, so that 32 bits of a result mean no more than 16
    if op == "linear":
        c.update(N=_log_int(rng, 64, 32768), norm=rng.random() < 0.5)
        c["out"] = "bf16" if c["norm"] else rng.choice(("bf16", "f32"))
        cost = c["K"] * c["N"]
    else:
        c.update(F=_log_int(rng, 64, 12288), out="bf16")
        cost = 3 * c["K"] * c["F"]
    most = max(1, min(8192, (8192 * 4096 * 6144) // cost))
    rows = _log_int(rng, 1, most)
    c["B"] = min(rows, _log_int(rng, 1, 64))
    c["T"] = max(1, rows // c["B"])
    return c


def _n_rows(case):
    """Valid rows of each request's block (ragged: from none to all T)."""
    T = case["T"]
    return [T if b == 0 or not case["ragged"] else (b * 5) % (T + 1) for b in range(case["B"])]


# ------------------------------------------------------------------ inputs

def _weight(g, N, K):
    """Codes [N, K] (rows on 16 bytes) and scales [N / 128, K / 128] of a random matrix whose columns differ in size."""
    dev = g.device
    codes = torch.zeros(N, -(-K // 16) * 16, dtype=torch.float8_e4m3fn, device=dev)[:, :K]
    scale = torch.empty(-(-N // BLOCK), -(-K // BLOCK), dtype=torch.float32, device=dev)
    for n in range(0, N, 1 << 14):
        m = min(1 << 14, N - n)
        w = torch.randn(m, K, generator=g, device=dev) * K ** -0.5 * torch.exp(0.3 * torch.randn(m, 1, generator=g, device=dev))
        w = F.pad(w, (0, -K % BLOCK, 0, -m % BLOCK)).view(-(-m // BLOCK), BLOCK, -(-K // BLOCK), BLOCK)
        s = w.abs().amax((1, 3)) / 448
        scale[n // BLOCK:n // BLOCK + len(s)] = s
        w = (w / s.clamp(min=1e-30)[:, None, :, None]).clamp(-448, 448).view(-1, scale.shape[1] * BLOCK)[:m, :K]
        codes[n:n + m].copy_(w.to(torch.float8_e4m3fn))
    return codes, scale


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    B, T, K = case["B"], case["T"], case["K"]
    dt = DTYPES[case["dtype"]]
    # activations: channels of different sizes, a few of them far larger
    chan = torch.exp(0.5 * torch.randn(K, generator=g, device=dev))
    chan[torch.randint(0, K, (max(1, K // 500),), generator=g, device=dev)] *= 20
    st = dict(case=case, x=(torch.randn(B, T, K, generator=g, device=dev) * chan).to(dt), n_rows=None)
    if case["ragged"]:
        st["n_rows"] = torch.tensor(_n_rows(case), dtype=torch.int32, device=dev)
    if case.get("norm", True):
        st["residual"] = (3 * torch.randn(B, T, K, generator=g, device=dev)).to(dt)
        st["gain"] = (1 + 0.2 * torch.randn(K, generator=g, device=dev)).to(dt)
        st["total"] = torch.zeros(B, T, K, dtype=dt, device=dev)
    if case["op"] == "linear":
        st["w"] = _weight(g, case["N"], K)
        cols = case["N"]
    else:
        st["wg"], st["wu"], st["wd"] = _weight(g, case["F"], K), _weight(g, case["F"], K), _weight(g, K, case["F"])
        cols = K
    st["out"] = torch.zeros(B, T, cols, dtype=DTYPES[case["out"]], device=dev)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return globals()["_%s_%s" % ("own" if own else "plain", st["case"]["op"])](st)


def _own_quantise(st):
    from history_free_speculative_gb300 import binding
    if "gain" not in st:
        return binding.fp8_quantise(st["x"], n_rows=st["n_rows"])
    return binding.fp8_quantise(st["x"], gain=st["gain"], eps=EPS, residual=st["residual"], total=st["total"], n_rows=st["n_rows"])


def _answer(st):
    return dict(out=st["out"], total=st["total"]) if "total" in st else dict(out=st["out"])


def _own_linear(st):
    from history_free_speculative_gb300 import binding
    codes, scale = _own_quantise(st)
    binding.fp8_linear(codes, scale, *st["w"], n_rows=st["n_rows"], out=st["out"])
    return _answer(st)


def _own_feed_forward(st):
    from history_free_speculative_gb300 import binding
    codes, scale = _own_quantise(st)
    codes, scale = binding.fp8_gated(codes, scale, *st["wg"], *st["wu"], n_rows=st["n_rows"])
    binding.fp8_linear(codes, scale, *st["wd"], n_rows=st["n_rows"], out=st["out"])
    return _answer(st)


def _valid(st):
    c = st["case"]
    t = torch.arange(c["T"], device=st["x"].device).expand(c["B"], -1)
    return (t >= 0 if st["n_rows"] is None else t < st["n_rows"][:, None])[..., None]


def _coded(x):
    """float32 x [..., K] as the values its 8-bit codes stand for."""
    K = x.shape[-1]
    y = F.pad(x, (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(y.abs().amax(-1, keepdim=True))       # amax = m 2^e, 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875)).clamp(min=-126)
    y = torch.ldexp(torch.ldexp(y, -e).to(torch.float8_e4m3fn).float(), e)
    return y.flatten(-2)[..., :K]


def _normed(st):
    """The residual sum, kept in the stream's type, and its norm; without a norm x as it comes."""
    x = st["x"].float()
    if "gain" not in st:
        return x
    total = (x + st["residual"].float()).to(st["x"].dtype)
    st["total"].copy_(torch.where(_valid(st), total, st["total"]))
    x = total.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["gain"].float()


def _product(x, w):
    codes, scale = w
    N, K = codes.shape
    full = scale.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return torch.matmul(x, (codes.float() * full).T)


def _finish(st, y):
    st["out"].copy_(torch.where(_valid(st), y.to(st["out"].dtype), st["out"]))
    return _answer(st)


def _plain_linear(st):
    return _finish(st, _product(_coded(_normed(st)), st["w"]))


def _plain_feed_forward(st):
    x = _coded(_normed(st))
    gate, up = _product(x, st["wg"]), _product(x, st["wu"])
    return _finish(st, _product(_coded(gate / (1 + torch.exp(-gate)) * up), st["wd"]))


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    n, K = sum(_n_rows(case)), case["K"]
    b, o = (2 if case[k] == "bf16" else 4 for k in ("dtype", "out"))
    by = n * K * b + (2 * n * K * b + K * b if case.get("norm", True) else 0)
    if case["op"] == "linear":
        N = case["N"]
        return dict(bytes=by + N * K + n * N * o, flops=2 * n * N * K)
    return dict(bytes=by + 3 * K * case["F"] + n * K * o, flops=6 * n * K * case["F"])


# ------------------------------------------------------------------ the definition, in 64 bits

def _grid(x):
    """The nearest numbers of the format, by its grid: eight steps between powers of two, steps of 2^-9 below 2^-6."""
    rows, K = x.shape
    out = torch.empty_like(x)
    for c in range(0, K, BLOCK):
        y = x[:, c:c + BLOCK]
        top = y.abs().amax(1, keepdim=True)
        s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -118) / 448)).clamp(min=-126))
        s = torch.where(top > 448 * s, 2 * s, torch.where((top <= 224 * s) & (s > 2.0 ** -126), s / 2, s))
        q = y / s
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, c:c + BLOCK] = torch.round(q / step) * step * s
    return out


def _wide(w):
    """A weight in 64 bits, a slice of its rows at a time."""
    codes, scale = w
    for n in range(0, codes.shape[0], 64 * BLOCK):
        c = codes[n:n + 64 * BLOCK].float().double()
        for i in range(0, c.shape[0], BLOCK):
            c[i:i + BLOCK] *= scale[(n + i) // BLOCK].double().repeat_interleave(BLOCK)[:c.shape[1]]
        yield c


def _times(x, w):
    return torch.cat([x @ c.T for c in _wide(w)], 1)


def exact(case, seed):
    st = prepare(case, seed)
    rows = torch.cat([torch.arange(n, device="cuda") + b * case["T"] for b, n in enumerate(_n_rows(case))])
    x, ans = st["x"].flatten(0, 1)[rows].double(), {}
    if "gain" in st:
        x = (x + st["residual"].flatten(0, 1)[rows].double()).to(DTYPES[case["dtype"]]).double()
        ans["total"] = torch.zeros(case["B"] * case["T"], case["K"], dtype=torch.float64, device="cuda")
        ans["total"][rows] = x
        ans["total"] = ans["total"].view(st["x"].shape)
        x = x / (x.pow(2).sum(1, keepdim=True) / case["K"] + EPS).sqrt() * st["gain"].double()
    x = _grid(x)
    if case["op"] == "feed_forward":
        g = _times(x, st["wg"])
        x = _grid(g * torch.sigmoid(g) * _times(x, st["wu"]))
    y = _times(x, st["w"] if case["op"] == "linear" else st["wd"])
    ans["out"] = torch.zeros(case["B"] * case["T"], y.shape[1], dtype=torch.float64, device="cuda")
    ans["out"][rows] = y
    ans["out"] = ans["out"].view(st["out"].shape)
    return ans
