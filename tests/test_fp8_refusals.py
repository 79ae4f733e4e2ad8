"""Refusals of the products with 8-bit weights: argument errors come back before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from history_free_speculative_gb300 import binding, build

INVALID, SHAPE = -1, -2
P = 4096      # an aligned address nothing reads
FAR = (1 << 32) + 5
NAN, INF = float("nan"), float("inf")
X = dict(B=2, T=3, K=200, codes=P, codes_stride=208, scale=P)
CALLS = {
    "dlite_fp8_quantise": (binding.Fp8QuantiseArgs, dict(X, dtype=1, x=P, x_stride=200, eps=1e-6)),
    "dlite_fp8_weight": (binding.Fp8WeightArgs, dict(N=300, K=200, dtype=1, w=P, w_stride=200, codes=P, codes_stride=208, scale=P)),
    "dlite_fp8_linear": (binding.Fp8LinearArgs, dict(X, N=300, dtype=1, w=P, w_stride=208, w_scale=P, out=P, out_stride=300)),
    "dlite_fp8_gated": (binding.Fp8GatedArgs, dict(X, F=300, gate=P, gate_stride=208, gate_scale=P, up=P, up_stride=208, up_scale=P, out_codes=P,
                                                   out_stride=304, out_scale=P)),
}
ROWS = [({"B": 0}, INVALID), ({"T": -1}, INVALID), ({"K": 0}, INVALID), ({"codes": None}, INVALID), ({"scale": None}, INVALID),
        ({"codes_stride": 192}, INVALID), ({"codes_stride": 200}, INVALID), ({"codes": P + 8}, INVALID), ({"K": (1 << 20) + 1, "codes_stride": 1 << 21,
                                                                                                         "w_stride": 1 << 21, "x_stride": 1 << 21, "gate_stride": 1 << 21, "up_stride": 1 << 21}, SHAPE)]
BAD = {
    "dlite_fp8_quantise": ROWS + [({"x": None}, INVALID), ({"dtype": 2}, INVALID), ({"x_stride": 199}, INVALID), ({"residual": P}, INVALID),
                                  ({"total": P}, INVALID), ({"residual": P, "total": P + 4096, "residual_stride": 199, "total_stride": 200}, INVALID),
                                  ({"residual": P, "total": P + 4096, "residual_stride": 200, "total_stride": 0}, INVALID),
                                  ({"residual": P + 4096, "total": P + 4096, "residual_stride": 200, "total_stride": 208}, INVALID),
                                  ({"residual": P + 4096, "total": P, "residual_stride": 200, "total_stride": 208}, INVALID),
                                  ({"gain": P, "eps": -1.0}, INVALID), ({"gain": P, "eps": NAN}, INVALID), ({"gain": P, "eps": INF}, INVALID),
                                  ({"B": 1 << 30, "T": 4}, SHAPE), ({"B": 1, "T": (1 << 31) - 1}, SHAPE), ({"B": (1 << 22) + 1, "T": 1}, SHAPE)],
    "dlite_fp8_weight": [({"N": 0}, INVALID), ({"K": 0}, INVALID), ({"w": None}, INVALID), ({"codes": None}, INVALID), ({"scale": None}, INVALID),
                         ({"dtype": -1}, INVALID), ({"w_stride": 199}, INVALID), ({"codes_stride": 200}, INVALID), ({"codes_stride": 192}, INVALID),
                         ({"N": (1 << 22) + 1}, SHAPE), ({"K": (1 << 20) + 1, "w_stride": 1 << 21, "codes_stride": 1 << 21}, SHAPE)],
    "dlite_fp8_linear": ROWS + [({"w": None}, INVALID), ({"w_scale": None}, INVALID), ({"out": None}, INVALID), ({"N": 0}, INVALID), ({"dtype": 2}, INVALID),
                                ({"w_stride": 200}, INVALID), ({"w_stride": 192}, INVALID), ({"out_stride": 299}, INVALID),
                                ({"N": (1 << 22) + 1, "out_stride": 1 << 23}, SHAPE), ({"B": 1 << 20, "T": 5}, SHAPE), ({"w_stride": 1 << 40}, SHAPE),
                                ({"codes_stride": 1 << 40}, SHAPE)],
    "dlite_fp8_gated": ROWS + [({n: None}, INVALID) for n in ("gate", "gate_scale", "up", "up_scale", "out_codes", "out_scale")] +
                       [({"F": 0}, INVALID), ({"gate_stride": 200}, INVALID), ({"up_stride": 192}, INVALID), ({"out_stride": 288}, INVALID),
                        ({"out_stride": 300}, INVALID), ({"F": (1 << 22) + 1, "out_stride": 1 << 23}, SHAPE), ({"B": 1 << 22, "T": 2}, SHAPE)],
}
POINTERS = {      # pointer fields and what they are aligned to
    "dlite_fp8_quantise": dict(x=2, residual=2, total=2, gain=2, codes=16, scale=4, n_rows=4, status=4),
    "dlite_fp8_weight": dict(w=2, codes=16, scale=4, status=4),
    "dlite_fp8_linear": dict(codes=16, scale=4, w=16, w_scale=4, out=2, n_rows=4, status=4),
    "dlite_fp8_gated": dict(codes=16, scale=4, gate=16, gate_scale=4, up=16, up_scale=4, out_codes=16, out_scale=4, n_rows=4, status=4),
}


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("name,change,code", [(n, c, k) for n, l in BAD.items() for c, k in l], ids=str)
def test_bad_arguments(lib, name, change, code):
    cls, good = CALLS[name]
    fields = {n for n, _ in cls._fields_}
    a = cls(**dict(good, **{n: v for n, v in change.items() if n in fields}))
    assert getattr(lib, name)(ctypes.byref(a), None) == code
    assert getattr(lib, name)(None, None) == INVALID


@pytest.mark.parametrize("name,field,size", [(n, f, s) for n, d in POINTERS.items() for f, s in d.items()])
def test_misaligned_pointers(lib, name, field, size):
    cls, good = CALLS[name]
    assert set(POINTERS[name]) == {n for n, t in cls._fields_ if t is ctypes.c_void_p}
    kw = dict(good, **{field: P + size // 2})
    if field in ("residual", "total"):
        kw = dict(kw, residual_stride=200, total_stride=200, **{"total" if field == "residual" else "residual": P})
    assert getattr(lib, name)(ctypes.byref(cls(**kw)), None) == INVALID


# ---------------------------------------------------------------- the binding

@pytest.fixture
def closed(monkeypatch):
    """Tensors that stand for device tensors; no call may reach the library."""
    class Closed:
        def __getattr__(self, name):
            raise AssertionError(f"{name} reached")

    monkeypatch.setattr(binding, "load", lambda: Closed())
    monkeypatch.setattr(binding, "_here", lambda stream, *t: (0, None))
    monkeypatch.setattr(binding, "_new", lambda s, shape, dtype, zero=False: torch.empty(shape, dtype=dtype, device="meta"))
    monkeypatch.setattr(binding, "_new_strided", lambda s, shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype, device="meta"))


def _codes(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="meta").view(torch.float8_e4m3fn)


def _far(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda: binding.fp8_quantise(_far(1, FAR, 8)), lambda: binding.fp8_quantise(_far(1, 1, FAR)), lambda: binding.fp8_weight(_far(FAR, 8)),
    lambda: binding.fp8_weight(_far(8, FAR)), lambda: binding.fp8_linear(_codes(1, FAR, 16), _far(1, FAR, 1), _codes(8, 16), _far(1, 1)),
    lambda: binding.fp8_linear(_codes(1, 1, 16), _far(1, 1, 1), _codes(FAR, 16), _far(-(-FAR // 128), 1)),
    lambda: binding.fp8_gated(_codes(1, 1, 16), _far(1, 1, 1), _codes(FAR, 16), _far(-(-FAR // 128), 1), _codes(FAR, 16), _far(-(-FAR // 128), 1)),
], ids=range(7))
def test_sizes_outside_32_bits(closed, call):
    with pytest.raises(ValueError, match="outside 32 bits"):
        call()


def test_the_bindings_checks(closed):
    x, c, s, w, ws = _far(2, 3, 160), _codes(2, 3, 160), torch.empty_strided((2, 3, 2), (3, 1, 6), device="meta"), _codes(50, 160), _far(1, 2)
    bad = [
        lambda: binding.fp8_quantise(x[0]), lambda: binding.fp8_quantise(x[:, :2]), lambda: binding.fp8_quantise(x[..., ::2]),
        lambda: binding.fp8_quantise(x.to(torch.float16)), lambda: binding.fp8_quantise(x, total=x), lambda: binding.fp8_quantise(x, residual=x[:, :1]),
        lambda: binding.fp8_quantise(x, residual=x.bfloat16()), lambda: binding.fp8_quantise(x, gain=x[0, 0, :100]),
        lambda: binding.fp8_quantise(x, gain=x[0, 0].bfloat16()), lambda: binding.fp8_quantise(x, codes=c[..., :100]),
        lambda: binding.fp8_quantise(x, codes=x), lambda: binding.fp8_quantise(x, scale=s[..., :1]), lambda: binding.fp8_quantise(x, scale=s.double()),
        lambda: binding.fp8_quantise(x, scale=_far(2, 3, 2)), lambda: binding.fp8_linear(c, _far(2, 3, 2), w, ws),
        lambda: binding.fp8_quantise(x, n_rows=torch.zeros(3, dtype=torch.int32)), lambda: binding.fp8_quantise(x, n_rows=torch.zeros(2)),
        lambda: binding.fp8_quantise(x[:1].expand(2, 3, 160)),
        lambda: binding.fp8_weight(x), lambda: binding.fp8_weight(x[0].t()), lambda: binding.fp8_weight(x[0].double()),
        lambda: binding.fp8_linear(x, s, w, ws), lambda: binding.fp8_linear(c, s, w[:, :100], ws), lambda: binding.fp8_linear(c, s, x[0, :, :160], ws),
        lambda: binding.fp8_linear(c, s[..., :1], w, ws), lambda: binding.fp8_linear(c, s, w, ws[:, :1]), lambda: binding.fp8_linear(c, s, w, ws, out=_far(2, 3, 49)),
        lambda: binding.fp8_linear(c, s, w, ws, out=_far(2, 3, 50).double()), lambda: binding.fp8_linear(c, s, w, ws, out=_far(2, 50, 3).transpose(1, 2)),
        lambda: binding.fp8_linear(c, s, w, ws, dtype=torch.float16),
        lambda: binding.fp8_gated(c, s, w, ws, w[:49], ws), lambda: binding.fp8_gated(c, s, w, ws, w, ws, out=_codes(2, 3, 49)),
        lambda: binding.fp8_gated(c, s, w, ws, w, ws, out=_far(2, 3, 50)), lambda: binding.fp8_gated(c, s, w, ws, w, ws, out_scale=s),
        lambda: binding.fp8_gated(c, s, w, ws, w, ws.double()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")


def test_the_binding_wants_device_tensors():
    x, c = torch.zeros(1, 1, 128), torch.zeros(1, 1, 128).to(torch.float8_e4m3fn)
    s = torch.zeros(1, 1, 1)
    for call in (lambda: binding.fp8_quantise(x), lambda: binding.fp8_weight(x[0]), lambda: binding.fp8_linear(c, s, c[0], s[0]),
                 lambda: binding.fp8_gated(c, s, c[0], s[0], c[0], s[0])):
        with pytest.raises(ValueError):
            call()
