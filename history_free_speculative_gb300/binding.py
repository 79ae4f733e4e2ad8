"""Thin ctypes binding of libdlite.so (argument marshalling only).

Every step of the round runs in the CUDA library; this module only turns
torch tensors into device pointers and checks return codes. It fails loudly
when the library is missing: there is no fallback path.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libdlite.so")

DLITE_F32, DLITE_BF16 = 0, 1
MAX_LAYERS = 8

STATUS = {
    0: "ok", -1: "invalid argument", -2: "unsupported shape", -3: "CUDA runtime error",
    -4: "device wait timed out", -5: "id out of range on the device", -6: "device allocation failed",
}


class DliteError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({code})")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("B_max", "D", "m", "K", "L_D", "n_q", "n_kv", "d_h", "F", "R", "V", "dtype")] + \
               [("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float), ("anchor_group", ctypes.c_int),
                ("head_type", ctypes.c_int), ("history", ctypes.c_int), ("act_planes", ctypes.c_int),
                ("head_warmup", ctypes.c_int)]


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("g_attn", "Wq", "Wk", "Wv", "Wo", "g_ffn", "Wg", "Wu", "Wd")]


GATED_FIELDS = ("E_R", "W_s", "b_s", "W_h", "b_h", "W_o")


class GatedWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in GATED_FIELDS]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("e_depth", "g_stage", "e_ph", "E", "g_final", "Q", "P")] + \
               [("layer", LayerWeights * MAX_LAYERS), ("gated", GatedWeights)]


VERIFY_GREEDY, VERIFY_SAMPLE, VERIFY_MATCH = 0, 1, 2


class VerifyArgs(ctypes.Structure):
    """dlite_verify_args (include/dlite.h)."""
    _fields_ = [("mode", ctypes.c_int), ("B", ctypes.c_int), ("n_verify", ctypes.c_int),
                ("candidates", ctypes.c_void_p), ("target_tokens", ctypes.c_void_p),
                ("qstats", ctypes.c_void_p), ("hs", ctypes.c_void_p), ("target_probs", ctypes.c_void_p),
                ("temperature", ctypes.c_float), ("seed", ctypes.c_uint64), ("pos", ctypes.c_void_p),
                ("accepted", ctypes.c_void_p), ("commits", ctypes.c_void_p), ("n_commit", ctypes.c_void_p),
                ("next_anchor", ctypes.c_void_p)]


ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}
KV_PAGE = 64
DEV_TIMEOUT, DEV_BOUNDS, DEV_NONFINITE = 1, 2, 4


class RopeConfig(ctypes.Structure):
    """dlite_rope_config (include/dlite.h)."""
    _fields_ = [("rot", ctypes.c_int), ("scaling", ctypes.c_int)] + \
               [(n, ctypes.c_double) for n in ("theta", "factor", "orig_len", "beta_fast", "beta_slow", "attn_factor")]


class RopeArgs(ctypes.Structure):
    """dlite_rope_args."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "heads", "d_h", "rot", "layout", "dtype", "n_pos")] + \
               [("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("pos", ctypes.c_void_p), ("n_rows", ctypes.c_void_p), ("table", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class KvCacheDesc(ctypes.Structure):
    """dlite_kv_cache."""
    _fields_ = [("pages", ctypes.c_void_p), ("block_table", ctypes.c_void_p)] + \
               [(n, ctypes.c_int) for n in ("n_pages", "n_kv", "d_h", "max_pages", "k_exp", "v_exp")]


class KvAppendArgs(ctypes.Structure):
    """dlite_kv_append_args."""
    _fields_ = [("cache", KvCacheDesc)] + [(n, ctypes.c_int) for n in ("B", "T", "dtype", "rot", "layout", "n_pos")] + \
               [("k", ctypes.c_void_p), ("k_stride", ctypes.c_int64), ("v", ctypes.c_void_p), ("v_stride", ctypes.c_int64),
                ("pos", ctypes.c_void_p), ("n_rows", ctypes.c_void_p), ("table", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class KvReadArgs(ctypes.Structure):
    """dlite_kv_read_args."""
    _fields_ = [("cache", KvCacheDesc)] + [(n, ctypes.c_int) for n in ("B", "T", "dtype")] + \
               [("k_out", ctypes.c_void_p), ("k_stride", ctypes.c_int64), ("v_out", ctypes.c_void_p), ("v_stride", ctypes.c_int64),
                ("pos", ctypes.c_void_p), ("n_rows", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class KvAttentionArgs(ctypes.Structure):
    """dlite_kv_attention_args."""
    _fields_ = [("cache", KvCacheDesc)] + [(n, ctypes.c_int) for n in ("B", "T", "n_q", "dtype", "window")] + \
               [("scale", ctypes.c_float), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64), ("lse", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("n_rows", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p)]


class LogprobsArgs(ctypes.Structure):
    """dlite_logprobs_args."""
    _fields_ = [(n, ctypes.c_int) for n in ("rows", "V", "n_top", "dtype")] + \
               [("temperature", ctypes.c_float), ("logits", ctypes.c_void_p), ("stride", ctypes.c_int64)] + \
               [(n, ctypes.c_void_p) for n in ("tokens", "logprob", "entropy", "top_ids", "top_logprobs", "status")]


class Fp8QuantiseArgs(ctypes.Structure):
    """dlite_fp8_quantise_args."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "K", "dtype")] + \
               [("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64),
                ("total", ctypes.c_void_p), ("total_stride", ctypes.c_int64), ("gain", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("codes", ctypes.c_void_p), ("codes_stride", ctypes.c_int64), ("scale", ctypes.c_void_p), ("n_rows", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class Fp8WeightArgs(ctypes.Structure):
    """dlite_fp8_weight_args."""
    _fields_ = [(n, ctypes.c_int) for n in ("N", "K", "dtype")] + \
               [("w", ctypes.c_void_p), ("w_stride", ctypes.c_int64), ("codes", ctypes.c_void_p), ("codes_stride", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class Fp8LinearArgs(ctypes.Structure):
    """dlite_fp8_linear_args."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "K", "N", "dtype")] + \
               [("codes", ctypes.c_void_p), ("codes_stride", ctypes.c_int64), ("scale", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("w_stride", ctypes.c_int64), ("w_scale", ctypes.c_void_p), ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("n_rows", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class Fp8GatedArgs(ctypes.Structure):
    """dlite_fp8_gated_args."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "K", "F")] + \
               [("codes", ctypes.c_void_p), ("codes_stride", ctypes.c_int64), ("scale", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_stride", ctypes.c_int64), ("gate_scale", ctypes.c_void_p), ("up", ctypes.c_void_p), ("up_stride", ctypes.c_int64),
                ("up_scale", ctypes.c_void_p), ("out_codes", ctypes.c_void_p), ("out_stride", ctypes.c_int64), ("out_scale", ctypes.c_void_p),
                ("n_rows", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class Taps(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("z", "x", "b", "hs")]


_lib = None

# name -> (restype, argtypes)
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_U64 = ctypes.c_uint64
_SIGS = {
    "dlite_create": (_I, [ctypes.POINTER(Config), ctypes.POINTER(Weights), ctypes.POINTER(_P)]),
    "dlite_destroy": (None, [_P]),
    "dlite_draft_round": (_I, [_P, _I, _P, _P, _F, _U64, _P, _P, _P, _P]),
    "dlite_draft_round_taps": (_I, [_P, _I, _P, _P, _F, _U64, _P, _P, _P, ctypes.POINTER(Taps), _P]),
    "dlite_backbone": (_I, [_P, _I, _P, _P, _P, _P]),
    "dlite_seq_head": (_I, [_P, _I, _P, _P, _P]),
    "dlite_lm_head": (_I, [_P, _I, _P, _F, _U64, _P, _P, _P, _P]),
    "dlite_verify": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _P]),
    "dlite_verify_sample": (_I, [_P, _I, _P, _P, _P, _P, _F, _U64, _P, _P, _P, _P, _P, _P]),
    "dlite_verify_ex": (_I, [_P, ctypes.POINTER(VerifyArgs), _P]),
    "dlite_advance": (_I, [_P, _I, _P, _P, _P]),
    "dlite_shift_group": (_I, [_P, _I, _P, _P, _P, _P]),
    "dlite_history_reset": (_I, [_P, _P]),
    "dlite_history_read": (_I, [_P, _I, _I, _I, _P, ctypes.POINTER(ctypes.c_int32), _P]),
    "dlite_verify_sample_static": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _F, _U64, _P, _P, _P,
                                        _P, _P, _P]),
    "dlite_round_host": (_I, [_P, _I, _P, _P, _P, _P, _P, _F, _U64, _P, _P, _P, _P, _P]),
    "dlite_synthetic_target": (_I, [_I, _I, _I, _P, _P, _I, _P, _U64, _P, _P, _P]),
    "dlite_rope_table": (_I, [ctypes.POINTER(RopeConfig), _I, _P, _P]),
    "dlite_rope": (_I, [ctypes.POINTER(RopeArgs), _P]),
    "dlite_kv_append": (_I, [ctypes.POINTER(KvAppendArgs), _P]),
    "dlite_kv_read": (_I, [ctypes.POINTER(KvReadArgs), _P]),
    "dlite_kv_attention_workspace": (ctypes.c_size_t, [ctypes.POINTER(KvAttentionArgs)]),
    "dlite_kv_attention": (_I, [ctypes.POINTER(KvAttentionArgs), _P]),
    "dlite_token_logprobs": (_I, [ctypes.POINTER(LogprobsArgs), _P]),
    "dlite_fp8_quantise": (_I, [ctypes.POINTER(Fp8QuantiseArgs), _P]),
    "dlite_fp8_weight": (_I, [ctypes.POINTER(Fp8WeightArgs), _P]),
    "dlite_fp8_linear": (_I, [ctypes.POINTER(Fp8LinearArgs), _P]),
    "dlite_fp8_gated": (_I, [ctypes.POINTER(Fp8GatedArgs), _P]),
    "dlite_selftest_wait": (_I, [_P, _U64, _P, _P]),
    "dlite_selftest_ring": (_I, [_U64, _P, _P, _P]),
    "dlite_device_status": (_I, [_P, _I, ctypes.POINTER(_I), _P]),
    "dlite_status_string": (ctypes.c_char_p, [_I]),
    "dlite_last_cuda_error": (ctypes.c_char_p, []),
    "dlite_launch_count": (_I, [_P, _I, _F]),
    "dlite_counters": (_I, [_P, _I, ctypes.POINTER(ctypes.c_int64), _P]),
    "dlite_selftest_gemm": (_I, [_I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P,
                                 ctypes.POINTER(ctypes.c_int), _P]),
    "dlite_stage_times": (_I, [_P, _I, _P, _P, _F, _U64, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                               _P, ctypes.POINTER(ctypes.c_char_p), _I, _P]),
}

EXPORTED = tuple(_SIGS)


def load(path=None):
    """Load libdlite.so (built by history_free_speculative_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libdlite.so not built ({path}); run `python -m "
                           "history_free_speculative_gb300.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return ctypes.c_void_p(t.data_ptr())


def _hptr(t):
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("contiguous host tensor expected")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(code, what):
    if code != 0:
        if code == -3 and _lib is not None:   # DLITE_ERR_CUDA: name the runtime error
            what = f"{what} [{_lib.dlite_last_cuda_error().decode()}]"
        raise DliteError(code, what)


def selftest_gemm(X, W, rows=None, stream=None, plan=None, part=None, outs=None):
    """Tensor-core product X[:rows] @ W^T through the round's GEMM engine.

    X, W: lists of 1 or 2 bf16 device planes ([x_rows, K] with x_rows a multiple
    of 128; W in the tiled weight layout, rows padded to 64). Returns
    (fp32 [rows, outs] device tensor, status).
    """
    lib = load()
    rows = X[0].shape[0] if rows is None else rows
    wrows, K = W[0].shape
    outs = wrows if outs is None else outs
    if part is None:
        part = torch.zeros(16 * rows * outs, dtype=torch.float32, device=X[0].device)
    st = torch.zeros(1, dtype=torch.int32, device=X[0].device)
    ov = (ctypes.c_int * 3)(*plan) if plan is not None else None
    S = lib.dlite_selftest_gemm(rows, outs, K, len(X), len(W), _ptr(X[0]),
                                _ptr(X[1]) if len(X) > 1 else None, X[0].shape[0], _ptr(W[0]),
                                _ptr(W[1]) if len(W) > 1 else None, _ptr(part), _ptr(st), ov,
                                _stream(stream))
    if S < 0:
        raise DliteError(S, "dlite_selftest_gemm")
    return part[:S * rows * outs].view(S, rows, outs).sum(0), st


def verify_sample_static(cand, qstats, hs, E, probs, temperature, seed, pos, accepted, commits,
                         n_commit, next_anchor, stream=None):
    """Allocation-free sampling verification (no handle; E float32 row-major [V, D])."""
    lib = load()
    B, K = cand.shape
    V, D = E.shape
    want = ((cand, torch.int32, (B, K)), (qstats, torch.float32, (B, K, 2)), (hs, torch.float32, (B, K, D)),
            (E, torch.float32, (V, D)), (probs, torch.float32, (B, K + 1, V)), (pos, torch.int64, (B,)),
            (accepted, torch.int32, (B,)), (commits, torch.int32, (B, K + 1)), (n_commit, torch.int32, (B,)),
            (next_anchor, torch.int32, (B,)))
    for t, dt, shape in want:
        if t.dtype != dt or tuple(t.shape) != shape:
            raise ValueError(f"verify_sample_static: expected {dt} {shape}, got {t.dtype} {tuple(t.shape)}")
    _check(lib.dlite_verify_sample_static(B, K, V, D, _ptr(cand), _ptr(qstats), _ptr(hs), _ptr(E),
                                          _ptr(probs), temperature, seed, _ptr(pos), _ptr(accepted),
                                          _ptr(commits), _ptr(n_commit), _ptr(next_anchor),
                                          _stream(stream)), "dlite_verify_sample_static")


def synthetic_target(cand, accept_c, seed, pos, target_tokens, V, round_counter=None, stream=None):
    """Synthetic target tokens [B, K+1] (dlite_synthetic_target): accept_c is
    [n_tables, B, K] float32 on the device, round_counter a device int32 (or None)."""
    lib = load()
    B, K = cand.shape
    if accept_c.dtype != torch.float32 or accept_c.dim() != 3 or tuple(accept_c.shape[1:]) != (B, K):
        raise ValueError("accept_c must be float32 [n_tables, B, K]")
    if cand.dtype != torch.int32 or pos.dtype != torch.int64 or target_tokens.dtype != torch.int32:
        raise ValueError("candidates / target_tokens int32, pos int64 expected")
    if tuple(target_tokens.shape) != (B, K + 1) or tuple(pos.shape) != (B,):
        raise ValueError("target_tokens [B, K+1] and pos [B] expected")
    if round_counter is not None and round_counter.dtype != torch.int32:
        raise ValueError("round_counter must be a device int32")
    _check(lib.dlite_synthetic_target(B, K, V, _ptr(cand), _ptr(accept_c), accept_c.shape[0],
                                      _ptr(round_counter), seed, _ptr(pos), _ptr(target_tokens),
                                      _stream(stream)), "dlite_synthetic_target")


# ---------------------------------------------------------------- target-side operators
# (no handle; tensors and stream of the current device; see include/dlite.h)

_DTYPES = {torch.float32: DLITE_F32, torch.bfloat16: DLITE_BF16}


def _dtype(t, what):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: float32 or bfloat16 expected, got {t.dtype}")
    return code


_LEAST, _MOST = -(1 << 31), (1 << 31) - 1      # what a C int holds; of other numbers ctypes would keep the low 32 bits


def _int(v, what):
    if not _LEAST <= v <= _MOST:
        raise ValueError(f"{what}: {v} is outside 32 bits")
    return v


def _sizes(what, *n):
    """Refuses sizes of a tensor that C ints do not hold (called where one of them does not)."""
    raise ValueError(f"{what}: sizes {list(n)} are outside 32 bits")


def _here(stream, *tensors):
    """(pointer, stream or None) of the stream to launch on: None for the current one. Every tensor
    has to be on the current CUDA device."""
    if tensors and tensors[0].get_device() < 0:
        raise ValueError("device tensor expected")
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor on {t.device}, current device cuda:{dev}")
    cur = torch._C._cuda_getCurrentRawStream(dev)   # torch.cuda.current_stream().cuda_stream without the Stream object
    if stream is None or (stream.cuda_stream == cur and stream.device.index == dev):
        return cur, None
    if stream.device.index != dev:
        raise ValueError(f"stream on {stream.device}, current device cuda:{dev}")
    return stream.cuda_stream, stream


def _vec(t, dtype, shape, what):
    """Pointer of a dense tensor of this type and shape (None: a null pointer)."""
    if t is None:
        return None
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous {dtype} {list(shape)} expected, got {t.dtype} {list(t.shape)}")
    return t.data_ptr()


def _row_stride(t, what):
    """Elements between the rows (b, t) of [B, T, H, d]: dense columns, evenly spaced rows."""
    if t.dim() != 4:
        raise ValueError(f"{what}: [B, T, heads, d_h] expected, got {list(t.shape)}")
    B, T, H, d = t.shape
    if (B | T | H | d) >> 31:
        _sizes(what, B, T, H, d)
    sb, st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (H > 1 and sh != d):
        raise ValueError(f"{what}: the heads of a row have to be dense")
    row = st if T > 1 else (sb if B > 1 else H * d)
    if T > 1 and B > 1 and sb != T * st:
        raise ValueError(f"{what}: rows (b, t) have to be evenly spaced")
    if row < H * d:
        raise ValueError(f"{what}: rows overlap")
    return row


def _new(stream, shape, dtype, zero=False):
    """A new tensor that belongs to the stream it is written on (zeros where a call leaves rows out)."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device="cuda")
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device="cuda")


def rope_table(n_pos, rot, theta=1e6, scaling="plain", factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0,
               attn_factor=0.0, stream=None):
    """(cos, sin) of positions 0..n_pos-1, float32 [n_pos, rot / 2, 2] on the current device
    (dlite_rope_table). scaling: "plain", "linear", "ntk" or "yarn"."""
    lib = load()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling: one of {sorted(ROPE_SCALINGS)} expected")
    n_pos, rot = _int(int(n_pos), "n_pos"), _int(int(rot), "rot")
    ptr, s = _here(stream)
    table = _new(s, (max(n_pos, 0), max(rot, 0) // 2, 2), torch.float32)
    cfg = RopeConfig(rot, ROPE_SCALINGS[scaling], theta, factor, orig_len, beta_fast, beta_slow, attn_factor)
    _check(lib.dlite_rope_table(ctypes.byref(cfg), n_pos, table.data_ptr() or None, ptr), "dlite_rope_table")
    return table


def _table(table, layout):
    """(rotated columns, layout code, positions) of a rope_table."""
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout: one of {sorted(ROPE_LAYOUTS)} expected")
    if table.dtype != torch.float32 or table.dim() != 3 or table.shape[2] != 2 or not table.is_contiguous():
        raise ValueError("table: contiguous float32 [n_pos, rot / 2, 2] expected")
    n_pos, half, _ = table.shape
    if (n_pos | 2 * half) >> 31:
        _sizes("table", n_pos, 2 * half)
    return 2 * half, ROPE_LAYOUTS[layout], n_pos


def rope(x, pos, table, layout="half", n_rows=None, out=None, status=None, stream=None):
    """x [B, T, heads, d_h] with the first columns of every head rotated by the angles of
    position pos[b] + t (dlite_rope). out: None (a new tensor), x itself, or another tensor of
    x's shape; rows t >= n_rows[b] of it are left as they were (zeros in a new one). Returns out."""
    lib = load()
    ptr, s = _here(stream, x, pos, table, n_rows, out, status)
    xs = _row_stride(x, "x")
    B, T, H, d = x.shape
    if out is None:
        out = _new(s, x.shape, x.dtype, zero=n_rows is not None)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out: x's shape and type expected")
    rot, lay, n_pos = _table(table, layout)
    a = RopeArgs(B, T, H, d, rot, lay, _dtype(x, "x"), n_pos, x.data_ptr(), xs, out.data_ptr(), _row_stride(out, "out"),
                 _vec(pos, torch.int64, (B,), "pos"), _vec(n_rows, torch.int32, (B,), "n_rows"), table.data_ptr(),
                 _vec(status, torch.int32, (1,), "status"))
    _check(lib.dlite_rope(ctypes.byref(a), ptr), "dlite_rope")
    return out


def kv_pages(n_pages, n_kv, d_h, device="cuda"):
    """Memory of a paged 4-bit cache: uint8 [n_pages, n_kv, 72 d_h], one record of 64 tokens per
    (page, head). The zeros it starts with stand for zero keys and values."""
    return torch.zeros(n_pages, n_kv, 72 * d_h, dtype=torch.uint8, device=device)


def _kv_desc(pages, block_table, B, k_exp, v_exp):
    if pages.dtype != torch.uint8 or pages.dim() != 3 or not pages.is_contiguous():
        raise ValueError("pages: contiguous uint8 [n_pages, n_kv, 72 d_h] expected")
    n_pages, n_kv, rec = pages.shape
    if rec % 72:
        raise ValueError("pages: records of 72 d_h bytes expected")
    if block_table.dim() != 2:
        raise ValueError("block_table: int32 [B, max_pages] expected")
    max_pages = block_table.shape[1]
    bt = _vec(block_table, torch.int32, (B, max_pages), "block_table")
    if (n_pages | n_kv | rec | max_pages) >> 31:
        _sizes("pages, block_table", n_pages, n_kv, rec, max_pages)
    if not (_LEAST <= k_exp <= _MOST and _LEAST <= v_exp <= _MOST):
        _int(k_exp, "k_exp"), _int(v_exp, "v_exp")
    return KvCacheDesc(pages.data_ptr(), bt, n_pages, n_kv, rec // 72, max_pages, k_exp, v_exp)


def kv_append(pages, block_table, k, v, pos, table=None, layout="half", n_rows=None, k_exp=0, v_exp=0, status=None, stream=None):
    """Append k, v [B, T, n_kv, d_h] to the cache at positions pos[b] + t, the keys rotated on
    the way when a rope_table is given (dlite_kv_append). block_table is int32 [B, max_pages]."""
    lib = load()
    ptr, s = _here(stream, pages, block_table, k, v, pos, table, n_rows, status)
    ks, vs = _row_stride(k, "k"), _row_stride(v, "v")
    B, T, H, d = k.shape
    desc = _kv_desc(pages, block_table, B, k_exp, v_exp)
    if v.shape != k.shape or v.dtype != k.dtype or H != desc.n_kv or d != desc.d_h:
        raise ValueError("k, v: [B, T, n_kv, d_h] of the cache's heads and one type expected")
    rot, lay, n_pos = _table(table, layout) if table is not None else (0, 0, 0)
    a = KvAppendArgs(desc, B, T, _dtype(k, "k"), rot, lay, n_pos, k.data_ptr(), ks, v.data_ptr(), vs,
                     _vec(pos, torch.int64, (B,), "pos"), _vec(n_rows, torch.int32, (B,), "n_rows"),
                     table.data_ptr() if table is not None else None, _vec(status, torch.int32, (1,), "status"))
    _check(lib.dlite_kv_append(ctypes.byref(a), ptr), "dlite_kv_append")


def kv_read(pages, block_table, pos, T, n_rows=None, k_exp=0, v_exp=0, dtype=torch.bfloat16, k_out=None, v_out=None,
            status=None, stream=None):
    """The values the cache holds at positions pos[b] + t, t < T: (k, v) [B, T, n_kv, d_h]
    (dlite_kv_read). New outputs start as zeros where rows are not read."""
    lib = load()
    ptr, s = _here(stream, pages, block_table, pos, n_rows, k_out, v_out, status)
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out: both or neither expected")
    B = block_table.shape[0]
    desc = _kv_desc(pages, block_table, B, k_exp, v_exp)
    if not _LEAST <= T <= _MOST:
        _int(T, "T")
    shape = (B, T, desc.n_kv, desc.d_h)
    if k_out is None:
        k_out, v_out = (_new(s, shape, dtype, zero=True) for _ in range(2))
    elif tuple(k_out.shape) != shape or tuple(v_out.shape) != shape or v_out.dtype != k_out.dtype:
        raise ValueError(f"k_out, v_out: {list(shape)} of one type expected")
    a = KvReadArgs(desc, B, T, _dtype(k_out, "k_out"), k_out.data_ptr(), _row_stride(k_out, "k_out"), v_out.data_ptr(),
                   _row_stride(v_out, "v_out"), _vec(pos, torch.int64, (B,), "pos"), _vec(n_rows, torch.int32, (B,), "n_rows"),
                   _vec(status, torch.int32, (1,), "status"))
    _check(lib.dlite_kv_read(ctypes.byref(a), ptr), "dlite_kv_read")
    return k_out, v_out


def kv_attention(q, pages, block_table, pos, scale=None, window=0, n_rows=None, k_exp=0, v_exp=0, out=None, lse=None,
                 workspace=None, status=None, stream=None):
    """Attention of q [B, T, n_q, d_h] (rows at positions pos[b] + t, their keys already
    appended) over the cache (dlite_kv_attention); scale None: d_h^-1/2. lse: None (not wanted), True (a new
    tensor) or float32 [B, T, n_q]. workspace: None (a new one for this call) or a uint8 tensor of at least
    kv_attention_workspace(...) bytes. Returns (out, lse); rows t >= n_rows[b] are left as
    they were (zeros in new outputs)."""
    lib = load()
    ptr, s = _here(stream, q, pages, block_table, pos, n_rows, out, None if lse is True else lse, workspace, status)
    qs = _row_stride(q, "q")
    B, T, H, d = q.shape
    desc = _kv_desc(pages, block_table, B, k_exp, v_exp)
    if d != desc.d_h:
        raise ValueError(f"q: heads of {desc.d_h} columns expected")
    if out is None:
        out = _new(s, q.shape, q.dtype, zero=n_rows is not None)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out: q's shape and type expected")
    if lse is True:
        lse = _new(s, (B, T, H), torch.float32, zero=n_rows is not None)
    if not _LEAST <= window <= _MOST:
        _int(window, "window")
    a = KvAttentionArgs(desc, B, T, H, _dtype(q, "q"), window, d ** -0.5 if scale is None else scale, q.data_ptr(), qs,
                        out.data_ptr(), _row_stride(out, "out"), _vec(lse, torch.float32, (B, T, H), "lse"),
                        _vec(pos, torch.int64, (B,), "pos"), _vec(n_rows, torch.int32, (B,), "n_rows"), None, 0,
                        _vec(status, torch.int32, (1,), "status"))
    need = lib.dlite_kv_attention_workspace(ctypes.byref(a))
    if need:
        if workspace is None:
            workspace = _new(s, (need,), torch.uint8)
        elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace: contiguous uint8 expected")
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(lib.dlite_kv_attention(ctypes.byref(a), ptr), "dlite_kv_attention")
    return out, lse


def kv_attention_workspace(B, T, n_q, n_kv, d_h, max_pages, dtype=torch.bfloat16):
    """Bytes of workspace a kv_attention call of these sizes needs on the current device (0: none)."""
    for n, what in ((B, "B"), (T, "T"), (n_q, "n_q"), (n_kv, "n_kv"), (d_h, "d_h"), (max_pages, "max_pages")):
        _int(n, what)
    a = KvAttentionArgs(KvCacheDesc(16, 16, 1, n_kv, d_h, max_pages, 0, 0), B, T, n_q, _DTYPES[dtype], 0, 1.0, 16, n_q * d_h,
                        16, n_q * d_h, None, 16, None, None, 0, None)
    return load().dlite_kv_attention_workspace(ctypes.byref(a))


def token_logprobs(logits, tokens, temperature=1.0, n_top=0, logprob=None, entropy=None, top_ids=None, top_logprobs=None,
                   status=None, stream=None):
    """ln softmax(logits / temperature) of one token per row, the row's entropy and its n_top most
    likely alternatives (dlite_token_logprobs). logits [..., V] with dense, evenly spaced rows, tokens int32
    of the leading shape. Rows whose token is negative are not read: zeros, ids -1.
    Returns dict(logprob, entropy [...] float32, top_ids [..., n_top] int32, top_logprobs [..., n_top] float32)."""
    lib = load()
    ptr, s = _here(stream, logits, tokens, logprob, entropy, top_ids, top_logprobs, status)
    if logits.dim() < 1 or logits.shape[:-1] != tokens.shape:
        raise ValueError("logits [..., V] and tokens of the leading shape expected")
    lead, V = tuple(tokens.shape), logits.shape[-1]
    rows = tokens.numel()
    if V > 1 and logits.stride(-1) != 1:
        raise ValueError("logits: the ids of a row have to be dense")
    stride, span = V, None
    for n, st in reversed(list(zip(lead, logits.stride()))):
        if n > 1:
            if span is None:
                stride = st
            elif st != span:
                raise ValueError("logits: rows have to be evenly spaced")
            span = st * n
    n_top = int(n_top)
    if not _LEAST <= n_top <= _MOST:
        _int(n_top, "n_top")
    if (rows | V) >> 31:
        _sizes("logits", rows, V)
    at = lead + (max(n_top, 0),)
    outs = []
    for name, t, shape, dt in (("logprob", logprob, lead, torch.float32), ("entropy", entropy, lead, torch.float32),
                               ("top_ids", top_ids, at, torch.int32), ("top_logprobs", top_logprobs, at, torch.float32)):
        if t is None:
            t = _new(s, shape, dt)
        else:
            _vec(t, dt, shape, name)
        outs.append(t)
    a = LogprobsArgs(rows, V, n_top, _dtype(logits, "logits"), temperature, logits.data_ptr(), stride,
                     _vec(tokens, torch.int32, lead, "tokens"), *(t.data_ptr() for t in outs), _vec(status, torch.int32, (1,), "status"))
    _check(lib.dlite_token_logprobs(ctypes.byref(a), ptr), "dlite_token_logprobs")
    return dict(logprob=outs[0], entropy=outs[1], top_ids=outs[2], top_logprobs=outs[3])


# ---------------------------------------------------------------- products with 8-bit weights

FP8_BLOCK = 128
_E4M3 = torch.float8_e4m3fn


def _rows_of(t, what):
    """(B, T, C, elements between the rows) of [B, T, C]: dense columns, evenly spaced rows."""
    if t.dim() != 3:
        raise ValueError(f"{what}: [B, T, columns] expected, got {list(t.shape)}")
    B, T, C = t.shape
    if (B | T | C) >> 31:
        _sizes(what, B, T, C)
    if t.is_contiguous():
        return B, T, C, C
    sb, st, sc = t.stride()
    if C > 1 and sc != 1:
        raise ValueError(f"{what}: the columns of a row have to be dense")
    row = st if T > 1 else (sb if B > 1 else C)
    if T > 1 and B > 1 and sb != T * st:
        raise ValueError(f"{what}: rows (b, t) have to be evenly spaced")
    if row < C:
        raise ValueError(f"{what}: rows overlap")
    return B, T, C, row


def _like(t, other, what):
    """Row stride of t, which has to be of the shape and type of `other`."""
    if t.shape != other.shape or t.dtype != other.dtype:
        raise ValueError(f"{what}: {other.dtype} {list(other.shape)} expected, got {t.dtype} {list(t.shape)}")
    return _rows_of(t, what)[3]


def _codes_of(t, what):
    """(B, T, C, bytes between the rows) of e4m3 codes [B, T, C]; one row's may be anything."""
    if t.dtype != _E4M3:
        raise ValueError(f"{what}: float8_e4m3fn expected, got {t.dtype}")
    B, T, C, row = _rows_of(t, what)
    return B, T, C, row if row != C or B * T > 1 else -(-C // 16) * 16


def _scale_of(t, B, T, C, what):
    """Pointer of the scales [B, T, ceil(C / 128)] of rows, whose memory has the rows (b, t) of a block side by side."""
    n = -(-C // FP8_BLOCK)
    if t.dtype != torch.float32 or t.shape != (B, T, n) or t.stride() != (T, 1, B * T):
        sb, st, sn = t.stride() if t.dim() == 3 else (0, 0, 0)
        if t.dtype != torch.float32 or t.shape != (B, T, n) or (n > 1 and sn != B * T) or (T > 1 and st != 1) or (B > 1 and sb != T):
            raise ValueError(f"{what}: float32 {[B, T, n]} with strides {[T, 1, B * T]} expected, got {t.dtype} {list(t.shape)} with strides "
                             f"{list(t.stride())}")
    return t.data_ptr()


def _new_scale(stream, B, T, C):
    return _new_strided(stream, (B, T, -(-C // FP8_BLOCK)), (T, 1, B * T), torch.float32)


def fp8_scale(B, T, C, stream=None):
    """Memory for the scales of rows [B, T, C]: float32 [B, T, ceil(C / 128)] with strides (T, 1, B T), the rows (b, t) of a block side
    by side. What fp8_quantise and fp8_gated make where none is given."""
    return _new_scale(_here(stream)[1], _int(B, "B"), _int(T, "T"), _int(C, "C"))


def _weight_of(w, scale, K, what):
    """(N, pointer, bytes between the rows, pointer of the scales) of codes [N, K] and their scales."""
    if w.dtype != _E4M3 or w.dim() != 2 or w.shape[1] != K:
        raise ValueError(f"{what}: float8_e4m3fn [N, {K}] expected, got {w.dtype} {list(w.shape)}")
    N = w.shape[0]
    if N >> 31:
        _sizes(what, N, K)
    row, col = w.stride()
    if K > 1 and col != 1:
        raise ValueError(f"{what}: the columns of a row have to be dense")
    if N == 1:
        row = -(-K // 16) * 16
    if scale.dtype != torch.float32 or scale.shape != (-(-N // FP8_BLOCK), -(-K // FP8_BLOCK)) or not scale.is_contiguous():
        raise ValueError(f"{what}_scale: contiguous float32 {[-(-N // FP8_BLOCK), -(-K // FP8_BLOCK)]} expected, got {scale.dtype} "
                         f"{list(scale.shape)}")
    return N, w.data_ptr(), row, scale.data_ptr()


def _new_strided(stream, shape, strides, dtype):
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


def _new_codes(stream, B, T, C):
    """(codes [B, T, C], bytes between their rows): rows on 16 bytes."""
    pitch = -(-C // 16) * 16
    if pitch == C:
        return _new(stream, (B, T, C), _E4M3), C
    return _new_strided(stream, (B, T, C), (T * pitch, pitch, 1), _E4M3), pitch


def fp8_quantise(x, gain=None, eps=1e-6, residual=None, total=None, n_rows=None, codes=None, scale=None, status=None, stream=None):
    """x [B, T, K] as 8-bit codes (float8_e4m3fn [B, T, K]) and scales (float32 [B, T, ceil(K / 128)]), one per 128 columns
    (dlite_fp8_quantise); the scales' memory has the rows (b, t) of a block side by side (fp8_scale). With residual: total = x + residual is stored (total None: in residual's place) and takes x's place; with
    gain [K] it is normed by its root mean square. Rows t >= n_rows[b] are left as they were (in new outputs: anything).
    Returns (codes, scale)."""
    lib = load()
    ptr, s = _here(stream, x, gain, residual, total, n_rows, codes, scale, status)
    B, T, K, xs = _rows_of(x, "x")
    if residual is None:
        if total is not None:
            raise ValueError("total: goes with a residual")
        rs = ts = 0
    else:
        total = residual if total is None else total
        rs, ts = _like(residual, x, "residual"), _like(total, x, "total")
    if codes is None:
        codes, cs = _new_codes(s, B, T, K)
    elif codes.shape != x.shape:
        raise ValueError(f"codes: {list(x.shape)} expected, got {list(codes.shape)}")
    else:
        cs = _codes_of(codes, "codes")[3]
    if scale is None:
        scale = _new_scale(s, B, T, K)
    else:
        _scale_of(scale, B, T, K, "scale")
    a = Fp8QuantiseArgs(B, T, K, _dtype(x, "x"), x.data_ptr(), xs, None if residual is None else residual.data_ptr(), rs,
                        None if residual is None else total.data_ptr(), ts, _vec(gain, x.dtype, (K,), "gain"), eps, codes.data_ptr(),
                        cs, scale.data_ptr(), _vec(n_rows, torch.int32, (B,), "n_rows"), _vec(status, torch.int32, (1,), "status"))
    _check(lib.dlite_fp8_quantise(ctypes.byref(a), ptr), "dlite_fp8_quantise")
    return codes, scale


def fp8_weight(w, status=None, stream=None):
    """A weight [N, K] as 8-bit codes (float8_e4m3fn [N, K], rows on 16 bytes) and float32 scales of its 128 x 128 blocks
    (dlite_fp8_weight): once, where a model is loaded. Returns (codes, scale)."""
    lib = load()
    ptr, s = _here(stream, w, status)
    if w.dim() != 2 or (w.shape[1] > 1 and w.stride(1) != 1):
        raise ValueError(f"w: [N, K] with dense rows expected, got {list(w.shape)}")
    N, K = w.shape
    if (N | K) >> 31:
        _sizes("w", N, K)
    codes, cs = _new_codes(s, 1, N, K)
    codes = codes[0]
    scale = _new(s, (-(-N // FP8_BLOCK), -(-K // FP8_BLOCK)), torch.float32)
    a = Fp8WeightArgs(N, K, _dtype(w, "w"), w.data_ptr(), w.stride(0) if N > 1 else K, codes.data_ptr(), cs, scale.data_ptr(),
                      _vec(status, torch.int32, (1,), "status"))
    _check(lib.dlite_fp8_weight(ctypes.byref(a), ptr), "dlite_fp8_weight")
    return codes, scale


def fp8_linear(codes, scale, w, w_scale, dtype=torch.bfloat16, n_rows=None, out=None, status=None, stream=None):
    """x w^T [B, T, N] of rows in 8 bits (codes [B, T, K] and scale, fp8_quantise's or fp8_gated's) and a weight in 8 bits
    (codes [N, K], float32 scales of 128 x 128 blocks), summed in float32 (dlite_fp8_linear). Rows t >= n_rows[b] of out are
    left as they were (zeros in a new one). Returns out."""
    lib = load()
    ptr, s = _here(stream, codes, scale, w, w_scale, n_rows, out, status)
    B, T, K, cs = _codes_of(codes, "codes")
    N, wp, ws, wsp = _weight_of(w, w_scale, K, "w")
    if out is None:
        out = _new(s, (B, T, N), dtype, zero=n_rows is not None)
    elif tuple(out.shape) != (B, T, N):
        raise ValueError(f"out: {[B, T, N]} expected, got {list(out.shape)}")
    a = Fp8LinearArgs(B, T, K, N, _dtype(out, "out"), codes.data_ptr(), cs, _scale_of(scale, B, T, K, "scale"),
                      wp, ws, wsp, out.data_ptr(), _rows_of(out, "out")[3], _vec(n_rows, torch.int32, (B,), "n_rows"),
                      _vec(status, torch.int32, (1,), "status"))
    _check(lib.dlite_fp8_linear(ctypes.byref(a), ptr), "dlite_fp8_linear")
    return out


def fp8_gated(codes, scale, gate, gate_scale, up, up_scale, n_rows=None, out=None, out_scale=None, status=None, stream=None):
    """silu(x gate^T) (x up^T) of rows in 8 bits and two weights in 8 bits, in one kernel, as 8-bit rows again
    (dlite_fp8_gated): what fp8_linear takes for the down projection. Returns (codes [B, T, F], scale [B, T, ceil(F / 128)]); rows
    t >= n_rows[b] are left as they were (in new outputs: anything)."""
    lib = load()
    ptr, s = _here(stream, codes, scale, gate, gate_scale, up, up_scale, n_rows, out, out_scale, status)
    B, T, K, cs = _codes_of(codes, "codes")
    N, gp, gs, gsp = _weight_of(gate, gate_scale, K, "gate")
    n, pp, ps, psp = _weight_of(up, up_scale, K, "up")
    if n != N:
        raise ValueError(f"up: the gate's {N} rows expected, got {n}")
    if out is None:
        out, ocs = _new_codes(s, B, T, N)
    elif tuple(out.shape) != (B, T, N):
        raise ValueError(f"out: {[B, T, N]} expected, got {list(out.shape)}")
    else:
        ocs = _codes_of(out, "out")[3]
    if out_scale is None:
        out_scale = _new_scale(s, B, T, N)
    else:
        _scale_of(out_scale, B, T, N, "out_scale")
    a = Fp8GatedArgs(B, T, K, N, codes.data_ptr(), cs, _scale_of(scale, B, T, K, "scale"), gp, gs, gsp, pp, ps, psp,
                     out.data_ptr(), ocs, out_scale.data_ptr(), _vec(n_rows, torch.int32, (B,), "n_rows"), _vec(status, torch.int32, (1,), "status"))
    _check(lib.dlite_fp8_gated(ctypes.byref(a), ptr), "dlite_fp8_gated")
    return out, out_scale


def selftest_ring(limit_ns, status, result, stream=None):
    """Probe of the bounded waits of rows over a ring of copies (dlite_selftest_ring): result is a device int32 [3, 4]."""
    lib = load()
    ptr, _ = _here(stream, status, result)
    _check(lib.dlite_selftest_ring(int(limit_ns), _vec(status, torch.int32, (1,), "status"), _vec(result, torch.int32, (3, 4), "result"), ptr),
           "dlite_selftest_ring")


def config_struct(cfg, B_max):
    return Config(B_max=B_max, D=cfg.D, m=cfg.m, K=cfg.K, L_D=cfg.L_D, n_q=cfg.n_q,
                  n_kv=cfg.n_kv, d_h=cfg.d_h, F=cfg.F, R=cfg.R, V=cfg.V,
                  dtype=DLITE_F32 if cfg.dtype == "f32" else DLITE_BF16,
                  rms_eps=cfg.eps, rope_theta=cfg.theta, anchor_group=getattr(cfg, "G", 1),
                  head_type=1 if getattr(cfg, "head", "rnn") == "gated" else 0,
                  history=getattr(cfg, "history", 0), act_planes=getattr(cfg, "act_planes", 1),
                  head_warmup=getattr(cfg, "warmup", 0))


class Drafter:
    """A drafter handle on the current CUDA device.

    W is the weight dict of workload.make_weights (tensors on the device, in
    the config's dtype). The library copies and repacks them at creation.
    """

    def __init__(self, cfg, W, B_max):
        self.lib = load()
        self.cfg = cfg
        self.B_max = B_max
        c = config_struct(cfg, B_max)
        w = Weights()
        for n in ("e_depth", "g_stage", "e_ph", "E", "g_final", "Q", "P"):
            setattr(w, n, _ptr(W[n]).value)
        for i, L in enumerate(W["layers"]):
            for n in ("g_attn", "Wq", "Wk", "Wv", "Wo", "g_ffn", "Wg", "Wu", "Wd"):
                setattr(w.layer[i], n, _ptr(L[n]).value)
        if getattr(cfg, "head", "rnn") == "gated":
            for n in GATED_FIELDS:
                setattr(w.gated, n, _ptr(W[n]).value)
        h = ctypes.c_void_p()
        _check(self.lib.dlite_create(ctypes.byref(c), ctypes.byref(w), ctypes.byref(h)), "dlite_create")
        self.h = h

    def close(self):
        if self.h:
            self.lib.dlite_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- outputs helpers
    def new_outputs(self, B, device="cuda"):
        K = self.cfg.K
        return dict(
            cand=torch.empty(B, K, dtype=torch.int32, device=device),
            qstats=torch.empty(B, K, 2, dtype=torch.float32, device=device),
            accepted=torch.empty(B, dtype=torch.int32, device=device),
            commits=torch.empty(B, K + 1, dtype=torch.int32, device=device),
            n_commit=torch.empty(B, dtype=torch.int32, device=device),
            next_anchor=torch.empty(B, dtype=torch.int32, device=device),
        )

    # ---- calls
    def draft_round(self, hidden, anchor, temperature, seed, pos, cand, qstats, stream=None,
                    taps=None):
        B = hidden.shape[0]
        if taps is None:
            rc = self.lib.dlite_draft_round(self.h, B, _ptr(hidden), _ptr(anchor), temperature,
                                            seed, _ptr(pos), _ptr(cand), _ptr(qstats), _stream(stream))
        else:
            t = Taps(*(None if taps.get(k) is None else taps[k].data_ptr() for k in ("z", "x", "b", "hs")))
            rc = self.lib.dlite_draft_round_taps(self.h, B, _ptr(hidden), _ptr(anchor), temperature,
                                                 seed, _ptr(pos), _ptr(cand), _ptr(qstats),
                                                 ctypes.byref(t), _stream(stream))
        _check(rc, "dlite_draft_round")

    def backbone(self, hidden, anchor, b, stream=None):
        _check(self.lib.dlite_backbone(self.h, hidden.shape[0], _ptr(hidden), _ptr(anchor), _ptr(b),
                                       _stream(stream)), "dlite_backbone")

    def seq_head(self, b, hs, stream=None):
        _check(self.lib.dlite_seq_head(self.h, b.shape[0], _ptr(b), _ptr(hs), _stream(stream)),
               "dlite_seq_head")

    def lm_head(self, hs, temperature, seed, pos, cand, qstats, stream=None):
        _check(self.lib.dlite_lm_head(self.h, hs.shape[0], _ptr(hs), temperature, seed, _ptr(pos),
                                      _ptr(cand), _ptr(qstats), _stream(stream)), "dlite_lm_head")

    def verify(self, cand, target_tokens, accepted, commits, n_commit, next_anchor, stream=None):
        _check(self.lib.dlite_verify(self.h, cand.shape[0], _ptr(cand), _ptr(target_tokens),
                                     _ptr(accepted), _ptr(commits), _ptr(n_commit),
                                     _ptr(next_anchor), _stream(stream)), "dlite_verify")

    def verify_sample(self, cand, qstats, hs, probs, temperature, seed, pos, accepted, commits,
                      n_commit, next_anchor, stream=None):
        _check(self.lib.dlite_verify_sample(self.h, cand.shape[0], _ptr(cand), _ptr(qstats),
                                            _ptr(hs), _ptr(probs), temperature, seed, _ptr(pos),
                                            _ptr(accepted), _ptr(commits), _ptr(n_commit),
                                            _ptr(next_anchor), _stream(stream)),
               "dlite_verify_sample")

    def verify_ex(self, mode, cand, accepted, commits, n_commit, next_anchor, n_verify=None,
                  target_tokens=None, qstats=None, hs=None, probs=None, temperature=0.0, seed=0, pos=None,
                  stream=None):
        """dlite_verify_ex: greedy / sampling / match verification over the first
        n_verify candidates (default all K)."""
        a = VerifyArgs(mode=mode, B=cand.shape[0], n_verify=cand.shape[1] if n_verify is None else n_verify,
                       candidates=_ptr(cand), target_tokens=_ptr(target_tokens), qstats=_ptr(qstats),
                       hs=_ptr(hs), target_probs=_ptr(probs), temperature=temperature, seed=seed,
                       pos=_ptr(pos), accepted=_ptr(accepted), commits=_ptr(commits),
                       n_commit=_ptr(n_commit), next_anchor=_ptr(next_anchor))
        _check(self.lib.dlite_verify_ex(self.h, ctypes.byref(a), _stream(stream)), "dlite_verify_ex")

    def history_reset(self, stream=None):
        """Refill every draft-KV ring with the synthetic history; cursors to 0."""
        _check(self.lib.dlite_history_reset(self.h, _stream(stream)), "dlite_history_reset")

    def history_read(self, layer, request, which, stream=None):
        """One ring of the history-KV control: ([n_kv, H, d_h] bf16 on the device, cursor)."""
        c = self.cfg
        dst = torch.empty(c.n_kv, c.history, c.d_h, dtype=torch.bfloat16, device="cuda")
        cur = ctypes.c_int32(0)
        _check(self.lib.dlite_history_read(self.h, layer, request, which, _ptr(dst), ctypes.byref(cur),
                                           _stream(stream)), "dlite_history_read")
        return dst, int(cur.value)

    def shift_group(self, commits, n_commit, group, stream=None):
        _check(self.lib.dlite_shift_group(self.h, n_commit.shape[0], _ptr(commits), _ptr(n_commit), _ptr(group),
                                          _stream(stream)), "dlite_shift_group")

    def advance(self, n_commit, pos, stream=None):
        _check(self.lib.dlite_advance(self.h, n_commit.shape[0], _ptr(n_commit), _ptr(pos),
                                      _stream(stream)), "dlite_advance")

    def round_host(self, hidden_h, anchor_h, pos_h, tgt_h, probs_h, temperature, seed, out_h,
                   stream=None):
        _check(self.lib.dlite_round_host(self.h, hidden_h.shape[0], _hptr(hidden_h), _hptr(anchor_h),
                                         _hptr(pos_h), _hptr(tgt_h), _hptr(probs_h), temperature,
                                         seed, _hptr(out_h["accepted"]), _hptr(out_h["commits"]),
                                         _hptr(out_h["n_commit"]), _hptr(out_h["next_anchor"]),
                                         _stream(stream)), "dlite_round_host")

    def device_status(self, clear=True, stream=None):
        v = ctypes.c_int(0)
        rc = self.lib.dlite_device_status(self.h, 1 if clear else 0, ctypes.byref(v), _stream(stream))
        return rc, v.value

    def stage_times(self, hidden, anchor, temperature, seed, pos, out, target_tokens=None,
                    target_probs=None, stream=None, cap=128):
        """Per-launch CUDA-event times (ms) of one eager draft (+ verify): [(name, ms)]."""
        times = (ctypes.c_float * cap)()
        names = (ctypes.c_char_p * cap)()
        n = self.lib.dlite_stage_times(
            self.h, hidden.shape[0], _ptr(hidden), _ptr(anchor), temperature, seed, _ptr(pos),
            _ptr(target_tokens), _ptr(target_probs), _ptr(out["cand"]), _ptr(out["qstats"]),
            _ptr(out["accepted"]), _ptr(out["commits"]), _ptr(out["n_commit"]),
            _ptr(out["next_anchor"]), times, names, cap, _stream(stream))
        if n < 0:
            raise DliteError(n, "dlite_stage_times")
        return [(names[i].decode(), times[i]) for i in range(min(n, cap))]

    def selftest_wait(self, limit_ns, result, stream=None):
        """Bounded-wait probe (dlite_selftest_wait): result is a device int32 [3]."""
        _check(self.lib.dlite_selftest_wait(self.h, int(limit_ns), _ptr(result), _stream(stream)),
               "dlite_selftest_wait")

    def counters(self, reset=False, stream=None):
        """Sampling-verify counters: residual draws, proposals, fallbacks, bonus draws."""
        out = (ctypes.c_int64 * 5)()
        _check(self.lib.dlite_counters(self.h, 1 if reset else 0, out, _stream(stream)), "dlite_counters")
        return dict(residual=out[0], proposals=out[1], fallback=out[2], bonus=out[3],
                    lm_close_calls=out[4])

    def launch_count(self, B, temperature):
        return self.lib.dlite_launch_count(self.h, B, temperature)
