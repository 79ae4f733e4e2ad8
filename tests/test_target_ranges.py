"""The binding's integers: what a C int does not hold is refused, not cut to its low 32 bits (no GPU needed)."""
import pytest
import torch

from history_free_speculative_gb300 import binding, build

FAR = (1 << 32) + 5          # its low 32 bits: 5


@pytest.fixture
def calls(monkeypatch):
    """The calls with tensors that stand for device tensors; none of them may reach the library."""
    build.build()
    lib = binding.load()

    class Closed:
        def __getattr__(self, name):
            if name == "dlite_kv_attention_workspace":      # asks nothing of a device where sizes are refused
                return getattr(lib, name)
            raise AssertionError(f"{name} reached")

    monkeypatch.setattr(binding, "load", lambda: Closed())
    monkeypatch.setattr(binding, "_here", lambda stream, *t: (0, None))
    monkeypatch.setattr(binding, "_new", lambda s, shape, dtype, zero=False: torch.empty(shape, dtype=dtype, device="meta"))
    x, pos = torch.zeros(1, 1, 2, 64), torch.zeros(1, dtype=torch.int64)
    pages, bt = torch.zeros(1, 2, 72 * 64, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32)
    far = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    table, logits, tok = torch.zeros(4, 32, 2), torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    return {
        "attention window": lambda: binding.kv_attention(x, pages, bt, pos, window=FAR),
        "attention window below": lambda: binding.kv_attention(x, pages, bt, pos, window=-FAR),
        "attention k_exp": lambda: binding.kv_attention(x, pages, bt, pos, k_exp=FAR),
        "attention v_exp": lambda: binding.kv_attention(x, pages, bt, pos, v_exp=-FAR),
        "attention columns": lambda: binding.kv_attention(x, pages, far(1, FAR, dtype=torch.int32), pos),
        "attention rows": lambda: binding.kv_attention(far(1, FAR, 2, 64), pages, bt, pos),
        "attention pages": lambda: binding.kv_attention(x, far(FAR, 2, 72 * 64, dtype=torch.uint8), bt, pos),
        "workspace": lambda: binding.kv_attention_workspace(1, 1, 2, 2, 64, FAR),
        "append k_exp": lambda: binding.kv_append(pages, bt, x, x, pos, k_exp=FAR),
        "append v_exp": lambda: binding.kv_append(pages, bt, x, x, pos, v_exp=FAR),
        "append table": lambda: binding.kv_append(pages, bt, x, x, pos, table=far(FAR, 32, 2)),
        "read T": lambda: binding.kv_read(pages, bt, pos, FAR),
        "read k_exp": lambda: binding.kv_read(pages, bt, pos, 1, k_exp=FAR),
        "rope rows": lambda: binding.rope(far(FAR, 1, 1, 64), pos, table),
        "rope table": lambda: binding.rope(x, pos, far(FAR, 32, 2)),
        "rope_table n_pos": lambda: binding.rope_table(FAR, 2),
        "rope_table rot": lambda: binding.rope_table(1, FAR),
        "logprobs n_top": lambda: binding.token_logprobs(logits, tok, n_top=FAR),
        "logprobs rows": lambda: binding.token_logprobs(far(FAR, 8), far(FAR, dtype=torch.int32)),
        "logprobs V": lambda: binding.token_logprobs(far(2, FAR), tok),
    }


NAMES = ["attention window", "attention window below", "attention k_exp", "attention v_exp", "attention columns", "attention rows",
         "attention pages", "workspace", "append k_exp", "append v_exp", "append table", "read T", "read k_exp", "rope rows", "rope table",
         "rope_table n_pos", "rope_table rot", "logprobs n_top", "logprobs rows", "logprobs V"]


@pytest.mark.parametrize("name", NAMES)
def test_integers_outside_32_bits(calls, name):
    with pytest.raises(ValueError, match="outside 32 bits"):
        calls[name]()


def test_every_call_is_named(calls):
    assert list(calls) == NAMES
