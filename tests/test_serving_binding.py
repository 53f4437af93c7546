"""What the binding of the serving operators hands to the library, on the CPU: the library's calls are stand-ins that
note their arguments, the tensors are the host's."""

import pytest
import torch

from gguf_quant_block_amd import serving

# places of arguments of fc_gguf_kv_attend
TABLE_STRIDE, TABLE_WIDTH = 9, 10


@pytest.fixture
def kv(monkeypatch):
    """A cache of 2 key heads of 64 whose tensors lie on the host, and the calls that reach the library."""
    calls = []
    for name in ("fc_gguf_kv_append", "fc_gguf_kv_attend", "fc_gguf_logits"):
        monkeypatch.setitem(serving._calls, name, lambda *a, name=name: calls.append((name, a)) or 0)
    monkeypatch.setattr(serving, "_stream", lambda index: 0)
    kv = object.__new__(serving.PagedKv)
    kv.index, kv.head_dim, kv.kv_heads, kv.page_size, kv.pages = -1, 64, 2, 16, 4
    kv.dtype, kv.device, kv.scale, kv._h, kv.calls = torch.float16, torch.device("cpu"), 0.125, None, calls
    return kv


def _ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_rows_of_a_table_must_not_overlap(kv):
    q, cu, lens = torch.zeros((3, 4, 64), dtype=torch.float16), _ints(0, 1, 2, 3), _ints(5, 5, 5)
    row = _ints(0, 1, 2)
    for table in (row[None].expand(3, -1),                                   # one row for all: a stride of 0
                  _ints(0, 1, 2, 3, 4).as_strided((3, 3), (1, 1))):
        with pytest.raises(ValueError):
            kv.attend(q, cu, lens, table, 1)
    assert not kv.calls
    kv.attend(q, cu, lens, row.repeat(3, 2)[:, :3], 1)                       # wider rows than are used
    assert kv.calls[-1][1][TABLE_STRIDE:TABLE_WIDTH + 1] == (6, 3)
    kv.attend(q[:1], cu[:2], lens[:1], row[None].expand(1, -1), 1)           # (of one row the stride says nothing)
    assert kv.calls[-1][1][TABLE_STRIDE:TABLE_WIDTH + 1] == (3, 3)


def test_windows_past_32_bits_are_refused(kv):
    q, args = torch.zeros((1, 4, 64), dtype=torch.float16), (_ints(0, 1), _ints(5), _ints(0)[None], 1)
    for window in (2**31, 2**32 + 5, 2**40, -2**32 + 7):                     # (the call takes 32 bits of them)
        with pytest.raises(ValueError):
            kv.attend(q, *args, window=window)
    with pytest.raises(ValueError):
        kv.attend(q, *args[:3], 2**64 + 1)
    assert not kv.calls
    kv.attend(q, *args, window=2**30)
    assert len(kv.calls) == 1
