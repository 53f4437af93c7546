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


def test_outputs_that_overlap_inputs_are_refused(kv):
    flat = torch.zeros(4096, dtype=torch.float16)
    rows = lambda at, stride, heads=4, t=3: flat.as_strided((t, heads, 64), (stride, 64, 1), at)  # noqa: E731
    cu, lens, table = _ints(0, 3), _ints(5), _ints(0)[None]
    slots, k, v = _ints(0, 1, 2), torch.zeros((3, 2, 64), dtype=torch.float16), torch.zeros((3, 2, 64), dtype=torch.float16)
    for q, out, apart in ((rows(0, 256), rows(0, 256), False), (rows(0, 256), rows(256, 256), False), (rows(0, 256), rows(8, 256), False),
                          (rows(0, 256), rows(768, 256), True), (rows(768, 256), rows(0, 256), True),
                          (rows(0, 512), rows(256, 512), True), (rows(256, 512), rows(0, 512), True),     # columns of one matrix
                          (rows(0, 512), rows(248, 512), False), (rows(0, 512), rows(264, 512), False),
                          (rows(0, 1024), rows(256, 280), False), (rows(0, 1024), rows(256, 256), True),  # rows between its rows
                          (rows(1032, 1032), rows(0, 520), False),
                          (rows(0, 512, t=1), rows(256, 512, t=1), True), (rows(0, 512, t=1), rows(8, 512, t=1), False)):
        t = q.shape[0]
        kv.calls.clear()
        same = q.data_ptr() == out.data_ptr()
        args = (_ints(0, t), lens, table, t)
        if apart:
            kv.attend(q, *args, out=out)
            kv.append(q, k[:t], v[:t], slots[:t], out=out)
            kv.append(None if t == 3 else q, k[:t], v[:t], slots[:t], out=out)
            assert len(kv.calls) == 3
        else:
            with pytest.raises(ValueError):
                kv.attend(q, *args, out=out)
            if same:                                                         # append rotates in place
                kv.append(q, k[:t], v[:t], slots[:t], out=out)
            else:
                with pytest.raises(ValueError):
                    kv.append(q, k[:t], v[:t], slots[:t], out=out)
            assert len(kv.calls) == same
    # keys and values among the output's rows
    kv.calls.clear()
    q = torch.zeros((3, 4, 64), dtype=torch.float16)
    for part in (rows(0, 512, 2), rows(128, 512, 2), rows(392, 512, 2)):
        for kk, vv in ((part, v), (k, part)):
            with pytest.raises(ValueError):
                kv.append(q, kk, vv, slots, out=rows(0, 512))
    assert not kv.calls
    qkv = rows(0, 512, 8)
    kv.append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], slots, out=qkv[:, :4])    # one projection's rows, in place
    assert len(kv.calls) == 1


def test_logits_that_overlap_are_refused(monkeypatch):
    calls = []
    monkeypatch.setitem(serving._calls, "fc_gguf_logits", lambda *a: calls.append(a) or 0)
    monkeypatch.setattr(serving, "_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    flat = torch.zeros(1000, dtype=torch.float32)
    half = flat.view(torch.float16)
    x = flat.as_strided((3, 40), (80, 1))
    for out in (flat.as_strided((3, 40), (80, 1), 1), flat.as_strided((3, 40), (80, 1), 80), flat.as_strided((3, 40), (40, 1))):
        with pytest.raises(ValueError):
            serving.process_logits(x, out=out)
    with pytest.raises(ValueError):                                          # f16 logits, f32 outputs over them
        serving.process_logits(half.as_strided((3, 40), (80, 1)), out=flat.as_strided((3, 40), (40, 1)))
    assert not calls
    serving.process_logits(x, out=x)
    serving.process_logits(x, out=flat.as_strided((3, 40), (80, 1), 40))
    serving.process_logits(x, out=flat.as_strided((3, 40), (40, 1), 240))
    assert len(calls) == 3
