"""The serving operators of a decoder beside its FC layers: a paged key/value
cache with rotation and append, attention of new tokens over it, and the
processing of the output layer's logits (the fc_gguf_kv_* and fc_gguf_logits
calls of include/fc_gguf.h, which holds their contracts).

Argument marshalling only, as in binding.py: torch supplies device memory and
the current HIP stream.  The calls convert and copy nothing: a tensor of
another type, device or layout than the call takes is refused (ValueError
before the library is called, FcGgufError with the library's code otherwise).
"""

from __future__ import annotations

import ctypes
import math

import torch

from .binding import FcGgufError, lib

F16, BF16, F32 = 0, 1, 2
DTYPES = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}

_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_calls = {}


def _call(name):
    f = _calls.get(name)
    if f is None:
        f = _calls[name] = getattr(lib(), name)
    return f


def _check(code, what):
    if code != 0:
        raise FcGgufError(code, what)


def _stream(index):
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _heads(x, heads, dim, dtype, device, name):
    """[T, heads, dim] whose heads and dimensions lie next to each other: its row stride."""
    _need(x.dim() == 3 and x.dtype == dtype and x.device == device, f"{name}: a {dtype} tensor [T, heads, head_dim] on {device}")
    t, h, d = x.shape
    _need((heads is None or h == heads) and d == dim, f"{name}: [T, {heads or 'heads'}, {dim}], got {tuple(x.shape)}")
    row, head, one = x.stride()
    # strides of axes of length 0 or 1 say nothing
    _need(one == 1 and (head == d or h <= 1), f"{name}: heads and dimensions must be contiguous")
    return row if t > 1 else max(row, h * d) // 8 * 8


def _ints(x, device, name, dim=None):
    _need(x.dtype == torch.int32 and x.device == device and x.is_contiguous() and (dim is None or x.dim() == dim),
          f"{name}: a contiguous int32 tensor on {device}" + (f" of {dim} dimensions" if dim else ""))


def _floats(x, n, device, name):
    _need(x.dtype == torch.float32 and x.device == device and x.is_contiguous() and x.numel() == n,
          f"{name}: {n} contiguous float32 values on {device}")


class Rope:
    """A rotation: inv_freq f32[rot_dim/2] on the GPU, axis i32[rot_dim/2] (the
    position axis that turns each pair) or None, pairs (2j, 2j+1) if
    interleaved else (j, j + rot_dim/2), scale on sine and cosine."""

    def __init__(self, inv_freq, axis=None, interleaved=False, scale=1.0):
        _need(inv_freq.is_cuda, "inv_freq: a tensor on the GPU")
        _floats(inv_freq, inv_freq.numel(), inv_freq.device, "inv_freq")
        self.rot_dim = 2 * inv_freq.numel()
        if axis is not None:
            _ints(axis, inv_freq.device, "axis", 1)
            _need(axis.numel() == inv_freq.numel(), "axis: one entry for each pair")
        self.inv_freq, self.axis = inv_freq, axis
        self.interleaved, self.scale = bool(interleaved), float(scale)


class PagedKv:
    """One layer's paged key/value cache.

    k [pages, kv_heads, head_dim/8, page_size, 8] and v [pages, kv_heads,
    page_size/8, head_dim, 8], f16 or bf16 on the GPU, are allocated here
    (uninitialised) unless given.  They may be read, and whole pages copied in
    and out, like any tensors.
    """

    def __init__(self, pages, page_size, kv_heads, head_dim, dtype=torch.float16, *, device=None, k=None, v=None):
        if k is None or v is None:
            _need(k is None and v is None, "k and v: both or neither")
            _need(min(pages, page_size, kv_heads, head_dim) > 0 and head_dim % 8 == 0 and page_size % 8 == 0,
                  "pages, page_size, kv_heads, head_dim: positive, the sizes multiples of 8")
            if not torch.cuda.is_available():
                raise RuntimeError("no GPU visible: the library has no CPU path")
            device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
            k = torch.empty((pages, kv_heads, head_dim // 8, page_size, 8), dtype=dtype, device=device)
            v = torch.empty((pages, kv_heads, page_size // 8, head_dim, 8), dtype=dtype, device=device)
        _need(k.is_cuda and v.is_cuda and k.device == v.device and k.dtype == v.dtype == dtype, "k and v: of dtype, on one GPU")
        _need(k.is_contiguous() and v.is_contiguous() and tuple(k.shape) == (pages, kv_heads, head_dim // 8, page_size, 8)
              and tuple(v.shape) == (pages, kv_heads, page_size // 8, head_dim, 8), "k and v: contiguous, of the cache's shapes")
        self.k, self.v = k, v
        self.pages, self.page_size, self.kv_heads, self.head_dim = int(pages), int(page_size), int(kv_heads), int(head_dim)
        self.dtype, self.device = dtype, k.device
        self._h = ctypes.c_void_p()
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(_call("fc_gguf_kv_create")(pages, page_size, kv_heads, head_dim, DTYPES.get(dtype, -1), k.data_ptr(),
                                              v.data_ptr(), ctypes.byref(h)), "fc_gguf_kv_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _call("fc_gguf_kv_destroy")(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, q, k, v, slots, positions=None, rope=None, out=None):
        """Rotates q [T, heads, head_dim] and k [T, kv_heads, head_dim] by rope at
        positions i32 [T] or [axes, T] (None: no rotation) and appends k and v at
        slots i32 [T] (page * page_size + place; negative: not appended).  Returns
        the rotated q, in out (q itself, or None for a new tensor).  q may be None:
        keys and values only.  The three may be parts of one projection's rows."""
        dev, dim = self.device, self.head_dim
        t = k.shape[0]
        ks = _heads(k, self.kv_heads, dim, self.dtype, dev, "k")
        vs = _heads(v, self.kv_heads, dim, self.dtype, dev, "v")
        _ints(slots, dev, "slots", 1)
        _need(v.shape[0] == t and slots.shape[0] == t, "k, v and slots: one row for each token")
        qp, op, heads, qs, os = None, None, 0, 0, 0
        if q is not None:
            qs = _heads(q, None, dim, self.dtype, dev, "q")
            heads = q.shape[1]
            _need(q.shape[0] == t, "q: one row for each token")
            if out is None:
                out = torch.empty((t, heads, dim), dtype=self.dtype, device=dev)
            os = _heads(out, heads, dim, self.dtype, dev, "out")
            _need(out.shape[0] == t, "out: one row for each token")
            qp, op = q.data_ptr(), out.data_ptr()
            _need(qp != op or qs == os, "out: q itself, or other memory")
        pp, axes, fp, ap, rot, inter, scale = None, 1, None, None, 0, 0, 1.0
        if rope is not None:
            _need(positions is not None, "positions: needed with a rope")
            _ints(positions, dev, "positions")
            axes = 1 if positions.dim() == 1 else positions.shape[0]
            _need(positions.dim() in (1, 2) and positions.shape[-1] == t, "positions: [T] or [axes, T]")
            _need(rope.inv_freq.device == dev, f"rope: on {dev}")
            pp, fp, rot, inter, scale = positions.data_ptr(), rope.inv_freq.data_ptr(), rope.rot_dim, rope.interleaved, rope.scale
            ap = rope.axis.data_ptr() if rope.axis is not None else None
        rc = _call("fc_gguf_kv_append")(self._h, qp, qs, heads, k.data_ptr(), ks, v.data_ptr(), vs, t, slots.data_ptr(), pp,
                                        axes, fp, ap, rot, inter, scale, op, os, _stream(dev.index))
        if rc != 0:
            _check(rc, "fc_gguf_kv_append")
        return out

    def attend(self, q, cu_q, kv_lens, table, max_q, *, scale=None, window=0, out=None, lse=None):
        """Attention of q [T, heads, head_dim] over the cache: sequence s has rows
        cu_q[s] .. cu_q[s+1] (at most max_q) and kv_lens[s] keys, its new tokens
        the last of them, on pages table[s].  window > 0: each row sees its last
        `window` keys.  scale: 1 / sqrt(head_dim) unless given.  lse: f32 [T, heads]
        to fill, or None.  Returns the output, in out (None: a new tensor, zeros
        where no sequence has a row)."""
        dev, dim = self.device, self.head_dim
        qs = _heads(q, None, dim, self.dtype, dev, "q")
        t, heads = q.shape[0], q.shape[1]
        _ints(cu_q, dev, "cu_q", 1)
        _ints(kv_lens, dev, "kv_lens", 1)
        seqs = kv_lens.shape[0]
        _need(cu_q.shape[0] == seqs + 1, "cu_q: one entry more than kv_lens")
        _need(table.dtype == torch.int32 and table.device == dev and table.dim() == 2 and table.shape[0] == seqs,
              f"table: an int32 tensor [seqs, pages] on {dev}")
        width = table.shape[1]
        ts, one = table.stride()
        _need(one == 1 or width <= 1, "table: contiguous rows")
        if out is None:
            out = torch.zeros((t, heads, dim), dtype=self.dtype, device=dev)
        os = _heads(out, heads, dim, self.dtype, dev, "out")
        _need(out.shape[0] == t, "out: one row for each token")
        lp = None
        if lse is not None:
            _floats(lse, t * heads, dev, "lse")
            lp = lse.data_ptr()
        rc = _call("fc_gguf_kv_attend")(self._h, q.data_ptr(), qs, heads, t, cu_q.data_ptr(), kv_lens.data_ptr(), seqs,
                                        table.data_ptr(), max(ts, width), width, max_q,
                                        1.0 / math.sqrt(dim) if scale is None else scale, window, out.data_ptr(), os, lp,
                                        _stream(dev.index))
        if rc != 0:
            _check(rc, "fc_gguf_kv_attend")
        return out


def process_logits(x, *, tokens=None, lens=None, prompt_lens=None, repetition=None, frequency=None, presence=None,
                   bias_offsets=None, bias_ids=None, bias_values=None, mask=None, out=None):
    """Penalties for repeated tokens, biases and a grammar's mask on logits x
    [rows, vocab] (f16, bf16 or f32; rows may be strided).  tokens i32 [rows, n]
    (prompt first), lens and prompt_lens i32 [rows]; repetition, frequency and
    presence f32 [rows]; bias_offsets i32 [rows+1] into bias_ids i32 and
    bias_values f32; mask i32 [rows, words], bit v%32 of word v//32 allows token v.
    out: x itself, a tensor of x's type or f32, or None for a new f32 tensor.
    Returns out."""
    _need(x.is_cuda and x.dim() == 2 and x.dtype in DTYPES, "x: f16, bf16 or f32 [rows, vocab] on the GPU")
    dev = x.device
    rows, vocab = x.shape
    if out is None:
        out = torch.empty((rows, vocab), dtype=torch.float32, device=dev)
    _need(out.device == dev and out.shape == x.shape and out.dtype in DTYPES, f"out: [{rows}, {vocab}] on {dev}")
    strides = []
    for y, name in ((x, "x"), (out, "out")):
        row, one = y.stride()
        _need(one == 1 or vocab <= 1, f"{name}: contiguous rows")
        strides.append(row if rows > 1 else max(row, vocab))
    tp, ts, lp, pp = None, 0, None, None
    if tokens is not None:
        _ints(tokens, dev, "tokens", 2)
        _need(lens is not None and tokens.shape[0] == rows, "tokens: [rows, n], with lens")
        _ints(lens, dev, "lens", 1)
        _need(lens.shape[0] == rows, "lens: one for each row")
        tp, ts, lp = tokens.data_ptr(), tokens.shape[1], lens.data_ptr()
        if prompt_lens is not None:
            _ints(prompt_lens, dev, "prompt_lens", 1)
            _need(prompt_lens.shape[0] == rows, "prompt_lens: one for each row")
            pp = prompt_lens.data_ptr()
    factors = []
    for y, name in ((repetition, "repetition"), (frequency, "frequency"), (presence, "presence")):
        if y is not None:
            _floats(y, rows, dev, name)
        factors.append(None if y is None else y.data_ptr())
    bo, bi, bv, bn = None, None, None, 0
    if bias_offsets is not None:
        _need(bias_ids is not None and bias_values is not None, "bias_offsets: with bias_ids and bias_values")
        _ints(bias_offsets, dev, "bias_offsets", 1)
        _ints(bias_ids, dev, "bias_ids", 1)
        bn = bias_ids.shape[0]
        _floats(bias_values, bn, dev, "bias_values")
        _need(bias_offsets.shape[0] == rows + 1, "bias_offsets: one more than rows")
        bo, bi, bv = bias_offsets.data_ptr(), bias_ids.data_ptr(), bias_values.data_ptr()
    mp, ms = None, 0
    if mask is not None:
        _ints(mask, dev, "mask", 2)
        _need(mask.shape[0] == rows, "mask: one row for each of x's")
        mp, ms = mask.data_ptr(), mask.shape[1]
    _need(torch.cuda.current_device() == dev.index, f"x: on the current device, not on {dev}")
    rc = _call("fc_gguf_logits")(x.data_ptr(), strides[0], DTYPES[x.dtype], rows, vocab, tp, ts, lp, pp, *factors, bo, bi, bv,
                                 bn, mp, ms, out.data_ptr(), strides[1], DTYPES[out.dtype], _stream(dev.index))
    if rc != 0:
        _check(rc, "fc_gguf_logits")
    return out
