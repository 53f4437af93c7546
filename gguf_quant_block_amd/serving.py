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


# The checks of a call take most of its time on the host (an append of one
# token: 13.6 us with messages formatted ahead of the checks, of which 4.3 are
# the library's call), so they compare plain attributes and format a message
# only to raise it.  A tensor's device is compared by its index (-1: not on a
# GPU).

def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _heads(x, heads, dim, dtype, index, name):
    """[T, heads, dim] whose heads and dimensions lie next to each other: its row stride."""
    if x.dtype is not dtype or x.get_device() != index or x.dim() != 3:
        raise ValueError(f"{name}: a {dtype} tensor [T, heads, head_dim] on cuda:{index}")
    t, h, d = x.shape
    if d != dim or (heads is not None and h != heads):
        raise ValueError(f"{name}: [T, {heads or 'heads'}, {dim}], got {tuple(x.shape)}")
    row, head, one = x.stride()
    # strides of axes of length 0 or 1 say nothing
    if one != 1 or (head != d and h > 1):
        raise ValueError(f"{name}: heads and dimensions must be contiguous")
    return row if t > 1 else max(row, h * d) // 8 * 8


def _ints(x, index, name, dim=None):
    if x.dtype is not torch.int32 or x.get_device() != index or not x.is_contiguous() or (dim is not None and x.dim() != dim):
        raise ValueError(f"{name}: a contiguous int32 tensor on cuda:{index}" + (f" of {dim} dimensions" if dim else ""))


def _floats(x, n, index, name):
    if x.dtype is not torch.float32 or x.get_device() != index or not x.is_contiguous() or x.numel() != n:
        raise ValueError(f"{name}: {n} contiguous float32 values on cuda:{index}")


def _overlap(p, ps, pw, q, qs, qw, rows):
    """Whether rows of pw bytes, ps bytes apart from address p on, share memory
    with as many of qw bytes, qs apart from q on."""
    if p + (rows - 1) * ps + pw <= q or q + (rows - 1) * qs + qw <= p or rows == 0:
        return False
    if rows == 1:
        return True
    if ps < pw or qs < qw:                                # (no rows of the library's: it refuses them)
        return False
    if ps == qs:                                          # parts of one matrix's rows, as a rule: rows j and j + k
        return max((q - p - pw) // ps + 1, 1 - rows) <= min((q - p + qw - 1) // ps, rows - 1)
    return any(max((at - pw) // ps + 1, 0) <= min((at + qw - 1) // ps, rows - 1)
               for at in range(q - p, q - p + rows * qs, qs))


class Rope:
    """A rotation: inv_freq f32[rot_dim/2] on the GPU, axis i32[rot_dim/2] (the
    position axis that turns each pair) or None, pairs (2j, 2j+1) if
    interleaved else (j, j + rot_dim/2), scale on sine and cosine."""

    def __init__(self, inv_freq, axis=None, interleaved=False, scale=1.0):
        _need(inv_freq.is_cuda, "inv_freq: a tensor on the GPU")
        self.index = inv_freq.get_device()
        _floats(inv_freq, inv_freq.numel(), self.index, "inv_freq")
        self.rot_dim = 2 * inv_freq.numel()
        if axis is not None:
            _ints(axis, self.index, "axis", 1)
            _need(axis.numel() == inv_freq.numel(), "axis: one entry for each pair")
        self.inv_freq, self.axis = inv_freq, axis        # kept alive for their addresses
        self.freq_ptr, self.axis_ptr = inv_freq.data_ptr(), None if axis is None else axis.data_ptr()
        self.interleaved, self.scale = bool(interleaved), float(scale)


class PagedKv:
    """One layer's paged key/value cache.

    k [pages, kv_heads, head_dim/8, page_size, 8] and v [pages, kv_heads,
    page_size/8, head_dim, 8], f16 or bf16 on the GPU, are allocated here
    (uninitialised) unless given.  They may be read, and whole pages copied in
    and out, like any tensors.  A graph that captures attend is captured after
    one call of its largest sizes, and must not outlive the cache.
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
        self.dtype, self.device, self.index = dtype, k.device, k.get_device()
        self.scale = 1.0 / math.sqrt(head_dim)
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
        dev, dim, dtype = self.index, self.head_dim, self.dtype
        t = k.shape[0]
        ks = _heads(k, self.kv_heads, dim, dtype, dev, "k")
        vs = _heads(v, self.kv_heads, dim, dtype, dev, "v")
        _ints(slots, dev, "slots", 1)
        if v.shape[0] != t or slots.shape[0] != t:
            raise ValueError("k, v and slots: one row for each token")
        kp, vp = k.data_ptr(), v.data_ptr()
        qp = op = None
        heads = qs = os = 0
        if q is not None:
            qs = _heads(q, None, dim, dtype, dev, "q")
            rows, heads, _ = q.shape
            given = out is not None
            if not given:
                out = torch.empty((t, heads, dim), dtype=dtype, device=self.device)
            os = _heads(out, heads, dim, dtype, dev, "out")
            if rows != t or out.shape[0] != t:
                raise ValueError("q and out: one row for each token")
            qp, op = q.data_ptr(), out.data_ptr()
            if given:
                w, kw, n = 2 * heads * dim, 2 * self.kv_heads * dim, 2 * (t - 1)
                end = op + n * os + w                     # (most calls end at the comparisons of the whole ranges)
                if qp < end and op < qp + n * qs + w and (qp != op or qs != os) and _overlap(op, 2 * os, w, qp, 2 * qs, w, t):
                    raise ValueError("out: q itself, or other memory")
                if (kp < end and op < kp + n * ks + kw and _overlap(op, 2 * os, w, kp, 2 * ks, kw, t)
                        or vp < end and op < vp + n * vs + kw and _overlap(op, 2 * os, w, vp, 2 * vs, kw, t)):
                    raise ValueError("out: no memory of k or v")
        pp, axes, fp, ap, rot, inter, scale = None, 1, None, None, 0, 0, 1.0
        if rope is not None:
            _need(positions is not None, "positions: needed with a rope")
            _ints(positions, dev, "positions")
            shape = positions.shape
            if len(shape) == 2:
                axes = shape[0]
            if len(shape) not in (1, 2) or shape[-1] != t:
                raise ValueError("positions: [T] or [axes, T]")
            if rope.index != dev:
                raise ValueError(f"rope: on cuda:{dev}")
            pp, fp, rot, inter, scale = positions.data_ptr(), rope.freq_ptr, rope.rot_dim, rope.interleaved, rope.scale
            ap = rope.axis_ptr
        rc = _call("fc_gguf_kv_append")(self._h, qp, qs, heads, kp, ks, vp, vs, t, slots.data_ptr(), pp,
                                        axes, fp, ap, rot, inter, scale, op, os, _stream(dev))
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
        dev, dim, dtype = self.index, self.head_dim, self.dtype
        qs = _heads(q, None, dim, dtype, dev, "q")
        t, heads, _ = q.shape
        _ints(cu_q, dev, "cu_q", 1)
        _ints(kv_lens, dev, "kv_lens", 1)
        seqs = kv_lens.shape[0]
        if cu_q.shape[0] != seqs + 1:
            raise ValueError("cu_q: one entry more than kv_lens")
        if table.dtype is not torch.int32 or table.get_device() != dev or table.dim() != 2 or table.shape[0] != seqs:
            raise ValueError(f"table: an int32 tensor [seqs, pages] on cuda:{dev}")
        width = table.shape[1]
        ts, one = table.stride()
        if one != 1 and width > 1:
            raise ValueError("table: contiguous rows")
        if ts < width:
            if seqs > 1:
                raise ValueError("table: rows that do not overlap")
            ts = width
        given = out is not None
        if not given:
            out = torch.zeros((t, heads, dim), dtype=dtype, device=self.device)
        os = _heads(out, heads, dim, dtype, dev, "out")
        if out.shape[0] != t:
            raise ValueError("out: one row for each token")
        qp, op = q.data_ptr(), out.data_ptr()
        w = 2 * heads * dim
        if (given and qp < op + 2 * (t - 1) * os + w and op < qp + 2 * (t - 1) * qs + w
                and _overlap(op, 2 * os, w, qp, 2 * qs, w, t)):
            raise ValueError("out: no memory of q")
        # (the library's call takes 32 and 64 bits of them, and refuses what is out of its range in these)
        if not (-2**31 <= window < 2**31 and -2**63 <= max_q < 2**63):
            raise ValueError("window, max_q: out of range")
        lp = None
        if lse is not None:
            _floats(lse, t * heads, dev, "lse")
            lp = lse.data_ptr()
        rc = _call("fc_gguf_kv_attend")(self._h, qp, qs, heads, t, cu_q.data_ptr(), kv_lens.data_ptr(), seqs,
                                        table.data_ptr(), ts, width, max_q,
                                        self.scale if scale is None else scale, window, op, os, lp, _stream(dev))
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
    dev, dtype = x.get_device(), DTYPES.get(x.dtype)
    if dev < 0 or dtype is None or x.dim() != 2:
        raise ValueError("x: f16, bf16 or f32 [rows, vocab] on the GPU")
    rows, vocab = x.shape
    given = out is not None
    if not given:
        out = torch.empty((rows, vocab), dtype=torch.float32, device=x.device)
    out_dtype = DTYPES.get(out.dtype)
    if out_dtype is None or out.get_device() != dev or out.shape != x.shape:
        raise ValueError(f"out: [{rows}, {vocab}] on cuda:{dev}")
    xs, one = x.stride()
    os, out_one = out.stride()
    if (one != 1 or out_one != 1) and vocab > 1:
        raise ValueError("x and out: contiguous rows")
    if rows <= 1:
        xs, os = max(xs, vocab), max(os, vocab)
    xp, op = x.data_ptr(), out.data_ptr()
    if given and (xp != op or xs != os or dtype != out_dtype):
        size, out_size = 4 if dtype == F32 else 2, 4 if out_dtype == F32 else 2
        if _overlap(op, out_size * os, out_size * vocab, xp, size * xs, size * vocab, rows):
            raise ValueError("out: x itself, or other memory")
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
    rp = fp = sp = None
    if repetition is not None:
        _floats(repetition, rows, dev, "repetition")
        rp = repetition.data_ptr()
    if frequency is not None:
        _floats(frequency, rows, dev, "frequency")
        fp = frequency.data_ptr()
    if presence is not None:
        _floats(presence, rows, dev, "presence")
        sp = presence.data_ptr()
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
    if torch.cuda.current_device() != dev:
        raise ValueError(f"x: on the current device, not on cuda:{dev}")
    rc = _call("fc_gguf_logits")(xp, xs, dtype, rows, vocab, tp, ts, lp, pp, rp, fp, sp, bo, bi, bv, bn, mp, ms,
                                 op, os, out_dtype, _stream(dev))
    if rc != 0:
        _check(rc, "fc_gguf_logits")
    return out
