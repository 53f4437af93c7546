"""Norms of queries and keys for each head on their way into the cache, and the cache of 8 bits (append and attention)
through the binding, against the float64 oracle.

Tolerances, element by element, beside those of test_gpu_serving.py: a norm in f32 is off by (D / 2 + 8) 2^-24 (the sum
of D squares by D 2^-24 at most, halved by the root; division, root, two products), a code by half its step: 2^-4 of the
value, or 2^-10 of the scale below the codes' normal range.  Values are quantised without any arithmetic before, so
their codes are compared for equality.  Attention over 8 bits computes with values that the type holds exactly: the
tolerances are those of 16 bits.
"""

import numpy as np
import pytest
import torch

from helpers import guarded
from oracle import serving as o
from oracle import serving8 as o8
from test_gpu_serving import APPEND, BF16, F16, F32, ONES, _half, _i32, _layout, _near_attend, _np, _randn, _slots

pytestmark = pytest.mark.gpu


def _name(dtype):
    return str(dtype).replace("torch.", "")


def _bytes(t):
    torch.cuda.synchronize()
    return t.view(torch.uint8).cpu().numpy()


def _kv8(pages, ps, hk, D, dtype, seed=0):
    """A cache of 8 bits that holds arbitrary bytes."""
    from gguf_quant_block_amd.serving import PagedKv
    kv = PagedKv(pages, ps, hk, D, dtype, bits=8)
    tg = torch.Generator().manual_seed(seed)
    for x in (kv.k, kv.v, kv.k_scale, kv.v_scale):
        x.view(torch.uint8).copy_(torch.randint(0, 256, x.shape, dtype=torch.uint8, generator=tg))
    return kv


def _held(kv):
    return (o8.held(_bytes(kv.k), _bytes(kv.k_scale), _name(kv.dtype), False),
            o8.held(_bytes(kv.v), _bytes(kv.v_scale), _name(kv.dtype), True))


# ---------------------------------------------------------------- append

def _check_append(kv, before, q, k, v, slots, positions, f, inter, scale, norm, out, axis=None):
    dtype, ps = kv.dtype, kv.page_size
    D = k.shape[-1]
    eps = norm.eps if norm is not None else 0

    def want(x, w):
        x, plain = _np(x), w is None
        if w is not None:
            x = o8.head_norm(x, _np(w), eps)
        mag = np.zeros(x.shape)
        y = x
        if f is not None:
            y, mag = o.rotate(x, np.atleast_2d(positions), f, axis, inter, scale)
        err = 2.0 ** -21 * mag                                       # of f32, before the last rounding
        if w is not None:
            err = err + (D / 2 + 8) * 2.0 ** -24 * np.where(mag > 0, mag, np.abs(y))
        return y, err, plain & (mag == 0)

    def near(y, y0, err, same):
        tol = np.where(same, 0, err + _half(dtype) * (np.abs(y0) + err) + (2.0 ** -25 if dtype == F16 else 0))
        bad = np.abs(y - y0) > tol
        assert not bad.any(), (int(bad.sum()), float((np.abs(y - y0) - tol).max()))

    if out is not None:
        near(_np(out), *want(q, norm.q if norm is not None else None))
    k0, kerr, ksame = want(k, norm.k if norm is not None else None)
    there = [(t, int(s)) for t, s in enumerate(np.asarray(slots)) if 0 <= s < kv.pages * ps]
    now = [_bytes(x) if kv.bits == 8 else _np(x) for x in ((kv.k, kv.v, kv.k_scale, kv.v_scale) if kv.bits == 8 else (kv.k, kv.v))]
    touched = [np.zeros(x.shape, bool) for x in now]
    table = o8.e4m3_values()
    low, high = o8.LIMITS[_name(dtype)]
    vcodes, vexp = o8.quantise(_np(v), _name(dtype)) if kv.bits == 8 else (None, None)
    for t, s in there:
        pg, at = s // ps, s % ps
        touched[0][pg, :, :, at] = True
        touched[1][pg, :, at // 8, :, at % 8] = True
        if kv.bits == 16:
            near(o.key_slot(now[0], s), k0[t], kerr[t], ksame[t])
            assert np.array_equal(o.value_slot(now[1], s), _np(v)[t])
            continue
        touched[2][pg, :, at] = touched[3][pg, :, at] = True
        assert np.array_equal(now[3][pg, :, at].astype(int) - 127, vexp[t])
        assert np.array_equal(table[o.value_slot(now[1], s)], vcodes[t], equal_nan=True)
        e = now[2][pg, :, at].astype(int) - 127
        amax = np.abs(k0[t]).max(-1)
        slack = kerr[t].max(-1)
        assert ((low <= e) & (e <= high)).all()
        assert ((e == high) | (448 * 2.0 ** e >= amax - slack)).all() and ((e == low) | (448 * 2.0 ** (e - 1) < amax + slack)).all()
        by = 2.0 ** e[:, None]
        x = np.clip(k0[t], -240 * by, 240 * by) if (e == high).any() else k0[t]
        tol = kerr[t] + np.maximum((np.abs(x) + kerr[t]) * 2.0 ** -4, by * 2.0 ** -10)
        assert (np.abs(table[o.key_slot(now[0], s)] * by - x) <= tol).all()
    for x, b, m in zip(now, before, touched):
        assert np.array_equal(x[~m], b[~m], equal_nan=True)


def _before(kv):
    return [_bytes(x) for x in (kv.k, kv.v, kv.k_scale, kv.v_scale)] if kv.bits == 8 else [_np(kv.k), _np(kv.v)]


CASES = [(c, bits, norm) for i, c in enumerate(APPEND) for bits, norm in ((8, ("", "dim", "head", "k")[i % 4]), (16, ("dim", "head", "q")[i % 3]))]


@pytest.mark.parametrize("case,bits,kind", CASES, ids=lambda x: "-".join(str(y).replace("torch.", "") for y in x) if isinstance(x, tuple) else str(x))
def test_append(gpu_lib, case, bits, kind):
    from gguf_quant_block_amd.serving import HeadNorm, PagedKv, Rope
    dtype, hq, hk, D, rot, inter, axes, ps, T, how = case
    g = np.random.default_rng(sum(case[1:5]) + T)
    tg = torch.Generator().manual_seed(T)
    slots, pages = _slots(how, T, ps, g)
    if bits == 8:
        kv = _kv8(pages, ps, hk, D, dtype)
    else:
        kv = PagedKv(pages, ps, hk, D, dtype)
        kv.k.fill_(7.0)
        kv.v.fill_(7.0)
    before = _before(kv)
    qkv = _randn(tg, (T, (hq + 2 * hk) * D + 24), dtype, 3.0)
    q = qkv[:, :hq * D].unflatten(1, (hq, D)) if hq else None
    k = qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    v = qkv[:, (hq + hk) * D:(hq + 2 * hk) * D].unflatten(1, (hk, D))
    f = torch.tensor([10000.0 ** (-2 * j / rot) for j in range(rot // 2)], dtype=F32, device="cuda")
    axis = _i32(g.integers(0, axes, rot // 2)) if axes > 1 else None
    pos = g.integers(0, 200000, (axes, T))
    rope = Rope(f, axis=axis, interleaved=inter, scale=1.0 if axes > 1 else 1.19)
    w = lambda n: _randn(tg, (n, D) if kind == "head" else (D,), F32)  # noqa: E731
    norm = HeadNorm(w(hq) if kind != "k" and hq else None, w(hk) if kind != "q" or not hq else None, eps=1e-5) if kind else None
    out, guards = guarded((T, hq, D), dtype, seed=T) if hq else (None, lambda: None)
    got = kv.append(q, k, v, _i32(slots), _i32(pos if axes > 1 else pos[0]), rope, out=out, norm=norm)
    assert got is out
    guards()
    _check_append(kv, before, q if hq else k, k, v, slots, pos, _np(f), inter, rope.scale, norm, out, None if axis is None else _np(axis))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_append8_extremes(gpu_lib, dtype, D):
    """Heads of zeros, of the type's largest and smallest, at the scale's borders, infinite and NaN values among others."""
    T, hk, ps = 29, 3, 16
    g, tg = np.random.default_rng(D), torch.Generator().manual_seed(D)
    slots, pages = _slots("prompt", T, ps, g)
    kv = _kv8(pages, ps, hk, D, dtype)
    before = _before(kv)
    k = _randn(tg, (T, hk, D), dtype)
    top, small = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    for i, x in enumerate((0.0, -0.0, top, -top, small, small / 8, 448.0, 449.0, 1.75, 1.7578125, 3.5, 240 * 2.0 ** 8 if dtype == F16 else 240 * 2.0 ** 100)):
        k[i] = 0
        k[i, i % hk, i * 3 % D] = x
        k[i, (i + 1) % hk] = x
    k[14] *= 2.0 ** 12 if dtype == F16 else 2.0 ** 110
    k[15] *= 2.0 ** -13 if dtype == F16 else 2.0 ** -110
    v = k.flip(1).contiguous()
    finite = (k.clone(), v.clone())
    kv.append(None, k, v, _i32(slots))
    _check_append(kv, before, k, k, v, slots, None, None, False, 1.0, None, None)
    # and with infinite and NaN values: they become NaN, the others as if they were not there
    k[20, 0, 5], k[21, 1, D - 1], k[22, 2, 7] = float("inf"), float("-inf"), float("nan")
    k[23, 0], k[24, 1, ::2] = float("inf"), float("nan")
    v = k.flip(1).contiguous()
    before = _before(kv)
    kv.append(None, k, v, _i32(slots))
    now = _before(kv)
    table = o8.e4m3_values()
    kc, ke = o8.quantise(_np(k), _name(dtype))
    vc, ve = o8.quantise(_np(v), _name(dtype))
    for t, s in enumerate(slots):
        assert np.array_equal(now[2][s // ps, :, s % ps].astype(int) - 127, ke[t]) and np.array_equal(now[3][s // ps, :, s % ps].astype(int) - 127, ve[t])
        assert np.array_equal(table[o.key_slot(now[0], s)], kc[t], equal_nan=True)
        assert np.array_equal(table[o.value_slot(now[1], s)], vc[t], equal_nan=True)
    assert all(torch.isfinite(x).all() for x in finite)


def test_append_norm_in_place_zeros_and_no_rotation(gpu_lib):
    from gguf_quant_block_amd.serving import HeadNorm, PagedKv
    tg = torch.Generator().manual_seed(5)
    T, hq, hk, D = 9, 4, 2, 96
    kv = PagedKv(4, 16, hk, D, F16)
    kv.k.zero_()
    kv.v.zero_()
    q, k, v = (_randn(tg, (T, h, D), F16) for h in (hq, hk, hk))
    q[3] = 0
    k[4] = 0
    norm = HeadNorm(_randn(tg, (D,), F32), _randn(tg, (hk, D), F32), eps=1e-6)
    q0 = q.clone()
    before = _before(kv)
    assert kv.append(q, k, v, _i32(np.arange(T)), norm=norm, out=q) is q
    _check_append(kv, before, q0, k, v, np.arange(T), None, None, False, 1.0, norm, q)
    assert (_np(q)[3] == 0).all()


# ---------------------------------------------------------------- attend

def _fill8(kv, table, kvs, tg):
    """Keys and values of the sequences, quantised by append; arbitrary bytes elsewhere (as _kv8 leaves them)."""
    ps = kv.page_size
    slots = [int(table[s][j // ps]) * ps + j % ps for s, n in enumerate(kvs) for j in range(max(0, min(n, table.shape[1] * ps)))
             if 0 <= table[s][j // ps] < kv.pages]
    k, v = (_randn(tg, (len(slots), kv.kv_heads, kv.head_dim), kv.dtype) for _ in range(2))
    # scales of the tokens from 2^-6 to 2^6 apart
    by = 2.0 ** torch.randint(-6, 7, (len(slots), kv.kv_heads, 1), generator=tg)
    kv.append(None, k, (v * by.to("cuda", kv.dtype)), _i32(slots))


def _attend8_case(dtype, D, ps, hk, G, kvs, news, window=0, seed=0, table_edit=None, edit=None, scale=None, qscale=1.0, packed=False):
    g, tg = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    table, pages = _layout(kvs, ps, g)
    kv = _kv8(pages, ps, hk, D, dtype, seed)
    _fill8(kv, table, kvs, tg)
    if table_edit:
        table_edit(table)
    if edit:
        edit(kv, table)
    cu = np.concatenate([[0], np.cumsum(news)])
    T, H = int(cu[-1]), hk * G
    q = _randn(tg, (T, H + (2 if packed else 0), D), dtype, qscale)[:, :H]
    lse, lse_guard = guarded((T, H), F32, seed=seed)
    out, guard = guarded((T, H, D), dtype, seed=seed + 1)
    sc = D ** -0.5 if scale is None else scale
    assert kv.attend(q, _i32(cu), _i32(kvs), _i32(table), max(news), scale=scale, window=window, out=out, lse=lse) is out
    guard()
    lse_guard()
    with np.errstate(invalid="ignore"):
        r = o.attend(_np(q), *_held(kv), cu, kvs, table, sc, window)
    got = _np(out)
    # The sums are f32, of weights up to 2^12 (a bf16 row's reference point may lie so far below its largest score)
    # times up to 2^9 keys here: a value past 2^107 may take them past 2^128, whose result is infinite.
    big = (r["mass"] > 2.0 ** 107) & np.isinf(got)
    _near_attend(np.where(big, r["out"], got), _np(lse), r, dtype, D)
    return kv, q, cu, table, out, lse


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,ps,hk,G", [(64, 16, 2, 1), (96, 32, 3, 1), (128, 64, 1, 4), (256, 128, 1, 2), (128, 256, 2, 8),
                                       (64, 16, 1, 16), (96, 16, 1, 20)])
def test_attend8_single_tokens(gpu_lib, dtype, D, ps, hk, G):
    _attend8_case(dtype, D, ps, hk, G, ONES, [1] * len(ONES), seed=D + G)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,ps,hk,G,window", [(64, 16, 2, 3, 0), (96, 64, 1, 1, 0), (128, 32, 1, 8, 0), (256, 16, 1, 1, 0),
                                              (64, 32, 1, 4, 1), (128, 16, 2, 2, 33), (96, 16, 1, 5, 64), (256, 64, 1, 3, 7),
                                              (128, 64, 2, 2, 0), (96, 32, 1, 8, 0)])
def test_attend8_chunks_beside_single_tokens(gpu_lib, dtype, D, ps, hk, G, window):
    kvs, news = [77, 200, 301, 64, 5, 0, 3, 130, 40], [77, 65, 1, 33, 5, 1, 6, 0, 2]
    _attend8_case(dtype, D, ps, hk, G, kvs, news, window=window, seed=D + window)


@pytest.mark.parametrize("dtype,D,hk,G,kv,new,window", [(F16, 128, 1, 1, 5003, 1, 0), (BF16, 96, 2, 4, 3001, 3, 0),
                                                        (F16, 64, 1, 2, 4097, 9, 700), (BF16, 256, 1, 1, 2050, 2, 0),
                                                        (F16, 128, 1, 4, 2300, 150, 0), (BF16, 64, 1, 8, 1500, 70, 333),
                                                        (BF16, 128, 2, 2, 5000, 300, 0)])
def test_attend8_long_caches(gpu_lib, dtype, D, hk, G, kv, new, window):
    _attend8_case(dtype, D, 64 if new > 200 else 32, hk, G, [kv], [new], window=window, seed=kv)


@pytest.mark.parametrize("dtype,D,hk,G,new,window", [(F16, 64, 1, 1, 1, 0), (BF16, 96, 2, 3, 1, 100), (BF16, 128, 1, 8, 3, 0), (F16, 128, 3, 2, 1, 0),
                                                     (F16, 64, 1, 10, 2, 50)])
def test_attend8_many_short_sequences(gpu_lib, dtype, D, hk, G, new, window):
    # more sequences than CUs: workgroups of 4 waves
    kvs = [1 + 37 * i % 211 for i in range(300)]
    kvs[7], kvs[11], kvs[290] = 1000, 0, 513
    _attend8_case(dtype, D, 16, hk, G, kvs, [min(new, max(k, 1)) for k in kvs], window=window, seed=D + G)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attend8_peaked_and_flat_scores(gpu_lib, dtype):
    _attend8_case(dtype, 64, 16, 1, 2, [900, 33], [3, 33], qscale=40.0, seed=1)
    _attend8_case(dtype, 64, 16, 1, 2, [900, 33], [3, 33], qscale=0.0, seed=2)
    _attend8_case(dtype, 128, 16, 1, 1, [260, 300], [260, 1], scale=3.0, seed=3)
    _attend8_case(dtype, 128, 16, 1, 1, [260, 300], [260, 1], scale=1e-30, seed=3)


@pytest.mark.parametrize("new", [1, 3, 60])
def test_attend8_pages_outside_the_pool_take_no_part(gpu_lib, new):
    def edit(table):
        table[0, 1], table[0, 4], table[1, 0], table[2, :] = -1, 10**9, -2**31, 2**31 - 1

    _attend8_case(F16, 64, 16, 2, 2, [100, 90, 33], [new] * 3, seed=new, table_edit=edit)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("G,new", [(1, 40), (4, 3), (2, 200)])
def test_attend8_masked_nans_change_nothing(gpu_lib, dtype, G, new):
    kvs = [new + 30, new + 64]

    def edit(kv, table):
        for s, j in ((0, kvs[0] - 2), (1, kvs[1] - new // 2 - 1)):
            at = int(table[s][j // 16]) * 16 + j % 16
            kv.v.view(torch.uint8)[at // 16, :, (at % 16) // 8, ::3, at % 8] = 0x7F        # seen by the last rows only
            kv.v_scale.view(torch.uint8)[at // 16, :, at % 16] = 255                        # read as the largest that is stored
        at = int(table[0][(kvs[0] - 1) // 16]) * 16 + (kvs[0] - 1) % 16
        kv.k.view(torch.uint8)[at // 16, :, :, at % 16] = 0xFF

    kv, q, cu, table, out, lse = _attend8_case(dtype, 64, 16, 1, G, kvs, [new, new], edit=edit, seed=new)
    got = _np(out)
    assert np.isfinite(got[:new - 2]).all() and np.isnan(got[new - 1]).all()
    _attend8_case(dtype, 64, 16, 1, G, kvs, [new, new], edit=edit, seed=new, window=2)


def test_attend8_equals_16_bits_that_hold_the_same(gpu_lib):
    """The cache stands for values of the type exactly: attention over 16 bits that hold them differs by the order of its
    sums alone."""
    from gguf_quant_block_amd.serving import PagedKv
    for new, G in ((1, 4), (130, 2)):
        kv, q, cu, table, out, lse = _attend8_case(F16, 128, 64, 2, G, [900], [new], seed=new, packed=True)
        wide = PagedKv(kv.pages, 64, 2, 128, F16)
        k, v = _held(kv)
        for x, y in ((wide.k, k), (wide.v, v)):
            z = torch.from_numpy(y).cuda()
            x.copy_(z.half())
            live = torch.isfinite(z)
            assert torch.equal(x.double()[live], z[live])
        other = wide.attend(q, _i32(cu), _i32([900]), _i32(table), new)
        assert (other.double() - out.double()).abs().max() <= 2.0 ** -9 * out.double().abs().max()


def test_kv8_past_32_bit_offsets(gpu_lib):
    hk, D, ps = 8, 128, 64
    pages = 5 * 2**30 // (hk * D * ps)
    from gguf_quant_block_amd.serving import PagedKv
    kv, small = PagedKv(pages, ps, hk, D, F16, bits=8), _kv8(4, ps, hk, D, F16)
    tg = torch.Generator().manual_seed(6)
    last, n = [pages - 1, pages - 3], 100
    K, V = _randn(tg, (n, hk, D), F16), _randn(tg, (n, hk, D), F16)
    kv.append(None, K, V, _i32([last[j // ps] * ps + j % ps for j in range(n)]))
    small.append(None, K, V, _i32([(3 if j < ps else 1) * ps + j % ps for j in range(n)]))
    for m in (2, 70):
        q = _randn(tg, (m, hk, D), F16)
        out = kv.attend(q, _i32([0, m]), _i32([n]), _i32([last]), m)
        assert torch.equal(out, small.attend(q, _i32([0, m]), _i32([n]), _i32([[3, 1]]), m))


@pytest.mark.parametrize("new", [1, 70])
def test_kv8_graph_replays(gpu_lib, new):
    """Norm, rotation, append into 8 bits and attention in one captured graph, replayed with other places and lengths."""
    from gguf_quant_block_amd.serving import HeadNorm, Rope
    g, tg = np.random.default_rng(8), torch.Generator().manual_seed(8)
    hk, D, ps, room = 2, 64, 16, 1600
    table, pages = _layout([room], ps, g)
    kv = _kv8(pages, ps, hk, D, BF16)
    _fill8(kv, table, [room], tg)
    q, k, v = (_randn(tg, (new, h, D), BF16) for h in (4, hk, hk))
    rope = Rope(torch.tensor([1.0 / (i + 1) for i in range(32)], device="cuda"))
    norm = HeadNorm(_randn(tg, (4, D), F32), _randn(tg, (hk, D), F32))
    lens, cu, tab, slots, pos = _i32([900]), _i32([0, new]), _i32(table), _i32([0] * new), _i32([0] * new)
    y, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((new, 4), device="cuda")

    def step():
        kv.append(q, k, v, slots, pos, rope, out=y, norm=norm)
        kv.attend(y, cu, lens, tab, new, out=out, lse=lse)

    def place(n):
        at = np.arange(n - new, n)
        slots.copy_(_i32(table[0][at // ps] * ps + at % ps))
        pos.copy_(_i32(at))
        lens.fill_(n)

    place(room)
    step()
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        step()
    torch.cuda.synchronize()
    for n in (900, 75, 1501, room):
        place(n)
        q.mul_(0.75)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, out, lse, kv.k.view(torch.uint8), kv.k_scale.view(torch.uint8))]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, out, lse, kv.k.view(torch.uint8), kv.k_scale.view(torch.uint8))))
        _near_attend(_np(out), _np(lse), o.attend(_np(y), *_held(kv), [0, new], [n], table, D ** -0.5), BF16, D)


def test_two_caches_of_8_bits_on_two_streams(gpu_lib):
    cases = [_attend8_case(F16, 128, 16, 2, 4, [3000], [1], seed=s) for s in (11, 12)]
    outs = []
    torch.cuda.synchronize()
    for (kv, q, cu, table, out, lse), st in zip(cases, [torch.cuda.Stream() for _ in cases]):
        with torch.cuda.stream(st):
            outs.append([kv.attend(q, _i32(cu), _i32([3000]), _i32(table), 1) for _ in range(5)])
    torch.cuda.synchronize()
    for (_, _, _, _, out, _), got in zip(cases, outs):
        assert all(torch.equal(x, out) for x in got)


def test_refusals(gpu_lib):
    from gguf_quant_block_amd.binding import FcGgufError
    from gguf_quant_block_amd.serving import HeadNorm, PagedKv
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    k, v = u8(4, 2, 8, 16, 8).view(torch.float8_e4m3fn), u8(4, 2, 2, 64, 8).view(torch.float8_e4m3fn)
    s = u8(4, 2, 16).view(torch.float8_e8m0fnu)
    for kw in ({"bits": 4}, {"bits": 8, "k": k, "v": v}, {"bits": 8, "k": k.half(), "v": v.half(), "k_scale": s, "v_scale": s},
               {"k_scale": s, "v_scale": s}, {"bits": 8, "k": k, "v": v, "k_scale": s, "v_scale": s.view(torch.uint8)},
               {"bits": 8, "k": k, "v": v, "k_scale": s, "v_scale": u8(4, 2, 8).view(torch.float8_e8m0fnu)}):
        with pytest.raises(ValueError):
            PagedKv(4, 16, 2, 64, F16, **kw)
    kv = PagedKv(4, 16, 2, 64, F16, bits=8, k=k, v=v, k_scale=s, v_scale=s.clone())
    x, q, slots = torch.ones((3, 2, 64), dtype=F16, device="cuda"), torch.ones((3, 4, 64), dtype=F16, device="cuda"), _i32([0, 1, 2])
    with pytest.raises(ValueError):
        HeadNorm()
    for bad in (torch.ones(64), torch.ones(64, device="cuda", dtype=F16), torch.ones((2, 2, 64), device="cuda")):
        with pytest.raises(ValueError):
            HeadNorm(bad)
    one = torch.ones(64, device="cuda")
    for norm in (HeadNorm(torch.ones(96, device="cuda")), HeadNorm(torch.ones((2, 64), device="cuda")), HeadNorm(one, torch.ones((4, 64), device="cuda"))):
        with pytest.raises(ValueError):
            kv.append(q, x, x, slots, norm=norm)
    for norm in (HeadNorm(one, eps=-1.0), HeadNorm(one, eps=float("nan")), HeadNorm(one, eps=float("inf")),
                 HeadNorm(torch.ones(65, device="cuda")[1:])):          # weights 4 bytes past 16
        with pytest.raises(FcGgufError) as e:
            kv.append(q, x, x, slots, norm=norm)
        assert e.value.code == -1
    assert not _bytes(kv.k).any()
    kv.append(q[:0], x[:0], x[:0], slots[:0], norm=HeadNorm(one))
