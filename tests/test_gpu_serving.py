"""The serving operators (paged cache with rotation and append, attention over
it, logits processing) through the binding, against the float64 oracle.

Tolerances come from the formats and the order of the arithmetic, element by
element: a rounding to a type is off by half a step (finfo.eps / 2 of the
value; 2^-25 for f16 below its normal range), an f32 operation by 2^-24, an
f32 sum of n products by n 2^-24 of the sum of magnitudes (2^-23 is taken for
sums inside the matrix instructions).
"""

import numpy as np
import pytest
import torch

from helpers import guarded
from oracle import serving as o

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _np(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _kv(pages, ps, hk, D, dtype, fill=None):
    from gguf_quant_block_amd.serving import PagedKv
    kv = PagedKv(pages, ps, hk, D, dtype)
    if fill is not None:
        kv.k.fill_(fill)
        kv.v.fill_(fill)
    return kv


# ---------------------------------------------------------------- append

def _check_append(kv, k0, v0, q, k, v, slots, positions, f, axis, inter, scale, out):
    dtype = kv.dtype
    half = _half(dtype)
    wants = []
    for x in (q, k):
        if f is None:
            wants.append((_np(x), np.zeros(x.shape)))
        else:
            wants.append(o.rotate(_np(x), np.atleast_2d(positions), f, axis, inter, scale))

    def near(y, want, mag):
        tol = half * np.abs(want) * (mag > 0) + 2.0 ** -21 * mag + (2.0 ** -25 if dtype == F16 else 0) * (mag > 0)
        assert (np.abs(y - want) <= tol).all(), float((np.abs(y - want) - tol).max())

    if out is not None:
        near(_np(out), *wants[0])
    kp, vp, vn = _np(kv.k), _np(kv.v), _np(v)
    touched_k, touched_v = np.zeros(kp.shape, bool), np.zeros(vp.shape, bool)
    ps = kv.page_size
    for t, s in enumerate(np.asarray(slots)):
        if 0 <= s < kv.pages * ps:
            near(o.key_slot(kp, s), wants[1][0][t], wants[1][1][t])
            assert np.array_equal(o.value_slot(vp, s), vn[t])
            touched_k[s // ps, :, :, s % ps] = True
            touched_v[s // ps, :, (s % ps) // 8, :, s % 8] = True
    assert np.array_equal(kp[~touched_k], k0[~touched_k]) and np.array_equal(vp[~touched_v], v0[~touched_v])


# (dtype, heads, kv heads, D, rot, interleaved, axes, page size, tokens, how slots run)
APPEND = [
    (F16, 32, 32, 96, 96, False, 1, 64, 1, "step"),
    (F16, 4, 1, 64, 64, True, 1, 16, 2, "prompt"),
    (BF16, 5, 5, 128, 128, False, 1, 16, 67, "prompt"),
    (BF16, 16, 2, 128, 64, False, 3, 32, 131, "prompt"),
    (F16, 6, 3, 256, 256, True, 3, 256, 40, "step"),
    (F16, 8, 4, 64, 16, True, 1, 128, 33, "holes"),
    (BF16, 2, 1, 96, 48, False, 2, 32, 2100, "prompt"),
    (F16, 2, 2, 64, 32, False, 1, 16, 4500, "holes"),
    (BF16, 0, 2, 128, 128, True, 1, 64, 19, "prompt"),
]


def _slots(how, T, ps, g):
    """Slots of T tokens and a page count: scattered, in order from the middle of
    a page, or in order with gaps, skipped tokens and a step back."""
    if how == "step":
        pages = T + 2
        return np.argsort(g.random(pages))[:T] * ps + g.integers(0, ps, T), pages
    pages = (T + 5) // ps + 4
    order = np.argsort(g.random(pages))
    at = 5 + np.arange(T)
    s = order[at // ps] * ps + at % ps
    if how == "holes":
        s[g.random(T) < 0.15] = -1
        s[T // 2] = pages * ps                  # the first slot past the cache
        s[T // 3:T // 3 + 6] = s[T // 3:T // 3 + 6][::-1].copy()
    return s, pages


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_append(gpu_lib, case):
    from gguf_quant_block_amd.serving import Rope
    dtype, hq, hk, D, rot, inter, axes, ps, T, how = case
    g = np.random.default_rng(sum(case[1:5]) + T)
    tg = torch.Generator().manual_seed(T)
    slots, pages = _slots(how, T, ps, g)
    kv = _kv(pages, ps, hk, D, dtype, fill=7.0)
    k0, v0 = _np(kv.k), _np(kv.v)
    # one projection's rows, and a few unused columns after them
    qkv = _randn(tg, (T, (hq + 2 * hk) * D + 24), dtype)
    q = qkv[:, :hq * D].unflatten(1, (hq, D)) if hq else None
    k = qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    v = qkv[:, (hq + hk) * D:(hq + 2 * hk) * D].unflatten(1, (hk, D))
    f = torch.tensor([10000.0 ** (-2 * j / rot) for j in range(rot // 2)], dtype=F32, device="cuda")
    axis = _i32(g.integers(0, axes, rot // 2)) if axes > 1 else None
    pos = g.integers(0, 200000, (axes, T))
    rope = Rope(f, axis=axis, interleaved=inter, scale=1.0 if axes > 1 else 1.19)
    out, guards = guarded((T, hq, D), dtype, seed=T) if hq else (None, lambda: None)
    got = kv.append(q, k, v, _i32(slots), _i32(pos if axes > 1 else pos[0]), rope, out=out)
    assert got is out
    guards()
    _check_append(kv, k0, v0, q if hq else k, k, v, slots, pos, _np(f), None if axis is None else _np(axis), inter,
                  rope.scale, out)


def test_append_in_place_without_rotation_and_far_positions(gpu_lib):
    from gguf_quant_block_amd.serving import Rope
    tg = torch.Generator().manual_seed(3)
    T, hq, hk, D, ps = 21, 4, 2, 64, 16
    f = torch.tensor([1.0, 0.37] * 16, dtype=F32, device="cuda")
    for rope, pos in ((None, None), (Rope(f), np.array([2**31 - 1 - i for i in range(T)])), (Rope(f), -np.arange(T))):
        slots, pages = _slots("prompt", T, ps, np.random.default_rng(0))
        kv = _kv(pages, ps, hk, D, F16, fill=0.0)
        q, k, v = (_randn(tg, (T, h, D), F16) for h in (hq, hk, hk))
        q_before = q.clone()
        y = kv.append(q, k, v, _i32(slots), None if pos is None else _i32(pos), rope, out=q)
        assert y is q
        z = np.zeros
        _check_append(kv, z(kv.k.shape), z(kv.v.shape), q_before, k, v, slots, pos, None if rope is None else _np(f), None,
                      False, 1.0, y)


def test_append_nothing(gpu_lib):
    kv = _kv(2, 16, 1, 64, F16, fill=1.0)
    e = torch.empty((0, 1, 64), dtype=F16, device="cuda")
    assert kv.append(e, e, e, _i32([])).shape == (0, 1, 64)
    assert (_np(kv.k) == 1).all()


# ---------------------------------------------------------------- attend

def _layout(kvs, ps, g, spare=3):
    """A table of shuffled pages for kvs keys (entries past a sequence's last: -1)."""
    used = [-(-max(n, 0) // ps) for n in kvs]
    pages = sum(used) + spare
    order = np.argsort(g.random(pages))
    table = np.full((len(kvs), max(max(used), 1)), -1)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    return table, pages


def _fill(kv, table, kvs, tg, scale=1.0, stale=float("nan")):
    """Random keys and values where the sequences have them; `stale` elsewhere."""
    kv.k.copy_(_randn(tg, kv.k.shape, kv.dtype, scale))
    kv.v.copy_(_randn(tg, kv.v.shape, kv.dtype))
    ps = kv.page_size
    live = torch.zeros((kv.pages, ps), dtype=torch.bool)
    for s, n in enumerate(kvs):
        for p in range(-(-max(n, 0) // ps)):
            if 0 <= table[s][p] < kv.pages:
                live[int(table[s][p]), :max(0, min(ps, n - p * ps))] = True
    dead = ~live.cuda()
    kv.k.masked_fill_(dead[:, None, None, :, None], stale)
    kv.v.masked_fill_(dead.view(kv.pages, 1, ps // 8, 1, 8), stale)


def _near_attend(out, lse, r, dtype, D):
    half = _half(dtype)
    want, keys = r["out"], r["keys"][..., None]
    score = (D + 8) * 2.0 ** -23 * r["score"][..., None]          # error of a score
    weight = 2 * score + 2.0 ** -21 + (keys + 64) * 2.0 ** -23    # of a weight and of the sums, relative
    tol = r["mass"] * (1.01 * half + weight) + half * np.abs(want)
    if dtype == F16:
        tol = tol + 2.0 ** -25 * (1 + r["vsum"])
    fine = np.isfinite(want)                                      # where it is not, the same infinity or NaN
    assert np.array_equal(out[~fine], want[~fine], equal_nan=True)
    err = np.where(fine, np.abs(np.where(fine, out, 0) - np.where(fine, want, 0)), 0)
    ok = ~fine | (err <= tol)
    assert ok.all(), f"{int((~ok).sum())} of {ok.size} off, worst {float(np.nanmax(err / np.maximum(tol, 1e-30))):.2f} tolerances"
    if lse is not None:
        tl = score[..., 0] + 2.0 ** -20 + (r["keys"] + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0))
        fine = np.isfinite(r["lse"])
        assert np.array_equal(lse[~fine], r["lse"][~fine], equal_nan=True)
        assert (np.abs(lse - r["lse"])[fine] <= tl[fine]).all()


def _attend_case(dtype, D, ps, hk, G, kvs, news, window=0, seed=0, table_edit=None, value_edit=None, max_q=None,
                 scale=None, stale=float("nan"), qscale=1.0, packed=False):
    g, tg = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    table, pages = _layout(kvs, ps, g)
    kv = _kv(pages, ps, hk, D, dtype)
    if table_edit:
        table_edit(table)
    _fill(kv, table, kvs, tg, stale=stale)
    if value_edit:
        value_edit(kv, table)
    cu = np.concatenate([[0], np.cumsum(news)])
    T, H = int(cu[-1]), hk * G
    q = _randn(tg, (T, H + (2 if packed else 0), D), dtype, qscale)[:, :H]
    lse, lse_guard = guarded((T, H), F32, seed=seed)
    out, guard = guarded((T, H, D), dtype, seed=seed + 1)
    sc = D ** -0.5 if scale is None else scale
    got = kv.attend(q, _i32(cu), _i32(kvs), _i32(table), max(news) if max_q is None else max_q, scale=scale, window=window,
                    out=out, lse=lse)
    assert got is out
    guard()
    lse_guard()
    r = o.attend(_np(q), _np(kv.k), _np(kv.v), cu, kvs, table, sc, window)
    _near_attend(_np(out), _np(lse), r, dtype, D)
    return kv, q, cu, table, out, lse


ONES = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,ps,hk,G", [(64, 16, 2, 1), (96, 32, 3, 1), (128, 64, 1, 4), (256, 128, 1, 2), (128, 256, 2, 8),
                                       (64, 16, 1, 16), (96, 16, 1, 20)])
def test_attend_single_tokens(gpu_lib, dtype, D, ps, hk, G):
    _attend_case(dtype, D, ps, hk, G, ONES, [1] * len(ONES), seed=D + G)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,ps,hk,G,window", [(64, 16, 2, 3, 0), (96, 64, 1, 1, 0), (128, 32, 1, 8, 0), (256, 16, 1, 1, 0),
                                              (64, 32, 1, 4, 1), (128, 16, 2, 2, 33), (96, 16, 1, 5, 64), (256, 64, 1, 3, 7)])
def test_attend_chunks_beside_single_tokens(gpu_lib, dtype, D, ps, hk, G, window):
    # whole prompts, chunks over earlier keys, single tokens, nothing new, no keys, more rows than keys
    kvs, news = [77, 200, 301, 64, 5, 0, 3, 130, 40], [77, 65, 1, 33, 5, 1, 6, 0, 2]
    _attend_case(dtype, D, ps, hk, G, kvs, news, window=window, seed=D + window)


@pytest.mark.parametrize("dtype,D,hk,G,kv,new,window", [(F16, 128, 1, 1, 5003, 1, 0), (BF16, 96, 2, 4, 3001, 3, 0),
                                                        (F16, 64, 1, 2, 4097, 9, 700), (BF16, 256, 1, 1, 2050, 2, 0),
                                                        (F16, 128, 1, 4, 2300, 150, 0), (BF16, 64, 1, 8, 1500, 70, 333)])
def test_attend_long_caches(gpu_lib, dtype, D, hk, G, kv, new, window):
    _attend_case(dtype, D, 32, hk, G, [kv], [new], window=window, seed=kv)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attend_peaked_and_flat_scores(gpu_lib, dtype):
    # scores far apart (one key takes nearly all), growing maxima, and all equal
    _attend_case(dtype, 64, 16, 1, 2, [900, 33], [3, 33], qscale=40.0, seed=1)
    _attend_case(dtype, 64, 16, 1, 2, [900, 33], [3, 33], qscale=0.0, seed=2)
    _attend_case(dtype, 128, 16, 1, 1, [260, 300], [260, 1], scale=3.0, seed=3)
    _attend_case(dtype, 128, 16, 1, 1, [260, 300], [260, 1], scale=1e-30, seed=3)

    def rising(kv, table):          # each key's score above the one before
        for j in range(700):
            s = int(table[0][j // 16]) * 16 + j % 16
            kv.k[s // 16, :, :, s % 16] = j / 64

    _attend_case(dtype, 64, 16, 1, 1, [700], [130], value_edit=rising, seed=4)


@pytest.mark.parametrize("new", [1, 3, 60])
def test_attend_pages_outside_the_pool_take_no_part(gpu_lib, new):
    def edit(table):
        table[0, 1], table[0, 4], table[1, 0], table[2, :] = -1, 10**9, -2**31, 2**31 - 1

    _attend_case(F16, 64, 16, 2, 2, [100, 90, 33], [new] * 3, seed=new, table_edit=edit)


def test_attend_lengths_past_the_table_and_rows_past_max_q(gpu_lib):
    g, tg = np.random.default_rng(5), torch.Generator().manual_seed(5)
    table, pages = _layout([64, 64], 16, g)
    kv = _kv(pages, 16, 1, 64, F16)
    _fill(kv, table, [64, 64], tg)
    q = _randn(tg, (12, 2, 64), F16)
    cu, kvs = [0, 5, 12], [70, 64]                # 70 keys, 64 of them in the table
    out, lse = torch.full((12, 2, 64), 9.0, dtype=F16, device="cuda"), torch.full((12, 2), 9.0, device="cuda")
    kv.attend(q, _i32(cu), _i32(kvs), _i32(table), 6, out=out, lse=lse)
    r = o.attend(_np(q), _np(kv.k), _np(kv.v), cu, kvs, table, 0.125, max_q=6)
    got, gl = _np(out), _np(lse)
    assert (got[11] == 9).all() and (gl[11] == 9).all() and np.isnan(r["out"][11]).all()
    keep = slice(0, 11)
    _near_attend(got[keep], gl[keep], {k: x[keep] for k, x in r.items()}, F16, 64)
    # row offsets out of order or out of range read and write nothing outside q
    kv.attend(q, _i32([-3, 40, 2]), _i32(kvs), _i32(table), 6, out=out)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("G,new", [(1, 40), (4, 3), (2, 200)])
def test_attend_masked_infinities_change_nothing(gpu_lib, dtype, bad, G, new):
    kvs = [new + 30, new + 64]

    def edit(kv, table):
        for s, j in ((0, kvs[0] - 2), (1, kvs[1] - new // 2 - 1)):
            at = int(table[s][j // 16]) * 16 + j % 16
            kv.v[at // 16, :, (at % 16) // 8, ::3, at % 8] = bad          # seen by the last rows only
        at = int(table[0][(kvs[0] - 1) // 16]) * 16 + (kvs[0] - 1) % 16
        kv.k[at // 16, :, :, at % 16] = float("nan")

    kv, q, cu, table, out, lse = _attend_case(dtype, 64, 16, 1, G, kvs, [new, new], value_edit=edit, seed=new)
    got = _np(out)
    assert np.isfinite(got[:new - 2]).all() and np.isnan(got[new - 1]).all()      # the last row sees a NaN key
    # and with a window, keys that fall out of it
    _attend_case(dtype, 64, 16, 1, G, kvs, [new, new], value_edit=edit, seed=new, window=2)


def test_attend_strided_queries_and_default_output(gpu_lib):
    kv, q, cu, table, out, lse = _attend_case(BF16, 128, 32, 2, 4, [300, 20], [40, 2], seed=9, packed=True)
    again = kv.attend(q, _i32(cu), _i32([300, 20]), _i32(table), 40)
    assert torch.equal(again, out)
    wide = torch.zeros((42, 12, 128), dtype=BF16, device="cuda")
    kv.attend(q, _i32(cu), _i32([300, 20]), _i32(table), 40, out=wide[:, 2:10])
    assert torch.equal(wide[:, 2:10], out) and not wide[:, :2].any() and not wide[:, 10:].any()


def test_attend_past_32_bit_offsets(gpu_lib):
    # the last pages of a pool of 5 GB of keys and as much of values
    hk, D, ps, dtype = 8, 128, 64, F16
    page_bytes = hk * D * ps * 2
    pages = 5 * 2**30 // page_bytes
    kv = _kv(pages, ps, hk, D, dtype)
    tg = torch.Generator().manual_seed(6)
    last = [pages - 1, pages - 3]
    n = 100
    K, V = _randn(tg, (n, hk, D), dtype), _randn(tg, (n, hk, D), dtype)
    q = _randn(tg, (2, hk, D), dtype)
    slots = [last[j // ps] * ps + j % ps for j in range(n)]
    kv.append(None, K, V, _i32(slots))
    out = kv.attend(q, _i32([0, 2]), _i32([n]), _i32([last]), 2)
    small = _kv(4, ps, hk, D, dtype)
    small.append(None, K, V, _i32([(3 if j < ps else 1) * ps + j % ps for j in range(n)]))
    want = small.attend(q, _i32([0, 2]), _i32([n]), _i32([[3, 1]]), 2)
    assert torch.equal(out, want)
    assert torch.equal(kv.k[last[0]], small.k[3]) and torch.equal(kv.v[last[0]], small.v[3])


@pytest.mark.parametrize("new", [1, 70])
def test_attend_graph_replays_with_other_lengths(gpu_lib, new):
    g, tg = np.random.default_rng(8), torch.Generator().manual_seed(8)
    kvs = [1500, 700]
    table, pages = _layout(kvs, 16, g)
    kv = _kv(pages, 16, 2, 64, F16)
    _fill(kv, table, kvs, tg)
    q = _randn(tg, (2 * new, 4, 64), F16)
    lens, cu, tab = _i32(kvs), _i32([0, new, 2 * new]), _i32(table)
    out, lse = torch.empty_like(q), torch.empty((2 * new, 4), device="cuda")
    kv.attend(q, cu, lens, tab, new, out=out, lse=lse)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        kv.attend(q, cu, lens, tab, new, out=out, lse=lse)
    torch.cuda.synchronize()
    for now in (kvs, [70, 650], [1499, 0], kvs):
        lens.copy_(_i32(now))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got, gl = out.clone(), lse.clone()
        kv.attend(q, cu, lens, tab, new, out=out, lse=lse)
        assert torch.equal(got, out) and torch.equal(gl, lse)
        _near_attend(_np(out), _np(lse), o.attend(_np(q), _np(kv.k), _np(kv.v), [0, new, 2 * new], now, table, 0.125), F16, 64)


def test_two_caches_on_two_streams(gpu_lib):
    cases = [_attend_case(F16, 128, 16, 2, 4, [3000], [1], seed=s) for s in (11, 12)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    torch.cuda.synchronize()
    for (kv, q, cu, table, out, lse), st in zip(cases, streams):
        with torch.cuda.stream(st):
            outs.append([kv.attend(q, _i32(cu), _i32([3000]), _i32(table), 1) for _ in range(5)])
    torch.cuda.synchronize()
    for (_, _, _, _, out, _), got in zip(cases, outs):
        assert all(torch.equal(x, out) for x in got)


# ---------------------------------------------------------------- logits

def _logits_case(dtype, out_dtype, rows, vocab, hist, bias_n=0, mask=False, penalties=True, seed=0, in_place=False, pad=0):
    from gguf_quant_block_amd.serving import process_logits
    g, tg = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    x = _randn(tg, (rows, vocab + pad), dtype, 4.0)[:, :vocab]
    x0 = _np(x)
    kw, okw = {}, {}
    if hist:
        tokens = np.minimum((g.random((rows, hist)) ** 2 * vocab).astype(np.int64), vocab - 1)
        tokens[:, ::7] = vocab + 5
        tokens[:, 3::11] = -4
        lens = g.integers(0, hist + 1, rows)
        lens[0] = hist + 9                                   # clamped
        prompts = lens // 3
        kw |= {"tokens": _i32(tokens), "lens": _i32(lens), "prompt_lens": _i32(prompts)}
        okw |= {"tokens": tokens, "lens": lens, "prompt_lens": prompts}
        if penalties:
            for name in ("repetition", "frequency", "presence"):
                y = torch.tensor(g.uniform(0.7, 1.4, rows), dtype=F32)
                kw[name], okw[name] = y.cuda(), y.double().numpy()
    if bias_n:
        ids = g.integers(0, vocab, rows * bias_n)            # repeated ids among them
        ids[::9] = vocab
        vals = torch.tensor(g.normal(size=rows * bias_n) * 3, dtype=F32)
        offs = np.concatenate([[0], np.sort(g.integers(0, rows * bias_n + 1, rows - 1)), [rows * bias_n]])
        kw |= {"bias_offsets": _i32(offs), "bias_ids": _i32(ids), "bias_values": vals.cuda()}
        okw["bias"] = [list(zip(ids[offs[r]:offs[r + 1]], vals.double().numpy()[offs[r]:offs[r + 1]])) for r in range(rows)]
    if mask:
        words = g.integers(-2**31, 2**31, (rows, -(-vocab // 32) + 1))
        words[-1] = 0                                        # a grammar that leaves nothing
        kw["mask"], okw["mask"] = _i32(words), words
    out = x if in_place else guarded((rows, vocab), out_dtype, seed=seed)
    guard = (lambda: None) if in_place else out[1]
    out = out if in_place else out[0]
    assert process_logits(x, out=out, **kw) is out
    guard()
    want, mag = o.logits(x0, **okw)
    got = _np(out)
    half = _half(out.dtype)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    f = np.isfinite(want)
    entries = bias_n * rows + 8
    tol = half * np.abs(want) + entries * 2.0 ** -24 * mag + (2.0 ** -25 if out.dtype == F16 else 0)
    assert (np.abs(got - want)[f] <= tol[f]).all()


@pytest.mark.parametrize("dtype,out_dtype", [(F16, F32), (F16, F16), (BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("rows,vocab,hist,bias_n,mask", [(1, 1, 3, 0, False), (1, 31, 40, 2, True), (3, 4097, 300, 70, True),
                                                         (2, 9001, 0, 3, False), (5, 1000, 17, 0, True), (2, 5000, 900, 0, False)])
def test_logits(gpu_lib, dtype, out_dtype, rows, vocab, hist, bias_n, mask):
    _logits_case(dtype, out_dtype, rows, vocab, hist, bias_n, mask, seed=vocab + hist, pad=5)


def test_logits_in_place_strided_and_without_factors(gpu_lib):
    _logits_case(F16, F16, 3, 700, 20, 4, True, in_place=True, pad=9, seed=1)
    _logits_case(F32, F32, 3, 700, 20, 4, True, in_place=True, seed=2)
    _logits_case(BF16, F32, 2, 300, 30, penalties=False, seed=3)
    _logits_case(F16, F32, 2, 40000, 0, seed=4)


def test_logits_infinities_and_repeated_biases(gpu_lib):
    from gguf_quant_block_amd.serving import process_logits
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[inf, -inf, nan, 1.0, nan, 2.0]], device="cuda")
    y = process_logits(x, mask=_i32([[0b101111]]), tokens=_i32([[1, 3, 3]]), lens=_i32([3]),
                       repetition=torch.tensor([2.0], device="cuda"), presence=torch.tensor([0.25], device="cuda"))
    got = _np(y)[0]
    assert got[0] == inf and got[1] == -inf and np.isnan(got[2]) and got[3] == 0.25 and got[4] == -inf and got[5] == 2.0
    # entries of one id are added in their order, over more than one wave's 64: (0.1f * 130 times)
    n = 130
    offs, ids = _i32([0, n]), _i32([7] * n)
    vals = torch.full((n,), 0.1, device="cuda")
    y = process_logits(torch.zeros((1, 16), device="cuda"), bias_offsets=offs, bias_ids=ids, bias_values=vals)
    s = np.float32(0)
    for _ in range(n):
        s += np.float32(0.1)
    assert _np(y)[0, 7] == float(s) and (_np(y)[0, :7] == 0).all()


def test_append_and_logits_graph_replays(gpu_lib):
    from gguf_quant_block_amd.serving import Rope, process_logits
    tg = torch.Generator().manual_seed(4)
    kv = _kv(8, 16, 2, 64, F16, fill=0.0)
    q, k, v = (_randn(tg, (9, h, 64), F16) for h in (4, 2, 2))
    slots, pos = _i32(np.arange(9) + 3), _i32(np.arange(9))
    rope = Rope(torch.rand(32, device="cuda"))
    x = torch.randn((3, 5000), device="cuda")
    tok, lens = _i32(np.arange(300).reshape(3, 100) % 60), _i32([100, 50, 0])
    freq = torch.full((3,), 0.3, device="cuda")
    out, y = torch.empty_like(q), torch.empty_like(x)

    def step():
        kv.append(q, k, v, slots, pos, rope, out=out)
        process_logits(x, tokens=tok, lens=lens, frequency=freq, out=y)

    step()
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        step()
    torch.cuda.synchronize()
    for i in range(3):
        slots.copy_(_i32(np.arange(9) + 3 + 9 * i))
        pos.add_(5)
        lens.sub_(10 * i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, y, kv.k, kv.v)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, y, kv.k, kv.v)))


# ---------------------------------------------------------------- refusals

def test_refusals(gpu_lib, monkeypatch):
    from gguf_quant_block_amd.binding import FcGgufError
    from gguf_quant_block_amd.serving import PagedKv, Rope, process_logits
    for bad, code in (((4, 24, 1, 64), -1), ((4, 8, 1, 64), -1), ((4, 512, 1, 64), -1), ((4, 16, 1, 80), -2)):
        with pytest.raises(FcGgufError) as e:
            PagedKv(*bad)
        assert e.value.code == code
    with pytest.raises(FcGgufError):
        PagedKv(4, 16, 1, 64, torch.float32)
    with pytest.raises(ValueError):
        PagedKv(4, 16, 1, 64, F16, k=torch.empty(4, 1, 8, 16, 8, dtype=F16, device="cuda"))
    kv = _kv(4, 16, 2, 64, F16, fill=3.0)
    x = torch.zeros((3, 2, 64), dtype=F16, device="cuda")
    q = torch.zeros((3, 4, 64), dtype=F16, device="cuda")
    slots = _i32([0, 1, 2])
    rope = Rope(torch.ones(32, device="cuda"))
    for args in ((q.float(), x, x, slots), (q, x[:2], x, slots), (q, x, x, slots.long()), (q, x, x, slots[:2]),
                 (q.cpu(), x, x, slots), (q, x.transpose(1, 2), x, slots), (q, x, x, slots, None, rope),
                 (q, x, x, slots, _i32([0, 1]), rope)):
        with pytest.raises(ValueError):
            kv.append(*args)
    wide = Rope(torch.ones(64, device="cuda"))             # 128 rotated dimensions of 64
    odd = Rope(torch.ones(12, device="cuda"))              # 24: not a multiple of 16
    for r in (wide, odd):
        with pytest.raises(FcGgufError) as e:
            kv.append(q, x, x, slots, slots, r)
        assert e.value.code == -1
    off = torch.zeros(3 * 2 * 64 + 8, dtype=F16, device="cuda")[1:1 + 384].view(3, 2, 64)
    with pytest.raises(FcGgufError):                        # 2 bytes past a 16-byte piece
        kv.append(q, off, x, slots)
    assert (_np(kv.k) == 3).all() and (_np(kv.v) == 3).all()
    cu, lens, table = _i32([0, 3]), _i32([3]), _i32([[0]])
    for kw in ({"scale": 0.0}, {"scale": float("nan")}, {"scale": -1.0}, {"window": -1}):
        with pytest.raises(FcGgufError):
            kv.attend(q, cu, lens, table, 3, **kw)
    with pytest.raises(FcGgufError):                        # 3 query heads over 2 key heads
        kv.attend(q[:, :3], cu, lens, table, 3)
    for args in ((q, cu.long(), lens, table, 3), (q, cu, lens, table[0], 3), (q, _i32([0, 3, 3]), lens, table, 3),
                 (q.bfloat16(), cu, lens, table, 3)):
        with pytest.raises(ValueError):
            kv.attend(*args)
    assert kv.attend(q[:0], _i32([0, 0]), lens, table, 1).shape == (0, 4, 64)
    lg = torch.zeros((2, 40), device="cuda")
    for kw in ({"tokens": _i32([[1], [2]])}, {"mask": _i32([[1, 1]])}, {"out": lg.double()}, {"repetition": torch.ones(3, device="cuda")},
               {"bias_offsets": _i32([0, 0, 0])}):
        with pytest.raises(ValueError):
            process_logits(lg, **kw)
    with pytest.raises(FcGgufError):                        # 40 bits need 2 words
        process_logits(lg, mask=_i32([[1], [1]]))
    with pytest.raises(FcGgufError) as e:                   # f32 into f16
        process_logits(lg, out=lg.half())
    assert e.value.code == -2
    # no workspace: refused, and correct once there is memory again
    long = _kv(400, 16, 2, 64, F16, fill=1.0)
    q1, tab = torch.ones((1, 2, 64), dtype=F16, device="cuda"), _i32(np.arange(400)[None])
    monkeypatch.setenv("FC_GGUF_TEST_FAIL_ALLOC", "workspace")
    with pytest.raises(FcGgufError) as e:
        long.attend(q1, _i32([0, 1]), _i32([6400]), tab, 1)
    assert e.value.code == -3
    monkeypatch.delenv("FC_GGUF_TEST_FAIL_ALLOC")
    assert (_np(long.attend(q1, _i32([0, 1]), _i32([6400]), tab, 1)) == 1).all()
    long.close()
    long.close()
