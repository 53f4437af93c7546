"""Attention over the paged cache on every path of its kernels: tiles of 256 rows (both halves of their waves), split
tiles and their joining, the shares of the streaming kernel over few, many and empty sequences, sequences that are not
split, and calls of changing sizes on one handle.  Against float64 on the GPU; the tolerances are those of
test_gpu_serving (half a step for each rounding, the f32 sums by their length)."""

import numpy as np
import pytest
import torch

from test_gpu_serving import BF16, F16, F32, _fill, _i32, _kv, _layout, _near_attend, _np

pytestmark = pytest.mark.gpu


def _reference(q, kv, cu, kvs, table, scale, window):
    """As oracle.serving.attend, a sequence and key head at a time in float64 torch."""
    T, H, D = q.shape
    hk, ps = kv.kv_heads, kv.page_size
    G = H // hk
    r = {"out": torch.full((T, H, D), float("nan")), "lse": torch.full((T, H), float("nan")), "mass": torch.zeros(T, H, D),
         "vsum": torch.zeros(T, H, D), "score": torch.zeros(T, H), "keys": torch.zeros(T, H)}
    r = {k: x.double().cuda() for k, x in r.items()}
    for s, n in enumerate(kvs):
        a, b = int(cu[s]), int(cu[s + 1])
        if a == b:
            continue
        if n <= 0:                                  # no keys: zeros
            r["out"][a:b], r["lse"][a:b] = 0.0, -float("inf")
            continue
        pos = n - (b - a) + torch.arange(b - a, device="cuda")
        held = min(n, table.shape[1] * ps)
        page = torch.tensor(np.repeat(table[s], ps)[:held], device="cuda").long()
        good = (page >= 0) & (page < kv.pages)
        key = torch.arange(held, device="cuda")
        place = page.clamp(0, kv.pages - 1)
        see = good & (key <= pos[:, None]) & (key > pos[:, None] - window if window else True)
        for h in range(hk):
            k = torch.where(good[:, None], kv.k[place, h, :, key % ps].flatten(1).double(), 0.0)
            v = torch.where(good[:, None], kv.v[place, h, key % ps // 8, :, key % 8].double(), 0.0)
            x = q[a:b, h * G:(h + 1) * G].double().transpose(0, 1).contiguous()
            z = (scale * (x.flatten(0, 1) @ k.t())).view(G, b - a, -1).masked_fill(~see, -float("inf"))
            m = z.amax(-1, keepdim=True).clamp(min=-1e300)
            e = (z - m).exp()
            t = e.sum(-1, keepdim=True)
            w = e / torch.where(t == 0, 1.0, t)
            rows = (slice(a, b), slice(h * G, (h + 1) * G))
            put = lambda name, y: r[name].__setitem__(rows, y.transpose(0, 1))  # noqa: E731
            mm = lambda y, u: (y.flatten(0, 1) @ u).unflatten(0, (G, b - a))  # noqa: E731
            put("out", mm(w, v))
            put("lse", (m + t.log()).squeeze(-1))
            put("mass", mm(w, v.abs()))
            put("vsum", mm(see.double().expand(G, -1, -1).contiguous(), v.abs()) / torch.where(t == 0, 1.0, t))
            put("score", (scale * (x.abs().flatten(0, 1) @ k.abs().t()).view(G, b - a, -1)).masked_fill(~see, 0.0).amax(-1))
            put("keys", see.sum(-1).double().expand(G, -1).clone())
    return {k: x.cpu().numpy() for k, x in r.items()}


def _case(dtype, D, ps, hk, G, kvs, news, window=0, seed=0, edit=None, kv=None, scale=None, max_q=None, qscale=1.0):
    g, tg = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    table, pages = _layout(kvs, ps, g)
    if edit:
        edit(table)
    if kv is None:
        kv = _kv(pages, ps, hk, D, dtype)
    assert kv.pages >= pages
    _fill(kv, table, kvs, tg)
    cu = np.concatenate([[0], np.cumsum(news)])
    T, H = int(cu[-1]), hk * G
    q = (torch.randn((T, H, D), generator=tg) * qscale).to(dtype).cuda()
    out, lse = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda"), torch.full((T, H), 7.0, device="cuda")
    sc = D ** -0.5 if scale is None else scale
    kv.attend(q, _i32(cu), _i32(kvs), _i32(table), max(news) if max_q is None else max_q, scale=scale, window=window, out=out, lse=lse)
    r = _reference(q, kv, cu, kvs, table, sc, window)
    _near_attend(_np(out), _np(lse), r, dtype, D)
    return kv, q, cu, table, out, lse


# enough rows for tiles of 256: T * group / 256 * kv_heads of at least the number of CUs
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,ps,hk,G,kvs,news,window", [
    (128, 16, 64, 4, [333], [256], 0),
    (64, 64, 64, 4, [700, 40], [255, 17], 0),
    (128, 128, 32, 8, [300, 300, 90], [150, 61, 90], 0),
    (64, 32, 128, 2, [1100], [260], 100),
    (128, 64, 64, 1, [1030], [1030], 65),
    (96, 32, 64, 4, [520, 64], [250, 64], 0),
])
def test_wide_tiles(gpu_lib, dtype, D, ps, hk, G, kvs, news, window):
    _case(dtype, D, ps, hk, G, kvs, news, window=window, seed=D + ps)


def test_wide_tiles_growing_maxima_and_missing_pages(gpu_lib):
    def edit(table):
        table[0, 2], table[0, 11] = -1, 10**9

    _case(F16, 128, 16, 64, 4, [400], [256], seed=2, edit=edit, qscale=20.0)
    _case(BF16, 64, 16, 64, 4, [400], [256], seed=3, edit=edit, scale=1e-30)
    _case(F16, 64, 16, 64, 4, [400], [256], seed=4, qscale=0.0)
    # keys that grow along the sequence: the reference point has to follow in nearly every tile
    kv, q, cu, table, out, lse = _case(F16, 64, 16, 64, 4, [512], [256], seed=5)
    for j in range(512):
        kv.k[int(table[0][j // 16]), :, :, j % 16] = j / 16
    q.fill_(0.5)
    kv.attend(q, _i32(cu), _i32([512]), _i32(table), 256, out=out, lse=lse)
    _near_attend(_np(out), _np(lse), _reference(q, kv, cu, [512], table, 0.125, 0), F16, 64)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_wide_tiles_masked_infinities(gpu_lib, bad):
    for D, dtype in ((64, BF16), (128, F16)):
        kv, q, cu, table, out, lse = _case(dtype, D, 16, 64, 4, [300], [256], seed=D)
        place = (int(table[0][250 // 16]), slice(None), 250 % 16 // 8, slice(0, D, 3), 250 % 8)
        kept = kv.v[place].clone()
        want = _np(out)
        kv.v[place] = bad
        kv.attend(q, _i32(cu), _i32([300]), _i32(table), 256, out=out, lse=lse)
        got, seen = _np(out), np.arange(44, 300) >= 250
        assert np.array_equal(got[~seen], want[~seen])
        cols = np.zeros(D, bool)
        cols[::3] = True
        hit = got[seen][:, :, cols]
        assert np.isnan(hit).all() if np.isnan(bad) else (hit == bad).all()
        assert np.array_equal(got[seen][:, :, ~cols], want[seen][:, :, ~cols])
        kv.v[place] = kept


@pytest.mark.parametrize("dtype,D,ps,hk,G,kvs,news,window", [
    (F16, 128, 16, 2, 8, [9000], [64], 0),                 # a few tiles of long key ranges: split, and joined
    (BF16, 64, 64, 1, 4, [5000, 700], [40, 300], 0),
    (F16, 256, 32, 1, 2, [3000], [100], 0),
    (BF16, 96, 16, 1, 12, [4100, 90], [9, 33], 2000),
    (F16, 64, 16, 1, 1, [2000] + [60] * 70, [200] + [40] * 70, 0),   # more sequences than a wave has lanes
])
def test_split_tiles(gpu_lib, dtype, D, ps, hk, G, kvs, news, window):
    _case(dtype, D, ps, hk, G, kvs, news, window=window, seed=sum(news))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("seqs,most,D,hk,G", [(1, 20000, 64, 2, 4), (5, 4000, 128, 4, 1), (70, 1500, 64, 1, 3), (300, 1300, 96, 1, 1),
                                              (40, 3000, 64, 8, 17), (33, 2500, 256, 1, 2), (700, 900, 64, 2, 2)])
def test_shares(gpu_lib, dtype, seqs, most, D, hk, G):
    g = np.random.default_rng(seqs)
    kvs = np.exp(g.uniform(0, np.log(most), seqs)).astype(int)
    kvs[0] = most
    kvs[seqs // 2] = 0 if seqs > 1 else most
    news = np.where(g.random(seqs) < 0.1, 0, 1)            # some sequences have nothing new
    news[0] = 1
    kv, q, cu, table, out, lse = _case(dtype, D, 16, hk, G, kvs.tolist(), news.tolist(), seed=seqs)
    for _ in range(3):                                     # the same bits again: pieces are joined in one order
        again, l2 = torch.empty_like(out), torch.empty_like(lse)
        kv.attend(q, _i32(cu), _i32(kvs), _i32(table), 1, out=again, lse=l2)
        assert torch.equal(again, out) and torch.equal(l2, lse)


def test_one_handle_many_sizes(gpu_lib):
    """The workspace and its counters serve calls of growing and shrinking sizes."""
    kv = _kv(700, 16, 2, 64, F16)
    sizes = [([3000], [1]), ([50] * 90, [1] * 90), ([2000, 1500, 10], [1, 1, 1]), ([600], [300]), ([4000], [2]),
             ([100] * 60, [2] * 60), ([5000], [40]), ([3000], [1])]
    for i, (kvs, news) in enumerate(sizes):
        _case(F16, 64, 16, 2, 4, kvs, news, seed=i, kv=kv)


def test_short_sequences_where_all_could_be_long(gpu_lib):
    # max_q rows for every sequence by T, but cu_q leaves some of them with one or none, and rows of no sequence
    g, tg = np.random.default_rng(0), torch.Generator().manual_seed(0)
    kvs, cu = [300, 70, 40], [0, 1, 1, 90]
    table, pages = _layout(kvs, 16, g)
    kv = _kv(pages, 16, 1, 64, BF16)
    _fill(kv, table, kvs, tg)
    q = torch.randn((300, 4, 64), generator=tg).to(BF16).cuda()
    out, lse = torch.full((300, 4, 64), 7.0, dtype=BF16, device="cuda"), torch.full((300, 4), 7.0, dtype=F32, device="cuda")
    kv.attend(q, _i32(cu), _i32(kvs), _i32(table), 100, out=out, lse=lse)
    r = _reference(q[:90], kv, cu, kvs, table, 0.125, 0)
    _near_attend(_np(out)[:90], _np(lse)[:90], r, BF16, 64)
    assert (_np(out)[90:] == 7).all() and (_np(lse)[90:] == 7).all()


@pytest.mark.parametrize("rows,vocab", [(1, 32064), (3, 1025), (128, 9003), (600, 1030)])
def test_logits_slices(gpu_lib, rows, vocab):
    from test_gpu_serving import _logits_case
    _logits_case(F32, F32, rows, vocab, 40, 0, True, seed=rows)




def test_growth_in_a_capture_is_refused(gpu_lib):
    from gguf_quant_block_amd.binding import FcGgufError
    g = np.random.default_rng(1)
    table, pages = _layout([3000], 16, g)
    kv = _kv(pages, 16, 1, 64, F16, fill=1.0)
    q, args = torch.ones((1, 2, 64), dtype=F16, device="cuda"), (_i32([0, 1]), _i32([3000]), _i32(table), 1)
    out, y = torch.zeros_like(q), torch.zeros(4, device="cuda")
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        with pytest.raises(FcGgufError) as e:
            kv.attend(q, *args, out=out)
        y.add_(1.0)
    assert e.value.code == -3
    graph.replay()
    kv.attend(q, *args, out=out)
    assert (_np(out) == 1).all() and (_np(y) == 1).all()
