"""The choice of the next token through the binding, against rows sorted and summed in float64.

A token's weight is rounded to 2^-33 of its octave (off by 2^-34 of itself), so a running sum is off by 2^-34 of itself
and a border between two results by 2^-33 of the sum: rows whose oracle came within 2^-32 of another result say nothing
(a share below 10^-4 of them for the numbers drawn here: at most one of a case may).  The logarithm of a share is off
by 2^-33 and its rounding to f32.
"""

import numpy as np
import pytest
import torch

from helpers import guarded
from oracle import sampling as o

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _f32(x):
    return torch.tensor(np.asarray(x), dtype=F32, device="cuda")


def _check(x, u, out, logprobs, temperature=None, top_k=None, top_p=None, min_p=None):
    torch.cuda.synchronize()
    rows = x.shape[0]
    z, us = x.double().cpu().numpy(), u.double().cpu().numpy()
    get = lambda t, d: [d] * rows if t is None else t.double().cpu().numpy()  # noqa: E731
    got, lp = out.cpu().numpy(), logprobs.double().cpu().numpy()
    unsure = 0
    for r, (t, k, p, m) in enumerate(zip(get(temperature, 1.0), get(top_k, 0), get(top_p, 1.0), get(min_p, 0.0))):
        want, share, kept, margin = o.choose(z[r], us[r], t, k, p, m)
        if margin < 2.0 ** -32:
            unsure += 1
            continue
        assert got[r] == want, (r, got[r], want, kept, margin, t, k, p, m, us[r])
        assert lp[r] == share or abs(lp[r] - share) <= 2.0 ** -32 + 2.0 ** -24 * abs(share), (r, lp[r], share)
    assert unsure <= 1, unsure


def _run(x, u, **kw):
    from gguf_quant_block_amd.serving import sample
    rows = x.shape[0]
    out, guard = guarded((rows,), torch.int32, seed=rows)
    lp, lp_guard = guarded((rows,), F32, seed=rows + 1)
    assert sample(x, u, out=out, logprobs=lp, **kw) is out
    guard()
    lp_guard()
    _check(x, u, out, lp, **kw)
    return out, lp


def _case(dtype, rows, vocab, spread, seed, hidden=0.0, pad=0, **kw):
    tg = torch.Generator().manual_seed(seed)
    x = (torch.randn((rows, vocab + pad), generator=tg) * spread).to(dtype)
    if hidden:
        x[torch.rand(x.shape, generator=tg) < hidden] = -float("inf")
    x = x.cuda()[:, :vocab]
    u = torch.rand(rows, generator=tg).cuda()
    return _run(x, u, **{k: (v(rows, tg) if callable(v) else v) for k, v in kw.items() if v is not None})


def _near(a, b):
    return lambda n, g: (torch.rand(n, generator=g) * (b - a) + a).cuda()


def _whole(a, b):
    return lambda n, g: torch.randint(a, b, (n,), dtype=torch.int32, generator=g).cuda()


FILTERS = [{}, {"temperature": _near(0.3, 1.8)}, {"top_k": _whole(1, 60)}, {"top_p": _near(0.3, 0.99)}, {"min_p": _near(0.01, 0.4)},
           {"temperature": _near(0.5, 1.2), "top_k": _whole(2, 400), "top_p": _near(0.5, 0.99), "min_p": _near(0.001, 0.1)},
           {"top_k": _whole(300, 3000), "top_p": _near(0.9, 0.999)}, {"top_p": _near(0.9, 0.9999), "min_p": _near(1e-4, 1e-2)}]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 63), (5, 1000), (7, 4097), (2, 20011), (3, 50257)])
@pytest.mark.parametrize("spread", [0.0, 0.3, 2.0, 9.0])
def test_filters(gpu_lib, dtype, rows, vocab, spread):
    for i, kw in enumerate(FILTERS):
        _case(dtype, rows, vocab, spread, seed=vocab + i, pad=3 * (i % 3), hidden=0.5 if i % 2 and vocab > 60 else 0.0, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large(gpu_lib, dtype):
    for spread, kw in ((1.5, {"top_p": _near(0.9, 0.99)}), (0.05, {}), (4.0, {"temperature": _near(0.5, 1.0), "top_k": _whole(1, 2000)}),
                       (0.0, {"top_p": _near(0.2, 0.9)}), (0.5, {"top_k": _whole(20000, 90000), "min_p": _near(0.1, 0.3)})):
        _case(dtype, 4, 131073, spread, seed=int(spread * 10), **kw)


@pytest.mark.parametrize("rows", [1, 20, 130, 300])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_parts(gpu_lib, dtype, rows):
    """Rows whose tokens have to be read again, in as many parts as there are idle workgroups, and what a part finds too
    large to hand over: sorted rows, whose tokens of a bin stand in one part, and rows of few different logits."""
    tg = torch.Generator().manual_seed(rows)
    few = min(rows, 6)
    for vocab in (20000, 70001):
        x = torch.randn((few, vocab), generator=tg) * 1.2
        x = torch.cat([x.sort(dim=-1, descending=True)[0][:few // 2], x.sort(dim=-1)[0][few // 2:]])
        ties = torch.randint(0, 5, (few, vocab), generator=tg).float()
        for z in (x, ties):
            z = z.to(dtype).cuda().repeat(-(-rows // few), 1)[:rows].contiguous()
            u = torch.rand(few, generator=tg).cuda().repeat(-(-rows // few))[:rows].contiguous()
            n = min(rows, 4)
            for kw in ({}, {"top_p": 0.8}, {"top_k": 3000}, {"min_p": 0.05}, {"top_k": 9000, "top_p": 0.9, "min_p": 0.01}):
                full = {k: torch.full((rows,), v, dtype=torch.int32 if k == "top_k" else F32, device="cuda") for k, v in kw.items()}
                from gguf_quant_block_amd.serving import sample
                lp = torch.empty(rows, device="cuda")
                out = sample(z, u, logprobs=lp, **full)
                _check(z[:n], u[:n], out[:n], lp[:n], **{k: v[:n] for k, v in full.items()})
                assert all(torch.equal(out[i::few], out[i:i + 1].expand_as(out[i::few])) for i in range(few))


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("temperature", [4.0, 30.0, 1e4])
def test_bins_about_zero(gpu_lib, dtype, temperature):
    """Wide bins about 0, where logits stand many exponents apart, are taken apart over several levels."""
    tg = torch.Generator().manual_seed(int(temperature))
    for vocab, spread in ((2048, 0.73), (5000, 0.05), (40000, 1.0)):
        x = torch.randn((60, vocab), generator=tg) * spread * 10.0 ** (torch.randn((60, vocab), generator=tg) * 0.5)
        x, u = x.to(dtype).cuda(), torch.rand(60, generator=tg).cuda()
        t = torch.full((60,), temperature, device="cuda")
        for kw in ({}, {"top_p": torch.full_like(t, 0.9)}, {"top_k": _i32([vocab // 3] * 60)}, {"min_p": torch.full_like(t, 0.8)}):
            out, lp = _run(x, u, temperature=t, **kw)
            again, _ = _run(x, u, temperature=t, **kw)
            assert torch.equal(out, again)


@pytest.mark.parametrize("vocab", [4097, 33001, 131073])
def test_logits_next_to_each_other(gpu_lib, vocab):
    """Equal logits, and f32 steps from 1: the ids, or the last bits, say what the order is.  131073 steps of 2^-23 are 2^-6:
    weights differ by 1.6 %, and the share of the first k tokens from k / vocab by less."""
    u = _f32([0.0, 0.1, 0.5, 0.77, 0.999])
    equal = torch.full((5, vocab), 0.25, device="cuda")
    steps = torch.arange(vocab, dtype=torch.float64).mul(2.0**-23).add(1.0).float().flip(0).repeat(5, 1).cuda()
    for x in (equal, steps):
        for kw in ({}, {"top_p": _f32([0.3] * 5)}, {"top_k": _i32([vocab // 2] * 5)}):
            out, _ = _run(x, u, **kw)
            part = 0.3 if "top_p" in kw else 0.5 if "top_k" in kw else 1.0
            assert ((out.double() / vocab - u.double() * part).abs() < 2.0**-5 + 2 / vocab).all()


def test_borders(gpu_lib):
    """Settings at their ends, random numbers at theirs, ties across borders."""
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[1.0, 3.0, 3.0, -2.0, 3.0, 0.5, 1.0, -inf]], device="cuda").repeat(12, 1)
    u = _f32([0.0, 0.999999940395, 1.0, -1.0, nan, 0.3, 0.5, 0.7, 0.9, 0.95, 0.97, 0.99])
    _run(x, u)
    for k in range(0, 10):
        _run(x, u, top_k=_i32([k] * 12))
    for k in (-3, 2**31 - 1, -2**31):
        out, _ = _run(x, u, top_k=_i32([k] * 12))
    for p in (0.0, -1.0, 1e-30, 0.29, 0.31, 0.6, 0.9, 1.0, 2.0, nan, inf):
        out, lp = _run_loose(x, u, top_p=_f32([p] * 12))
        if p <= 0 or p == 1e-30:
            assert (out == 1).all() and (lp == 0).all()
    for m in (0.0, -1.0, 1e-30, 0.1, 0.2, 1.0, 1.5, nan):
        out, lp = _run_loose(x, u, min_p=_f32([m] * 12))
        if m == 1.5:
            assert (out == 1).all() and (lp == 0).all()
        if m == 1.0:
            assert set(out.tolist()) == {1, 2, 4}
    for t in (0.0, -0.0, -1.0, nan):
        out, lp = _run(x, u, temperature=_f32([t] * 12))
        assert (out == 1).all() and (lp == 0).all()
    for t in (1e-45, 1e-30, 1e-3, 1e30, 3e38, inf):
        _run_loose(x, u, temperature=_f32([t] * 12))
        _run_loose(x, u, temperature=_f32([t] * 12), top_p=_f32([0.7] * 12), min_p=_f32([0.3] * 12), top_k=_i32([5] * 12))


def _run_loose(x, u, **kw):
    """As _run, for settings whose borders may stand on a tie: run, and compare what is not at one."""
    from gguf_quant_block_amd.serving import sample
    lp = torch.empty(x.shape[0], device="cuda")
    out = sample(x, u, logprobs=lp, **kw)
    torch.cuda.synchronize()
    z, us = x.double().cpu().numpy(), u.double().cpu().numpy()
    k = {n: v.double().cpu().numpy() for n, v in kw.items()}
    for r in range(x.shape[0]):
        one = {n: v[r] for n, v in k.items()}
        if np.isnan(one.get("top_p", 0)):
            one["top_p"] = 1.0
        if one.get("top_p", 1) <= 0 or one.get("min_p", 0) > 1:
            continue
        want, share, _, margin = o.choose(z[r], us[r], **one)
        if margin >= 2.0 ** -32:
            assert out[r].item() == want, (r, out[r].item(), want, one, us[r])
            assert abs(lp[r].item() - share) <= 2.0 ** -32 + 2.0 ** -24 * abs(share)
    return out, lp


def test_infinities_and_nan(gpu_lib):
    inf, nan = float("inf"), float("nan")
    rows = [[-inf] * 6, [nan] * 6, [nan, -inf, nan, 2.0, nan, -inf], [inf, 1.0, inf, nan, -inf, 5.0], [-inf, 1.0, nan, 1.5, -inf, nan],
            [3.4e38, -3.4e38, 0.0, 3.3e38, 1.0, nan], [0.0, -0.0, 0.0, -0.0, -1.0, 0.0]]
    for dtype in (F32, BF16):
        x = torch.tensor(rows, device="cuda").to(dtype)
        for v in (0.0, 0.2, 0.4, 0.6, 0.8, 0.99):
            u = _f32([v] * len(rows))
            for kw in ({}, {"top_k": _i32([2] * len(rows))}, {"top_p": _f32([0.8] * len(rows))}, {"min_p": _f32([0.5] * len(rows))},
                       {"temperature": _f32([0.0] * len(rows))}):
                out, lp = _run(x, u, **kw)
                assert out[:2].tolist() == [-1, -1] and torch.isneginf(lp[:2]).all() and out[2].item() == 3
                assert out[3].item() in (0, 2)
    # across slices: the largest far above the others' and in another slice
    x = torch.zeros((2, 40000), device="cuda")
    x[0, 39999], x[1, 20000] = inf, 1e30
    out, lp = _run(x, _f32([0.9, 0.9]))
    assert out.tolist() == [39999, 20000] and (lp == 0).all()


def test_every_share(gpu_lib):
    """With u in the middles of a grid the counts of the tokens are their shares."""
    from gguf_quant_block_amd.serving import sample
    n, vocab = 4096, 37
    tg = torch.Generator().manual_seed(2)
    row = torch.randn(vocab, generator=tg) * 2
    x = row.cuda()[None].expand(n, vocab).contiguous()
    out = sample(x, (torch.arange(n, device="cuda") + 0.5) / n)
    want = torch.softmax(row.double(), 0)
    got = torch.bincount(out.long().cpu(), minlength=vocab) / n
    assert ((got - want).abs() <= 1.0 / n + 1e-9).all()


def test_a_row_depends_on_itself_alone(gpu_lib):
    """The same bits whatever other rows there are (and so however rows are sliced), on every call."""
    from gguf_quant_block_amd.serving import sample
    tg = torch.Generator().manual_seed(7)
    x, u = torch.randn((300, 30011), generator=tg).cuda() * 2, torch.rand(300, generator=tg).cuda()
    p = torch.full((300,), 0.95, device="cuda")
    lp = torch.empty(300, device="cuda")
    out = sample(x, u, top_p=p, logprobs=lp)
    for n in (1, 2, 40, 300):
        l2 = torch.empty(n, device="cuda")
        assert torch.equal(sample(x[:n], u[:n], top_p=p[:n], logprobs=l2), out[:n]) and torch.equal(l2, lp[:n])
    assert sample(x[:0], u[:0]).shape == (0,)


def test_graph_replays_and_streams(gpu_lib):
    from gguf_quant_block_amd.serving import process_logits, sample
    tg = torch.Generator().manual_seed(9)
    x, u = torch.randn((5, 20000), generator=tg).cuda() * 3, torch.rand(5, generator=tg).cuda()
    y, out, lp = torch.empty_like(x), torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(5, device="cuda")
    p, mask = torch.full((5,), 0.9, device="cuda"), _i32(np.random.default_rng(1).integers(-2**31, 2**31, (5, 625)))

    def step():
        process_logits(x, mask=mask, out=y)
        sample(y, u, top_p=p, out=out, logprobs=lp)

    step()
    torch.cuda.synchronize()
    graphs, stream = [torch.cuda.CUDAGraph() for _ in range(2)], torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for graph in graphs:
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            step()
    torch.cuda.synchronize()
    for i in range(4):
        u.copy_(torch.rand(5, generator=tg))
        x.mul_(0.8)
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        got = out.clone(), lp.clone()
        out.fill_(-7)
        step()
        assert torch.equal(got[0], out) and torch.equal(got[1], lp)
        _check(y, u, out, lp, top_p=p)
    # two at once
    other = torch.randn((64, 50001), generator=tg).cuda()
    v = torch.rand(64, generator=tg).cuda()
    want = sample(other, v), sample(y, u, top_p=p)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            outs[0].append(sample(other, v))
        with torch.cuda.stream(streams[1]):
            outs[1].append(sample(y, u, top_p=p))
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for got, w in zip(outs, want) for a in got)


def test_refusals(gpu_lib):
    from gguf_quant_block_amd.binding import FcGgufError
    from gguf_quant_block_amd.serving import sample
    x, u = torch.zeros((2, 40), device="cuda"), torch.zeros(2, device="cuda")
    i = _i32([1, 1])
    for args, kw in (((x.double(), u), {}), ((x[0], u), {}), ((x.cpu(), u), {}), ((x, u[:1]), {}), ((x, u.double()), {}), ((x.t(), u), {}),
                     ((x, u), {"temperature": u[:1]}), ((x, u), {"top_k": u}), ((x, u), {"top_k": i.long()}), ((x, u), {"top_p": i}),
                     ((x, u), {"min_p": u.cpu()}), ((x, u), {"out": i.long()}), ((x, u), {"out": i[:1]}), ((x, u), {"logprobs": i}),
                     ((x, u), {"out": x.view(-1)[:2].view(torch.int32)}), ((x, u), {"logprobs": u}),
                     ((x, u), {"out": u.view(torch.int32)}), ((x, u), {"out": i, "logprobs": i.view(F32)}), ((x, u), {"out": i, "top_k": i})):
        with pytest.raises(ValueError):
            sample(*args, **kw)
    for shape, code in (((2, 0), -1), ((65536, 1), -5)):
        with pytest.raises(FcGgufError) as e:
            sample(torch.zeros(shape, device="cuda"), torch.zeros(shape[0], device="cuda"))
        assert e.value.code == code
