"""The serving operators between the fully-connected layers of a decoder, as cases to be measured: appending
rotated keys and values to a paged cache, attention of new tokens over that cache, and the processing of the
output layer's logits.  `run` computes a case in elementary torch operations, or, where `own` is true, through
the package's entry points."""

import math
import random

import torch

own = False

DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    append = {"op": "append", "dtype": "float16", "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128,
              "interleaved": False, "axes": 1, "page": 64}
    attend = {"op": "attend", "dtype": "float16", "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "seqs": 1,
              "ragged": False, "window": 0}
    logits = {"op": "logits", "dtype": "float16", "out": "float32", "ragged": True}
    return [
        # one token of one conversation, every query head with a key head of its own: latency is all that counts
        {**append, "name": "append-1", "kv_heads": 32, "head_dim": 96, "rot": 96, "tokens": 1, "start": 4095},
        # one decode step of a busy server: each token goes to another sequence's page
        {**append, "name": "append-batch-128", "dtype": "bfloat16", "rot": 64, "tokens": 128, "start": 30011, "step": True},
        # a chunk of a long prompt, which begins in the middle of a page
        {**append, "name": "append-prompt-4096", "tokens": 4096, "start": 8197},
        # the patches of an image among text: time, height and width, pairs next to each other, pages of 16
        {**append, "name": "append-image-3-axes", "dtype": "bfloat16", "interleaved": True, "axes": 3, "page": 16,
         "tokens": 2500, "start": 333},
        # one token of one conversation, every query head with a key head of its own
        {**attend, "name": "attend-1", "kv_heads": 32, "head_dim": 96, "kv": 1003, "new": 1},
        # one decode step of a busy server, conversations of all lengths
        {**attend, "name": "attend-batch-64", "dtype": "bfloat16", "seqs": 64, "kv": 8192, "new": 1, "ragged": True},
        # one token over a long document
        {**attend, "name": "attend-long-1", "kv": 131072, "new": 1},
        # a few drafted tokens of some sequences are verified at once
        {**attend, "name": "attend-draft-8x5", "dtype": "bfloat16", "seqs": 8, "kv": 6001, "new": 5, "page": 16,
         "ragged": True},
        # a chunk of a prompt over what was cached before
        {**attend, "name": "attend-chunk-4096", "kv": 8192, "new": 4096},
        # chunks and single tokens in one step, keys inside a window
        {**attend, "name": "attend-mixed-window", "dtype": "bfloat16", "heads": 16, "kv_heads": 4, "head_dim": 64,
         "seqs": 12, "kv": 5003, "new": 1031, "page": 32, "ragged": True, "window": 2047},
        # the next token of one conversation
        {**logits, "name": "logits-1", "rows": 1, "vocab": 32064, "history": 700, "bias": 5, "mask": True},
        # one decode step of a busy server, a larger vocabulary
        {**logits, "name": "logits-batch-128", "dtype": "float32", "rows": 128, "vocab": 131073, "history": 4096,
         "bias": 40, "mask": True},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "logits"))
    dtype = rng.choice(("float16", "bfloat16"))
    if op == "logits":
        rows = _spread(rng, 1, 128)
        return {"op": op, "dtype": rng.choice(("float16", "bfloat16", "float32")), "out": "float32", "rows": rows,
                "vocab": _spread(rng, 1009, 131073), "history": _spread(rng, 1, 4096), "bias": _spread(rng, 1, 40),
                "mask": rng.random() < 0.5, "ragged": True}
    head_dim = rng.choice((64, 96, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    c = {"op": op, "dtype": dtype, "kv_heads": kv_heads, "heads": kv_heads * rng.choice((1, 2, 3, 4, 8)),
         "head_dim": head_dim, "page": rng.choice((16, 32, 64, 128))}
    if c["heads"] * head_dim > 4096:
        c["heads"] = kv_heads
    if op == "append":
        c |= {"rot": rng.choice((head_dim, head_dim // 2)), "interleaved": rng.random() < 0.5,
              "axes": rng.choice((1, 1, 3)), "tokens": _spread(rng, 1, 4096), "start": _spread(rng, 1, 100000)}
        c["step"] = c["tokens"] <= 256 and rng.random() < 0.5
        return c
    if rng.random() < 0.5:  # single and drafted tokens
        seqs = _spread(rng, 1, 64)
        c |= {"seqs": seqs, "kv": _spread(rng, 17, 131072 // seqs), "new": rng.choice((1, 1, 1, 2, 5, 11))}
    else:                   # chunks
        seqs = rng.choice((1, 2, 3, 8))
        c |= {"seqs": seqs, "kv": _spread(rng, 33, 8192 // seqs)}
        c["new"] = _spread(rng, 16, min(c["kv"], 4096 // seqs))
    c |= {"ragged": rng.random() < 0.7, "window": rng.choice((0, 0, 129, 1024))}
    return c


def _lengths(case):
    """Keys and new tokens of each sequence of an attention case; the first sequence has the largest of both."""
    kv, new, n = case["kv"], min(case["new"], case["kv"]), case["seqs"]
    if not case["ragged"]:
        return [kv] * n, [new] * n
    rng = random.Random("%d %d %d" % (kv, new, n))
    kvs = [kv] + [_spread(rng, max(1, kv // 16), kv) for _ in range(n - 1)]
    # every other sequence decodes one token beside the chunks
    news = [new] + [min(k, 1 if i % 2 else _spread(rng, 1, new)) for i, k in enumerate(kvs[1:])]
    return kvs, news


def _seen(case):
    """(pairs, keys): query-key pairs that the mask leaves, and keys that some query sees, over the sequences."""
    pairs = keys = 0
    w = case["window"]
    for kv, new in zip(*_lengths(case)):
        first = kv - new
        if w:
            pairs += sum(min(p + 1, w) for p in range(first, kv))
            keys += kv - max(0, first - w + 1)
        else:
            pairs += new * first + new * (new + 1) // 2
            keys += kv
    return pairs, keys


def work(case):
    if case["op"] == "append":
        t, d = case["tokens"], case["head_dim"]
        return {"bytes": t * ((case["heads"] + 2 * case["kv_heads"]) * d * 2 * 2 + 4 * case["axes"] + 4),
                "flops": t * (case["heads"] + case["kv_heads"]) * case["rot"] // 2 * 6}
    if case["op"] == "attend":
        pairs, keys = _seen(case)
        t, d, h = sum(_lengths(case)[1]), case["head_dim"], case["heads"]
        return {"bytes": 2 * t * h * d * 2 + t * h * 4 + keys * case["kv_heads"] * d * 2 * 2,
                "flops": 4 * d * h * pairs}
    n, size = case["rows"] * case["vocab"], {"float32": 4}
    return {"bytes": n * (size.get(case["dtype"], 2) + 4) + (n // 8 if case["mask"] else 0)
            + sum(_history(case)) * 4 + case["rows"] * case["bias"] * 8, "flops": 6 * n}


def _history(case):
    rng = random.Random("%d %d" % (case["rows"], case["history"]))
    return [case["history"]] + [_spread(rng, 1, case["history"]) for _ in range(case["rows"] - 1)]


# ---------------------------------------------------------------- what a program has in hand

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"append": _prepare_append, "attend": _prepare_attend, "logits": _prepare_logits}[case["op"]](case, g)


def _normal(g, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(0.0, scale, generator=g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(case, pages):
    """The package's cache object and its two tensors: keys [pages, kv_heads, head_dim/8, page, 8] and values
    [pages, kv_heads, page/8, head_dim, 8]."""
    h, d, p, dtype = case["kv_heads"], case["head_dim"], case["page"], DTYPES[case["dtype"]]
    if own:
        from gguf_quant_block_amd.serving import PagedKv
        cache = PagedKv(pages, p, h, d, dtype)
        return cache, cache.k, cache.v
    return None, torch.empty((pages, h, d // 8, p, 8), dtype=dtype, device="cuda"), \
        torch.empty((pages, h, p // 8, d, 8), dtype=dtype, device="cuda")


def _prepare_append(case, g):
    t, h, hk, d, page = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    dtype, rot, axes = DTYPES[case["dtype"]], case["rot"], case["axes"]
    step = case.get("step", False)
    # a step's tokens belong to as many sequences, each with a page of its own; a prompt's follow each other
    pages = t + 2 if step else (case["start"] % page + t) // page + 3
    cache, k_pages, v_pages = _cache(case, pages)
    k_pages.normal_(0.0, 1.0, generator=g)
    v_pages.normal_(0.0, 1.0, generator=g)
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    if step:
        slots = order[i] * page + torch.randint(0, page, (t,), generator=g, device="cuda")
        positions = torch.randint(0, case["start"] + 1, (t,), generator=g, device="cuda")
    else:
        at = case["start"] % page + i
        slots = order[at // page] * page + at % page
        positions = case["start"] + i
    if axes > 1:  # a square image: time stands still, height and width walk over its patches
        side = max(1, math.isqrt(t))
        positions = torch.stack([torch.full_like(positions, case["start"]), case["start"] + i // side,
                                 case["start"] + i % side])
    qkv = _normal(g, (t, (h + 2 * hk) * d), dtype)     # the projection's output, as it stands
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([h * d, hk * d, hk * d], dim=1))
    inv_freq = torch.tensor([10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float32, device="cuda")
    # sections of the pairs for time, height and width
    axis = _ints([0 if j < rot // 8 else 1 + (j - rot // 8) * (axes - 1) // (rot // 2 - rot // 8) for j in range(rot // 2)])
    s = {"op": "append", "cache": cache, "k_pages": k_pages, "v_pages": v_pages, "q": q, "k": k, "v": v,
         "slots": slots.int(), "positions": positions.int(), "inv_freq": inv_freq, "axis": axis if axes > 1 else None,
         "interleaved": case["interleaved"], "out": torch.empty((t, h, d), dtype=dtype, device="cuda")}
    if own:
        from gguf_quant_block_amd.serving import Rope
        s["rope"] = Rope(inv_freq, axis=s["axis"], interleaved=case["interleaved"])
    return s


def _prepare_attend(case, g):
    h, hk, d, page, dtype = case["heads"], case["kv_heads"], case["head_dim"], case["page"], DTYPES[case["dtype"]]
    kvs, news = _lengths(case)
    used = [-(-n // page) for n in kvs]
    pages = sum(used) + 3
    cache, k_pages, v_pages = _cache(case, pages)
    k_pages.normal_(0.0, 1.0, generator=g)
    v_pages.normal_(0.0, 1.0, generator=g)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(kvs), max(used)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return {"op": "attend", "cache": cache, "k_pages": k_pages, "v_pages": v_pages, "window": case["window"],
            "q": _normal(g, (cu[-1], h, d), dtype, 1.5), "cu_q": _ints(cu), "kv_lens": _ints(kvs), "table": table,
            "max_q": max(news), "out": torch.empty((cu[-1], h, d), dtype=dtype, device="cuda"),
            "lse": torch.empty((cu[-1], h), dtype=torch.float32, device="cuda")}


def _prepare_logits(case, g):
    b, n, hist, nb = case["rows"], case["vocab"], case["history"], case["bias"]
    lens = _history(case)
    # generated text repeats itself: the square of an even number lies near the start of the vocabulary
    tokens = (torch.rand((b, hist), generator=g, device="cuda").square() * n).int().clamp_(max=n - 1)
    uniform = lambda low, high: torch.empty(b, device="cuda").uniform_(low, high, generator=g)  # noqa: E731
    # the biased ids of a row are distinct
    ids = torch.rand((b, n), generator=g, device="cuda").topk(nb, dim=1).indices.int().reshape(-1)
    s = {"op": "logits", "x": _normal(g, (b, n), DTYPES[case["dtype"]], 4.0), "tokens": tokens, "lens": _ints(lens),
         "prompt_lens": _ints([n // 3 for n in lens]), "repetition": uniform(1.0, 1.3), "frequency": uniform(0.0, 0.3),
         "presence": uniform(0.0, 0.3), "bias_offsets": _ints([nb * i for i in range(b + 1)]), "bias_ids": ids,
         "bias_values": _normal(g, (b * nb,), torch.float32, 3.0), "mask": None,
         "out": torch.empty((b, n), dtype=DTYPES[case["out"]], device="cuda")}
    if case["mask"]:  # a grammar leaves about a quarter of the tokens
        word = lambda: torch.randint(-2**31, 2**31, (b, -(-n // 32)), generator=g, device="cuda")  # noqa: E731
        s["mask"] = (word() & word()).int()
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return {"append": _append, "attend": _attend, "logits": _logits}[state["op"]](state)


def _append(s):
    if own:
        s["cache"].append(s["q"], s["k"], s["v"], s["slots"], s["positions"], s["rope"], out=s["out"])
        return s["out"], s["k_pages"], s["v_pages"]
    k_pages, v_pages, inv_freq = s["k_pages"], s["v_pages"], s["inv_freq"]
    page, half = k_pages.shape[3], inv_freq.numel()
    pos = s["positions"] if s["axis"] is None else s["positions"][s["axis"].long()].t()
    angle = pos.reshape(s["q"].shape[0], 1, -1).double() * inv_freq.double()
    c, n = angle.cos().float(), angle.sin().float()

    def rotate(x):
        x = x.float()
        turned, rest = x[..., :2 * half], x[..., 2 * half:]
        if s["interleaved"]:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * c - b * n, b * c + a * n], dim=-1).flatten(-2)
        else:
            a, b = turned[..., :half], turned[..., half:]
            turned = torch.cat([a * c - b * n, b * c + a * n], dim=-1)
        return torch.cat([turned, rest], dim=-1)

    slot = s["slots"].long()
    at, off = slot // page, slot % page
    s["out"].copy_(rotate(s["q"]))
    k_pages[at, :, :, off] = rotate(s["k"]).to(k_pages.dtype).unflatten(-1, (-1, 8))
    v_pages[at, :, off // 8, :, off % 8] = s["v"]
    return s["out"], k_pages, v_pages


def _attend(s):
    if own:
        s["cache"].attend(s["q"], s["cu_q"], s["kv_lens"], s["table"], s["max_q"], window=s["window"], out=s["out"],
                          lse=s["lse"])
        return s["out"], s["lse"]
    q, cu, kv_lens, most = s["q"], s["cu_q"].long(), s["kv_lens"].long(), s["max_q"]
    (t, h, d), (seqs, hk) = q.shape, (cu.numel() - 1, s["k_pages"].shape[1])
    table = s["table"].clamp(min=0).long()
    k = s["k_pages"][table].permute(0, 2, 3, 5, 1, 4).reshape(seqs, hk, d, -1).float()
    v = s["v_pages"][table].permute(0, 2, 1, 3, 5, 4).reshape(seqs, hk, -1, d).float()
    i = torch.arange(most, device=q.device)
    new = cu[1:] - cu[:-1]
    row = torch.where(i < new[:, None], cu[:-1, None] + i, t)    # rows past a sequence's last go to a row of their own
    x = q[row.clamp(max=t - 1)].float().unflatten(2, (hk, -1)).permute(0, 2, 3, 1, 4).reshape(seqs, hk, -1, d)
    score = torch.matmul(x * d ** -0.5, k).unflatten(2, (-1, most))
    pos = (kv_lens - new)[:, None, None] + i[:, None]
    j = torch.arange(k.shape[3], device=q.device)
    seen = j <= pos
    if s["window"]:
        seen &= j > pos - s["window"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = (score - top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.flatten(2, 3), v).unflatten(2, (-1, most)) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    out, lses = q.new_empty((t + 1, h, d)), s["lse"].new_empty((t + 1, h))
    out[row] = o.permute(0, 3, 1, 2, 4).reshape(seqs, most, h, d).to(q.dtype)
    lses[row] = lse.permute(0, 3, 1, 2).reshape(seqs, most, h)
    return out[:t], lses[:t]


def _logits(s):
    if own:
        from gguf_quant_block_amd.serving import process_logits
        process_logits(s["x"], tokens=s["tokens"], lens=s["lens"], prompt_lens=s["prompt_lens"],
                       repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                       bias_offsets=s["bias_offsets"], bias_ids=s["bias_ids"], bias_values=s["bias_values"],
                       mask=s["mask"], out=s["out"])
        return s["out"]
    x, tokens = s["x"].float(), s["tokens"].long()
    b, n = x.shape
    i = torch.arange(tokens.shape[1], device=x.device)
    there = i < s["lens"][:, None]
    written = there & (i >= s["prompt_lens"][:, None])
    seen = torch.zeros_like(x).scatter_add_(1, tokens, there.float())
    count = torch.zeros_like(x).scatter_add_(1, tokens, written.float())
    r = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - (s["frequency"][:, None] * count + s["presence"][:, None] * (count > 0))
    row = torch.searchsorted(s["bias_offsets"][1:].contiguous(),
                             torch.arange(s["bias_ids"].numel(), dtype=torch.int32, device=x.device), right=True)
    x.index_put_((row, s["bias_ids"].long()), s["bias_values"], accumulate=True)
    if s["mask"] is not None:
        token = torch.arange(n, device=x.device)
        x.masked_fill_((s["mask"][:, token // 32] >> (token % 32).int() & 1) == 0, -math.inf)
    return x.to(s["out"].dtype)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "logits": _exact_logits}[case["op"]](s)


def _exact_append(s):
    half, page = s["inv_freq"].numel(), s["k_pages"].shape[3]
    t, _, d = s["k"].shape
    out, k_pages, v_pages = s["q"].double().clone(), s["k_pages"].double(), s["v_pages"].double()
    k = s["k"].double().clone()
    for j in range(half):
        pos = s["positions"][int(s["axis"][j])] if s["axis"] is not None else s["positions"]
        turn = torch.polar(torch.ones(t, dtype=torch.float64, device=pos.device), pos.double() * s["inv_freq"][j].double())
        a, b = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + half)
        for x in (out, k):
            z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
            x[..., a], x[..., b] = z.real, z.imag
    k_flat = k_pages.permute(0, 3, 1, 2, 4).reshape(-1, k.shape[1], d)       # a row for each slot
    v_flat = v_pages.permute(0, 2, 4, 1, 3).reshape(-1, k.shape[1], d)
    k_flat[s["slots"].long()] = k
    v_flat[s["slots"].long()] = s["v"].double()
    k_pages = k_flat.reshape(-1, page, k.shape[1], d // 8, 8).permute(0, 2, 3, 1, 4)
    v_pages = v_flat.reshape(-1, page // 8, 8, k.shape[1], d).permute(0, 3, 1, 4, 2)
    return out, k_pages, v_pages


def _exact_attend(s):
    q, page, hk = s["q"], s["k_pages"].shape[3], s["k_pages"].shape[1]
    t, h, d = q.shape
    out = torch.zeros((t, h, d), dtype=torch.float64, device=q.device)
    lse = torch.full((t, h), -math.inf, dtype=torch.float64, device=q.device)
    cu, kvs = s["cu_q"].tolist(), s["kv_lens"].tolist()
    for i, kv in enumerate(kvs):
        a, b = cu[i], cu[i + 1]
        if a == b:
            continue
        pages = s["table"][i, :-(-kv // page)].long()
        pos = torch.arange(kv - (b - a), kv, device=q.device)[:, None]
        key = torch.arange(kv, device=q.device)[None]
        hidden = (key > pos) | ((key <= pos - s["window"]) if s["window"] else False)
        for x in range(h):
            y = x // (h // hk)
            k = s["k_pages"][pages, y].double().movedim(1, 2).flatten(2).flatten(0, 1)[:kv]
            v = s["v_pages"][pages, y].double().movedim(2, 3).flatten(0, 2)[:kv]
            for at in range(a, b, 1024):        # some rows at a time
                part = slice(at, min(at + 1024, b))
                z = q[part, x].double() @ k.t() / math.sqrt(d)
                z = z.masked_fill(hidden[part.start - a:part.stop - a], -math.inf)
                out[part, x] = torch.softmax(z, -1) @ v
                lse[part, x] = torch.logsumexp(z, -1)
    return out, lse


def _exact_logits(s):
    x = s["x"].double()
    b, n = x.shape
    lens, prompts, offsets = s["lens"].tolist(), s["prompt_lens"].tolist(), s["bias_offsets"].tolist()
    for i in range(b):
        row, said = x[i], s["tokens"][i, :lens[i]].long()
        past = torch.bincount(said, minlength=n)
        count = torch.bincount(said[prompts[i]:], minlength=n)
        r = s["repetition"][i].double()
        row = torch.where(past > 0, torch.where(row > 0, row / r, row * r), row)
        row = row - s["frequency"][i].double() * count - s["presence"][i].double() * count.clamp(max=1)
        at = slice(offsets[i], offsets[i + 1])
        x[i] = row.index_add(0, s["bias_ids"][at].long(), s["bias_values"][at].double())
    if s["mask"] is not None:
        bits = torch.stack([s["mask"] >> k & 1 for k in range(32)], dim=-1).flatten(1)[:, :n]
        x = torch.where(bits == 1, x, -math.inf)
    return x
