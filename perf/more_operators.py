"""More operators between the fully-connected layers of a decoder, as cases to be measured: appending to the paged
cache with norms of queries and keys for each head, or into a cache of 8 bits; attention over a cache of 8 bits; and
the choice of the next token.  `run` computes a case in elementary torch operations, or, where `own` is true, through
the package's entry points."""

import math
import random

import torch

own = False

DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}

# A head of a token in 8 bits: e4m3 codes times a power of two, its exponent between the two of the type (so that every
# code stands for a value that the type holds), its codes up to 448, or 240 at the upper exponent.
EXPONENTS = {torch.float16: (-14, 8), torch.bfloat16: (-110, 120)}
BIAS = 127              # of a stored exponent
EPS = 1e-6              # of the norms


# ---------------------------------------------------------------- the cases

def listed():
    append = {"op": "append", "dtype": "float16", "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128,
              "interleaved": False, "page": 64, "bits": 16, "norm": "dim"}
    attend = {"op": "attend", "dtype": "float16", "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "seqs": 1,
              "ragged": False, "window": 0}
    sample = {"op": "sample", "dtype": "float32", "spread": 4.0, "hidden": 0.0, "temperature": 0.8, "top_k": 0,
              "top_p": 1.0, "min_p": 0.0}
    return [
        # one token of one conversation whose queries and keys are normalised: latency is all that counts
        {**append, "name": "norm-append-1", "tokens": 1, "start": 4095},
        # a chunk of a long prompt that begins in the middle of a page, norms with weights of their own for each head
        {**append, "name": "norm-append-prompt-4096", "dtype": "bfloat16", "tokens": 4096, "start": 8197, "norm": "head"},
        # one decode step of a busy server into 8 bits, each token into another sequence's page, half of a head rotated
        {**append, "name": "append8-batch-128", "dtype": "bfloat16", "rot": 64, "bits": 8, "tokens": 128, "start": 30011,
         "step": True},
        # a chunk of a long prompt into 8 bits
        {**append, "name": "append8-prompt-4096", "bits": 8, "norm": "", "tokens": 4096, "start": 8197},
        # one token of one conversation, every query head with a key head of its own
        {**attend, "name": "attend8-1", "heads": 24, "kv_heads": 24, "head_dim": 96, "kv": 1003, "new": 1},
        # one decode step of a busy server, conversations of all lengths
        {**attend, "name": "attend8-batch-64", "dtype": "bfloat16", "seqs": 64, "kv": 8192, "new": 1, "ragged": True},
        # one token over a long document
        {**attend, "name": "attend8-long-1", "kv": 131072, "new": 1},
        # a few drafted tokens of some sequences are verified at once
        {**attend, "name": "attend8-draft-8x5", "dtype": "bfloat16", "seqs": 8, "kv": 6001, "new": 5, "page": 16,
         "ragged": True},
        # a chunk of a prompt over what was cached before
        {**attend, "name": "attend8-chunk-4096", "kv": 8192, "new": 4096},
        # the next token of one conversation
        {**sample, "name": "sample-1", "rows": 1, "vocab": 32064, "top_k": 40, "top_p": 0.95, "min_p": 0.05},
        # one decode step of a busy server, a larger vocabulary, a nucleus of each row
        {**sample, "name": "sample-batch-128", "rows": 128, "vocab": 131073, "top_p": 0.9},
        # the same under a grammar that hides most tokens, logits in 16 bits that are nearly flat and repeat each other
        {**sample, "name": "sample-flat-masked-33", "dtype": "bfloat16", "rows": 33, "vocab": 131073, "spread": 1.5,
         "hidden": 0.75, "temperature": 1.0, "min_p": 0.01, "top_p": 0.97},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("append", "append", "attend", "attend", "sample"))
    if op == "sample":
        return {"op": op, "dtype": rng.choice(("float16", "bfloat16", "float32")), "rows": _spread(rng, 1, 128),
                "vocab": _spread(rng, 1009, 131073), "spread": rng.choice((0.5, 1.5, 4.0)),
                "hidden": rng.choice((0.0, 0.0, 0.75)), "temperature": rng.choice((0.3, 0.8, 1.0, 1.7)),
                "top_k": rng.choice((0, _spread(rng, 1, 1000))), "top_p": rng.choice((1.0, rng.uniform(0.5, 0.99))),
                "min_p": rng.choice((0.0, rng.uniform(0.01, 0.2)))}
    head_dim = rng.choice((64, 96, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    c = {"op": op, "dtype": rng.choice(("float16", "bfloat16")), "kv_heads": kv_heads,
         "heads": kv_heads * rng.choice((1, 2, 3, 4, 8)), "head_dim": head_dim, "page": rng.choice((16, 32, 64, 128))}
    if c["heads"] * head_dim > 4096:
        c["heads"] = kv_heads
    if op == "append":
        bits = rng.choice((8, 8, 16))
        c |= {"rot": rng.choice((head_dim, head_dim // 2)), "interleaved": rng.random() < 0.5, "bits": bits,
              "norm": rng.choice(("dim", "head") if bits == 16 else ("", "dim", "head")),
              "tokens": _spread(rng, 1, 4096), "start": _spread(rng, 1, 100000)}
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
        t, d, h, hk = case["tokens"], case["head_dim"], case["heads"], case["kv_heads"]
        kept = 2 * hk * (d * 2 if case["bits"] == 16 else d + 1)
        return {"bytes": t * ((h + 2 * hk) * d * 2 + h * d * 2 + kept + 8),
                "flops": t * (h + hk) * (case["rot"] // 2 * 6 + (4 * d if case["norm"] else 0))}
    if case["op"] == "attend":
        pairs, keys = _seen(case)
        t, d, h = sum(_lengths(case)[1]), case["head_dim"], case["heads"]
        return {"bytes": 2 * t * h * d * 2 + t * h * 4 + keys * case["kv_heads"] * (d + 1) * 2,
                "flops": 4 * d * h * pairs}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4 if case["dtype"] == "float32" else 2) + case["rows"] * 28, "flops": 4 * n}


# ---------------------------------------------------------------- what a program has in hand

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"append": _prepare_append, "attend": _prepare_attend, "sample": _prepare_sample}[case["op"]](case, g)


def _normal(g, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(0.0, scale, generator=g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _quantise(x, dtype):
    """x [..., head_dim] in f32 or f64 as (codes, stored exponents [...]): the definition of the cache of 8 bits."""
    low, high = EXPONENTS[dtype]
    m, e = torch.frexp(x.abs().amax(-1))                        # amax = m 2^e, 0.5 <= m < 1; 448 is 0.875 * 2^9
    e = torch.where(m == 0, low, e - 9 + (m > 0.875)).clamp(low, high)
    most = torch.where(e == high, 240.0, 448.0)[..., None].to(x.dtype)
    codes = (x * torch.exp2(-e.to(x.dtype))[..., None]).clamp(-most, most)
    return codes, e + BIAS


def _cache(case, pages):
    """The package's cache object and its tensors: keys [pages, kv_heads, head_dim/8, page, 8], values [pages, kv_heads,
    page/8, head_dim, 8] and, in 8 bits, the scales of both [pages, kv_heads, page]."""
    h, d, p, bits = case["kv_heads"], case["head_dim"], case["page"], case.get("bits", 8)
    dtype = DTYPES[case["dtype"]]
    if own:
        from gguf_quant_block_amd.serving import PagedKv
        cache = PagedKv(pages, p, h, d, dtype, bits=bits)
        return {"cache": cache, "k_pages": cache.k, "v_pages": cache.v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    held = dtype if bits == 16 else torch.float8_e4m3fn
    empty = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    return {"k_pages": empty((pages, h, d // 8, p, 8), held), "v_pages": empty((pages, h, p // 8, d, 8), held),
            "k_scale": empty((pages, h, p), torch.float8_e8m0fnu) if bits == 8 else None,
            "v_scale": empty((pages, h, p), torch.float8_e8m0fnu) if bits == 8 else None}


def _fill(s, g, dtype):
    """What earlier calls left in the cache: normal keys and values."""
    pages, h, d8, page, _ = s["k_pages"].shape
    if s["k_scale"] is None:
        s["k_pages"].normal_(0.0, 1.0, generator=g)
        s["v_pages"].normal_(0.0, 1.0, generator=g)
        return
    for name in ("k", "v"):
        codes, e = _quantise(_normal(g, (pages, h, page, d8 * 8), dtype).float(), dtype)
        codes = codes.unflatten(-1, (-1, 8)).transpose(2, 3) if name == "k" else codes.unflatten(2, (-1, 8)).transpose(3, 4)
        s[name + "_pages"].copy_(codes.contiguous())
        s[name + "_scale"].view(torch.uint8).copy_(e)


def _prepare_append(case, g):
    t, h, hk, d, page = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    dtype, rot = DTYPES[case["dtype"]], case["rot"]
    step = case.get("step", False)
    # a step's tokens belong to as many sequences, each with a page of its own; a prompt's follow each other
    pages = t + 2 if step else (case["start"] % page + t) // page + 3
    s = _cache(case, pages)
    _fill(s, g, dtype)
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    if step:
        slots = order[i] * page + torch.randint(0, page, (t,), generator=g, device="cuda")
        positions = torch.randint(0, case["start"] + 1, (t,), generator=g, device="cuda")
    else:
        at = case["start"] % page + i
        slots = order[at // page] * page + at % page
        positions = case["start"] + i
    qkv = _normal(g, (t, (h + 2 * hk) * d), dtype)     # the projection's output, as it stands
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([h * d, hk * d, hk * d], dim=1))
    inv_freq = torch.tensor([10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float32, device="cuda")
    s |= {"op": "append", "q": q, "k": k, "v": v, "slots": slots.int(), "positions": positions.int(), "inv_freq": inv_freq,
          "interleaved": case["interleaved"], "out": torch.empty((t, h, d), dtype=dtype, device="cuda"), "norms": None}
    if case["norm"]:
        shape = (lambda n: (n, d)) if case["norm"] == "head" else (lambda n: (d,))
        s["norms"] = [_normal(g, shape(n), torch.float32, 0.2).add_(1.0) for n in (h, hk)]
    if own:
        from gguf_quant_block_amd.serving import HeadNorm, Rope
        s["rope"] = Rope(inv_freq, interleaved=case["interleaved"])
        s["norm"] = HeadNorm(*s["norms"], eps=EPS) if case["norm"] else None
    return s


def _prepare_attend(case, g):
    h, d, page, dtype = case["heads"], case["head_dim"], case["page"], DTYPES[case["dtype"]]
    kvs, news = _lengths(case)
    used = [-(-n // page) for n in kvs]
    pages = sum(used) + 3
    s = _cache(case, pages)
    _fill(s, g, dtype)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(kvs), max(used)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return s | {"op": "attend", "window": case["window"], "q": _normal(g, (cu[-1], h, d), dtype, 1.5), "cu_q": _ints(cu),
                "kv_lens": _ints(kvs), "table": table, "max_q": max(news),
                "out": torch.empty((cu[-1], h, d), dtype=dtype, device="cuda"),
                "lse": torch.empty((cu[-1], h), dtype=torch.float32, device="cuda")}


def _prepare_sample(case, g):
    b, n = case["rows"], case["vocab"]
    uniform = lambda low, high: torch.empty(b, device="cuda").uniform_(low, high, generator=g)  # noqa: E731
    x = _normal(g, (b, n), DTYPES[case["dtype"]], case["spread"])
    if case["hidden"]:
        x.masked_fill_(torch.rand((b, n), generator=g, device="cuda") < case["hidden"], -math.inf)
    # every request has settings of its own, near the case's
    s = {"op": "sample", "x": x, "u": torch.rand(b, generator=g, device="cuda"),
         "temperature": case["temperature"] * uniform(0.9, 1.1), "top_k": None, "top_p": None, "min_p": None,
         "out": torch.empty(b, dtype=torch.int32, device="cuda"), "logprobs": torch.empty(b, device="cuda")}
    s["temperature"][b // 2:b // 2 + b // 16] = 0.0              # some of a batch take the largest
    if case["top_k"]:
        s["top_k"] = (case["top_k"] * uniform(0.7, 1.3)).ceil().int()
    if case["top_p"] < 1:
        s["top_p"] = 1.0 - (1.0 - case["top_p"]) * uniform(0.5, 1.5)
    if case["min_p"]:
        s["min_p"] = case["min_p"] * uniform(0.5, 1.5)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return {"append": _append, "attend": _attend, "sample": _sample}[state["op"]](state)


def _held(s):
    return (s["k_pages"], s["v_pages"]) + ((s["k_scale"], s["v_scale"]) if s["k_scale"] is not None else ())


def _append(s):
    if own:
        s["cache"].append(s["q"], s["k"], s["v"], s["slots"], s["positions"], s["rope"], out=s["out"], norm=s["norm"])
        return s["out"], *_held(s)
    k_pages, v_pages, inv_freq = s["k_pages"], s["v_pages"], s["inv_freq"]
    page, half = k_pages.shape[3], inv_freq.numel()
    angle = s["positions"].reshape(-1, 1, 1).double() * inv_freq.double()
    c, n = angle.cos().float(), angle.sin().float()

    def normed(x, weight):
        x = x.float()
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight

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

    q, k, v = s["q"], s["k"], s["v"]
    if s["norms"]:
        q, k = normed(q, s["norms"][0]), normed(k, s["norms"][1])
    s["out"].copy_(rotate(q))
    k = rotate(k)
    slot = s["slots"].long()
    at, off = slot // page, slot % page
    if s["k_scale"] is None:
        k, v = k.to(k_pages.dtype), v
    else:
        (k, ke), (v, ve) = _quantise(k, s["out"].dtype), _quantise(v.float(), s["out"].dtype)
        s["k_scale"].view(torch.uint8)[at, :, off] = ke.to(torch.uint8)
        s["v_scale"].view(torch.uint8)[at, :, off] = ve.to(torch.uint8)
        k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        k_pages, v_pages = k_pages.view(torch.uint8), v_pages.view(torch.uint8)
    k_pages[at, :, :, off] = k.unflatten(-1, (-1, 8))
    v_pages[at, :, off // 8, :, off % 8] = v
    return s["out"], *_held(s)


def _attend(s):
    if own:
        s["cache"].attend(s["q"], s["cu_q"], s["kv_lens"], s["table"], s["max_q"], window=s["window"], out=s["out"],
                          lse=s["lse"])
        return s["out"], s["lse"]
    q, cu, kv_lens, most = s["q"], s["cu_q"].long(), s["kv_lens"].long(), s["max_q"]
    (t, h, d), (seqs, hk) = q.shape, (cu.numel() - 1, s["k_pages"].shape[1])
    page = s["k_pages"].shape[3]
    table = s["table"].clamp(min=0).long()
    held = lambda name: s[name].view(torch.uint8)[table]  # noqa: E731
    k = held("k_pages").view(torch.float8_e4m3fn).float()
    k = k * held("k_scale").view(torch.float8_e8m0fnu).float()[:, :, :, None, :, None]
    k = k.permute(0, 2, 3, 5, 1, 4).reshape(seqs, hk, d, -1)
    v = held("v_pages").view(torch.float8_e4m3fn).float()
    v = v * held("v_scale").view(torch.float8_e8m0fnu).float().view(seqs, -1, hk, page // 8, 1, 8)
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(seqs, hk, -1, d)
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


def _sample(s):
    if own:
        from gguf_quant_block_amd.serving import sample
        sample(s["x"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
               out=s["out"], logprobs=s["logprobs"])
        return s["out"], s["logprobs"]
    # sums of many weights next to the border that u draws: 64 bits
    z, order = s["x"].double().sort(dim=-1, descending=True, stable=True)
    b, n = z.shape
    greedy = s["temperature"] <= 0
    rank = torch.arange(n, device=z.device)
    most = s["top_k"] if s["top_k"] is not None else torch.full((b,), n, dtype=torch.int32, device=z.device)
    most = torch.where(greedy, 1, torch.where(most > 0, most, n))
    w = ((z - z[:, :1]) / torch.where(greedy, 1.0, s["temperature"].double())[:, None]).exp()
    w = torch.where(rank < most[:, None], w, 0.0)
    c = w.cumsum(-1)
    kept = w > 0
    if s["top_p"] is not None:
        kept &= c - w < s["top_p"].double()[:, None] * c[:, -1:]
    if s["min_p"] is not None:
        kept &= w >= s["min_p"].double()[:, None]
    count = kept.sum(-1, keepdim=True)
    total = c.gather(-1, count - 1)
    at = torch.minimum((c <= s["u"].double()[:, None] * total).sum(-1, keepdim=True), count - 1)
    s["out"].copy_(order.gather(-1, at)[:, 0])
    s["logprobs"].copy_((w.gather(-1, at) / total).log()[:, 0])
    return s["out"], s["logprobs"]


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s)


def _exact_append(s):
    half, page = s["inv_freq"].numel(), s["k_pages"].shape[3]
    t, hk, d = s["k"].shape
    out, k, v = s["q"].double().clone(), s["k"].double().clone(), s["v"].double()
    for x, weight in zip((out, k), s["norms"] or ()):
        x.copy_(x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * weight.double())
    for j in range(half):
        turn = torch.polar(torch.ones(t, dtype=torch.float64, device=out.device),
                           s["positions"].double() * s["inv_freq"][j].double())
        a, b = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + half)
        for x in (out, k):
            z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
            x[..., a], x[..., b] = z.real, z.imag
    k_pages, v_pages, slots = s["k_pages"].double(), s["v_pages"].double(), s["slots"].long()
    scales = []
    if s["k_scale"] is not None:         # codes before their rounding, and the scales
        low, high = EXPONENTS[s["out"].dtype]
        for name in ("k", "v"):
            x = k if name == "k" else v.clone()
            big = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -200)
            scale = torch.exp2(torch.ceil(torch.log2(big / 448)).clamp(low, high))
            x.div_(scale)
            if name == "v":
                v = x
            whole = s[name + "_scale"].double().transpose(1, 2).reshape(-1, hk)
            whole[slots] = scale[..., 0]
            scales.append(whole.reshape(-1, page, hk).transpose(1, 2))
    k_flat = k_pages.permute(0, 3, 1, 2, 4).reshape(-1, hk, d)               # a row for each slot
    v_flat = v_pages.permute(0, 2, 4, 1, 3).reshape(-1, hk, d)
    k_flat[slots], v_flat[slots] = k, v
    k_pages = k_flat.reshape(-1, page, hk, d // 8, 8).permute(0, 2, 3, 1, 4)
    v_pages = v_flat.reshape(-1, page // 8, 8, hk, d).permute(0, 3, 1, 4, 2)
    return out, k_pages, v_pages, *scales


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
        for y in range(hk):
            scales = [s[n].view(torch.uint8)[pages, y].view(torch.float8_e8m0fnu).double().reshape(-1, 1) for n in ("k_scale", "v_scale")]
            k = s["k_pages"].view(torch.uint8)[pages, y].view(torch.float8_e4m3fn).double().movedim(1, 2).flatten(2).flatten(0, 1)
            v = s["v_pages"].view(torch.uint8)[pages, y].view(torch.float8_e4m3fn).double().movedim(2, 3).flatten(0, 2)
            k, v = (k * scales[0])[:kv], (v * scales[1])[:kv]
            for x in range(y * (h // hk), (y + 1) * (h // hk)):
                for at in range(a, b, 1024):        # some rows at a time
                    part = slice(at, min(at + 1024, b))
                    z = q[part, x].double() @ k.t() / math.sqrt(d)
                    z = z.masked_fill(hidden[part.start - a:part.stop - a], -math.inf)
                    out[part, x] = torch.softmax(z, -1) @ v
                    lse[part, x] = torch.logsumexp(z, -1)
    return out, lse


def _exact_sample(s):
    tokens, logprobs = [], []
    for i in range(s["x"].shape[0]):
        x, t = s["x"][i].double(), float(s["temperature"][i])
        ids = torch.argsort(-x, stable=True)
        ids = ids[:int((x > -math.inf).sum())]
        if s["top_k"] is not None and s["top_k"][i] > 0:
            ids = ids[:int(s["top_k"][i])]
        if t <= 0:
            ids, t = ids[:1], 1.0
        p = torch.softmax(x[ids] / t, 0)
        if s["top_p"] is not None:
            before = torch.cat([p.new_zeros(1), p.cumsum(0)[:-1]])
            p = p[before < s["top_p"][i].double()]
        if s["min_p"] is not None:
            p = p[p >= s["min_p"][i].double() * p[0]]
        p = p / p.sum()
        at = min(int(torch.searchsorted(p.cumsum(0), s["u"][i].double(), right=True)), p.numel() - 1)
        tokens.append(int(ids[at]))
        logprobs.append(float(p[at].log()))
    return torch.tensor(tokens), torch.tensor(logprobs, dtype=torch.float64)
