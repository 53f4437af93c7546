"""A small decoder on GGUF K-quant weights, served: prompts in chunks, then one token of every sequence at a time.

    python examples/decode.py

Every projection is an FcGguf on synthetic Q5_K and Q6_K blocks.  Between them stand the serving operators: PagedKv.append
(norms of queries and keys for each head where the model has them, rotation, and the cache in 16 or 8 bits),
PagedKv.attend (chunks and single tokens in one call), process_logits, and sample for the next token.  Norms of rows, the
gate and the embedding are plain torch.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gguf_quant_block_amd import synth  # noqa: E402
from gguf_quant_block_amd.binding import FcGguf  # noqa: E402
from gguf_quant_block_amd.serving import HeadNorm, PagedKv, Rope, process_logits, sample  # noqa: E402

LAYERS, HIDDEN, HEADS, KV_HEADS, HEAD_DIM, FFN, VOCAB = 2, 512, 8, 2, 64, 1024, 2048
GAIN = 1.0 / 64        # of the norms: synthetic weights have a standard deviation near 2


def shapes():
    """(name, N, K, qtype) of every projection, in the order of their seeds."""
    out = []
    for i in range(LAYERS):
        out += [(f"{i}.qkv", (HEADS + 2 * KV_HEADS) * HEAD_DIM, HIDDEN, "q6_k"), (f"{i}.o", HIDDEN, HEADS * HEAD_DIM, "q6_k"),
                (f"{i}.gate_up", 2 * FFN, HIDDEN, "q6_k"), (f"{i}.down", HIDDEN, FFN, "q6_k")]
    return out + [("output", VOCAB, HIDDEN, "q6_k")]


def weights(seed=0):
    """The blocks of every projection, and the embedding."""
    blocks = {name: synth.blocks(q, n, k, synth.rng(seed, i, synth.TAG_BLOCKS)) for i, (name, n, k, q) in enumerate(shapes())}
    return blocks, torch.from_numpy(synth.normal_f16((VOCAB, HIDDEN), synth.rng(seed, 0, synth.TAG_A)))


def norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * GAIN).half()


class Decoder:
    """The model with a cache of `pages` pages that its sequences share.  bits: of the cache; head_norm: weights of all
    heads' norms of queries and keys, a pair of lists of HEAD_DIM numbers, or None."""

    def __init__(self, pages=64, page_size=16, path=None, seed=0, bits=16, head_norm=None):
        blocks, embedding = weights(seed)
        self.fc = {name: FcGguf(n, k, q, blocks[name]) for name, n, k, q in shapes()}
        if path:
            for fc in self.fc.values():
                fc.set_path(path)
        self.embedding = embedding.cuda()
        self.page_size, self.free = page_size, list(range(pages))
        self.kv = [PagedKv(pages, page_size, KV_HEADS, HEAD_DIM, bits=bits) for _ in range(LAYERS)]
        self.head_norm = head_norm and HeadNorm(*(torch.tensor(w, dtype=torch.float32, device="cuda") for w in head_norm))
        self.rope = Rope(torch.tensor([10000.0 ** (-2 * j / HEAD_DIM) for j in range(HEAD_DIM // 2)], dtype=torch.float32,
                                      device="cuda"))
        self.tables, self.lens = [], []

    def add(self):
        """A new, empty sequence: its number."""
        self.tables.append([])
        self.lens.append(0)
        return len(self.lens) - 1

    def forward(self, new):
        """Runs new tokens {sequence: [tokens]} and returns the logits [sequences, VOCAB] after the last of each."""
        seqs = [s for s in new if new[s]]
        slots, positions, cu = [], [], [0]
        for s in seqs:
            for p in range(self.lens[s], self.lens[s] + len(new[s])):
                if p // self.page_size == len(self.tables[s]):
                    self.tables[s].append(self.free.pop())
                slots.append(self.tables[s][p // self.page_size] * self.page_size + p % self.page_size)
                positions.append(p)
            self.lens[s] += len(new[s])
            cu.append(len(slots))
        width = max(len(self.tables[s]) for s in seqs)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        table = ints([self.tables[s] + [-1] * (width - len(self.tables[s])) for s in seqs])
        lens, slots, positions, cu_q = ints([self.lens[s] for s in seqs]), ints(slots), ints(positions), ints(cu)
        most = max(len(new[s]) for s in seqs)

        x = self.embedding[ints([t for s in seqs for t in new[s]]).long()]
        for i in range(LAYERS):
            qkv = self.fc[f"{i}.qkv"](norm(x)).view(-1, HEADS + 2 * KV_HEADS, HEAD_DIM)
            q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
            q = self.kv[i].append(q, k, v, slots, positions, self.rope, norm=self.head_norm)
            a = self.kv[i].attend(q, cu_q, lens, table, most)
            x = self.fc[f"{i}.o"](a.view(-1, HEADS * HEAD_DIM), x)
            gate, up = self.fc[f"{i}.gate_up"](norm(x)).chunk(2, dim=-1)
            x = self.fc[f"{i}.down"]((torch.nn.functional.silu(gate.float()) * up.float()).half(), x)
        return self.fc["output"](norm(x[cu_q[1:].long() - 1]))


def generate(model, prompts, steps, chunk=32, repetition=1.2, allowed=None, temperature=0.0, top_k=0, top_p=1.0, min_p=0.0, seed=0):
    """Tokens after each prompt, `steps` of them, the largest or, with a temperature, drawn.  allowed: a mask as of
    process_logits, [sequences, words]."""
    seqs = [model.add() for _ in prompts]
    history = [list(p) for p in prompts]
    todo = {s: list(p) for s, p in zip(seqs, prompts)}
    last = {}
    while len(last) < len(seqs):            # prompts, a chunk of each at a time
        now = {s: todo[s][:chunk] for s in seqs if todo[s]}
        logits = model.forward(now)
        for i, s in enumerate(now):
            todo[s] = todo[s][chunk:]
            if not todo[s]:
                last[s] = logits[i]
    logits = torch.stack([last[s] for s in seqs])
    prompt_lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    each = lambda x: torch.full((len(seqs),), x, device="cuda")  # noqa: E731
    factor, generator = each(repetition), torch.Generator(device="cuda").manual_seed(seed)
    settings = {"temperature": each(float(temperature)), "top_k": each(int(top_k)).int(), "top_p": each(float(top_p)), "min_p": each(float(min_p))}
    for step in range(steps):
        longest = max(map(len, history))
        tokens = torch.tensor([h + [0] * (longest - len(h)) for h in history], dtype=torch.int32, device="cuda")
        lens = torch.tensor([len(h) for h in history], dtype=torch.int32, device="cuda")
        processed = process_logits(logits, tokens=tokens, lens=lens, prompt_lens=prompt_lens, repetition=factor, mask=allowed)
        u = torch.rand(len(seqs), generator=generator, device="cuda")
        choice = sample(processed, u, **settings).tolist()
        for h, t in zip(history, choice):
            h.append(t)
        if step + 1 < steps:
            logits = model.forward({s: [t] for s, t in zip(seqs, choice)})
    return [h[len(p):] for h, p in zip(history, prompts)]


def main():
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, VOCAB, (n,), generator=g).tolist() for n in (70, 5, 33)]
    # a grammar that leaves the even tokens only
    allowed = torch.full((len(prompts), VOCAB // 32), 0x55555555, dtype=torch.int32, device="cuda")
    for p, out in zip(prompts, generate(Decoder(), prompts, 12, allowed=allowed)):
        print(f"{len(p)} prompt tokens -> {out}")
    ones = [1.0] * HEAD_DIM
    drawn = generate(Decoder(bits=8, head_norm=(ones, ones)), prompts, 12, allowed=allowed, temperature=0.8, top_k=40, top_p=0.95, min_p=0.05)
    for p, out in zip(prompts, drawn):
        print(f"{len(p)} prompt tokens, head norms, 8 bits, drawn -> {out}")


if __name__ == "__main__":
    main()
