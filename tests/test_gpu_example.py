"""The serving example: FC layers, append, attention and logits processing together, against the same decoder in
float64 on dequantised weights.

Each FC is within 2e-3 of its float64 value (relative Frobenius), the other steps round to f16 (2^-11): nine FCs one
after the other stay within 2e-2, and 5e-2 leaves room for the softmax and the norms between them."""

import os
import sys

import numpy as np
import pytest
import torch

from oracle import kquant
from oracle import serving as o

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _reference(tokens):
    """Logits after every token of one sequence, in float64."""
    import decode as d
    blocks, embedding = d.weights()
    W = {name: kquant.dequantize(blocks[name], q).astype(np.float64) for name, n, k, q in d.shapes()}
    norm = lambda x: x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * d.GAIN  # noqa: E731
    f = np.array([10000.0 ** (-2 * j / d.HEAD_DIM) for j in range(d.HEAD_DIM // 2)])
    x = embedding.double().numpy()[tokens]
    n, pos = len(tokens), [np.arange(len(tokens))]
    for i in range(d.LAYERS):
        qkv = (norm(x) @ W[f"{i}.qkv"].T).reshape(n, -1, d.HEAD_DIM)
        q, k, v = np.split(qkv, [d.HEADS, d.HEADS + d.KV_HEADS], axis=1)
        q, k = o.rotate(q, pos, f)[0], o.rotate(k, pos, f)[0]
        a = np.zeros_like(q)
        for h in range(d.HEADS):
            z = q[:, h] @ k[:, h // (d.HEADS // d.KV_HEADS)].T / np.sqrt(d.HEAD_DIM)
            z[np.triu_indices(n, 1)] = -np.inf
            e = np.exp(z - z.max(-1, keepdims=True))
            a[:, h] = e / e.sum(-1, keepdims=True) @ v[:, h // (d.HEADS // d.KV_HEADS)]
        x = x + a.reshape(n, -1) @ W[f"{i}.o"].T
        gate, up = np.split(norm(x) @ W[f"{i}.gate_up"].T, 2, axis=-1)
        x = x + (gate / (1 + np.exp(-gate)) * up) @ W[f"{i}.down"].T
    return norm(x) @ W["output"].T


def test_decoder_against_float64(gpu_lib):
    import decode as d
    g = np.random.default_rng(3)
    tokens = [g.integers(0, d.VOCAB, n).tolist() for n in (61, 9)]
    want = [_reference(t) for t in tokens]
    model = d.Decoder(path="prefill")
    a, b = model.add(), model.add()
    # a chunk, a chunk beside a whole prompt, single tokens of both
    for new in ({a: tokens[0][:40]}, {a: tokens[0][40:57], b: tokens[1][:5]}, *({a: [tokens[0][57 + i]], b: [tokens[1][5 + i]]} for i in range(4))):
        got = model.forward(new).double().cpu().numpy()
        for i, s in enumerate(new):
            ref = want[s][model.lens[s] - 1]
            assert np.linalg.norm(got[i] - ref) <= 5e-2 * np.linalg.norm(ref)


def test_generation(gpu_lib):
    import decode as d
    prompts = [list(range(3, 73)), [7, 8]]
    allowed = torch.full((2, d.VOCAB // 32), 0x55555555, dtype=torch.int32, device="cuda")
    out = d.generate(d.Decoder(), prompts, 5, allowed=allowed)
    assert [len(x) for x in out] == [5, 5] and all(t % 2 == 0 for x in out for t in x)
    # the same tokens when a prompt is read in other chunks of at least 8 rows, and beside nothing else
    alone = d.generate(d.Decoder(), prompts[:1], 1, chunk=70, allowed=allowed[:1])
    assert alone[0] == out[0][:1]
