"""A long chunk beside hundreds of single tokens in one call."""

import numpy as np
import pytest

from test_gpu_attend_paths import _case
from test_gpu_serving import BF16, F16

pytestmark = pytest.mark.gpu


# rows of the chunk times the sequences, over all key heads, are more than a grid of every sequence's longest could hold
@pytest.mark.parametrize("dtype,D,hk,G,chunk,seqs,window", [(F16, 64, 32, 16, 512, 512, 0), (BF16, 128, 16, 8, 700, 1500, 50)])
def test_chunk_beside_many_single_tokens(gpu_lib, dtype, D, hk, G, chunk, seqs, window):
    g = np.random.default_rng(seqs)
    kvs = [chunk + 100] + g.integers(1, 60, seqs - 1).tolist()
    news = [chunk] + [1] * (seqs - 1)
    at = seqs // 3                                  # among the others
    kvs[0], kvs[at] = kvs[at], kvs[0]
    news[0], news[at] = news[at], news[0]
    _case(dtype, D, 16, hk, G, kvs, news, window=window, seed=seqs)
