"""CPU reference of the serving operators in float64 (test infrastructure).

Plain NumPy loops over tokens and heads from the operators' definitions; shares
nothing with the HIP path.  Besides each result stand the sums of magnitudes
that error bounds are made of.
"""

import numpy as np


def rotate(x, positions, inv_freq, axis=None, interleaved=False, scale=1.0):
    """x [T, H, D] rotated at positions [axes, T]; (result, magnitude), where
    magnitude is |x0| + |x1| of each rotated pair (0 where nothing is rotated)."""
    x = np.asarray(x, dtype=np.float64)
    out, mag = x.copy(), np.zeros_like(x)
    half = len(inv_freq)
    for j in range(half):
        pos = np.asarray(positions)[0 if axis is None else int(axis[j])].astype(np.float64)
        a = pos * np.float64(inv_freq[j])
        c, s = scale * np.cos(a)[:, None], scale * np.sin(a)[:, None]
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        out[:, :, i0] = x[:, :, i0] * c - x[:, :, i1] * s
        out[:, :, i1] = x[:, :, i1] * c + x[:, :, i0] * s
        mag[:, :, i0] = mag[:, :, i1] = abs(scale) * (np.abs(x[:, :, i0]) + np.abs(x[:, :, i1]))
    return out, mag


def key_slot(k_pages, slot):
    """The key [kv_heads, D] at a slot of k_pages [pages, kv_heads, D/8, ps, 8]."""
    ps = k_pages.shape[3]
    return k_pages[slot // ps, :, :, slot % ps].reshape(k_pages.shape[1], -1)


def value_slot(v_pages, slot):
    """The value [kv_heads, D] at a slot of v_pages [pages, kv_heads, ps/8, D, 8]."""
    ps = v_pages.shape[2] * 8
    return v_pages[slot // ps, :, (slot % ps) // 8, :, slot % 8]


def attend(q, k_pages, v_pages, cu_q, kv_lens, table, scale, window=0, max_q=None):
    """q [T, H, D] over the pages, sequence by sequence.  Returns a dict: out
    [T, H, D], lse [T, H]; mass (sum of weights times |value|), score (largest
    scale * sum |q_i k_i| of a row), vsum (sum of |value| / total), keys (number
    seen); rows of no sequence are NaN."""
    T, H, D = q.shape
    hk, ps, pages = k_pages.shape[1], k_pages.shape[3], k_pages.shape[0]
    r = {"out": np.full((T, H, D), np.nan), "lse": np.full((T, H), np.nan), "mass": np.zeros((T, H, D)),
         "vsum": np.zeros((T, H, D)), "score": np.zeros((T, H)), "keys": np.zeros((T, H))}
    q = np.asarray(q, dtype=np.float64)
    for s, kv in enumerate(kv_lens):
        a, b = int(cu_q[s]), int(cu_q[s + 1])
        kv, n = int(kv), b - a
        held = [j for j in range(min(kv, table.shape[1] * ps)) if 0 <= table[s][j // ps] < pages]
        slots = np.array([int(table[s][j // ps]) * ps + j % ps for j in held], dtype=np.int64)
        held = np.array(held, dtype=np.int64)
        if len(held):
            K = k_pages[slots // ps, :, :, slots % ps].reshape(len(held), hk, D).astype(np.float64)
            V = v_pages[slots // ps, :, (slots % ps) // 8, :, slots % 8].astype(np.float64)
        for i in range(n if max_q is None else min(n, max_q)):
            p = kv - n + i
            see = (held <= p) & ((held > p - window) if window else True)
            for h in range(H):
                if not see.any():
                    r["out"][a + i, h], r["lse"][a + i, h] = 0.0, -np.inf
                    continue
                k, v = K[see, h // (H // hk)], V[see, h // (H // hk)]
                z = scale * (k @ q[a + i, h])
                m = z.max()
                e = np.exp(z - m)
                t = e.sum()
                r["out"][a + i, h] = e @ v / t
                r["lse"][a + i, h] = m + np.log(t)
                r["mass"][a + i, h] = e @ np.abs(v) / t
                r["vsum"][a + i, h] = np.abs(v).sum(0) / t
                r["score"][a + i, h] = scale * (np.abs(k) @ np.abs(q[a + i, h])).max()
                r["keys"][a + i, h] = see.sum()
    return r


def logits(x, tokens=None, lens=None, prompt_lens=None, repetition=None, frequency=None, presence=None, bias=None,
           mask=None):
    """Logits x [rows, vocab] processed token by token; bias: per row a list of
    (id, value).  (result, magnitude): magnitude is the sum of the magnitudes
    that were added up."""
    x = np.array(x, dtype=np.float64)
    mag = np.abs(x)
    rows, vocab = x.shape
    for r in range(rows):
        if tokens is not None:
            said = [int(t) for t in tokens[r][:max(0, int(lens[r]))]]
            first = 0 if prompt_lens is None else max(0, int(prompt_lens[r]))
            for v in set(said):
                if not 0 <= v < vocab:
                    continue
                n = sum(t == v for t in said[first:])
                f = 1.0 if repetition is None else float(repetition[r])
                x[r, v] = x[r, v] / f if x[r, v] > 0 else x[r, v] * f
                mag[r, v] = abs(x[r, v])
                less = n * (0.0 if frequency is None else float(frequency[r]))
                less2 = (0.0 if presence is None or n == 0 else float(presence[r]))
                x[r, v] -= less + less2
                mag[r, v] += abs(less) + abs(less2)
        for v, b in (bias[r] if bias is not None else []):
            if 0 <= v < vocab:
                x[r, v] += float(b)
                mag[r, v] += abs(float(b))
        if mask is not None:
            for v in range(vocab):
                if not int(mask[r][v // 32]) >> (v % 32) & 1:
                    x[r, v] = -np.inf
    return x, mag
