"""CPU reference in float64 of the head norms and of the cache of 8 bits (test infrastructure): from the definitions,
element by element, sharing nothing with the HIP path."""

import numpy as np

LIMITS = {"float16": (-14, 8), "bfloat16": (-110, 120)}    # of a scale's exponent
BIAS = 127


def e4m3_values():
    """What the 256 codes stand for: sign, 4 bits of exponent (bias 7), 3 of fraction; all ones: NaN."""
    out = np.empty(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = np.nan if e == 15 and f == 7 else f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = -x if c >> 7 else x
    return out


def nearest(y):
    """The nearest finite values of a code (ties to the even fraction); y within +-448."""
    y = np.asarray(y, dtype=np.float64)
    mag = np.abs(y)
    exponent = np.floor(np.log2(np.where(mag > 0, mag, 1.0)))
    step = 2.0 ** (np.maximum(exponent, -6) - 3)
    return np.where(mag > 0, np.rint(y / step) * step, 0.0)


def quantise(x, dtype):
    """x [..., D] as (values of the codes, NaN among them; exponents [...])."""
    low, high = LIMITS[dtype]
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x)
    amax = np.where(fine, np.abs(x), 0).max(-1)
    e = np.full(amax.shape, low)
    for i in np.ndindex(amax.shape):
        while e[i] < high and amax[i] > 448 * 2.0 ** e[i]:
            e[i] += 1
    most = np.where(e == high, 240.0, 448.0)[..., None]
    y = np.clip(np.where(fine, x, 0) / 2.0 ** e[..., None], -most, most)
    return np.where(fine, nearest(y), np.nan), e


def held(codes, scales, dtype, values):
    """What a cache stands for: codes u8 pages of keys [pages, heads, D/8, ps, 8] or values [pages, heads, ps/8, D, 8],
    scales u8 [pages, heads, ps]."""
    low, high = LIMITS[dtype]
    e = np.clip(scales.astype(np.int64) - BIAS, low, high)
    by = 2.0 ** e.astype(np.float64)
    pages, heads, ps = scales.shape
    by = by.reshape(pages, heads, ps // 8, 1, 8) if values else by[:, :, None, :, None]
    x = e4m3_values()[codes] * by
    # (what append never stores: codes past 240 at the upper exponent are infinite in dtype)
    return np.where(np.abs(x) > 240 * 2.0 ** high, np.copysign(np.inf, x), x)


def head_norm(x, weight, eps):
    """x [T, H, D] with weight [D] or [H, D]."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
