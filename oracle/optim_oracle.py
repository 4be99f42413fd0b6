"""CPU restatement of the weights' update (test infrastructure only; it shares no
code with the CUDA path): the step in fp64, and the narrow moments' codes from the
fp32 arithmetic that the interface fixes.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
U32 = np.uint64(0xFFFFFFFF)


def mix(h):
    """32 random bits of each number below 2^32 (uint64 arithmetic modulo 2^32)."""
    h = np.asarray(h, dtype=np.uint64) & U32
    h = (h ^ (h >> np.uint64(15))) * np.uint64(0x6A09E667) & U32
    h = (h ^ (h >> np.uint64(13))) * np.uint64(0xBB67AE85) & U32
    return h ^ (h >> np.uint64(16))


def words(positions, t: int, seed: int):
    """The random word of each flat position in step t."""
    key = mix(mix((t + 0x9E3779B9) & 0xFFFFFFFF) + np.uint64(seed))
    i = np.asarray(positions, dtype=np.uint64)
    low = (i & U32) * np.uint64(0x9E3779B9) & U32
    high = (i >> np.uint64(32)) * np.uint64(0x3C6EF373) & U32
    return mix(low + high + key)


def e4m3_values():
    """The value of each of the 256 codes."""
    v = np.zeros(256)
    for c in range(128):
        e, f = c >> 3, c & 7
        v[c] = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
    v[127] = np.nan
    v[128:] = -v[:128]
    return v


VALUES = e4m3_values()


def narrow(a, random, least):
    """(codes, scales) of fp32 values `a` (a multiple of BLOCK of them, finite): the code below |a| / scale, or the
    next one where the place between the two, in units of 2^-20, and the 20 random bits carry."""
    a = np.asarray(a, dtype=np.float32).reshape(-1, BLOCK)
    scale = np.maximum(np.abs(a).max(1) * np.float32(1 / 448), np.float32(2.0 ** -120))
    y = np.minimum(np.abs(a) / scale[:, None], np.float32(448)).astype(np.float32).reshape(-1)
    # below 2^-6 the fp32 sum with 2^-6 is what the place is taken from
    y = np.where(y < 2.0 ** -6, (y + np.float32(2.0 ** -6)).astype(np.float32).astype(np.float64) - 2.0 ** -6, y)
    code = np.searchsorted(VALUES[:127], y, side="right") - 1
    step = np.where(code < 126, VALUES[np.minimum(code + 1, 126)] - VALUES[code], 1.0)
    place = np.floor((y - VALUES[code]) / step * 2.0 ** 20)
    code = code + (place + np.asarray(random, dtype=np.float64) >= 2.0 ** 20)
    flat = a.reshape(-1)
    code = np.where(flat != 0, np.maximum(code, least), 0)
    return (code + np.where(flat < 0, 128, 0)).astype(np.uint8), scale


def moments32(m, v, g, scale, beta1, beta2):
    """The new moments with every product and sum rounded to fp32."""
    f = np.float32
    m, v, g = (np.asarray(t, dtype=f) for t in (m, v, g))
    g = g * f(scale)
    return f(beta1) * m + f(1 - beta1) * g, f(beta2) * v + f(1 - beta2) * g * g


def step(p, m, v, g, t, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, decay=0.01, scale=1.0):
    """(p, m, v) after step number t, in fp64."""
    p, m, v, g = (np.asarray(a, dtype=np.float64) for a in (p, m, v, g))
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    update = m / (1 - beta1 ** t) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p - lr * decay * p - lr * update, m, v
