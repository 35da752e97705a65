"""AdamW step with 8-bit states, operation by operation in float32 (numpy), as include/puro_ops.h defines it.

States are E4M3 codes with one float32 scale for 128 consecutive elements: the first moment, and the root of the second.
Every operation below is one IEEE float32 operation, so that codes and scales are defined to the bit.
"""
from __future__ import annotations

import numpy as np

from . import e4m3

GROUP = 128
M32 = np.uint64(0xFFFFFFFF)


def mix(h):
    """The 32-bit finalizer of MurmurHash3 (A. Appleby), of numbers held in 64 bits."""
    h = np.asarray(h, dtype=np.uint64)
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & M32
    h = ((h ^ (h >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & M32
    return h ^ (h >> np.uint64(16))


def xorshift(x):
    """One step of the 32-bit xorshift generator (G. Marsaglia, 2003; 13, 17, 5), of numbers held in 64 bits."""
    x = (x ^ (x << np.uint64(13))) & M32
    x = x ^ (x >> np.uint64(17))
    return (x ^ (x << np.uint64(5))) & M32


def random_words(seed: int, step: int, place: int, n: int, first: int = 0) -> np.ndarray:
    """The random word (uint64 below 2^32) of the elements first .. first + n - 1 (first a multiple of 8) of a list's tensor
    number `place`: its low 16 bits round the moment, its high 16 bits the root."""
    key = np.uint64(0)
    for word in (seed & 0xFFFFFFFF, seed >> 32, step & 0xFFFFFFFF, place):
        key = mix(key ^ np.uint64(word))
    k = np.arange(first // 8, first // 8 + (n + 7) // 8, dtype=np.uint64)
    x = mix(((key ^ (k >> np.uint64(32))) + (k & M32) * np.uint64(0x9E3779B9)) & M32) | np.uint64(1)
    words = []
    for _ in range(8):
        x = xorshift(x)
        words.append(x)
    return np.stack(words, axis=1).reshape(-1)[:n]


def blocks(v: np.ndarray) -> np.ndarray:
    """[ceil(n / 128), 128], the last one filled up with zeros."""
    out = np.zeros(-(-v.size // GROUP) * GROUP, dtype=v.dtype)
    out[: v.size] = v.reshape(-1)
    return out.reshape(-1, GROUP)


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    v = e4m3.decode(blocks(codes)).astype(np.float32) * scales[:, None]
    return v.reshape(-1)[: codes.size]


def encode(v: np.ndarray, chance: np.ndarray, root: bool):
    """(codes, scales) of float32 values with 16 random bits each."""
    b = blocks(v)
    amax = np.fmax.reduce(np.abs(b), axis=1, initial=np.float32(0))      # a NaN does not enter
    a = np.maximum(amax, np.float32(2.0 ** -96))
    s, r = a * (np.float32(1) / np.float32(448)), np.float32(448) * (np.float32(1) / a)
    y = (b * r[:, None]).reshape(-1)[: v.size]
    bits = y.view(np.uint32).astype(np.uint64) + (chance.astype(np.uint64) << np.uint64(4))
    cut = (bits & np.uint64(0xFFF00000)).astype(np.uint32).view(np.float32)
    cut = np.where(np.isnan(y), y, cut)
    if root:
        cut = np.where((v > 0) & (cut < np.float32(2.0 ** -9)), np.float32(2.0 ** -9), cut)
    return np.where(np.isnan(cut), np.uint8(0x7F), e4m3.encode_nearest(np.where(np.isnan(cut), np.float32(0), cut))), s


def states(grad, m, v, beta1: float, beta2: float, coef=np.float32(1)):
    """(m', v') in float32 from float32 gradients and states."""
    f = np.float32
    g = grad * f(coef)
    return f(beta1) * m + f(1 - beta1) * g, f(beta2) * v + f(1 - beta2) * g * g


def step8(grad, avg, sq, avg_scale, sq_scale, beta1: float, beta2: float, seed: int, step: int, place: int, coef=np.float32(1)):
    """New (avg, sq, avg_scale, sq_scale) of one tensor, and the float32 (m', root) that the parameters' step takes."""
    m, root = decode(avg, avg_scale), decode(sq, sq_scale)
    m, v = states(grad.reshape(-1), m, root * root, beta1, beta2, coef)
    root = np.sqrt(v)
    word = random_words(seed, step, place, m.size)
    qa, sa = encode(m, word & np.uint64(0xFFFF), False)
    qr, sr = encode(root, word >> np.uint64(16), True)
    return qa, qr, sa, sr, m, root
