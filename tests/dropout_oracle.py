"""The dropout mask from its definition, in numpy on 64-bit words (host only)."""

import math

import numpy as np
import torch

M32 = 0xFFFFFFFF


def philox(counter, key):
    """Philox4x32, ten rounds: arrays (or numbers) of four counter words, two key words."""
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    k = [int(w) for w in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & np.uint64(M32),
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & np.uint64(M32)]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def threshold(p):
    return math.floor(p * 65536 + 0.5)


def keep(T, D, p, seed, step, site):
    """(kept [T, D] as a bool tensor, factor of the kept ones)."""
    n = T * D
    g = np.arange((n + 7) // 8, dtype=np.uint64)
    w = philox((g & np.uint64(M32), g >> np.uint64(32), site, step & M32), (seed & M32, (seed >> 32) & M32))
    words = np.stack([np.broadcast_to(x, g.shape) for x in w], 1).astype("<u4").view("<u2").reshape(-1)[:n]
    t = threshold(p)
    return torch.from_numpy(words >= t).view(T, D), 0.0 if t == 65536 else 65536.0 / (65536 - t)
