"""Philox4x32 in numpy's unsigned integers, and the dropout mask of the library's definition: the tests' own
restatement (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)."""
import numpy as np

LOW = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key, rounds):
    """counter: [..., 4], key: [2], 32-bit words as uint64; returns [..., 4] uint64."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & LOW, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1)


def threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def keep_mask(seed, offset, p, M, N, rows=None):
    """[M, N] booleans (of the rows [a, b) when `rows` says so)."""
    seed, offset = int(seed) % 2**64, int(offset) % 2**64
    a, b = rows or (0, M)
    e = np.arange(a * N, b * N, dtype=np.uint64)
    if e.size == 0:
        return np.zeros((b - a, N), dtype=bool)
    g = np.arange(int(e[0]) // 8, int(e[-1]) // 8 + 1, dtype=np.uint64)
    ctr = np.stack([g & LOW, g >> np.uint64(32), np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, offset >> 32)], -1)
    w = philox4x32(ctr, (seed & 0xFFFFFFFF, seed >> 32), 7)
    half = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(-1)
    at = (e - g[0] * np.uint64(8)).astype(np.int64)
    return (half[at] >= threshold(p)).reshape(b - a, N)
