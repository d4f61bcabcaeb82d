"""Philox4x32-10 in numpy's uint64, and dropout's masks from it."""
import numpy as np


def philox(counter, key):
    """counter: four arrays, key: two numbers; the four output words as uint64 below 2^32."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def numbers(rows, n, seed, step):
    """The 16-bit numbers of all elements, [rows, n]."""
    g = (n + 7) // 8
    seed, step = seed % 2 ** 64, step % 2 ** 64
    r, c = np.meshgrid(np.arange(rows), np.arange(g), indexing="ij")
    w = philox((c, r, np.full_like(c, step % 2 ** 32), np.full_like(c, step >> 32)), (seed % 2 ** 32, seed >> 32))
    halves = [h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))]
    return np.stack(halves, 2).reshape(rows, 8 * g)[:, :n].astype(np.int64)


def factors(rows, n, p, seed, step):
    """0 for dropped elements, else 65536 / (65536 - t), float64."""
    t = int(np.rint(65536 * p))
    return np.where(numbers(rows, n, seed, step) >= t, 65536.0 / (65536 - t), 0.0)
