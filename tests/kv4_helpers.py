"""Plain references of the operators around the 4-bit cache, in binary64 (or,
where a result is defined by binary32 steps, those steps one by one in numpy),
sharing no code with the CUDA path."""
import numpy as np

GROUP, TILE = 64, 16


def bf16(x):
    """float64 values rounded to bfloat16 (nearest even), as float64."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def quantise(x):
    """Codes [..., D], scales and zeros [..., D / 64] of bfloat16 values, by the
    formula's binary32 steps."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = np.minimum(g.min(-1), np.float32(0)), np.maximum(g.max(-1), np.float32(0))
    s16 = np.minimum((hi - lo) / np.float32(15), np.float32(65504)).astype(np.float16)
    s = s16.astype(np.float32)
    ok = s > 0
    safe = np.where(ok, s, np.float32(1))
    z = np.where(ok, np.clip(np.rint(-lo / safe), 0, 15), 0).astype(np.float32) + np.float32(0)   # +0, not -0
    q = np.clip(np.rint(g / safe[..., None]) + z[..., None], 0, 15) * ok[..., None]
    return q.reshape(x.shape).astype(np.uint8), s16, z.astype(np.float16)


class Cache:
    """A 4-bit cache on the host: bytes in the library's layout."""

    def __init__(self, blocks, Hkv, bs, D, fill=0):
        self.blocks, self.H, self.bs, self.D = blocks, Hkv, bs, D
        self.raw = np.full((blocks, Hkv, bs // TILE, 18 * D), fill, np.uint8)

    def put(self, part, slot, h, codes, s, z):
        D, r = self.D, slot % TILE
        tile = self.raw[slot // self.bs, h, slot % self.bs // TILE]
        for g in range(D // GROUP):
            c = codes[g * GROUP:(g + 1) * GROUP]
            at = part * 8 * D + (g * TILE + r) * 32
            tile[at:at + 32] = c[0::2] | (c[1::2] << 4)
            at = (16 + part) * D + (g * TILE + r) * 4
            tile[at:at + 4] = np.array([s[g], z[g]], np.float16).view(np.uint8)

    def append(self, k, v, slots):
        for part, x in ((0, k), (1, v)):
            c, s, z = quantise(x)
            for t, slot in enumerate(slots):
                if 0 <= slot < self.blocks * self.bs:
                    for h in range(self.H):
                        self.put(part, int(slot), h, c[t, h], s[t, h], z[t, h])

    def values(self, part, slot, h):
        D, r = self.D, slot % TILE
        tile = self.raw[slot // self.bs, h, slot % self.bs // TILE]
        out = np.empty(D)
        for g in range(D // GROUP):
            at = part * 8 * D + (g * TILE + r) * 32
            b = tile[at:at + 32]
            at = (16 + part) * D + (g * TILE + r) * 4
            s, z = tile[at:at + 4].view(np.float16).astype(np.float64)
            c = np.empty(GROUP)
            c[0::2], c[1::2] = b & 15, b >> 4
            out[g * GROUP:(g + 1) * GROUP] = (c - z) * s
        return out


def norm_rope(x, w, cos_sin, positions, eps=1e-6, offset=0.0, interleaved=False):
    """[T, H, D] in binary64, and a bound of |a| + |b| of each rotated pair."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (np.asarray(w, np.float64) + offset)
    size = np.abs(x)
    if cos_sin is None:
        return x, size
    rot = cos_sin.shape[1]
    y, h = x.copy(), rot // 2
    inside = (positions >= 0) & (positions < cos_sin.shape[0])
    row = np.asarray(cos_sin, np.float64)[np.where(inside, positions, 0)][:, None]
    c, s = row[..., :h], row[..., h:]
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(h), np.arange(h, rot))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size = size.copy()
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    y[~inside] = 0
    return y, size


def attention(q, cache, table, seq_lens, cu, scale, window=0, sinks=0):
    """out [T, Hq, D] in binary64 and a bound of the kernels' error.

    The bound: one BF16 rounding of the result (8 significant bits: 2^-8 of it
    at most); each weight of the sum over V
    rounded once to binary16 (2^-11) and each value at most once (2^-12); each
    key at most once to binary16 (a score error of 2^-12 scale sum |q k|), plus
    2^-20 of that sum for the binary32 sums; a score error e changes a
    normalised weight by at most a factor exp(2 e)."""
    T, Hq, D = q.shape
    G = Hq // cache.H
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b in range(len(seq_lens)):
        n = int(cu[b + 1] - cu[b])
        if n == 0:
            continue
        end = max(0, int(seq_lens[b]))
        end = min(end, table.shape[1] * cache.bs)
        slots = [int(table[b, j // cache.bs]) * cache.bs + j % cache.bs for j in range(end)]
        here = np.array([0 <= int(table[b, j // cache.bs]) < cache.blocks for j in range(end)], bool)
        for h in range(cache.H):
            zero = np.zeros(D)
            K = np.array([cache.values(0, s, h) if ok else zero for s, ok in zip(slots, here)]).reshape(end, D)
            V = np.array([cache.values(1, s, h) if ok else zero for s, ok in zip(slots, here)]).reshape(end, D)
            for i in range(n):
                t = int(cu[b]) + i
                p = int(seq_lens[b]) - n + i
                j = np.arange(end)
                see = here & (j <= p)
                if window > 0:
                    see &= (p - j < window) | (j < sinks)
                if not see.any():
                    continue
                k, v = K[see], V[see]
                for r in range(G):
                    x = q[t, h * G + r]
                    sc = scale * (k @ x)
                    e = (2.0 ** -12 + 2.0 ** -20) * abs(scale) * (np.abs(k) @ np.abs(x)).max()
                    w = np.exp(sc - sc.max())
                    w /= w.sum()
                    o = w @ v
                    out[t, h * G + r] = o
                    tol[t, h * G + r] = (2.0 ** -8 * np.abs(o) +
                                         (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -16 + np.expm1(2 * e)) * (w @ np.abs(v)) *
                                         (1 + 2.0 ** -8) + 1e-30)
    return out, tol
