"""Reference of the 4-bit key/value cache, in numpy and apart from the library: the cache format byte by byte, the
quantiser in fp32 (each operation rounded once, as the format defines it), and attention in fp64 with bounds on what
fp32 scores and fp16 probabilities may do to it."""
import numpy as np


def page_bytes(kv, D, P):
    return kv * P * (D + 8)


def quantise(x):
    """(codes u8, d, m fp16) of fp32 vectors x [..., D]."""
    x = np.asarray(x, np.float32)
    fine = np.isfinite(x).all(-1, keepdims=True)
    x = np.where(fine, x, np.float32(0))
    with np.errstate(over="ignore", divide="ignore"):
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        m = np.clip(-lo, np.float32(-65504), np.float32(65504)).astype(np.float16)
        d = np.minimum((hi - lo) * np.float32(1.0 / 15.0), np.float32(65504)).astype(np.float16)
        inv = np.where(d == 0, np.float32(0), np.float32(1) / np.where(d == 0, np.float16(1), d).astype(np.float32))
        q = np.clip(np.rint((x + m.astype(np.float32)) * inv), 0, 15)
    nan = np.float16(np.nan)
    return np.where(fine, q, 0).astype(np.uint8), np.where(fine, d, nan)[..., 0], np.where(fine, m, nan)[..., 0]


def places(D, P, t):
    """Byte and shift of the D codes of token t of a page's head block, and the byte of its pair, for keys and values."""
    W = min(4, D // 32)
    U = D // 8 // W
    e = np.arange(D)
    w = e // 8
    k = ((t // 16 * U + w // W) * 16 + t % 16) * W + w % W
    v = P * D // 8 + (t // 4 * (D // 8) + w) * 4 + t % 4
    return [(word * 4 + e % 8 // 2, e % 2 * 4, P * D + side * 4 * P + 4 * t) for side, word in enumerate((k, v))]


def write(block, D, P, t, side, q, d, m):
    """Put a vector's codes and pair into a head block (u8 array)."""
    byte, shift, at = places(D, P, t)[side]
    for i in range(D):
        block[byte[i]] = (int(block[byte[i]]) & ~(15 << shift[i]) & 255) | (int(q[i]) << shift[i])
    block[at:at + 4] = np.array([d, m], np.float16).view(np.uint8)


def read(block, D, P, t, side):
    """d q - m of a token, exact in fp64."""
    byte, shift, at = places(D, P, t)[side]
    d, m = block[at:at + 4].view(np.float16).astype(np.float64)
    return d * (block[byte] >> shift & 15) - m, d, m


class Cache:
    """A host image of a cache."""

    def __init__(self, image, kv, D, P):
        self.raw = np.asarray(image, np.uint8).reshape(-1, kv, P * (D + 8))
        self.kv, self.D, self.P = kv, D, P

    def at(self, table_row, pos):
        """(page, token) of a position, or None where it is absent."""
        j = pos // self.P
        if pos < 0 or j >= len(table_row) or not 0 <= table_row[j] < len(self.raw):
            return None
        return int(table_row[j]), pos % self.P

    def tokens(self, table_row, n):
        """Keys, values [n][kv][D] fp64, their pairs [n][kv][2] and presence [n] of positions 0..n-1."""
        D, P, kv = self.D, self.P, self.kv
        k, v = np.zeros((2, n, kv, D))
        dk, dv = np.zeros((2, n, kv, 2))
        here = np.zeros(n, bool)
        where = [places(D, P, t) for t in range(P)]
        for pos in range(n):
            at = self.at(table_row, pos)
            if at is None:
                continue
            here[pos] = True
            b = self.raw[at[0]]
            for side, (x, dm) in enumerate(((k, dk), (v, dv))):
                byte, shift, pair = where[at[1]][side]
                dm[pos] = b[:, pair:pair + 4].copy().view(np.float16).astype(np.float64)
                x[pos] = dm[pos][:, :1] * (b[:, byte] >> shift & 15) - dm[pos][:, 1:]
        return k, v, dk, dv, here


def attend(cache, table, start, lens, q, scale, causal=True, window=0):
    """Outputs [n][heads][D] and log sums [n][heads] in fp64, and for each row what bounds its error: the largest
    |score| sum, the mean |v|, the mean of 8 d, and the number of tokens."""
    n, heads, D = q.shape
    out, lse = np.full((n, heads, D), np.nan), np.full((n, heads), np.nan)
    size, mean, grid, seen = (np.zeros((n, heads)) for _ in range(4))
    for s in range(len(lens)):
        a, b, length = int(start[s]), int(start[s + 1]), max(int(lens[s]), 0)
        if a >= b:
            continue
        span = min(length, len(table[s]) * cache.P)
        k, v, dk, dv, here = cache.tokens(table[s], span)
        for i in range(a, b):
            pos = length - (b - a) + i - a
            j = np.arange(span)
            mask = here & (j <= pos if causal else j < length)
            if window:
                mask &= j > pos - window
            for h in range(heads):
                g = h * cache.kv // heads
                if not mask.any():
                    out[i, h], lse[i, h] = 0, -np.inf
                    continue
                kk, vv = k[mask, g], v[mask, g]
                x = kk @ q[i, h] * scale
                top = x.max()
                p = np.exp(x - top)
                out[i, h], lse[i, h] = p @ vv / p.sum(), top + np.log(p.sum())
                centre = dk[mask, g]
                size[i, h] = scale * np.max(np.abs(kk - (8 * centre[:, :1] - centre[:, 1:])) @ np.abs(q[i, h])
                                            + np.abs(8 * centre[:, 0] - centre[:, 1]) * np.abs(q[i, h]).sum())
                mean[i, h] = np.max(p @ np.abs(vv)) / p.sum()
                grid[i, h] = 8 * (p @ dv[mask, g, 0]) / p.sum()
                seen[i, h] = mask.sum() * 8 * dv[mask, g, 0].max() / p.sum()
    return out, lse, dict(size=size, mean=mean, grid=grid, seen=seen)


def attend_one(cache, table, length, q, scale, window):
    """attend() of one sequence whose tokens are all present, causal, by matrix products (for many rows)."""
    n, heads, _ = q.shape
    k, v, dk, dv, here = cache.tokens(table, length)
    assert here.all()
    shape = (n, heads)
    out, lse, by = np.zeros(q.shape), np.zeros(shape), {x: np.zeros(shape) for x in ("size", "mean", "grid", "seen")}
    pos, j = length - n + np.arange(n), np.arange(length)
    mask = (j <= pos[:, None]) & (j > pos[:, None] - window)
    for h in range(heads):
        g = h * cache.kv // heads
        kk, vv = k[:, g], v[:, g]
        x = np.where(mask, q[:, h] @ kk.T * scale, -np.inf)
        top = x.max(1)
        p = np.exp(x - top[:, None])
        total = p.sum(1)
        out[:, h], lse[:, h] = p @ vv / total[:, None], top + np.log(total)
        offset = 8 * dk[:, g, 0] - dk[:, g, 1]
        size = np.abs(q[:, h]) @ np.abs(kk - offset[:, None]).T + np.abs(q[:, h]).sum(1)[:, None] * np.abs(offset)
        by["size"][:, h] = scale * np.max(np.where(mask, size, 0), 1)
        by["mean"][:, h] = (p @ np.abs(vv)).max(1) / total
        by["grid"][:, h] = 8 * (p @ dv[:, g, 0]) / total
        by["seen"][:, h] = mask.sum(1) * 8 * np.max(np.where(mask, dv[:, g, 0], 0), 1) / total
    return out, lse, by


def bounds(ref, lse, by, D, bf16, many=False):
    """Largest errors of out and lse.  A score is a sum of D products and two more in fp32, each addition off by at
    most a last place (the matrix cores cut off): d = (D + 8) 2^-23 of the sum of magnitudes.  An output then moves by
    2 d of the mean |v|; p dv is rounded to fp16's 2^-11 (with its remainder, which fp16 results take along where a
    sequence has not many rows: 2^-21), as a factor of |c - 8| <= 8, or to 2^-25 where it is below 2^-20 of the largest (2^-31 after scaling: the reference lies at 2^6); the output is
    rounded to its type."""
    delta = (D + 8) * 2.0 ** -23 * by["size"] + 2.0 ** -21
    unit = 2.0 ** -8 if bf16 else 2.0 ** -11
    moved = 2 * delta * by["mean"] + (2.0 ** -11 if bf16 or many else 2.0 ** -21) * by["grid"] + 2.0 ** -30 * by["seen"]
    out = moved[..., None] * (1 + unit) + unit * np.abs(ref) + (0 if bf16 else 2.0 ** -25)
    with np.errstate(invalid="ignore"):
        return out, delta + 2.0 ** -21 * (1 + np.where(np.isfinite(lse), np.abs(lse), 0))
