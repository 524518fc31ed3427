"""Reference of the operators around long sequences of the 4-bit key/value cache, in numpy and apart from the library:
rotary positions, bounds and scores of pages, attention weights of pages, and which pages are given up."""
import math
from decimal import Decimal, getcontext

import numpy as np

import kv_ref as R

getcontext().prec = 60
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(pairs, base, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0):
    """Turns a position of each pair, to 60 digits."""
    b, k = Decimal(base), Decimal(factor)
    if scaling == "base":
        b *= (k.ln() * pairs / (pairs - 1)).exp()
    out = []
    if scaling == "index":
        at = lambda t: pairs * math.log(original / (2 * math.pi * t)) / math.log(base)
        lo, hi = Decimal(max(math.floor(at(high)), 0)), Decimal(min(math.ceil(at(low)), 2 * pairs - 1))
        hi += Decimal("0.001") if hi == lo else 0
    for i in range(pairs):
        f = (-b.ln() * i / pairs).exp()
        if scaling == "linear":
            f /= k
        if scaling == "index":
            r = min(max((i - lo) / (hi - lo), Decimal(0)), Decimal(1))
            f *= 1 - r + r / k
        if scaling == "turns":
            s = (Decimal(original) * f / TWO_PI - Decimal(low)) / (Decimal(high) - Decimal(low))
            s = min(max(s, Decimal(0)), Decimal(1))
            f *= s + (1 - s) / k
        out.append(f / TWO_PI)
    return out


def rope(x, pos, turn, halves, amplitude=1.0):
    """x [n][heads][D] turned, in fp64 (angles: the fraction of a turn to 60 digits)."""
    y = x.astype(np.float64).copy()
    n = len(turn)
    for i, t in enumerate(turn):
        angle = np.array([float((t * int(p)) % 1 * TWO_PI) for p in pos])[:, None]
        c, s = amplitude * np.cos(angle), amplitude * np.sin(angle)
        u, v = (i, i + n) if halves else (2 * i, 2 * i + 1)
        a, b = x[..., u].astype(np.float64), x[..., v].astype(np.float64)
        y[..., u], y[..., v] = a * c - b * s, a * s + b * c
    return y


def least_exponent(top):
    """The smallest e with top <= 127 * 2^e (0 for 0)."""
    if top == 0:
        return 0
    e = math.frexp(top)[1] - 8
    while top > 127 * 2.0 ** e:
        e += 1
    return e


def bounds_bytes(kv, D):
    return (kv * (2 * D + 4) + 15) // 16 * 16


def page_bounds(cache, page):
    """(hi, lo codes [kv][D], e [kv]) of a full page."""
    kv, D, P = cache.kv, cache.D, cache.P
    hi, lo, es = np.zeros((kv, D), np.int8), np.zeros((kv, D), np.int8), np.zeros(kv, np.int32)
    for h in range(kv):
        k = np.array([R.read(cache.raw[page, h], D, P, t, 0)[0] for t in range(P)])
        pairs = cache.raw[page, h, P * D:P * (D + 4)].copy().view(np.float16)
        if not np.isfinite(pairs).all():
            es[h] = 127
            continue
        k = k.astype(np.float32).astype(np.float64)
        most, least = k.max(0), k.min(0)
        e = least_exponent(max(np.abs(most).max(), np.abs(least).max()))
        hi[h], lo[h], es[h] = np.ceil(most / 2.0 ** e), np.floor(least / 2.0 ** e), e
    return hi, lo, es


def put_bounds(raw, kv, D, page, b):
    """Into a buffer [pages][bounds_bytes] of bytes."""
    hi, lo, es = b
    raw[page, :kv * 2 * D] = np.stack([hi, lo], 1).reshape(-1).view(np.uint8)
    raw[page, kv * 2 * D:kv * (2 * D + 4)] = es.view(np.uint8)


def scores(raw, kv, D, pages, g, q):
    """Scores of pages (numbers) for kv head g of its query heads q [group][D]."""
    q = np.asarray(q, np.float64)
    whole, power = [], []
    for x in q:
        top = np.abs(x).max() if np.isfinite(x).all() else 0.0
        e = least_exponent(top)
        whole.append(np.rint(x / 2.0 ** e) if top else np.zeros(D))
        power.append(e if top else None)
    most = max((e for e in power if e is not None), default=0)
    out = []
    for p in pages:
        code = raw[p, g * 2 * D:(g + 1) * 2 * D].view(np.int8).astype(np.float64).reshape(2, D)
        e = int(raw[p, kv * 2 * D + 4 * g:kv * 2 * D + 4 * g + 4].copy().view(np.int32)[0])
        best = -np.inf
        for z, k in zip(whole, power):
            s = np.maximum(z * code[0], z * code[1]).sum()
            best = max(best, s * 2.0 ** (max(k - most, -64) if k is not None else 0))
        out.append(np.inf if e == 127 else best * 2.0 ** e)
    return out


def select(raw, kv, D, P, n_pages, table, start, lens, q, first, last, take):
    """(lens [n], table [n][kv][take]) of rows q [n][heads][D]."""
    n, group = len(q), q.shape[1] // kv
    got, out = np.full((n, kv, take), -1, np.int32), np.zeros(n, np.int32)
    for s in range(len(lens)):
        for i in range(int(start[s]), int(start[s + 1])):
            pos = max(int(lens[s]), 0) - int(start[s + 1]) + i
            if pos < 0:
                continue
            own = pos // P
            have = [j for j in range(min(own, table.shape[1])) if 0 <= table[s, j] < n_pages]
            must = [j for j in have if j < first or j >= own - last]
            rest = [j for j in have if j not in set(must)]
            for g in range(kv):
                sc = scores(raw, kv, D, table[s, rest], g, q[i, g * group:(g + 1) * group])
                best = [j for _, j in sorted(zip([-x for x in sc], rest))][:take - 1 - len(must)]
                mine = sorted(must + best)
                got[i, g, :len(mine)] = table[s, mine]
                got[i, g, len(mine)] = table[s, own] if own < table.shape[1] else -1
            out[i] = len(mine) * P + pos % P + 1
    return out, got


def weigh(cache, table, start, lens, q, lse, scale, causal, window, stride):
    """Weights [seqs][kv][stride] in fp64 that the rows gave, which pages are weighed [seqs][stride], and bounds on
    what fp32 scores and sums may do to them."""
    n, heads, D = q.shape
    kv, P = cache.kv, cache.P
    w, used = np.zeros((len(lens), kv, stride)), np.zeros((len(lens), stride), bool)
    err = np.zeros_like(w)
    for s in range(len(lens)):
        a, b, length = int(start[s]), int(start[s + 1]), max(int(lens[s]), 0)
        if a >= b:
            continue
        used[s, :min(-(-length // P), stride)] = True
        span = min(length, table.shape[1] * P)
        k, _, dk, _, here = cache.tokens(table[s], span)
        j = np.arange(span)
        for i in range(a, b):
            pos = length - (b - a) + i - a
            mask = here & (j <= pos if causal else j < length)
            if window:
                mask &= j > pos - window
            for h in range(heads):
                g = h * kv // heads
                if not mask.any() or not np.isfinite(lse[i, h]):
                    continue
                x = k[mask, g] @ q[i, h] * scale
                p = np.exp(x - float(lse[i, h]))
                off = 8 * dk[mask, g, 0] - dk[mask, g, 1]
                size = scale * (np.abs(k[mask, g] - off[:, None]) @ np.abs(q[i, h]) + np.abs(off) * np.abs(q[i, h]).sum())
                keep = j[mask] // P < stride
                np.add.at(w[s, g], j[mask][keep] // P, p[keep])
                # a score is a sum of D products and some more in fp32; its place in an exponential is off by
                # 2^-24 of up to 2^5 (what lies lower is nothing), the exponential by a last place
                np.add.at(err[s, g], j[mask][keep] // P, (p * ((D + 8) * 2.0 ** -23 * size + 2.0 ** -18))[keep])
    # additions in a row: a lane's tokens of all rows, then the lanes
    chain = (n * heads // kv + 16) * (P // 16 + 1) // 4 + 64
    return w, used, err + w * chain * 2.0 ** -24


def evict(table, lens, weights, P, n_pages, keep, first, last):
    """(table, gone, count) after giving pages up; weights [seqs][kv][stride] fp32."""
    table = table.copy()
    gone, count = np.full_like(table, -1), np.zeros(len(lens), np.int32)
    for s in range(len(lens)):
        used = -(-max(int(lens[s]), 0) // P)
        have = [j for j in range(min(used, table.shape[1])) if 0 <= table[s, j] < n_pages]
        order = []
        for j in have:
            if not first <= j < used - last:
                continue
            x = 0.0
            if j < weights.shape[2]:
                for h in range(weights.shape[1]):
                    x += float(weights[s, h, j])
                x = float(np.float32(x))
            else:
                x = np.nan
            order.append((1, 0.0, j) if x != x else (0, x, j))
        drop = sorted(j for _, _, j in sorted(order)[:max(len(have) - keep, 0)])
        gone[s, :len(drop)] = table[s, drop]
        count[s] = len(drop)
        table[s, drop] = -1
    return table, gone, count
