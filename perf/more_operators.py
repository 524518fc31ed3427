"""Long sequences over the 4-bit key/value cache: what is measured of the operators around it.

rope:   rotary positions.  lw_rope turns pairs of dimensions of queries and keys by their position, in the types that
        the projections give and the cache takes.
sparse: attention over a few pages.  lw_kv_bounds keeps, for each full page and kv head, each channel's largest and
        smallest key in 8 bits, lw_kv_select scores the pages of a row's sequence with them and takes the best, and
        lw_kv_attend_selected attends over those.
weigh:  the attention weight that a call's rows gave to each page of their sequences (lw_kv_weigh).
evict:  the pages of least weight given up (lw_kv_evict).

Rotary positions.  Pair i of `pairs` is turned by pos * f_i: (a, b) -> g (a cos - b sin, a sin + b cos), where a and b
are dimensions i and i + pairs ("halves") or 2i and 2i + 1 ("pairs"), and dimensions past 2 pairs stay.
f_i = base^(-i / pairs), and for contexts longer than the `original` one
    linear  f / factor
    base    (base factor^(pairs / (pairs - 1)))^(-i / pairs)
    index   f (1 - r + r / factor), r = (i - lo) / (hi - lo) within 0..1, where lo = floor(at(high)) and
            hi = ceil(at(low)), kept within 0..2 pairs - 1, hi 0.001 more where they are equal, and
            at(turns) = pairs ln(original / (2 pi turns)) / ln(base)
    turns   f (s + (1 - s) / factor), s = (original f / 2 pi - low) / (high - low) within 0..1

The cache is the one of lw_kv_append: a page holds P tokens of every kv head, per head P*D/2 bytes of key codes, P*D/2
of value codes, P words d | m << 16 of the keys and P of the values, a vector being worth d*q - m.  Word w (eight codes,
the lowest dimension in the low nibble) of token t lies, for keys, at (((t/16) * U + w/W) * 16 + t%16) * W + w%W with
W = min(4, D/32) and U = D/8/W, and for values at ((t/4) * (D/8) + w) * 4 + t%4.  Row i of a sequence's n new tokens is
at position lens - n + i and sees the positions up to its own.

Bounds.  Of a page's P keys of a head, as lw_kv_read gives them in 32 bits: hi and lo, each channel's largest and
smallest, and e, the smallest whole number with all |hi|, |lo| <= 127 * 2^e (0 where they are 0).  Held: ceil(hi 2^-e)
and floor(lo 2^-e), D bytes each, head after head, then the heads' e as 32-bit numbers, padded to 16 bytes.

Scores.  A query head vector x is taken as whole numbers rint(x 2^-e), e as above (zeros where x has a NaN or an
infinity).  A head's score for a page is sum_d max(x_d hi_d, x_d lo_d) of those numbers times 2^max(e - top, -64), top
the largest e of the kv head's group (of its heads that are not zero), times 2^(the page's e), and the page's is the
largest of the group's heads': whole numbers times powers of two, exact in 32 bits.  A row takes the page of its own
position, the first `first` pages, the last `last` ones before its own, and of the others those of the highest scores,
the lowest position first among equals, until it has `take`.

Weights.  w[s][g][j] = decay * (what it was) + the sum, over the sequence's rows and the query heads of kv head g, and
over the tokens of page j that a row sees, of exp(scale q.k - lse).

Giving up.  Of a sequence's pages those with the lowest weights (summed over heads in 64 bits and rounded to 32), the
lowest position first among equals, but not the first `first` and the last `last`, until `keep` are left.
"""
import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
WIDTH = {"fp16": 2, "bf16": 2, "fp32": 4}


def listed():
    return [
        # one user's next token, from a coded projection's fp32 output to the fp16 that attention takes: latency
        dict(name="rope_1_token", op="rope", seqs=1, new_min=1, new_max=1, len_min=777, len_max=777, heads=40, dim=128, pairs=64, layout="halves", scaling="none", base=10000.0, factor=1.0, original=0, low=0.0, high=0.0, given=False, x="fp32", y="fp16"),
        # a step of a serving batch, a part of each head turned, neighbouring dimensions
        dict(name="rope_96_seqs", op="rope", seqs=96, new_min=1, new_max=2, len_min=33, len_max=40000, heads=33, dim=96, pairs=24, layout="pairs", scaling="linear", base=10000.0, factor=8.0, original=4096, low=0.0, high=0.0, given=True, x="bf16", y="bf16"),
        # prompts of several users, a context stretched 16 times
        dict(name="rope_prompts", op="rope", seqs=5, new_min=1001, new_max=8191, len_min=1001, len_max=131071, heads=40, dim=128, pairs=64, layout="halves", scaling="index", base=500000.0, factor=16.0, original=8192, low=1.0, high=32.0, given=False, x="fp32", y="bf16"),
        # one user's token on a medium conversation; it fills a page
        dict(name="sparse_1", op="sparse", seqs=1, new_min=1, new_max=1, len_min=5120, len_max=5120, heads=32, kv=8, dim=128, page=64, take=16, first=1, last=1, dtype="fp16"),
        # a serving batch of many lengths
        dict(name="sparse_16", op="sparse", seqs=16, new_min=1, new_max=1, len_min=501, len_max=32760, heads=32, kv=8, dim=128, page=64, take=32, first=1, last=2, dtype="bf16"),
        # one very long context
        dict(name="sparse_long", op="sparse", seqs=1, new_min=1, new_max=1, len_min=131071, len_max=131071, heads=64, kv=8, dim=128, page=32, take=128, first=2, last=4, dtype="fp16"),
        # a few guessed tokens a sequence checked at once, wide heads
        dict(name="sparse_verify", op="sparse", seqs=7, new_min=3, new_max=5, len_min=9000, len_max=50000, heads=16, kv=4, dim=256, page=128, take=12, first=1, last=1, dtype="fp16"),
        # what one user's token looked at on a long context
        dict(name="weigh_long", op="weigh", seqs=1, new_min=1, new_max=1, len_min=131071, len_max=131071, heads=64, kv=8, dim=128, page=64, decay=1.0, window=0, dtype="fp16"),
        # a step of a serving batch, older weights fading
        dict(name="weigh_16", op="weigh", seqs=16, new_min=1, new_max=3, len_min=501, len_max=8190, heads=32, kv=8, dim=128, page=32, decay=0.95, window=0, dtype="bf16"),
        # a prompt's piece over what the cache already has, before its pages are thinned out
        dict(name="weigh_prompt", op="weigh", seqs=2, new_min=1023, new_max=1024, len_min=3001, len_max=8192, heads=32, kv=8, dim=128, page=64, decay=1.0, window=0, dtype="bf16"),
        # one conversation past its budget
        dict(name="evict_1", op="evict", seqs=1, len_min=6001, len_max=6001, kv=8, page=64, keep=64, first=1, last=4),
        # a serving batch, long and short
        dict(name="evict_64", op="evict", seqs=64, len_min=100, len_max=131071, kv=8, page=32, keep=1000, first=2, last=8),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("rope", "sparse", "sparse", "weigh", "evict"))
    case = dict(op=op)
    if op == "rope":
        case["dim"] = rng.choice((64, 128, 128, 256, 80, 96, 112, 66))
        case["pairs"] = rng.choice((case["dim"] // 2, case["dim"] // 2, case["dim"] // 4, rng.randint(2, case["dim"] // 2)))
        case["heads"] = rng.choice((1, 2, 5, 8, 12, 24, 40, 72))
        case["seqs"] = log(1, 64)
        case["new_max"] = log(1, max(2, min(8192, 18000 * 40 * 128 // (case["seqs"] * case["heads"] * case["dim"]))))
        case["new_min"] = rng.randint(1, case["new_max"])
        case["len_min"] = case["new_max"] + log(1, 4000) - 1
        case["len_max"] = case["len_min"] + log(1, 200000) - 1
        case["layout"] = rng.choice(("halves", "pairs"))
        case["scaling"] = rng.choice(("none", "linear", "base", "index", "turns"))
        case["base"] = rng.choice((10000.0, 500000.0, 1000000.0))
        case["factor"] = 1.0 if case["scaling"] == "none" else rng.choice((2.0, 8.0, 32.0, 2.5))
        case["original"] = rng.choice((2048, 4096, 8192, 32768))
        case["low"], case["high"] = rng.choice(((1.0, 4.0), (1.0, 32.0)))
        case["given"] = rng.random() < 0.3
        case["x"], case["y"] = rng.choice(tuple(TYPES)), rng.choice(tuple(TYPES))
        return case
    case["kv"] = rng.choice((1, 2, 4, 8, 8, 16))
    case["page"] = rng.choice((32, 64, 128, 256))
    if op == "evict":
        case["seqs"] = log(1, 64)
        case["len_max"] = log(2, 131072)
        case["len_min"] = rng.randint(1, case["len_max"])
        case["keep"] = log(1, max(2, case["len_max"] // case["page"]))
        case["first"], case["last"] = rng.choice((0, 1, 4)), rng.choice((1, 2, 9))
        return case
    case["dim"] = rng.choice((64, 128, 128, 256))
    if case["dim"] == 256:
        case["kv"] = min(case["kv"], 4)
    case["heads"] = case["kv"] * rng.choice((1, 2, 4, 5, 8))
    case["dtype"] = rng.choice(("fp16", "bf16"))
    unit = case["kv"] * case["dim"]
    if op == "sparse":
        case["seqs"] = log(1, 32)
        case["new_max"] = rng.choice((1, 1, 1, 2, 5, 9))
        case["len_max"] = log(20, max(40, min(131072, 131072 * 1024 // (case["seqs"] * unit))))
        case["first"], case["last"] = rng.choice((0, 1, 2)), rng.choice((0, 1, 4))
        most = 16 * 32 * 64 * 1024 // (case["seqs"] * case["new_max"] * unit * case["page"])
        case["take"] = case["first"] + case["last"] + log(1, max(2, min(128, most)))
    else:
        case["decay"] = rng.choice((1.0, 0.95, 0.0))
        case["window"] = rng.choice((0, 0, log(16, 4096)))
        if rng.random() < 0.6:
            case["seqs"] = log(1, 64)
            case["new_max"] = rng.choice((1, 1, 2, 5, 9))
            case["len_max"] = log(20, max(40, min(131072, 131072 * 1024 // (case["seqs"] * unit * case["new_max"]))))
        else:
            case["seqs"] = log(1, 4)
            case["new_max"] = log(17, 1024)
            most = 2 * 1024 * 32 * 128 * 8192 // (case["seqs"] * case["new_max"] * case["heads"] * case["dim"])
            case["len_max"] = log(case["new_max"], max(case["new_max"] + 1, min(8192, most)))
    case["new_min"] = rng.randint(1, case["new_max"])
    case["len_min"] = max(case["new_max"], rng.randint(1, case["len_max"]))
    case["len_max"] = max(case["len_max"], case["len_min"])
    return case


def spread(lo, hi, n):
    """n whole numbers from lo to hi, the largest first and the others in no order."""
    return [hi if i == 0 else lo + (hi - lo) * ((i * 7919 + 13) % n) // n for i in range(n)]


def sizes(case):
    new = spread(case.get("new_min", 1), case.get("new_max", 1), case["seqs"])
    lens = [max(a, b) for a, b in zip(spread(case["len_min"], case["len_max"], case["seqs"]), new)]
    return new, lens


def bounds_bytes(kv, dim):
    return -(-kv * (2 * dim + 4) // 16) * 16


def work(case):
    new, lens = sizes(case)
    rows = sum(new)
    if case["op"] == "rope":
        n = rows * case["heads"]
        return {"bytes": n * case["dim"] * (WIDTH[case["x"]] + WIDTH[case["y"]]), "flops": n * case["pairs"] * 6}
    kv, page = case["kv"], case["page"]
    pages = [-(-n // page) for n in lens]
    if case["op"] == "evict":
        return {"bytes": sum(pages) * 4 * kv + 3 * 4 * max(pages) * case["seqs"], "flops": sum(pages) * kv}
    dim, heads = case["dim"], case["heads"]
    key, q = kv * (dim // 2 + 4), rows * heads * dim * 2
    if case["op"] == "weigh":
        pairs = seen = 0
        for n, length in zip(new, lens):
            w = case["window"] or length
            first, last = length - n + 1, length                 # keys at or before each new token
            full = max(0, last - max(first, w) + 1)              # rows whose window is full
            pairs += full * w + sum(range(first, min(last, w - 1) + 1))
            seen += length - max(0, first - w)
        return {"bytes": seen * key + q + rows * heads * 4 + 8 * kv * sum(pages), "flops": 2 * dim * heads * pairs}
    filled = sum(length // page - (length - n) // page for n, length in zip(new, lens))
    took = [min(p, case["take"]) for p in pages]
    read = sum(min(p, n * t) for p, n, t in zip(pages, new, took)) * page * kv * (dim + 8)
    held = (sum(pages) + filled) * kv * (2 * dim + 4) + filled * page * key
    return {"bytes": read + held + 2 * q + rows * (kv * case["take"] + heads + 1) * 4,
            "flops": sum(n * (t * page * 4 + 4 * p) for n, t, p in zip(new, took, pages)) * dim * heads}


# ------------------------------------------------------------------ the cache, as elementary operations

def quantise(x):
    """Codes and pairs (d, m) of vectors x[..., D], 32-bit."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    m, d = (-lo).half(), ((hi - lo) * (1.0 / 15.0)).half()
    q = torch.round((x + m.float()) / torch.where(d == 0, 1.0, d.float())).clamp(0.0, 15.0)
    return q, torch.cat((d, m), -1).contiguous().view(torch.int32).squeeze(-1)


def words(q):
    """32-bit words of codes q[..., D]."""
    q = q.unflatten(-1, (-1, 4, 2)).to(torch.uint8)
    return (q[..., 0] | q[..., 1] << 4).contiguous().view(torch.int32).squeeze(-1)


def head_words(kw, vw, kdm, vdm):
    """The words of a head's part of pages from words [..., P, D/8] and pairs [..., P] by token."""
    n = kw.shape[-1]
    w = min(4, n // 4)
    k = kw.unflatten(-1, (-1, w)).unflatten(-3, (-1, 16)).transpose(-3, -2)
    v = vw.unflatten(-2, (-1, 4)).transpose(-2, -1)
    return torch.cat((k.flatten(-4), v.flatten(-3), kdm, vdm), -1)


def worth(code_words, pairs):
    """d q - m of words [..., D/8] and pairs [...], each rounded once to 32 bits."""
    shifts = torch.arange(0, 32, 4, device=code_words.device, dtype=torch.int32)
    q = (code_words.unsqueeze(-1) >> shifts & 15).flatten(-2)
    dm = pairs.contiguous().view(torch.float16).unflatten(-1, (-1, 2))
    d, m = dm[..., :1], dm[..., 1:]
    return torch.addcmul(-m.float(), q.float(), d.float())


def keys_of(block, page, dim):
    """Keys [..., P, D] in 32 bits of heads' parts of pages."""
    w, n = min(4, dim // 32), page * dim // 8
    k = block[..., :n].unflatten(-1, (page // 16, -1, 16, w)).transpose(-3, -2).flatten(-2).flatten(-3, -2)
    return worth(k, block[..., 2 * n:2 * n + page])


def values_of(block, page, dim):
    n = page * dim // 8
    v = block[..., n:2 * n].unflatten(-1, (page // 4, dim // 8, 4)).transpose(-2, -1).flatten(-3, -2)
    return worth(v, block[..., 2 * n + page:])


def least_exponent(top):
    """The smallest e with top <= 127 * 2^e (0 for 0)."""
    f, e = torch.frexp(top)
    return torch.where(top == 0, 0, e - 7 + (f > 127.0 / 128.0))


def bounds_of(k):
    """Bounds [..., 2 D] int8 and exponents [...] of keys [..., P, D]."""
    hi, lo = k.amax(-2), k.amin(-2)
    e = least_exponent(torch.maximum(hi.abs().amax(-1), lo.abs().amax(-1)))
    unit = torch.exp2(-e.float())[..., None]
    return torch.cat((torch.ceil(hi * unit), torch.floor(lo * unit)), -1).to(torch.int8), e.to(torch.int32)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(seed)
    new, lens = sizes(case)
    seqs, rows, op = case["seqs"], sum(new), case["op"]
    start = torch.tensor([sum(new[:s]) for s in range(seqs + 1)], dtype=torch.int32, device=dev)
    state = dict(case, start=start, lens_=torch.tensor(lens, dtype=torch.int32, device=dev), rows=rows, new=new,
                 longest=max(lens), most_new=max(new), plens=lens)
    if op == "rope":
        # queries and keys lie side by side, the values after them, as one projection gives them
        wide = torch.randn((rows, case["heads"] + 8, case["dim"]), generator=g, device=dev).to(TYPES[case["x"]])
        state["x"] = wide[:, :case["heads"]]
        state["y"] = torch.empty((rows, case["heads"], case["dim"]), dtype=TYPES[case["y"]], device=dev)
        state["pos"] = None
        if case["given"]:
            _, _, at = rows_of(state)
            state["pos"] = at.to(torch.int32)
        else:
            state["table"] = torch.zeros((seqs, 1), dtype=torch.int32, device=dev)
        return state
    kv, page = case["kv"], case["page"]
    need = [-(-n // page) for n in lens]
    pool, wide = sum(need) + 3, max(need)
    at = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table, base = torch.full((seqs, wide), -1, dtype=torch.int32, device=dev), 0
    for s, n in enumerate(need):
        table[s, :n] = at[base:base + n]
        base += n
    state.update(table=table, pool=pool)
    if op == "evict":
        # a few pages were given up before; weights fall off with a heavy tail
        table.masked_fill_(torch.rand(table.shape, generator=g, device=dev) < 0.05, -1)
        state["weights"] = torch.randn((seqs, kv, wide), generator=g, device=dev).mul_(2.0).exp_()
        state["left"], state["gone"] = torch.empty_like(table), torch.empty_like(table)
        state["count"] = torch.empty(seqs, dtype=torch.int32, device=dev)
        state["dim"] = 64                                        # (what the pages hold is not looked at)
        state["pages"] = torch.empty(pool * kv * page * 72, dtype=torch.uint8, device=dev)
        return state
    dim, heads, kind = case["dim"], case["heads"], TYPES[case["dtype"]]
    pages = torch.empty((pool, kv, page * (dim + 8) // 4), dtype=torch.int32, device=dev)
    # keys with a few strong channels, values without
    loud = torch.where(torch.rand((kv, 1, dim), generator=g, device=dev) < 0.04, 4.0, 1.0)
    step = max(1, (1 << 26) // (kv * page * dim))
    for i in range(0, pool, step):
        n, sides = min(step, pool - i), []
        # a page's keys have something in common, so that some pages matter more than others
        theme = torch.randn((n, kv, 1, dim), generator=g, device=dev) * 0.5
        for gain, mean in ((loud, theme), (0.7, 0.0)):
            q, dm = quantise((torch.randn((n, kv, page, dim), generator=g, device=dev) + mean) * gain)
            sides.append((words(q), dm))
        pages[i:i + n] = head_words(sides[0][0], sides[1][0], sides[0][1], sides[1][1])
    state["pages"] = pages.view(torch.uint8).flatten()
    flat = torch.randn((rows, heads + 2 * kv, dim), generator=g, device=dev).to(kind)
    state["q"] = flat[:, :heads]
    if op == "weigh":
        state["lse"] = torch.cat([x for _, _, x in log_sums(state)])
        state["before"] = torch.rand((seqs, kv, wide), generator=g, device=dev)
        state["weights"] = torch.zeros_like(state["before"])
        return state
    take = case["take"]
    # what earlier steps have left: the bounds of every page filled so far
    bounds = torch.zeros((pool, bounds_bytes(kv, dim)), dtype=torch.uint8, device=dev)
    for s in range(seqs):
        put_bounds(state, bounds, table[s, :(lens[s] - new[s]) // page].long())
    state["bounds"] = bounds
    state["out"] = torch.empty((rows, heads, dim), dtype=kind, device=dev)
    state["lse"] = torch.empty((rows, heads), dtype=torch.float32, device=dev)
    state["some"] = torch.empty((rows, kv, take), dtype=torch.int32, device=dev)
    state["some_lens"] = torch.empty(rows, dtype=torch.int32, device=dev)
    state["some_start"] = torch.empty(rows + 1, dtype=torch.int32, device=dev)
    return state


def rows_of(state):
    """Sequence, number within it and position of each new token."""
    start = state["start"].long()
    row = torch.arange(state["rows"], device=start.device)
    seq = torch.searchsorted(start[1:], row, right=True)
    nth = row - start[seq]
    return seq, nth, state["lens_"].long()[seq] - (start[seq + 1] - start[seq]) + nth


def blocks(state):
    return state["pages"].view(torch.int32).view(-1, state["kv"], state["page"] * (state["dim"] + 8) // 4)


def put_bounds(state, bounds, pages):
    """Bounds of the pages (numbers) into the buffer."""
    kv, dim, page = state["kv"], state["dim"], state["page"]
    step = max(1, (1 << 27) // (kv * page * dim))
    for i in range(0, len(pages), step):
        some = pages[i:i + step]
        codes, e = bounds_of(keys_of(blocks(state)[some], page, dim))
        held = torch.cat((codes.flatten(1).view(torch.uint8), e.contiguous().view(torch.uint8)), 1)
        bounds[some, :held.shape[1]] = held


# ------------------------------------------------------------------ plain forms

def frequencies(case, dev):
    n = case["pairs"]
    i = torch.arange(n, dtype=torch.float64, device=dev)
    base, factor, kind = case["base"], case["factor"], case["scaling"]
    if kind == "base":
        base = base * factor ** (n / (n - 1))
    f = torch.pow(torch.tensor(base, dtype=torch.float64, device=dev), -i / n)
    if kind == "linear":
        f = f / factor
    if kind == "index":
        lo, hi = (n * math.log(case["original"] / (2 * math.pi * t)) / math.log(base) for t in (case["high"], case["low"]))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), 2 * n - 1)
        r = ((i - lo) / (hi - lo if hi != lo else 0.001)).clamp(0, 1)
        f = f * (1 - r + r / factor)
    if kind == "turns":
        s = ((case["original"] * f / (2 * math.pi) - case["low"]) / (case["high"] - case["low"])).clamp(0, 1)
        f = f * (s + (1 - s) / factor)
    return f


def amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "index" else 1.0


def plain_rope(state):
    n = state["pairs"]
    x = state["x"].float()
    at = rows_of(state)[2] if state["pos"] is None else state["pos"].long()
    if "turn" not in state:                                      # a table of the model's
        state["turn"] = frequencies(state, x.device)
    angle = at.double()[:, None] * state["turn"]
    g = amplitude(state)
    cos, sin = (angle.cos() * g).float()[:, None], (angle.sin() * g).float()[:, None]
    if state["layout"] == "halves":
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((turned, x[..., 2 * n:]), -1).to(state["y"].dtype)


def padded(state):
    """Queries [seqs, kv, group * most, D] in 32 bits and positions [seqs, most] (-1: no row)."""
    heads, kv, dim, most = state["heads"], state["kv"], state["dim"], state["most_new"]
    seq, nth, pos = rows_of(state)
    q = torch.zeros((state["seqs"], most, heads, dim), device=pos.device)
    q[seq, nth] = state["q"].float()
    where = torch.full((state["seqs"], most), -1, device=pos.device)
    where[seq, nth] = pos
    return q.transpose(1, 2).reshape(state["seqs"], kv, heads // kv * most, dim), where


def log_sums(state):
    """For each sequence: its scores [heads, n, tokens] (-infinity where hidden), its number and log sums [n, heads]."""
    page, dim, kv, heads = state["page"], state["dim"], state["kv"], state["heads"]
    at = 0
    for s, (n, length) in enumerate(zip(state["new"], state["plens"])):
        mine = state["table"][s, :-(-length // page)].long()
        k = keys_of(blocks(state)[mine], page, dim).transpose(0, 1).flatten(1, 2)[:, :length]
        q = state["q"][at:at + n].float().transpose(0, 1).reshape(kv, -1, dim)
        at += n
        score = ((q @ k.transpose(1, 2)) * dim ** -0.5).view(heads, n, length)
        j, p = torch.arange(length, device=k.device), torch.arange(length - n, length, device=k.device)[:, None]
        hidden = (j > p) | (j <= p - state["window"]) if state["window"] else j > p
        score.masked_fill_(hidden, float("-inf"))
        top = score.amax(-1, keepdim=True)
        yield s, score, ((score - top).exp_().sum(-1).log() + top.squeeze(-1)).T


def plain_weigh(state):
    heads, kv, page, dim, most, seqs = (state[x] for x in ("heads", "kv", "page", "dim", "most_new", "seqs"))
    seq, nth, _ = rows_of(state)
    q, where = padded(state)
    lse = torch.full((seqs, most, heads), float("inf"), device=q.device)
    lse[seq, nth] = state["lse"]
    lse = lse.transpose(1, 2).reshape(seqs, kv, -1, 1)
    table, wide = state["table"].long(), state["table"].shape[1]
    total = torch.empty((seqs, kv, wide), device=q.device)
    step = max(1, (1 << 28) // (seqs * heads * most * page))     # pages a time
    for j0 in range(0, wide, step):
        at = table[:, j0:j0 + step]
        k = keys_of(blocks(state)[at.clamp(min=0)], page, dim).transpose(1, 2).flatten(2, 3)
        score = (q @ k.transpose(2, 3)) * dim ** -0.5
        t = torch.arange(j0 * page, j0 * page + k.shape[2], device=q.device)
        sees = (t <= where[:, :, None]) & (at >= 0).repeat_interleave(page, 1)[:, None, :]
        if state["window"]:
            sees &= t > where[:, :, None] - state["window"]
        p = (score - lse).exp_().view(seqs, kv, -1, most, k.shape[2]).masked_fill_(~sees[:, None, None], 0.0)
        total[:, :, j0:j0 + step] = p.sum((2, 3)).unflatten(-1, (-1, page)).sum(-1)
    used = torch.arange(wide, device=q.device) * page < state["lens_"][:, None]
    kept = torch.where((used & (table >= 0))[:, None], total + state["decay"] * state["before"], 0.0)
    return {"weights": torch.where(used[:, None], kept, state["weights"])}


def first_of(key, count):
    """Which of [..., n] are the first `count` [...] of a descending order, the lowest place first among equals."""
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, torch.arange(key.shape[-1], device=key.device).expand_as(order))
    return rank < count[..., None]


def plain_evict(state):
    table, page, kv = state["table"], state["page"], state["kv"]
    wide = table.shape[1]
    j = torch.arange(wide, device=table.device)
    used = (-(-state["lens_"] // page))[:, None]
    here = (table >= 0) & (table < state["pool"]) & (j < used)
    total = torch.zeros((state["seqs"], wide), dtype=torch.float64, device=table.device)
    for h in range(kv):
        total += state["weights"][:, h].double()
    may = here & (j >= state["first"]) & (j < used - state["last"])
    key = torch.where(may, -total.float(), float("-inf"))
    out = first_of(key, here.sum(-1) - state["keep"]) & may
    place = torch.where(out, out.cumsum(-1) - 1, wide)
    gone = torch.full((state["seqs"], wide + 1), -1, dtype=torch.int32, device=table.device).scatter_(1, place, table)
    return {"table": torch.where(out, -1, table), "gone": torch.where(j < out.sum(-1, keepdim=True), gone[:, :-1], -1),
            "count": out.sum(-1).to(torch.int32)}


def plain_select(state):
    heads, kv, dim, page, take, seqs, most = (state[x] for x in ("heads", "kv", "dim", "page", "take", "seqs", "most_new"))
    seq, nth, pos = rows_of(state)
    q, _ = padded(state)
    q = q.view(seqs, kv, -1, most, dim)
    e = least_exponent(q.abs().amax(-1))                         # [seqs, kv, group, most]
    q = torch.round(torch.ldexp(q, -e[..., None]))
    some = (q != 0).any(-1)
    top = torch.where(some, e, -1000).amax(2, keepdim=True)
    share = torch.exp2((e - top).clamp(-64, 0).float())
    table, wide = state["table"].long(), state["table"].shape[1]
    n = kv * 2 * dim
    held = state["bounds"][table.clamp(min=0)]
    codes = held[..., :n].view(torch.int8).view(seqs, wide, kv, 2 * dim).permute(0, 2, 3, 1).float()
    pe = held[..., n:n + 4 * kv].contiguous().view(torch.int32).transpose(1, 2)
    both = torch.cat((q.clamp(min=0), q.clamp(max=0)), -1).flatten(2, 3)
    score = (both @ codes).view(seqs, kv, -1, most, wide) * share[..., None]
    score = (score.amax(2) * torch.exp2(pe.float())[:, :, None]).transpose(1, 2)[seq, nth]       # [rows, kv, pages]
    mine = (pos // page)[:, None]
    j = torch.arange(wide, device=q.device)
    may = ((table[seq] >= 0) & (j < mine))[:, None]
    forced = ((j < state["first"]) | (j >= mine - state["last"]))[:, None]
    key = torch.where(may, torch.where(forced, float("inf"), score), float("-inf"))
    chosen = first_of(key, torch.full(key.shape[:2], take - 1, device=q.device)) & may
    chosen |= (j == mine)[:, None]
    at = torch.where(chosen, j, wide).sort(-1).values[..., :take]
    got = torch.where(at < wide, table[seq][:, None].expand(-1, kv, -1).gather(2, at.clamp(max=wide - 1)), -1).to(torch.int32)
    got = torch.nn.functional.pad(got, (0, take - got.shape[-1]), value=-1)
    return got, ((chosen[:, 0].sum(-1) - 1) * page + pos % page + 1).to(torch.int32)


def plain_sparse(state):
    heads, kv, dim, page, take = (state[x] for x in ("heads", "kv", "dim", "page", "take"))
    for s, (n, length) in enumerate(zip(state["new"], state["plens"])):
        put_bounds(state, state["bounds"], state["table"][s, (length - n) // page:length // page].long())
    got, lens = plain_select(state)
    rows, outs, lses = state["rows"], [], []
    step = max(1, (1 << 28) // (kv * take * page * dim))
    for i in range(0, rows, step):
        block = blocks(state)[got[i:i + step].long().clamp(min=0), torch.arange(kv, device=got.device)[:, None]]
        q = state["q"][i:i + step].float().unflatten(1, (kv, -1))
        score = (q @ keys_of(block, page, dim).flatten(2, 3).transpose(2, 3)) * dim ** -0.5
        there = (got[i:i + step] >= 0).repeat_interleave(page, 2)
        there &= torch.arange(take * page, device=q.device) < lens[i:i + step, None, None]
        score.masked_fill_(~there[:, :, None], float("-inf"))
        top = score.amax(-1, keepdim=True)
        p = (score - top).exp_()
        total = p.sum(-1, keepdim=True)
        outs.append(((p @ values_of(block, page, dim).flatten(2, 3)) / total).flatten(1, 2))
        lses.append((total.log() + top).squeeze(-1).flatten(1, 2))
    return {"out": torch.cat(outs).to(state["q"].dtype), "lse": torch.cat(lses), "table": got, "lens": lens,
            "bounds": state["bounds"]}


# ------------------------------------------------------------------ the framework's calls

def handles(state):
    """The framework's handles, made at the first pass and kept as a user's program keeps them."""
    if "dg" in state:
        return state["dg"]
    import decode_gemv_amd as dg
    state["dg"] = dg
    if state["op"] == "rope":
        kinds = dict(none=dg.LW_ROPE_PLAIN, linear=dg.LW_ROPE_LINEAR, base=dg.LW_ROPE_BASE, index=dg.LW_ROPE_INDEX, turns=dg.LW_ROPE_TURNS)
        state["plan"] = dg.lw_rope_make(state["pairs"], dg.LW_ROPE_HALVES if state["layout"] == "halves" else dg.LW_ROPE_PAIRS,
                                        base=state["base"], scaling=kinds[state["scaling"]], factor=state["factor"],
                                        original=state["original"], low=state["low"], high=state["high"],
                                        amplitude=amplitude(state))
        if state["pos"] is None:
            state["batch"] = dg.KvBatch(state["start"], state["lens_"], state["table"], max_len=state["longest"])
        return dg
    state["batch"] = dg.KvBatch(state["start"], state["lens_"], state["table"], max_len=state["longest"])
    state["cache"] = dg.KvCache(state["pages"], state["kv"], state["dim"], state["page"])
    if state["op"] == "sparse":
        state["selection"] = dg.KvSelection(state["some_start"], state["some_lens"], state["some"])
        need = dg.lw_kv_select_scratch_bytes(state["cache"], state["batch"], state["rows"], state["heads"])
        state["work"] = torch.empty(max(need, 16), dtype=torch.uint8, device=state["pages"].device)
        need = dg.lw_kv_attend_selected_scratch_bytes(state["cache"], state["selection"], state["heads"])
        state["room"] = torch.empty(max(need, 16), dtype=torch.uint8, device=state["pages"].device)
    return dg


def run(state):
    if not own:
        return {"rope": lambda s: {"y": plain_rope(s)}, "sparse": plain_sparse, "weigh": plain_weigh, "evict": plain_evict}[state["op"]](state)
    dg = handles(state)
    if state["op"] == "rope":
        if state["pos"] is None:
            dg.lw_rope(state["plan"], state["x"], state["y"], batch=state["batch"])
        else:
            dg.lw_rope(state["plan"], state["x"], state["y"], pos=state["pos"])
        return {"y": state["y"]}
    if state["op"] == "evict":
        dg.lw_kv_evict(state["cache"], state["batch"], state["weights"], state["keep"], state["left"], state["gone"], state["count"],
                       first=state["first"], last=state["last"])
        return {"table": state["left"], "gone": state["gone"], "count": state["count"]}
    if state["op"] == "weigh":
        dg.lw_kv_weigh(state["cache"], state["batch"], state["q"], state["lse"], state["weights"], before=state["before"],
                       decay=state["decay"], window=state["window"])
        return {"weights": state["weights"]}
    dg.lw_kv_bounds(state["cache"], state["batch"], state["rows"], state["bounds"])
    dg.lw_kv_select(state["cache"], state["batch"], state["q"], state["bounds"], state["selection"], first=state["first"],
                    last=state["last"], work=state["work"])
    dg.lw_kv_attend_selected(state["cache"], state["selection"], state["q"], state["out"], lse=state["lse"], work=state["room"])
    return {"out": state["out"], "lse": state["lse"], "table": state["some"], "lens": state["some_lens"], "bounds": state["bounds"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact_rope(case, state):
    new, lens = sizes(case)
    n, x = case["pairs"], state["x"].double()
    at = torch.cat([torch.arange(b - a, b) for a, b in zip(new, lens)]).to(x.device).double()
    base = case["base"] * (case["factor"] ** (n / (n - 1)) if case["scaling"] == "base" else 1.0)
    edge = [n * math.log(case["original"] / (t * 2 * math.pi)) / math.log(base) for t in (case["high"], case["low"])] if case["scaling"] == "index" else None
    y = x.clone()
    g = 1.0 + math.log(case["factor"]) / 10 if case["scaling"] == "index" else 1.0
    for i in range(n):
        f = base ** (-i / n)
        if case["scaling"] == "linear":
            f /= case["factor"]
        elif case["scaling"] == "index":
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), 2 * n - 1)
            r = min(max((i - lo) / ((hi - lo) or 0.001), 0.0), 1.0)
            f = f * (1 - r) + f / case["factor"] * r
        elif case["scaling"] == "turns":
            s = min(max((case["original"] * f / (2 * math.pi) - case["low"]) / (case["high"] - case["low"]), 0.0), 1.0)
            f = f * s + f / case["factor"] * (1 - s)
        u, v = (i, i + n) if case["layout"] == "halves" else (2 * i, 2 * i + 1)
        turn = torch.polar(torch.full_like(at, g), at * f)[:, None]
        z = torch.complex(x[..., u], x[..., v]) * turn
        y[..., u], y[..., v] = z.real, z.imag
    return {"y": y}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rope":
        return exact_rope(case, state)
    new, lens = sizes(case)
    kv, page = case["kv"], case["page"]
    if case["op"] == "evict":
        table = state["table"].cpu()
        gone, count = torch.full_like(table, -1), []
        for s in range(case["seqs"]):
            used = -(-lens[s] // page)
            w = [0.0] * used
            for h in range(kv):
                w = [a + b for a, b in zip(w, state["weights"][s, h, :used].tolist())]
            w = torch.tensor(w, dtype=torch.float64).float().tolist()
            have = [j for j in range(used) if table[s, j] >= 0]
            may = sorted((j for j in have if case["first"] <= j < used - case["last"]), key=lambda j: (w[j], j))
            drop = sorted(may[:max(len(have) - case["keep"], 0)])
            gone[s, :len(drop)] = table[s, drop]
            table[s, drop] = -1
            count.append(len(drop))
        dev = state["table"].device
        return {"table": table.to(dev), "gone": gone.to(dev), "count": torch.tensor(count, dtype=torch.int32, device=dev)}
    dim, heads = case["dim"], case["heads"]
    raw = state["pages"].view(-1, kv, page * (dim + 8))
    i, t = torch.arange(dim, device=raw.device), torch.arange(page, device=raw.device)[:, None]
    wide = min(4, dim // 32)
    place = [((t // 16 * (dim // 8 // wide) + i // 8 // wide) * 16 + t % 16) * wide + i // 8 % wide, page * dim // 8 + (t // 4 * (dim // 8) + i // 8) * 4 + t % 4]

    def tokens(pages, h, side):
        """Keys (side 0) or values [pages, P, D] of head h, byte by byte from the layout."""
        some = raw[pages, h]
        byte = (place[side] * 4 + i % 8 // 2).flatten().expand(len(some), -1)
        code = (some.gather(1, byte).view(-1, page, dim) >> (i % 2 * 4).to(torch.uint8) & 15).double()
        at = page * (dim + 4 * side)
        dm = some[:, at:at + 4 * page].contiguous().view(torch.float16).double().view(-1, page, 2)
        return dm[..., :1] * code - dm[..., 1:]

    def fit(top):
        """The smallest e with top <= 127 * 2^e."""
        f, e = torch.frexp(top / 127)
        return torch.where(top == 0, 0, torch.where(f == 0.5, e - 1, e))

    if case["op"] == "weigh":
        w, at = state["weights"].double(), 0
        for s, (n, length) in enumerate(zip(new, lens)):
            mine = state["table"][s, :-(-length // page)].long()
            j, p = torch.arange(len(mine) * page, device=raw.device), torch.arange(length - n, length, device=raw.device)[:, None]
            hidden = (j > p) | (j <= p - (case["window"] or 1 << 40))
            for g in range(kv):
                k = tokens(mine, g, 0).flatten(0, 1)
                total = state["before"][s, g, :len(mine)].double() * case["decay"]
                for h in range(g * heads // kv, (g + 1) * heads // kv):
                    q = state["q"][at:at + n, h].double()
                    a = torch.exp(q @ k.T / math.sqrt(dim) - state["lse"][at:at + n, h].double()[:, None])
                    total += a.masked_fill_(hidden, 0.0).sum(0).view(-1, page).sum(1)
                w[s, g, :len(mine)] = total
            at += n
        return {"weights": w}

    held = torch.zeros_like(state["bounds"])
    codes = held[:, :kv * 2 * dim].view(torch.int8).view(-1, kv, 2, dim)
    power = torch.zeros((len(held), kv), dtype=torch.int32, device=raw.device)
    for s, length in enumerate(lens):
        full = state["table"][s, :length // page].long()
        for h in range(kv):
            for some in full.split(1 << 9):
                k = tokens(some, h, 0).float().double()
                most, least = k.max(1).values, k.min(1).values
                e = fit(torch.maximum(most.abs(), least.abs()).max(1).values)
                power[some, h] = e.to(torch.int32)
                codes[some, h] = torch.stack((torch.ceil(torch.ldexp(most, -e[:, None])), torch.floor(torch.ldexp(least, -e[:, None]))), 1).to(torch.int8)
    held[:, kv * 2 * dim:kv * (2 * dim + 4)] = power.view(torch.uint8).view(len(held), -1)
    some, some_lens = torch.full((sum(new), kv, case["take"]), -1, dtype=torch.int32), []
    outs, lses, row, per = [], [], 0, heads // kv
    for s, (n, length) in enumerate(zip(new, lens)):
        pages = state["table"][s].long()
        for pos in range(length - n, length):
            own_page = pos // page
            for g in range(kv):
                q = state["q"][row, g * per:(g + 1) * per].double()
                e = fit(q.abs().max(1).values)
                z = torch.round(torch.ldexp(q, -e[:, None]))
                e = torch.where((z == 0).all(1), -1000, e)
                b = codes[pages[:own_page], g].double()
                score = torch.maximum(z[:, None] * b[:, 0], z[:, None] * b[:, 1]).sum(-1)        # [group, pages]
                score = torch.ldexp(score, (e - e.max()).clamp(min=-64)[:, None]).max(0).values if own_page else score[0]
                score = torch.ldexp(score, power[pages[:own_page], g]).tolist()
                must = [j for j in range(own_page) if j < case["first"] or j >= own_page - case["last"]]
                rest = sorted((j for j in range(own_page) if j not in set(must)), key=lambda j: (-score[j], j))
                picks = sorted(must + rest[:case["take"] - 1 - len(must)]) + [own_page]
                mine = pages[picks]
                some[row, g, :len(picks)] = mine.to(torch.int32).cpu()
                k, v = tokens(mine, g, 0).flatten(0, 1), tokens(mine, g, 1).flatten(0, 1)
                last = (len(picks) - 1) * page + pos % page + 1
                x = q @ k[:last].T / math.sqrt(dim)
                lse = torch.logsumexp(x, -1)
                outs.append(torch.exp(x - lse[:, None]) @ v[:last])
                lses.append(lse)
            some_lens.append(last)
            row += 1
    return {"out": torch.stack(outs).view(sum(new), heads, dim), "lse": torch.stack(lses).view(sum(new), heads),
            "table": some.to(raw.device), "lens": torch.tensor(some_lens, dtype=torch.int32, device=raw.device), "bounds": held}
