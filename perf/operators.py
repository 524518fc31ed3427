"""The 4-bit key/value cache: what is measured of its three operators.

lw_kv_append quantises new keys and values into a paged cache, lw_kv_read
dequantises cached tokens, lw_kv_attend lets new tokens attend over the cache.
One key or value head vector x[0..D) is held as 4-bit codes q and an fp16
pair (d, m), worth d*q - m:

    m = fp16(-min x), d = fp16((max x - min x) / 15), both kept within +-65504
    q = clamp(rint((x + m) * (1 / d)), 0, 15)      (0 where d is 0)

and a vector with a NaN or an infinity has d = m = NaN.  A page holds P tokens
of every head: per head P*D/2 bytes of key codes, P*D/2 bytes of value codes,
then P words d | m << 16 of the keys and P of the values.  A word holds the
codes of eight dimensions, the lowest in the low nibble.  Word w of token t
lies, for keys, at (((t/16) * U + w/W) * 16 + t%16) * W + w%W with
W = min(4, D/32) and U = D/8/W, and for values at
((t/4) * (D/8) + w) * 4 + t%4.

A batch packs the new tokens of its sequences back to back: sequence s has
rows start[s] .. start[s+1], and they are the last ones of its lens[s] tokens.
table[s][i] names the page of its tokens i*P .. i*P + P - 1 (-1: no page, its
tokens are absent).  A causal row at position p sees keys j <= p, and with a
window w only keys j > p - w; a row that sees nothing gives zeros and a log
sum of -infinity.
"""
import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one user's next token: the call's latency is all there is
        dict(name="append_1_token", op="append", seqs=1, new_min=1, new_max=1, len_min=777, len_max=777, kv=8, dim=128, page=64, dtype="fp16"),
        # one step of a serving batch, sequences of many lengths
        dict(name="append_64_seqs", op="append", seqs=64, new_min=1, new_max=1, len_min=33, len_max=4096, kv=8, dim=128, page=64, dtype="bf16"),
        # prompts of several users entering the cache
        dict(name="append_prompts", op="append", seqs=5, new_min=1001, new_max=8191, len_min=1001, len_max=8191, kv=8, dim=128, page=128, dtype="fp16"),
        # a shared prefix taken out for another use
        dict(name="read_515", op="read", seqs=1, new_min=515, new_max=515, len_min=700, len_max=700, kv=8, dim=64, page=32, dtype="bf16"),
        # whole sequences read back, to move or to recompute with
        dict(name="read_sequences", op="read", seqs=8, new_min=2049, new_max=16384, len_min=2049, len_max=16384, kv=8, dim=128, page=64, dtype="fp16"),
        # one user's token on a short conversation: latency
        dict(name="decode_1_short", op="attend", seqs=1, new_min=1, new_max=1, len_min=300, len_max=300, heads=32, kv=8, dim=128, page=64, window=0, dtype="fp16"),
        # a serving batch of many lengths
        dict(name="decode_16", op="attend", seqs=16, new_min=1, new_max=1, len_min=501, len_max=8190, heads=32, kv=8, dim=128, page=64, window=0, dtype="bf16"),
        # one very long context
        dict(name="decode_long", op="attend", seqs=1, new_min=1, new_max=1, len_min=131071, len_max=131071, heads=64, kv=8, dim=128, page=128, window=0, dtype="fp16"),
        # every head with keys of its own, small heads, a sliding window
        dict(name="decode_window", op="attend", seqs=96, new_min=1, new_max=1, len_min=100, len_max=6000, heads=16, kv=16, dim=64, page=32, window=1024, dtype="bf16"),
        # a few guessed tokens a sequence checked at once, wide heads
        dict(name="verify_5", op="attend", seqs=7, new_min=3, new_max=5, len_min=900, len_max=5000, heads=16, kv=4, dim=256, page=64, window=0, dtype="fp16"),
        # a prompt over itself
        dict(name="prompt_2048", op="attend", seqs=1, new_min=2048, new_max=2048, len_min=2048, len_max=2048, heads=32, kv=8, dim=128, page=64, window=0, dtype="bf16"),
        # pieces of long prompts after what the cache already has
        dict(name="chunks_long", op="attend", seqs=3, new_min=511, new_max=1024, len_min=9000, len_max=16384, heads=64, kv=8, dim=128, page=64, window=0, dtype="fp16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("append", "read", "attend", "attend", "attend"))
    case = dict(op=op, dim=rng.choice((64, 128, 128, 256)), page=rng.choice((32, 64, 128, 256)), dtype=rng.choice(("fp16", "bf16")))
    case["kv"] = rng.choice((1, 2, 4, 8, 8, 16)) if case["dim"] < 256 else rng.choice((1, 2, 4))
    if op != "attend":
        case["dtype"] = rng.choice(("fp16", "bf16", "fp32"))
        case["seqs"] = log(1, 64)
        budget = 20000 * 1024 // (case["kv"] * case["dim"])      # tokens of the largest listed append
        case["new_max"] = log(1, max(2, min(16384, budget // case["seqs"])))
        case["new_min"] = rng.randint(1, case["new_max"])
        case["len_min"] = case["new_max"] + log(1, 2000) - 1
        case["len_max"] = case["len_min"] + log(1, 2000) - 1
        return case
    case["heads"] = case["kv"] * rng.choice((1, 2, 4, 5, 8))
    case["window"] = rng.choice((0, 0, 0, log(16, 4096)))
    if rng.random() < 0.65:                                      # single tokens, or a few guessed ones
        case["seqs"] = log(1, 96)
        case["new_max"] = rng.choice((1, 1, 1, 2, 5, 9))
        most = 131072 * 1024 // (case["seqs"] * case["kv"] * case["dim"])
        case["len_max"] = log(20, max(40, min(131072, most)))
    else:                                                        # prompts and pieces of them
        case["seqs"] = log(1, 4)
        case["new_max"] = log(17, 1024)
        most = 3 * 1024 * 64 * 128 * 8000 // (case["seqs"] * case["new_max"] * case["heads"] * case["dim"])
        case["len_max"] = log(case["new_max"], max(case["new_max"] + 1, min(16384, most)))
    case["new_min"] = rng.randint(1, case["new_max"])
    case["len_min"] = max(case["new_max"], rng.randint(1, case["len_max"]))
    case["len_max"] = max(case["len_max"], case["len_min"])
    return case


def spread(lo, hi, n):
    """n whole numbers from lo to hi, the largest first and the others in no order."""
    return [hi if i == 0 else lo + (hi - lo) * ((i * 7919 + 13) % n) // n for i in range(n)]


def sizes(case):
    new = spread(case["new_min"], case["new_max"], case["seqs"])
    lens = [max(a, b) for a, b in zip(spread(case["len_min"], case["len_max"], case["seqs"]), new)]
    return new, lens


def work(case):
    new, lens = sizes(case)
    kv, dim = case["kv"], case["dim"]
    wide = 4 if case["dtype"] == "fp32" else 2
    held = 2 * kv * (dim // 2 + 4)                               # bytes of one cached token
    dense = 2 * kv * dim * wide
    if case["op"] == "append":                                   # written, and what was written read back
        return {"bytes": sum(new) * (dense + held + held + dense), "flops": sum(new) * 2 * kv * dim * 8}
    if case["op"] == "read":
        return {"bytes": sum(new) * (held + dense), "flops": sum(new) * 2 * kv * dim * 2}
    pairs = seen = 0
    for n, length in zip(new, lens):
        w = case["window"] or length
        first, last = length - n + 1, length                     # keys at or before each new token
        full = max(0, last - max(first, w) + 1)                  # rows whose window is full
        pairs += full * w + sum(range(first, min(last, w - 1) + 1))
        seen += length - max(0, first - w)
    q = sum(new) * case["heads"] * dim * wide
    return {"bytes": 2 * q + seen * held, "flops": 4 * dim * case["heads"] * pairs}


def quantise(x):
    """Codes and pairs (d, m) of vectors x[..., D], 32-bit."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    m = (-lo).clamp(-65504.0, 65504.0).half()
    d = ((hi - lo) * (1.0 / 15.0)).clamp(max=65504.0).half()
    fine = torch.isfinite(x).all(-1, keepdim=True)
    nan = torch.full_like(d, float("nan"))
    d, m = torch.where(fine, d, nan), torch.where(fine, m, nan)
    inverse = torch.where(d == 0, torch.zeros_like(lo), 1.0 / d.float())
    q = torch.round((x + m.float()) * inverse).clamp(0.0, 15.0)
    return torch.where(fine, q, torch.zeros_like(q)).to(torch.uint8), d, m


def packed(q):
    """Words of codes q[..., D]."""
    q = q.unflatten(-1, (-1, 4, 2)).to(torch.uint8)
    q = (q[..., 0] | q[..., 1] << 4).contiguous()
    return q.view(torch.int32).squeeze(-1)


def joined(d, m):
    return torch.cat((d, m), -1).contiguous().view(torch.int32).squeeze(-1)


def block_words(kw, vw, kdm, vdm):
    """The words of head blocks from words and pairs by token: kw, vw [..., P, D/8], kdm, vdm [..., P]."""
    words = kw.shape[-1]
    w = min(4, words // 4)
    k = kw.unflatten(-1, (-1, w)).unflatten(-3, (-1, 16)).transpose(-3, -2)
    v = vw.unflatten(-2, (-1, 4)).transpose(-2, -1)
    return torch.cat((k.flatten(-4), v.flatten(-3), kdm, vdm), -1)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(seed)
    new, lens = sizes(case)
    kv, dim, page, seqs = case["kv"], case["dim"], case["page"], case["seqs"]
    need = [-(-n // page) for n in lens]
    pool, wide = sum(need) + 3, max(need)
    at = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.full((seqs, wide), -1, dtype=torch.int32, device=dev)
    left, base = torch.full((pool,), 0, dtype=torch.int32, device=dev), 0
    for s, n in enumerate(need):                                 # a page's tokens in use
        mine = at[base:base + n]
        table[s, :n] = mine
        left[mine.long()] = (lens[s] - page * torch.arange(n, device=dev, dtype=torch.int32)).clamp(max=page)
        base += n
    # what the pages hold: keys with a few strong channels, values without; NaN pairs where no token lies
    pages = torch.empty((pool, kv, page * (dim + 8) // 4), dtype=torch.int32, device=dev)
    loud = torch.where(torch.rand((kv, 1, dim), generator=g, device=dev) < 0.04, 4.0, 1.0)
    used = (torch.arange(page, device=dev) < left[:, None])[:, None, :]
    step = max(1, (1 << 26) // (kv * page * dim))
    for i in range(0, pool, step):
        n, sides = min(step, pool - i), []
        for gain in (loud, 0.7):
            x = torch.randn((n, kv, page, dim), generator=g, device=dev) * gain
            q, d, m = quantise(x)
            dm = torch.where(used[i:i + n], joined(d, m), 0x7E007E00)
            sides.append((packed(q), dm))
        pages[i:i + n] = block_words(sides[0][0], sides[1][0], sides[0][1], sides[1][1])
    rows, kind = sum(new), TYPES[case["dtype"]]
    start = torch.tensor([sum(new[:s]) for s in range(seqs + 1)], dtype=torch.int32, device=dev)
    state = dict(case, pages=pages.view(torch.uint8).flatten(), start=start, table=table,
                 lens_=torch.tensor(lens, dtype=torch.int32, device=dev), rows=rows, longest=max(lens), most_new=max(new))
    heads = case.get("heads", 0)
    # queries, keys and values of the new tokens lie side by side, as one projection gives them
    flat = torch.randn((rows, heads + 2 * kv, dim), generator=g, device=dev).to(kind)
    state["q"], state["k"], state["v"] = flat[:, :heads], flat[:, heads:heads + kv], flat[:, heads + kv:]
    state["k"].mul_(loud[:, 0].to(kind))
    state["out"] = torch.empty((rows, heads, dim), dtype=kind, device=dev)
    state["back"] = [torch.empty((rows, kv, dim), dtype=kind, device=dev) for _ in range(2)]
    state["lse"] = torch.empty((rows, heads), dtype=torch.float32, device=dev)
    return state


def rows_of(state):
    """Sequence, number within it and position of each new token."""
    start = state["start"].long()
    row = torch.arange(state["rows"], device=start.device)
    seq = torch.searchsorted(start[1:], row, right=True)
    nth = row - start[seq]
    return seq, nth, state["lens_"].long()[seq] - (start[seq + 1] - start[seq]) + nth


def dense(state, block):
    """Keys and values [..., P, D] in 32 bits of head blocks' words."""
    page, dim = state["page"], state["dim"]
    w, n = min(4, dim // 32), page * dim // 8
    shifts = torch.arange(0, 32, 4, device=block.device, dtype=torch.int32)
    k = block[..., :n].unflatten(-1, (page // 16, -1, 16, w)).transpose(-3, -2).flatten(-2).flatten(-3, -2)
    v = block[..., n:2 * n].unflatten(-1, (page // 4, dim // 8, 4)).transpose(-2, -1).flatten(-3, -2)
    got = []
    for words, at in ((k, 2 * n), (v, 2 * n + page)):
        dm = block[..., at:at + page].contiguous().view(torch.float16).unflatten(-1, (page, 2)).float()
        q = (words.unsqueeze(-1) >> shifts & 15).flatten(-2).float()
        got.append(q * dm[..., :1] - dm[..., 1:])
    return got


def gathered(state):
    """Keys and values [seqs, kv, tokens, D] of whole sequences, and which tokens exist."""
    table = state["table"].long()
    blocks = state["pages"].view(torch.int32).view(-1, state["kv"], state["page"] * (state["dim"] + 8) // 4)
    k, v = dense(state, blocks[table.clamp(min=0)])
    here = (table >= 0).repeat_interleave(state["page"], 1)
    here &= torch.arange(here.shape[1], device=here.device) < state["lens_"][:, None]
    return k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3), here


def plain_attend(state):
    heads, kv, dim, most = state["heads"], state["kv"], state["dim"], state["most_new"]
    k, v, here = gathered(state)
    k = torch.where(here[:, None, :, None], k, 0.0)
    v = torch.where(here[:, None, :, None], v, 0.0)
    seq, nth, pos = rows_of(state)
    seqs, tokens = here.shape
    q = torch.zeros((seqs, most, heads, dim), device=k.device)
    q[seq, nth] = state["q"].float()
    where = torch.full((seqs, most), -1, device=k.device)
    where[seq, nth] = pos
    q = q.transpose(1, 2).reshape(seqs, kv, heads // kv * most, dim)
    score = (q @ k.transpose(2, 3)) * dim ** -0.5
    j = torch.arange(tokens, device=k.device)
    sees = here[:, None, :] & (j <= where[:, :, None])
    if state["window"]:
        sees &= j > where[:, :, None] - state["window"]
    score = score.view(seqs, kv, heads // kv, most, tokens).masked_fill_(~sees[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(seqs, kv, -1, tokens) @ v).view(seqs, kv, heads // kv, most, dim) / torch.where(total == 0, 1.0, total)
    lse = (total.log() + top).squeeze(-1)
    out = out.flatten(1, 2).transpose(1, 2)[seq, nth]
    return {"out": out.to(state["q"].dtype), "lse": lse.flatten(1, 2).transpose(1, 2)[seq, nth]}


def plain_read(state):
    seq, _, pos = rows_of(state)
    page = state["table"].long()[seq, pos // state["page"]]
    kw, vw, kdm, vdm = places(state, page, pos % state["page"])
    words = state["pages"].view(torch.int32)
    shifts = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    kd, vd = (words[at].view(torch.float16).float().unflatten(-1, (-1, 2)) for at in (kdm, vdm))
    k = (words[kw].unsqueeze(-1) >> shifts & 15).flatten(-2).float() * kd[..., :1] - kd[..., 1:]
    v = (words[vw].unsqueeze(-1) >> shifts & 15).flatten(-2).float() * vd[..., :1] - vd[..., 1:]
    return {"k": k.to(state["k"].dtype), "v": v.to(state["v"].dtype)}


def places(state, page, t):
    """Word numbers in the pages of tokens' key and value words [n, kv, D/8] and pairs [n, kv]."""
    kv, dim, size = state["kv"], state["dim"], state["page"]
    words, w = dim // 8, min(4, dim // 32)
    base = (page[:, None] * kv + torch.arange(kv, device=page.device)) * (size * (dim + 8) // 4)
    i, t = torch.arange(words, device=page.device), t[:, None]
    k = ((t // 16 * (words // w) + i // w) * 16 + t % 16) * w + i % w
    v = (t // 4 * words + i) * 4 + t % 4
    n = size * words
    return base[..., None] + k[:, None], base[..., None] + n + v[:, None], base + 2 * n + t, base + 2 * n + size + t


def plain_append(state):
    seq, _, pos = rows_of(state)
    page = state["table"].long()[seq, pos // state["page"]]
    kw, vw, kdm, vdm = places(state, page, pos % state["page"])
    words = state["pages"].view(torch.int32)
    kq, kd, km = quantise(state["k"].float())
    vq, vd, vm = quantise(state["v"].float())
    words[kw], words[vw], words[kdm], words[vdm] = packed(kq), packed(vq), joined(kd, km), joined(vd, vm)


def handles(state):
    """The framework's cache and batch, made at the first pass and kept as a user's program keeps them."""
    if "cache" not in state:
        import decode_gemv_amd as dg
        state["dg"] = dg
        state["cache"] = dg.KvCache(state["pages"], state["kv"], state["dim"], state["page"])
        state["batch"] = dg.KvBatch(state["start"], state["lens_"], state["table"], max_len=state["longest"])
        if state["op"] == "attend":
            need = dg.lw_kv_attend_scratch_bytes(state["cache"], state["batch"], state["rows"], state["heads"])
            state["work"] = torch.empty(need, dtype=torch.uint8, device=state["pages"].device)
    return state["dg"], state["cache"], state["batch"]


def run(state):
    if own:
        dg, cache, batch = handles(state)
        if state["op"] == "attend":
            dg.lw_kv_attend(cache, batch, state["q"], state["out"], window=state["window"], lse=state["lse"], work=state["work"])
            return {"out": state["out"], "lse": state["lse"]}
        if state["op"] == "append":
            dg.lw_kv_append(cache, batch, state["k"], state["v"])
        dg.lw_kv_read(cache, batch, *state["back"])
        return dict(zip("kv", state["back"]))
    if state["op"] == "attend":
        return plain_attend(state)
    if state["op"] == "append":
        plain_append(state)
    return plain_read(state)


def exact(case, seed):
    state = prepare(case, seed)
    new, lens = sizes(case)
    kv, dim, page = case["kv"], case["dim"], case["page"]
    if case["op"] == "append":
        got = {}
        for name in "kv":
            x = state[name].double()
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            m, d = (-lo).half().double(), ((hi - lo) / 15).half().double()
            got[name] = d * ((x + m) / torch.where(d == 0, 1.0, d)).round().clamp(0, 15) - m
        return got
    raw = state["pages"].view(-1, kv, page * (dim + 8))
    i = torch.arange(dim, device=raw.device)

    def tokens(s, lo, hi):
        """Keys and values [kv, hi - lo, D] of sequence s, byte by byte from the layout."""
        t = torch.arange(lo, hi, device=raw.device)
        blocks = raw[state["table"][s, t // page].long()].transpose(0, 1)
        t = (t % page)[:, None]
        wide = min(4, dim // 32)
        word = [((t // 16 * (dim // 8 // wide) + i // 8 // wide) * 16 + t % 16) * wide + i // 8 % wide, page * dim // 8 + (t // 4 * (dim // 8) + i // 8) * 4 + t % 4]
        got = []
        for side in range(2):
            byte = (word[side] * 4 + i % 8 // 2).expand(kv, -1, -1)
            code = (blocks.gather(2, byte) >> (i % 2 * 4).to(torch.uint8) & 15).double()
            at = (page * (dim + 4 * side) + 4 * t + torch.arange(4, device=raw.device)).expand(kv, -1, -1)
            dm = blocks.gather(2, at).contiguous().view(torch.float16).double()
            got.append(dm[..., :1] * code - dm[..., 1:])
        return got

    if case["op"] == "read":
        parts = [tokens(s, lens[s] - n, lens[s]) for s, n in enumerate(new)]
        return {name: torch.cat([p[side] for p in parts], 1).transpose(0, 1) for side, name in enumerate("kv")}
    outs, lses, at = [], [], 0
    for s, n in enumerate(new):
        k, v = tokens(s, 0, lens[s])
        q = state["q"][at:at + n].double().transpose(0, 1)       # [heads, n, D]
        at += n
        j, p = torch.arange(lens[s], device=raw.device), torch.arange(lens[s] - n, lens[s], device=raw.device)[:, None]
        hidden = (j > p) | (j <= p - (case["window"] or 1 << 30))
        out, lse = [], []
        for h in range(case["heads"]):
            score = q[h] @ k[h * kv // case["heads"]].T / math.sqrt(dim)
            score.masked_fill_(hidden, float("-inf"))
            lse.append(torch.logsumexp(score, -1))
            out.append(torch.exp(score - lse[-1][:, None]) @ v[h * kv // case["heads"]])
        outs.append(torch.stack(out, 1))
        lses.append(torch.stack(lse, 1))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
