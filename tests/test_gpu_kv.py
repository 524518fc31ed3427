"""GPU: the 4-bit key/value cache through the C ABI.  What lw_kv_append writes and lw_kv_read gives is equal, bit for
bit, to the reference's; lw_kv_attend's outputs and log sums lie within bounds derived from the arithmetic (kv_ref.bounds)
of attention in fp64 over what the cache holds."""
import numpy as np
import pytest

import kv_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as T
    assert T.cuda.is_available(), "GPU tests need a GPU"
    return T


@pytest.fixture(scope="module")
def dg():
    import decode_gemv_amd as D
    return D


def say(*a):
    print(*a, flush=True)


TYPES = {"fp16": "float16", "bf16": "bfloat16", "fp32": "float32"}


def host(t):
    """A tensor's values as a numpy array (bf16 as fp32)."""
    import torch
    return (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


class Setup:
    """A cache of random bytes and a batch over a shuffled table."""

    def __init__(self, torch, dg, kv, D, P, new, lens, seed, extra=2, table=None, n_pages=None, before=0, after=0):
        rng = np.random.default_rng(seed)
        self.torch, self.dg, self.kv, self.D, self.P = torch, dg, kv, D, P
        need = [max(1, -(-max(n, 1) // P)) for n in lens]
        self.n_pages = n_pages or sum(need) + extra
        if table is None:
            order = rng.permutation(self.n_pages)
            table, at = np.full((len(lens), max(need)), -1, np.int32), 0
            for s, n in enumerate(need):
                table[s, :n] = order[at:at + n]
                at += n
        self.table = np.asarray(table, np.int32)
        self.start = before + np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.lens = np.asarray(lens, np.int32)
        self.rows = int(self.start[-1]) + after
        self.image = rng.integers(0, 256, self.n_pages * R.page_bytes(kv, D, P), dtype=np.uint8)
        self.pages = torch.from_numpy(self.image.copy()).cuda()
        self.cache = dg.KvCache(self.pages, kv, D, P)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.batch = dg.KvBatch(dev(self.start), dev(self.lens), dev(self.table), max_len=int(max(self.lens.max(), 0)))
        self.rng = rng

    def where(self, row):
        """(sequence, position) of a packed row, or None."""
        for s in range(len(self.lens)):
            if self.start[s] <= row < self.start[s + 1]:
                return s, max(int(self.lens[s]), 0) - int(self.start[s + 1] - row)
        return None

    def fill(self, gain=1.0):
        """Quantised random keys and values in every token of every page (vectorised, in the reference's layout)."""
        D, P = self.D, self.P
        raw = self.image.reshape(self.n_pages, self.kv, P * (D + 8))
        for t in range(P):
            for side, (byte, shift, at) in enumerate(R.places(D, P, t)):
                x = (self.rng.standard_normal((self.n_pages, self.kv, D)) * gain).astype(np.float32)
                if side == 0:
                    x[..., D // 3] *= 5                      # a channel that stands out, as keys have
                q, d, m = R.quantise(x)
                raw[:, :, byte[0::2]] = q[..., 0::2] | q[..., 1::2] << 4
                raw[:, :, at:at + 4] = np.stack([d, m], -1).view(np.uint8)
        self.pages.copy_(self.torch.from_numpy(self.image))
        return self

    def tensor(self, heads, dtype, how="dense", values=None):
        """A packed tensor [rows][heads][D]: dense, a slice of a fused one, or misaligned with odd strides."""
        torch = self.torch
        kind = getattr(torch, TYPES[dtype])
        n, D = self.rows, self.D
        if how == "dense":
            t = torch.empty((n, heads, D), dtype=kind, device="cuda")
        elif how == "fused":
            t = torch.empty((n, heads + 3, D), dtype=kind, device="cuda")[:, 1:1 + heads]
        elif how == "heads first":
            t = torch.empty((heads, n, D), dtype=kind, device="cuda").transpose(0, 1)
        else:
            flat = torch.empty(1 + n * (heads * (D + 1) + 5) + D, dtype=kind, device="cuda")
            t = flat[1:].as_strided((n, heads, D), (heads * (D + 1) + 5, D + 1, 1))
        if values is None:
            values = self.rng.standard_normal((n, heads, D)).astype(np.float32)
        t.copy_(torch.from_numpy(values).cuda())
        return t


APPENDS = [
    # kv, D, P, new, lens: one token, tokens that cross pages and tiles, rows of many sequences in one wavefront
    (1, 64, 32, [1], [1]), (3, 64, 32, [1, 2, 1, 1, 5], [33, 64, 1, 70, 5]), (2, 128, 64, [70, 0, 3], [130, 9, 67]),
    (8, 128, 128, [1, 1, 1], [129, 300, 128]), (2, 256, 32, [33, 1], [40, 65]), (1, 256, 256, [1, 7], [256, 260]),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"kv{c[0]}_D{c[1]}_P{c[2]}_n{sum(c[3])}")
def test_append_and_read_are_exact(torch, dg, case, dtype):
    kv, D, P, new, lens = case
    for how in ("dense", "fused", "heads first", "misaligned"):
        say("append", case, dtype, how)
        s = Setup(torch, dg, kv, D, P, new, lens, 11 + sum(new))
        k, v = s.tensor(kv, dtype, how), s.tensor(kv, dtype, how)
        dg.lw_kv_append(s.cache, s.batch, k, v)
        want = s.image.copy().reshape(s.n_pages, kv, -1)
        sides = [R.quantise(host(x)) for x in (k, v)]
        back = [np.zeros((s.rows, kv, D)) for _ in range(2)]
        ref = R.Cache(want, kv, D, P)
        for row in range(s.rows):
            seq, pos = s.where(row)
            page, t = ref.at(s.table[seq], pos)
            for h in range(kv):
                for side, (q, d, m) in enumerate(sides):
                    R.write(want[page, h], D, P, t, side, q[row, h], d[row, h], m[row, h])
                    back[side][row, h] = R.read(want[page, h], D, P, t, side)[0]
        torch.cuda.synchronize()
        got = s.pages.cpu().numpy().reshape(want.shape)
        assert np.array_equal(got, want), "the cache's bytes differ (or others than the tokens' were written)"
        ok, ov = s.tensor(kv, dtype, how), s.tensor(kv, dtype, how)
        dg.lw_kv_read(s.cache, s.batch, ok, ov)
        torch.cuda.synchronize()
        for got, ref64 in ((ok, back[0]), (ov, back[1])):
            exact = torch.from_numpy(ref64.astype(np.float32)).to(got.dtype)     # d q - m rounds once: fp32 holds it
            assert torch.equal(got.cpu(), exact)


def test_append_special_vectors(torch, dg):
    kv, D, P = 2, 128, 32
    s = Setup(torch, dg, kv, D, P, [9], [40], 21)
    x = s.rng.standard_normal((9, kv, D)).astype(np.float32)
    x[0] = 2.5
    x[1, 0, 7] = np.nan
    x[2, 1, 100] = np.inf
    x[3, 0, 3] = -np.inf
    x[4, 0, :2] = 3e38, -3e38
    x[5] *= 1e-7
    x[6] = 0
    x[7, 0] = 70000.0
    x[8, 1] = -1e-30
    k, v = s.tensor(kv, "fp32", "dense", x), s.tensor(kv, "bf16", "dense", x).float()
    dg.lw_kv_append(s.cache, s.batch, k, v)
    ok, ov = torch.empty_like(k), torch.empty_like(v)
    dg.lw_kv_read(s.cache, s.batch, ok, ov)
    torch.cuda.synchronize()
    for src, got in ((k, ok), (v, ov)):
        q, d, m = R.quantise(host(src))
        want = (d.astype(np.float64)[..., None] * q - m.astype(np.float64)[..., None]).astype(np.float32)
        assert np.array_equal(host(got), want, equal_nan=True)
    assert np.isnan(host(ok)[1, 0]).all() and np.isfinite(host(ok)[1, 1]).all()


def test_append_every_scale(torch, dg):
    """Vectors whose d is each finite fp16 there is, and values between and on the codes."""
    d = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float32)
    rng = np.random.default_rng(12)
    x = rng.uniform(0, 15, (len(d), 1, 64)).astype(np.float32) * d[:, None, None]
    x[:, 0, 0], x[:, 0, 1], x[:, 0, 2] = 0, 15 * d, 7.5 * d
    x -= (rng.integers(0, 16, len(d)) * d).astype(np.float32)[:, None, None]
    s = Setup(torch, dg, 1, 64, 256, [len(d)], [len(d)], 58)
    k = s.tensor(1, "fp32", "dense", x)
    dg.lw_kv_append(s.cache, s.batch, k, k)
    ok, ov = torch.empty_like(k), torch.empty_like(k)
    dg.lw_kv_read(s.cache, s.batch, ok, ov)
    q, sd, m = R.quantise(x)
    assert len(np.unique(sd.view(np.uint16))) > 30000
    want = (sd.astype(np.float64)[..., None] * q - m.astype(np.float64)[..., None]).astype(np.float32)
    assert np.array_equal(host(ok), want) and np.array_equal(host(ov), want)


def test_absent_tokens_and_rows_of_no_sequence(torch, dg):
    """Pages of -1 or past the pool, positions before 0 and past the table: not written, read as zeros; rows before
    start[0] and from start[n] on keep what they held; pages that no table names keep theirs."""
    kv, D, P = 2, 64, 32
    table = [[0, -1, 2], [9, 3, 1 << 30], [4, 4, 4]]
    s = Setup(torch, dg, kv, D, P, [40, 40, 3], [90, 100, 2], 31, table=table, n_pages=6, before=2, after=3)
    k, v = s.tensor(kv, "fp16"), s.tensor(kv, "fp16")
    dg.lw_kv_append(s.cache, s.batch, k, v)
    ok, ov = (torch.full_like(k, 7.0) for _ in range(2))
    dg.lw_kv_read(s.cache, s.batch, ok, ov)
    torch.cuda.synchronize()
    want = s.image.copy().reshape(6, kv, -1)
    ref = R.Cache(want, kv, D, P)
    q = [R.quantise(host(x)) for x in (k, v)]
    for row in range(s.rows):
        at = s.where(row)
        place = ref.at(s.table[at[0]], at[1]) if at else None
        for side, got in enumerate((ok, ov)):
            for h in range(kv):
                if place:
                    R.write(want[place[0], h], D, P, place[1], side, *(a[row, h] for a in q[side]))
                    exact = R.read(want[place[0], h], D, P, place[1], side)[0].astype(np.float16)
                    assert np.array_equal(host(got)[row, h], exact)
                else:
                    assert np.all(host(got)[row, h] == (7.0 if at is None else 0.0)), row
    assert np.array_equal(s.pages.cpu().numpy().reshape(want.shape), want)


# ------------------------------------------------------------------ attention

def check(s, q, out, lse, dtype, rows=None, **kw):
    ref, rl, by = R.attend(R.Cache(s.pages.cpu().numpy(), s.kv, s.D, s.P), s.table, s.start, s.lens,
                           host(q).astype(np.float64), s.D ** -0.5, **kw)
    many = q.shape[0] * (q.shape[1] // s.kv) > 64 * len(s.lens)      # of the tiles of 128 rows
    tol, tl = R.bounds(ref, rl, by, s.D, dtype == "bf16", many)
    rows = np.isfinite(ref).all((1, 2)) if rows is None else rows
    got, gl = host(out).astype(np.float64)[rows], host(lse)[rows]
    ref, rl, tol, tl = ref[rows], rl[rows], tol[rows], tl[rows]
    assert np.isfinite(got).all()
    off = np.abs(got - ref)
    assert np.all(off <= tol), f"out {np.max(off[off > tol] / tol[off > tol])} of its bound"
    empty = np.isneginf(rl)
    assert np.array_equal(empty, np.isneginf(gl)) and np.all(got[empty] == 0)
    off = np.abs(gl[~empty] - rl[~empty]) / tl[~empty]
    assert np.all(off <= 1), f"lse {off.max()} of its bound"


def run(s, q, dtype, work=True, how="dense", **kw):
    torch, dg = s.torch, s.dg
    out = s.tensor(q.shape[1], dtype, how, np.full(tuple(q.shape), np.nan, np.float32))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    need = dg.lw_kv_attend_scratch_bytes(s.cache, s.batch, s.rows, q.shape[1]) if work is True else work
    mem = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    dg.lw_kv_attend(s.cache, s.batch, q, out, lse=lse, work=mem, **kw)
    torch.cuda.synchronize()
    return out, lse


ATTENDS = [
    # kv, group, P, new, lens: rows of one tile in part, in full and over; tiles of 8, 16 and 32 rows; first tokens;
    # sequences without new tokens; steps and pages that end inside
    (1, 1, 32, [1], [1]), (2, 1, 32, [1, 1, 1], [31, 32, 33]), (2, 4, 64, [1, 1], [300, 129]), (1, 8, 32, [1], [257]),
    (2, 5, 32, [1, 0, 1], [70, 40, 100]), (1, 16, 64, [1, 1], [65, 200]), (2, 3, 32, [5, 3], [90, 3]),
    (1, 7, 128, [9, 1, 20], [200, 64, 20]), (2, 2, 32, [40], [40]), (1, 40, 64, [2], [90]), (1, 1, 32, [67], [99]),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: f"kv{c[0]}x{c[1]}_P{c[2]}_n{'_'.join(map(str, c[3]))}")
def test_attend(torch, dg, case, D, dtype):
    kv, group, P, new, lens = case
    say("attend", case, D, dtype)
    s = Setup(torch, dg, kv, D, P, new, lens, 100 + sum(lens)).fill()
    q = s.tensor(kv * group, dtype, "fused")
    for kw in (dict(), dict(window=17), dict(causal=False), dict(causal=False, window=40)):
        out, lse = run(s, q, dtype, **kw)
        check(s, q, out, lse, dtype, **kw)


@pytest.mark.parametrize("D,group,new", [(128, 4, 1), (64, 1, 1), (256, 8, 1), (128, 9, 1), (128, 8, 6)])
def test_attend_in_chunks(torch, dg, D, group, new):
    """Long sequences beside short ones, cut into many chunks, few, or one: as the scratch allows."""
    kv, P = 1, 64
    s = Setup(torch, dg, kv, D, P, [new] * 3, [3000, 33, 1027], 7 + D).fill()
    q = s.tensor(kv * group, "fp16")
    whole = dg.lw_kv_attend_scratch_bytes(s.cache, s.batch, s.rows, kv * group)
    assert whole > 0
    for nb in (whole, whole // 3, 64, 0):
        say("chunks", D, group, new, nb)
        out, lse = run(s, q, "fp16", work=nb)
        check(s, q, out, lse, "fp16")
        again, lse2 = run(s, q, "fp16", work=nb)
        assert torch.equal(out, again) and torch.equal(lse, lse2), "not deterministic"


@pytest.mark.parametrize("seqs,kv,group,new", [(64, 1, 2, 1), (65, 2, 4, 1), (130, 1, 3, 4), (200, 3, 1, 1)])
def test_ragged_batches_in_chunks(torch, dg, seqs, kv, group, new):
    """Sequences of all lengths, some without new tokens, cut into chunks of one size for the batch."""
    rng = np.random.default_rng(seqs)
    lens = [int(rng.integers(new, 1300)) if i % 3 else new for i in range(seqs)]
    lens[seqs // 2], lens[-1] = 2600, 1100
    count = [0 if i % 7 == 5 else 1 + i % new for i in range(seqs)]
    s = Setup(torch, dg, kv, 64, 64, count, lens, 19 + seqs).fill()
    q = s.tensor(kv * group, "bf16")
    for kw in (dict(), dict(window=1500), dict(causal=False)):
        say("ragged", seqs, kv, group, new, kw)
        out, lse = run(s, q, "bf16", **kw)
        check(s, q, out, lse, "bf16", **kw)


@pytest.mark.parametrize("how", ["fused", "heads first", "misaligned"])
def test_attend_strides(torch, dg, how):
    s = Setup(torch, dg, 2, 128, 32, [3, 1], [80, 40], 55).fill()
    q = s.tensor(8, "bf16", how)
    dense = s.tensor(8, "bf16", "dense", host(q))
    out, lse = run(s, q, "bf16", how=how)
    want, want_lse = run(s, dense, "bf16")
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    check(s, q, out, lse, "bf16")


def test_attend_scale_and_large_queries(torch, dg):
    # a scale of its own is folded into the queries of the reference; large and small queries, a row of zeros
    s = Setup(torch, dg, 1, 64, 32, [4], [70], 56).fill()
    x = s.rng.standard_normal((4, 2, 64)).astype(np.float32)
    x[0] *= 300
    x[1] *= 1e-4
    x[2] = 0
    q = s.tensor(2, "fp16", "dense", x)
    out, lse = run(s, q, "fp16")
    check(s, q, out, lse, "fp16")
    out, lse = run(s, q, "fp16", scale=0.03125)               # a quarter of 64 ** -0.5: exact on the queries
    check(s, q.float() * 0.25, out, lse, "fp16")


def test_rows_that_see_nothing(torch, dg):
    """More new tokens than the sequence has, windows over pages given up, and whole sequences without pages."""
    table = [[0, -1, -1, 1], [2, 2, 2, 2], [-1, 99, -5, -1]]
    for D, group, P in ((128, 4, 32), (64, 20, 32)):
        for dtype in ("fp16", "bf16"):
            s = Setup(torch, dg, 1, D, P, [2, 5, 3], [90, 2, 128], 61, table=table, n_pages=3).fill()
            q = s.tensor(group, dtype)
            for kw in (dict(), dict(window=20), dict(causal=False)):
                say("nothing", D, group, dtype, kw)
                out, lse = run(s, q, dtype, **kw)
                check(s, q, out, lse, dtype, **kw)
            assert torch.isneginf(lse[-3:]).all()
            out, lse = run(s, q, dtype, window=20)
            assert torch.isneginf(lse[:2]).all()              # positions 69..89 lie in pages given up
            assert torch.isneginf(lse[2:5]).all()             # positions -3..-1


def test_hidden_tokens_may_hold_anything(torch, dg):
    """NaN and infinite pairs past the length, before the window and after a row's position; a visible NaN reaches the
    rows that see it and no other."""
    kv, D, P = 1, 128, 32
    for group in (1, 12, 40):
        s = Setup(torch, dg, kv, D, P, [3], [50], 71).fill()
        raw = s.image.reshape(s.n_pages, kv, -1)
        clean = R.Cache(s.image.copy(), kv, D, P)
        def spoil(pos, bits):
            page, t = clean.at(s.table[0], pos)
            for _, _, at in R.places(D, P, t):
                raw[page, 0, at:at + 4] = np.array([bits, bits], np.uint16).view(np.uint8)
        for pos in range(50, 64):
            spoil(pos, 0x7E00 if pos % 2 else 0x7C00)
        for pos in range(0, 20):
            spoil(pos, 0x7E00)
        s.pages.copy_(torch.from_numpy(s.image))
        q = s.tensor(group, "fp16")
        out, lse = run(s, q, "fp16", window=25)
        check(s, q, out, lse, "fp16", window=25)
        spoil(49, 0x7E00)                                     # the last token: only the last row sees it
        s.pages.copy_(torch.from_numpy(s.image))
        bad, bad_lse = run(s, q, "fp16", window=25)
        assert torch.equal(bad[:2], out[:2]) and torch.equal(bad_lse[:2], lse[:2])
        assert torch.isnan(bad[2]).all() and torch.isnan(bad_lse[2]).all()


def test_query_with_nan_or_infinity(torch, dg):
    s = Setup(torch, dg, 1, 64, 32, [1, 1, 1], [40, 40, 40], 72).fill()
    x = s.rng.standard_normal((3, 4, 64)).astype(np.float32)
    x[0, 1, 5] = np.nan
    x[1, 2, 6] = np.inf
    out, lse = run(s, s.tensor(4, "bf16", "dense", x), "bf16")
    bad = torch.zeros((3, 4), dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.isfinite(out[~bad]).all() and torch.isfinite(lse[~bad]).all()


def test_values_of_very_different_sizes(torch, dg):
    """Value pairs from 2^-20 to 2^10 in one sequence, the large ones late: the offset moves with them."""
    s = Setup(torch, dg, 1, 64, 32, [1], [160], 73)
    s.fill()
    raw = s.image.reshape(s.n_pages, 1, -1)
    for pos in range(160):
        page, t = R.Cache(s.image, 1, 64, 32).at(s.table[0], pos)
        at = R.places(64, 32, t)[1][2]
        d = np.float16(2.0 ** (-20 + 30 * pos / 160))
        raw[page, 0, at:at + 4] = np.array([d, np.float16(7.5) * d], np.float16).view(np.uint8)
    s.pages.copy_(torch.from_numpy(s.image))
    for dtype in ("fp16", "bf16"):
        q = s.tensor(4, dtype)
        out, lse = run(s, q, dtype)
        check(s, q, out, lse, dtype)


# ------------------------------------------------- attention of many rows
# Tiles of 128 rows are taken where 128 rows times tokens make 2^19 and more, by the tokens that the batch is planned for:
# a table with room for many does that for short sequences, too.

def planned_for(s, tokens):
    wide = np.full((len(s.lens), tokens // s.P), -1, np.int32)
    wide[:, :s.table.shape[1]] = s.table
    s.batch = s.dg.KvBatch(s.batch.start, s.batch.lens, s.torch.from_numpy(wide).cuda())
    return s


MANY = [
    # kv, group, P, new, lens: part of a tile, one and several; pages that end inside a tile of tokens; first tokens;
    # no new tokens; fewer tokens than a wavefront takes
    (1, 1, 32, [67], [99]), (2, 2, 32, [40], [40]), (1, 40, 64, [2], [90]), (1, 1, 64, [130], [131]),
    (2, 1, 128, [200, 70], [260, 500]), (1, 5, 256, [100, 0, 31], [700, 10, 31]), (1, 128, 32, [1], [1]),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", MANY, ids=lambda c: f"kv{c[0]}x{c[1]}_P{c[2]}_n{'_'.join(map(str, c[3]))}")
def test_many_rows(torch, dg, case, D, dtype):
    kv, group, P, new, lens = case
    say("many", case, D, dtype)
    s = planned_for(Setup(torch, dg, kv, D, P, new, lens, 200 + sum(lens)).fill(), 1 << 19)
    q = s.tensor(kv * group, dtype, "fused")
    for kw in (dict(), dict(causal=False)):
        for work in (True, 0):
            out, lse = run(s, q, dtype, work=work, **kw)
            check(s, q, out, lse, dtype, **kw)


@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_in_chunks(torch, dg, D):
    s = planned_for(Setup(torch, dg, 1, D, 64, [128], [3000], 31 + D).fill(), 1 << 17)
    q = s.tensor(4, "fp16")
    whole = dg.lw_kv_attend_scratch_bytes(s.cache, s.batch, s.rows, 4)
    for nb in (whole, whole // 40, 0):                        # 1024 tokens a chunk, 43690, all
        say("many rows in chunks", D, nb)
        out, lse = run(s, q, "fp16", work=nb)
        check(s, q, out, lse, "fp16")
        again, lse2 = run(s, q, "fp16", work=nb)
        assert torch.equal(out, again) and torch.equal(lse, lse2), "not deterministic"


@pytest.mark.parametrize("how", ["heads first", "misaligned"])
def test_many_rows_strides(torch, dg, how):
    s = planned_for(Setup(torch, dg, 2, 128, 32, [33], [80], 57).fill(), 1 << 19)
    q = s.tensor(8, "bf16", how)
    out, lse = run(s, q, "bf16", how=how)
    want, want_lse = run(s, s.tensor(8, "bf16", "dense", host(q)), "bf16")
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    check(s, q, out, lse, "bf16")


def test_many_rows_that_see_nothing(torch, dg):
    table = [[0, -1, -1, 1], [2, 2, 2, 2], [-1, 99, -5, -1]]
    for D in (64, 128):
        for dtype in ("fp16", "bf16"):
            s = Setup(torch, dg, 1, D, 32, [2, 5, 3], [90, 2, 128], 63, table=table, n_pages=3).fill()
            planned_for(s, 1 << 18)
            q = s.tensor(40, dtype)
            for kw in (dict(), dict(causal=False)):
                say("many, nothing", D, dtype, kw)
                out, lse = run(s, q, dtype, **kw)
                check(s, q, out, lse, dtype, **kw)
            assert torch.isneginf(lse[-3:]).all()


def test_many_rows_special_values(torch, dg):
    """What hidden tokens hold, one NaN that the last rows see, a query with a NaN and one with an infinity, and value
    pairs of very different sizes."""
    s = planned_for(Setup(torch, dg, 1, 128, 32, [3], [50], 75).fill(), 1 << 19)
    raw = s.image.reshape(s.n_pages, 1, -1)
    def pair(pos, side, d, m):
        page, t = R.Cache(s.image, 1, 128, 32).at(s.table[0], pos)
        at = R.places(128, 32, t)[side][2]
        raw[page, 0, at:at + 4] = np.array([d, m], np.float16).view(np.uint8)
    for pos in range(50, 64):
        for side in (0, 1):
            pair(pos, side, np.nan if pos % 2 else np.inf, np.nan)
    for pos in range(50):
        d = np.float16(2.0 ** (-20 + 30 * pos / 50))
        pair(pos, 1, d, np.float16(7.5) * d)
    s.pages.copy_(torch.from_numpy(s.image))
    x = s.rng.standard_normal((3, 40, 128)).astype(np.float32)
    q = s.tensor(40, "fp16", "dense", x)
    out, lse = run(s, q, "fp16")
    check(s, q, out, lse, "fp16")
    for side in (0, 1):
        kept = s.image.copy()
        pair(49, side, np.nan, np.nan)
        s.pages.copy_(torch.from_numpy(s.image))
        bad, bad_lse = run(s, q, "fp16")
        assert torch.equal(bad[:2], out[:2]) and torch.equal(bad_lse[:2], lse[:2])
        assert torch.isnan(bad[2]).all()
        s.image[:] = kept
    s.pages.copy_(torch.from_numpy(s.image))
    x[0, 7, 5], x[1, 31, 6] = np.nan, np.inf
    bad, bad_lse = run(s, s.tensor(40, "fp16", "dense", x), "fp16")
    spoiled = torch.zeros((3, 40), dtype=torch.bool, device="cuda")
    spoiled[0, 7] = spoiled[1, 31] = True
    assert torch.isnan(bad[spoiled]).all() and torch.isnan(bad_lse[spoiled]).all()
    assert torch.equal(bad[~spoiled], out[~spoiled]) and torch.equal(bad_lse[~spoiled], lse[~spoiled])


@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_many_rows_in_a_window(torch, dg, D, dtype):
    """Rows enough that a window's tokens make the work: 1100 new tokens of 64 heads on 2, on a sequence of 1731."""
    kv, heads, window = 2, 64, 900
    s = Setup(torch, dg, kv, D, 32, [1100], [1731], 91 + D).fill()
    q = s.tensor(heads, dtype)
    out, lse = run(s, q, dtype, window=window)
    ref, rl, by = R.attend_one(R.Cache(s.pages.cpu().numpy(), kv, D, 32), s.table[0], 1731, host(q).astype(np.float64),
                               D ** -0.5, window)
    tol, tl = R.bounds(ref, rl, by, D, dtype == "bf16", True)
    assert np.all(np.abs(host(out) - ref) <= tol) and np.all(np.abs(host(lse) - rl) <= tl)


def test_batches_of_many_sequences(torch, dg):
    # more sequences than the 64 a lookup takes at a time, some without new tokens
    rng = np.random.default_rng(81)
    n = 150
    lens = rng.integers(1, 60, n)
    new = np.minimum(rng.integers(0, 3, n), lens)
    s = Setup(torch, dg, 1, 64, 32, list(new), list(lens), 82).fill()
    k, v, q = s.tensor(1, "bf16"), s.tensor(1, "bf16"), s.tensor(2, "bf16")
    dg.lw_kv_append(s.cache, s.batch, k, v)
    ok, ov = torch.empty_like(k), torch.empty_like(v)
    dg.lw_kv_read(s.cache, s.batch, ok, ov)
    out, lse = run(s, q, "bf16")
    check(s, q, out, lse, "bf16")
    for x, got in ((k, ok), (v, ov)):
        c, d, m = R.quantise(host(x))
        want = (d.astype(np.float64)[..., None] * c - m.astype(np.float64)[..., None]).astype(np.float32)
        assert torch.equal(got.cpu(), torch.from_numpy(want).bfloat16())


def test_tens_of_thousands_of_sequences(torch, dg):
    """40000 sequences that share pages, some without new tokens: three steps of looking for one, and more row tiles
    than one dimension of a grid; a sample of the rows is compared."""
    rng = np.random.default_rng(85)
    n, pages = 40000, 29
    lens, new = 1 + np.arange(n) % 31, np.where(np.arange(n) % 5 == 3, 0, 1)
    s = Setup(torch, dg, 1, 64, 32, list(new), list(lens), 86, table=(np.arange(n) % pages)[:, None], n_pages=pages).fill()
    q = s.tensor(2, "bf16")
    out, lse = run(s, q, "bf16")
    some = np.sort(rng.choice(np.flatnonzero(new), 400, replace=False))
    rows = s.start[some]
    ref, rl, by = R.attend(R.Cache(s.pages.cpu().numpy(), 1, 64, 32), s.table[some], np.arange(401), s.lens[some],
                           host(q).astype(np.float64)[rows], 64 ** -0.5)
    tol, tl = R.bounds(ref, rl, by, 64, True)
    assert np.all(np.abs(host(out)[rows] - ref) <= tol) and np.all(np.abs(host(lse)[rows] - rl) <= tl)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # new keys of 5000 sequences that share pages, each in a place of its own
    few = Setup(torch, dg, 1, 64, 32, [1] * 5000, [1 + i % 32 for i in range(5000)], 87,
                table=(np.arange(5000) // 32)[:, None], n_pages=5000 // 32 + 1)
    k, v = few.tensor(1, "bf16"), few.tensor(1, "bf16")
    dg.lw_kv_append(few.cache, few.batch, k, v)
    ok, ov = torch.empty_like(k), torch.empty_like(v)
    dg.lw_kv_read(few.cache, few.batch, ok, ov)
    for x, got in ((k, ok), (v, ov)):
        c, d, m = R.quantise(host(x))
        want = (d.astype(np.float64)[..., None] * c - m.astype(np.float64)[..., None]).astype(np.float32)
        assert torch.equal(got.cpu(), torch.from_numpy(want).bfloat16())


def test_lens_past_the_bound_given(torch, dg):
    # max_len is a hint: a longer sequence is served in full
    s = Setup(torch, dg, 1, 128, 32, [1, 1], [900, 40], 83).fill()
    q = s.tensor(4, "fp16")
    for hint in (1, 300, 0):
        s.batch = dg.KvBatch(s.batch.start, s.batch.lens, s.batch.table, max_len=hint)
        out, lse = run(s, q, "fp16")
        check(s, q, out, lse, "fp16")


def test_offsets_past_32_bits(torch, dg):
    """Pages more than 4 GiB into the cache."""
    kv, D, P = 8, 256, 256
    size = R.page_bytes(kv, D, P)
    n_pages = (9 << 29) // size + 2                           # 4.5 GiB
    pages = torch.empty(n_pages * size, dtype=torch.uint8, device="cuda")
    table = np.array([[n_pages - 1, n_pages - 2]], np.int32)
    small = Setup(torch, dg, kv, D, P, [300], [300], 84, table=[[0, 1]], n_pages=2)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    big_cache = dg.KvCache(pages, kv, D, P)
    big_batch = dg.KvBatch(small.batch.start, small.batch.lens, dev(table))
    k, v, q = small.tensor(kv, "fp16"), small.tensor(kv, "fp16"), small.tensor(kv, "fp16")
    dg.lw_kv_append(small.cache, small.batch, k, v)
    dg.lw_kv_append(big_cache, big_batch, k, v)
    assert torch.equal(pages[-size:][:P * (D + 8)], small.pages[:P * (D + 8)])
    outs = []
    for cache, batch in ((small.cache, small.batch), (big_cache, big_batch)):
        ok, ov, out = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
        dg.lw_kv_read(cache, batch, ok, ov)
        dg.lw_kv_attend(cache, batch, q, out)
        outs.append((ok, ov, out))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_another_stream_and_graph_replays(torch, dg):
    """A step (append, attend, lengths moved on by the program) on a side stream, captured and replayed: every replay
    follows the arrays' contents and equals the eager call."""
    kv, D, P, steps = 2, 128, 32, 4
    s = Setup(torch, dg, kv, D, P, [1, 1, 1], [40, 5, 500], 91, table=np.arange(3 * 17).reshape(3, 17), n_pages=51).fill()
    s.batch = dg.KvBatch(s.batch.start, s.batch.lens, s.batch.table)
    ks, vs = ([s.tensor(kv, "bf16") for _ in range(steps)] for _ in range(2))
    qs = [s.tensor(8, "bf16") for _ in range(steps)]
    work = torch.empty(dg.lw_kv_attend_scratch_bytes(s.cache, s.batch, 3, 8), dtype=torch.uint8, device="cuda")
    k, v, q, out = ks[0].clone(), vs[0].clone(), qs[0].clone(), torch.empty_like(qs[0])
    lse = torch.empty((3, 8), device="cuda")
    pages0, lens0 = s.pages.clone(), s.batch.lens.clone()

    def step():
        dg.lw_kv_append(s.cache, s.batch, k, v)
        dg.lw_kv_attend(s.cache, s.batch, q, out, work=work, lse=lse)

    def whole(go):
        s.pages.copy_(pages0)
        s.batch.lens.copy_(lens0)
        got = []
        for i in range(steps):
            k.copy_(ks[i]), v.copy_(vs[i]), q.copy_(qs[i])
            out.fill_(float("nan"))
            torch.cuda.synchronize()
            go()
            torch.cuda.synchronize()
            got.append((out.clone(), lse.clone()))
            s.batch.lens.add_(1)
        return got + [(s.pages.clone(), s.batch.lens.clone())]

    eager = whole(step)
    side = torch.cuda.Stream()

    def on_side():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
    streamed = whole(on_side)
    s.batch.lens.copy_(lens0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        replayed = whole(graph.replay)
        for a, b, c in zip(eager, streamed, replayed):
            for x, y, z in zip(a, b, c):
                assert torch.equal(x, y) and torch.equal(x, z)


def test_python_refusals(torch, dg):
    s = Setup(torch, dg, 2, 64, 32, [2], [40], 92)
    k = s.tensor(2, "fp16")
    dev = s.batch
    bad = [lambda: dg.lw_kv_append(s.cache, dev, k.cpu(), k), lambda: dg.lw_kv_append(s.cache, dev, k[:, :1], k[:, :1]),
           lambda: dg.lw_kv_append(s.cache, dev, k, k.bfloat16()), lambda: dg.lw_kv_append(s.cache, dev, k, k[:1]),
           lambda: dg.lw_kv_append(s.cache, dev, k.int(), k.int()), lambda: dg.lw_kv_append(s.cache, dev, k[..., ::2], k[..., ::2]),
           lambda: dg.lw_kv_read(s.cache, dev, k[0], k[0]), lambda: dg.lw_kv_attend(s.cache, dev, k.float(), k.float()),
           lambda: dg.lw_kv_attend(s.cache, dev, k, k, lse=torch.empty(3, device="cuda")),
           lambda: dg.lw_kv_attend(s.cache, dev, k[:, :1], k[:, :1]), lambda: dg.lw_kv_attend(s.cache, dev, k, k, scale=0.0),
           lambda: dg.KvCache(s.pages[:-1], 2, 64, 32), lambda: dg.KvCache(s.pages, 2, 96, 32),
           lambda: dg.KvBatch(dev.start, dev.lens.long(), dev.table), lambda: dg.KvBatch(dev.start[:1], dev.lens, dev.table),
           lambda: dg.KvBatch(dev.start, dev.lens, dev.table[0])]
    before = s.pages.clone()
    for i, f in enumerate(bad):
        with pytest.raises(dg.LwError):
            f()
            say("not refused:", i)
    torch.cuda.synchronize()
    assert torch.equal(before, s.pages)


@pytest.mark.parametrize("args", [[], ["--prompt", "33", "--steps", "3", "--batch", "5"]])
def test_example_cached_decode(torch, dg, args):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import cached_decode
    # fp16 outputs (2^-11) of fp32 scores
    assert cached_decode.main(args) < 1e-3
