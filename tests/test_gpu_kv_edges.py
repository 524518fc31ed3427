"""GPU: corners of the 4-bit key/value cache's attention, against fp64 (kv_ref) with bounds derived from the arithmetic."""
import numpy as np
import pytest

import kv_ref as R
from test_gpu_kv import ATTENDS, MANY, Setup, dg, host, planned_for, run, say, torch  # noqa: F401  (dg and torch are fixtures)
from test_kv_plan import plan

pytestmark = pytest.mark.gpu


def tight(ref, rl, by, D, bf16):
    """kv_ref.bounds with p dv held to 2^-21 whatever the result's type; a bf16 result is rounded to 2^-8."""
    tol, tl = R.bounds(ref, rl, by, D, False)
    return (tol + 2.0 ** -8 * (np.abs(ref) + tol) if bf16 else tol), tl


def compare(s, q, out, lse, dtype, **kw):
    """Rows whose reference is finite lie within tight(); rows that see nothing are zeros and -infinity."""
    ref, rl, by = R.attend(R.Cache(s.pages.cpu().numpy(), s.kv, s.D, s.P), s.table, s.start, s.lens,
                           host(q).astype(np.float64), kw.pop("scale", s.D ** -0.5), **kw)
    tol, tl = tight(ref, rl, by, s.D, dtype == "bf16")
    fine = np.isfinite(ref).all(-1)
    got, gl = host(out).astype(np.float64), host(lse).astype(np.float64)
    out_of = ~(np.abs(got - ref) <= tol) & fine[..., None]
    assert not out_of.any(), f"{out_of.sum()} values out of their bounds, {np.argwhere(out_of)[:4].tolist()}"
    empty = np.isneginf(rl) & fine
    assert np.all(np.isneginf(gl[empty])) and np.all(got[empty] == 0)
    some = fine & ~empty
    assert np.all(np.abs(gl[some] - rl[some]) <= tl[some])
    return ref, fine


def cancelling(torch, dg, kv, D, group, planned, dtype, n):
    """A token of no value, and values in pairs under equal weights, 4 d and -3 (4 d / 3): what is left of them is the
    roundings of d (fp16) and, if p d were rounded to fp16 too, that rounding, some ten times the bound."""
    s = Setup(torch, dg, kv, D, 32, [1], [n], 300 + D + n).fill()
    raw = s.image.reshape(s.n_pages, kv, -1)
    at = [R.Cache(s.image, kv, D, 32).at(s.table[0], pos) for pos in range(n)]

    def put(pos, h, side, q, d, m):
        R.write(raw[at[pos][0], h], D, 32, at[pos][1], side, np.broadcast_to(q, D), d, m)
    for h in range(kv):
        put(0, h, 1, 0, np.float16(0), np.float16(0))
        for pos in range(1, n, 2):
            key = R.quantise(s.rng.standard_normal(D).astype(np.float32))
            d = np.float16(s.rng.uniform(0.2, 0.9))
            for i, code in ((0, 12), (1, 5)):
                put(pos + i, h, 0, *key)                      # one key for both
                put(pos + i, h, 1, code, d, np.float16(8) * d)
                d = np.float16(np.float64(d) * 4 / 3)
    s.pages.copy_(torch.from_numpy(s.image))
    if planned:
        planned_for(s, planned)
    x = np.zeros((1, kv * group, D), np.float32)              # queries of one element: scores of a few roundings
    x[0, np.arange(kv * group), s.rng.integers(0, D, kv * group)] = s.rng.uniform(-1, 1, kv * group)
    q = s.tensor(kv * group, dtype, "dense", x)
    out, lse = run(s, q, dtype)
    compare(s, q, out, lse, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_rounding_leaves_is_of_the_rounded_value(torch, dg, D):
    """Values that cancel under 40 thousand weights: some p dv lie between two roundings (of the product, and of the product
    rounded to 32 bits), which have to be the same one in both parts of p dv."""
    cancelling(torch, dg, 64, D, 32, 0, "fp16", 21)


# group (rows of the one new token), tokens that the batch is planned for: tiles of 8, 16, 32 and 128 rows
TILES = [(8, 0), (16, 0), (32, 0), (128, 1 << 19)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("group,planned", TILES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_cancel(torch, dg, D, group, planned, dtype):
    for n in (3, 23):
        say("cancel", D, group, dtype, n)
        cancelling(torch, dg, 1, D, group, planned, dtype, n)


@pytest.mark.parametrize("group,planned", TILES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_far_below_one(torch, dg, D, group, planned):
    """Queries and scales whose product is below the smallest normal number: all seen tokens weigh the same, and those that
    are hidden still nothing."""
    for dtype, size, scale in (("bf16", 1e-22, 1e-20), ("bf16", 1e-39, 1e-3), ("fp16", 6e-8, 1e-37), ("bf16", 1e-38, 1e-38)):
        say("tiny scores", D, group, dtype, size, scale)
        s = Setup(torch, dg, 1, D, 32, [2], [5], 401 + D).fill()
        if planned:
            planned_for(s, planned)
        q = s.tensor(group // 2, dtype, "dense", (s.rng.standard_normal((2, group // 2, D)) * size).astype(np.float32))
        out, lse = run(s, q, dtype, scale=scale)
        _, fine = compare(s, q, out, lse, dtype, scale=scale)
        assert fine.all()


@pytest.mark.parametrize("work", [True, 0])
@pytest.mark.parametrize("group", [8, 128])
def test_a_table_of_2_to_26_pages(torch, dg, group, work):
    s = Setup(torch, dg, 1, 64, 256, [1], [300], 35).fill()
    wide = torch.full((1, 1 << 26), -1, dtype=torch.int32, device="cuda")
    wide[:, :2] = torch.from_numpy(s.table).cuda()
    s.batch = dg.KvBatch(s.batch.start, s.batch.lens, wide)
    q = s.tensor(group, "bf16")
    out, lse = run(s, q, "bf16", work=work)
    compare(s, q, out, lse, "bf16")


@pytest.mark.parametrize("D,group,planned", [(D, g, p) for D in (64, 128, 256) for g, p in ((2, 0), (5, 0), (10, 0), (48, 1 << 19))])
def test_values_that_are_not_numbers(torch, dg, D, group, planned):
    """A value pair of NaN, its key as it was: the outputs of the rows that see it are NaN, and no log sum is."""
    s = Setup(torch, dg, 1, D, 32, [3], [100], 501 + D).fill()
    if planned:
        planned_for(s, planned)
    q = s.tensor(group, "fp16")
    clean = s.image.copy()
    ref, rl, by = R.attend(R.Cache(clean, 1, D, 32), s.table, s.start, s.lens, host(q).astype(np.float64), D ** -0.5)
    tol, tl = tight(ref, rl, by, D, False)
    for pos, sees in ((99, 2), (98, 1), (97, 0), (70, 0), (5, 0)):            # the first row that sees it
        say("not numbers", D, group, pos)
        s.image[:] = clean
        page, t = R.Cache(clean, 1, D, 32).at(s.table[0], pos)
        at = R.places(D, 32, t)[1][2]
        s.image.reshape(s.n_pages, -1)[page, at:at + 4] = np.array([np.nan, np.nan], np.float16).view(np.uint8)
        s.pages.copy_(torch.from_numpy(s.image))
        out, lse = run(s, q, "fp16")
        assert np.isnan(host(out)[sees:]).all()
        assert np.all(np.abs(host(out)[:sees] - ref[:sees]) <= tol[:sees])
        assert np.all(np.abs(host(lse) - rl) <= tl)


def tile(s, heads, window=0):
    """Rows of a tile that the call takes."""
    longest = min(s.batch.desc.max_len or 1 << 62, s.batch.desc.table_stride * s.P)
    return plan(s.D, s.kv, heads // s.kv, len(s.lens), s.rows, longest, window).tile


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case,planned", [(c, 0) for c in ATTENDS] + [(c, 1 << 19) for c in MANY])
def test_p_dv_in_two_parts(torch, dg, case, planned, D, dtype):
    """The calls of the other tests' tiles of 8, 16 and 128 rows within the bounds of a p dv that is held to 2^-21."""
    kv, group, P, new, lens = case
    s = Setup(torch, dg, kv, D, P, new, lens, 700 + sum(lens)).fill()
    if planned:
        planned_for(s, planned)
    q = s.tensor(kv * group, dtype)
    say("two parts", case, D, dtype, tile(s, kv * group))
    assert tile(s, kv * group) in ((32, 128) if planned and D < 256 else (8, 16))
    for kw in (dict(), dict(causal=False)):
        out, lse = run(s, q, dtype, **kw)
        compare(s, q, out, lse, dtype, **kw)


# ------------------------------------------------------------------ tiles of 32 rows

TALL = [
    # kv, group, P, new, lens: 17 to 32 rows a sequence on average; tiles in part, in full and several of a sequence; pages
    # that end inside a step; first tokens; sequences without new tokens
    (1, 1, 32, [20], [20]), (2, 5, 32, [5, 4], [70, 40]), (1, 17, 64, [1], [257]), (1, 32, 32, [1], [1]),
    (2, 3, 128, [9, 1, 20], [200, 64, 20]), (1, 4, 32, [8], [33]), (1, 8, 64, [0, 6], [40, 300]), (1, 2, 256, [40, 0, 3], [97, 30, 3]),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", TALL, ids=lambda c: f"kv{c[0]}x{c[1]}_P{c[2]}_n{'_'.join(map(str, c[3]))}")
def test_tall_tiles(torch, dg, case, D, dtype):
    kv, group, P, new, lens = case
    say("tall", case, D, dtype)
    s = Setup(torch, dg, kv, D, P, new, lens, 600 + sum(lens)).fill()
    q = s.tensor(kv * group, dtype, "fused")
    for kw in (dict(), dict(window=17), dict(causal=False), dict(causal=False, window=40)):
        assert tile(s, kv * group, kw.get("window", 0)) == 32
        out, lse = run(s, q, dtype, **kw)
        compare(s, q, out, lse, dtype, **kw)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [33, 64])
def test_tall_tiles_of_more_rows_and_much_work(torch, dg, rows, D, dtype):
    s = planned_for(Setup(torch, dg, 1, D, 64, [rows], [150], 610 + D + rows).fill(), 1 << 19)
    q = s.tensor(1, dtype)
    assert tile(s, 1) == 32
    for work in (True, 0):
        out, lse = run(s, q, dtype, work=work)
        compare(s, q, out, lse, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_tall_tiles_in_chunks(torch, dg, D, dtype):
    """Long sequences beside short ones, cut into many chunks, few, or one."""
    s = Setup(torch, dg, 1, D, 64, [6, 1, 5], [3000, 33, 1027], 620 + D).fill()
    q = s.tensor(7, dtype)
    assert tile(s, 7) == 32
    whole = dg.lw_kv_attend_scratch_bytes(s.cache, s.batch, s.rows, 7)
    assert whole > 0
    for nb in (whole, whole // 3, 64, 0):
        for kw in (dict(), dict(window=1500)):
            say("tall chunks", D, nb, kw)
            out, lse = run(s, q, dtype, work=nb, **kw)
            compare(s, q, out, lse, dtype, **kw)
            again, lse2 = run(s, q, dtype, work=nb, **kw)
            assert torch.equal(out, again) and torch.equal(lse, lse2), "not deterministic"


@pytest.mark.parametrize("how", ["heads first", "misaligned"])
def test_tall_tiles_strides(torch, dg, how):
    s = Setup(torch, dg, 2, 128, 32, [5, 3], [80, 40], 631).fill()
    q = s.tensor(10, "bf16", how)
    assert tile(s, 10) == 32
    out, lse = run(s, q, "bf16", how=how)
    want, want_lse = run(s, s.tensor(10, "bf16", "dense", host(q)), "bf16")
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    compare(s, q, out, lse, "bf16")


def test_tall_tiles_that_see_nothing(torch, dg):
    """More new tokens than the sequence has, windows over pages given up, and whole sequences without pages."""
    table = [[0, -1, -1, 1], [2, 2, 2, 2], [-1, 99, -5, -1]]
    for D in (64, 128):
        for dtype in ("fp16", "bf16"):
            s = Setup(torch, dg, 1, D, 32, [2, 5, 3], [90, 2, 128], 641, table=table, n_pages=3).fill()
            q = s.tensor(8, dtype)
            assert tile(s, 8) == 32
            for kw in (dict(), dict(window=20), dict(causal=False)):
                say("tall, nothing", D, dtype, kw)
                out, lse = run(s, q, dtype, **kw)
                compare(s, q, out, lse, dtype, **kw)
                assert torch.isneginf(lse[-3:]).all()
            out, lse = run(s, q, dtype, window=20)
            assert torch.isneginf(lse[:2]).all() and torch.isneginf(lse[2:5]).all()


def test_tall_tiles_special_values(torch, dg):
    """NaN and infinite pairs past the length, before the window and after a row's position, a visible NaN, queries with a
    NaN and an infinity, and value pairs of very different sizes."""
    for D in (64, 128):
        s = Setup(torch, dg, 1, D, 32, [3], [50], 651).fill()
        def pair(pos, side, d, m):
            page, t = R.Cache(s.image, 1, D, 32).at(s.table[0], pos)
            at = R.places(D, 32, t)[side][2]
            s.image.reshape(s.n_pages, -1)[page, at:at + 4] = np.array([d, m], np.float16).view(np.uint8)
        for pos in range(50):
            d = np.float16(2.0 ** (-20 + 30 * pos / 50))
            pair(pos, 1, d, np.float16(7.5) * d)
        for pos in list(range(50, 64)) + list(range(20)):
            for side in (0, 1):
                pair(pos, side, np.nan if pos % 2 else np.inf, np.nan)
        s.pages.copy_(torch.from_numpy(s.image))
        x = s.rng.standard_normal((3, 10, D)).astype(np.float32)
        q = s.tensor(10, "fp16", "dense", x)
        assert tile(s, 10, 25) == 32
        out, lse = run(s, q, "fp16", window=25)
        compare(s, q, out, lse, "fp16", window=25)
        clean = s.image.copy()
        pair(49, 0, np.nan, np.nan)                           # only the last rows see it
        s.pages.copy_(torch.from_numpy(s.image))
        bad, bad_lse = run(s, q, "fp16", window=25)
        assert torch.equal(bad[:2], out[:2]) and torch.equal(bad_lse[:2], lse[:2])
        assert torch.isnan(bad[2]).all() and torch.isnan(bad_lse[2]).all()
        s.pages.copy_(torch.from_numpy(clean))
        x[0, 7, 5], x[1, 3, 6] = np.nan, np.inf
        bad, bad_lse = run(s, s.tensor(10, "fp16", "dense", x), "fp16", window=25)
        spoiled = torch.zeros((3, 10), dtype=torch.bool, device="cuda")
        spoiled[0, 7] = spoiled[1, 3] = True
        assert torch.isnan(bad[spoiled]).all() and torch.isnan(bad_lse[spoiled]).all()
        assert torch.equal(bad[~spoiled], out[~spoiled]) and torch.equal(bad_lse[~spoiled], lse[~spoiled])


# ------------------------------------------------------------------ batches of many workgroups

@pytest.mark.parametrize("kv,group,seqs,long_", [(8, 2, 130, 4400), (16, 1, 70, 2500), (4, 9, 300, 12000)])
def test_one_long_sequence_among_many(torch, dg, kv, group, seqs, long_):
    """More workgroups than the chip has places for, cut into chunks for the sake of one sequence."""
    lens = [1 + i * 7 % 40 for i in range(seqs)]
    lens[seqs // 3] = long_
    s = Setup(torch, dg, kv, 64, 256, [1] * seqs, lens, 800 + seqs).fill()
    assert plan(64, kv, group, seqs, seqs, long_).target > 0 and seqs * kv >= 1024
    q = s.tensor(kv * group, "bf16")
    for kw in (dict(), dict(window=1200)):
        out, lse = run(s, q, "bf16", **kw)
        compare(s, q, out, lse, "bf16", **kw)


def test_log_sums_are_fp32_by_token_and_head(torch, dg):
    from decode_gemv_amd import lw
    s = Setup(torch, dg, 2, 64, 32, [3], [40], 95).fill()
    q = s.tensor(8, "fp16")
    out = torch.empty_like(q)
    for bad in (torch.zeros((3, 8), dtype=torch.int32, device="cuda"), torch.zeros((8, 3), device="cuda"),
                torch.zeros(24, device="cuda"), torch.zeros((3, 8), dtype=torch.float64, device="cuda"),
                torch.zeros((3, 8), dtype=torch.float16, device="cuda"), torch.zeros((8, 3), device="cuda").T):
        with pytest.raises(dg.LwError):
            dg.lw_kv_attend(s.cache, s.batch, q, out, lse=bad)
        assert not bad.any()
    lw._KV_TYPES.clear()                                      # as in a process's first call
    lse = torch.zeros((3, 8), device="cuda")
    dg.lw_kv_attend(s.cache, s.batch, q, out, lse=lse)
    compare(s, q, out, lse, "fp16")


@pytest.mark.parametrize("how", [0, 1, 2])
def test_starts_that_decrease(torch, dg, how):
    """An error of the caller's, in device memory, that no host check sees: results are anything, but nothing outside of
    the call's tensors is touched, whatever the workspace held."""
    starts = [[0, 9, 2, 12, 1, 20, 3], [30, 20, 10, 5, 0, -7, 40], [0, 1 << 30, -(1 << 31), 17, 40, 2, (1 << 31) - 1]]
    s = Setup(torch, dg, 2, 64, 64, [6] * 6, [3000, 700, 1500, 64, 2000, 900], 97 + how).fill()
    rows, heads, pad = 36, 6, 4096
    start = torch.tensor(starts[how], dtype=torch.int32, device="cuda")
    batch = dg.KvBatch(start, s.batch.lens, s.batch.table, max_len=3000)
    need = dg.lw_kv_attend_scratch_bytes(s.cache, batch, rows, heads)
    assert need and plan(64, 2, 3, 6, rows, 3000).target
    q = s.tensor(heads, "fp16")
    for fill in (0, 0xFF, 0x7F, None):
        say("decreasing", how, fill)
        mem = torch.full((need + 2 * pad,), fill or 0, dtype=torch.uint8, device="cuda")
        if fill is None:
            mem.copy_(torch.from_numpy(s.rng.integers(0, 256, need + 2 * pad, dtype=np.uint8)))
        before = mem.clone()
        big = torch.full((rows * heads * 64 + 2 * pad,), 7.0, dtype=torch.float16, device="cuda")
        out = big[pad:-pad].view(rows, heads, 64)
        sums = torch.full((rows * heads + 2 * pad,), 7.0, device="cuda")
        dg.lw_kv_attend(s.cache, batch, q, out, lse=sums[pad:-pad].view(rows, heads), work=mem[pad:-pad])
        k, v = s.tensor(2, "fp16"), s.tensor(2, "fp16")
        dg.lw_kv_read(s.cache, batch, k, v)
        torch.cuda.synchronize()
        for x, y in ((mem, before), (big, torch.full_like(big, 7.0)), (sums, torch.full_like(sums, 7.0))):
            assert torch.equal(x[:pad], y[:pad]) and torch.equal(x[-pad:], y[-pad:])
    assert np.array_equal(s.pages.cpu().numpy(), s.image)


@pytest.mark.parametrize("group,planned", TILES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_near_the_largest_number(torch, dg, D, group, planned):
    """bf16 queries whose elements' sum has no fp32 number, under a scale that brings the scores back."""
    s = Setup(torch, dg, 1, D, 32, [1], [70], 403 + D).fill()
    if planned:
        planned_for(s, planned)
    x = s.rng.uniform(0.6, 1, (1, group, D)) * np.where(np.arange(group) % 3, 1, -1)[:, None]
    q = s.tensor(group, "bf16", "dense", (x * 3e38).astype(np.float32))
    out, lse = run(s, q, "bf16", scale=1e-39)
    _, fine = compare(s, q, out, lse, "bf16", scale=1e-39)
    assert fine.all()


@pytest.mark.parametrize("group,planned", TILES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_far_from_zero(torch, dg, D, group, planned):
    """Scores so large that fp32 tells them apart by more than an exponential can bear: the largest takes all the weight, also
    where it is far below zero.  Rows whose two largest are closer than what fp32 scores are off by are left out."""
    for dtype, size, gain, n in (("fp16", 3e4, 1, 40), ("fp16", 6e4, 300, 40), ("bf16", 1e8, 1, 70), ("bf16", 1e20, 1, 33),
                                 ("bf16", 1e33, 1, 40), ("bf16", 1e33, 1, 1), ("bf16", 1e31, 1, 2), ("fp16", 6e4, 300, 1),
                                 ("bf16", 1e12, 1, 1500)):
        say("large scores", D, group, dtype, size, gain, n)
        s = Setup(torch, dg, 1, D, 64, [1], [n], 404 + D).fill(gain)
        if planned:
            planned_for(s, planned)
        q = s.tensor(group, dtype, "dense", np.clip(s.rng.standard_normal((1, group, D)) * size, -3e38 if dtype == "bf16" else -65504,
                                                     3e38 if dtype == "bf16" else 65504).astype(np.float32))
        out, lse = run(s, q, dtype)
        cache = R.Cache(s.pages.cpu().numpy(), 1, D, 64)
        ref, rl, by = R.attend(cache, s.table, s.start, s.lens, host(q).astype(np.float64), D ** -0.5)
        k, v, _, dv, _ = cache.tokens(s.table[0], n)
        x = np.sort(host(q)[0].astype(np.float64) @ k[:, 0].T * D ** -0.5, -1)
        delta = (D + 8) * 2.0 ** -23 * by["size"][0]
        clear = np.ones(group, bool) if n == 1 else x[:, -1] - x[:, -2] > 2 * delta + 40
        assert clear.sum() >= group // 4
        top = np.abs(dv[:, 0, 0]).max() * 8
        tol = 2.0 ** (-8 if dtype == "bf16" else -11) * np.abs(ref[0]) + 2.0 ** -20 * top + 2.0 ** -25
        assert np.all(np.abs(host(out)[0] - ref[0])[clear] <= tol[clear])
        assert np.all(np.abs(host(lse)[0] - rl[0]) <= delta + 2.0 ** -21 * (1 + np.abs(rl[0])))
