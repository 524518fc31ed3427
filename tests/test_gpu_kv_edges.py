"""GPU: corners of the 4-bit key/value cache's attention, against fp64 (kv_ref) with bounds derived from the arithmetic."""
import numpy as np
import pytest

import kv_ref as R
from test_gpu_kv import Setup, dg, host, planned_for, run, say, torch  # noqa: F401  (dg and torch are fixtures)

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
