"""GPU: bounds of pages, the choice of pages and attention over them, through the C ABI.  Bounds and selections are equal,
bit for bit, to the reference's (kv_long_ref); outputs lie within kv_ref.bounds of attention in fp64 over the chosen pages."""
import numpy as np
import pytest

import kv_long_ref as L
import kv_ref as R
from test_gpu_kv import Setup, host, say

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


def all_bounds(s, fill=0xA5):
    """The bounds of every page as the reference has them, host bytes."""
    cache = R.Cache(s.image, s.kv, s.D, s.P)
    raw = np.full((s.n_pages, L.bounds_bytes(s.kv, s.D)), fill, np.uint8)
    for p in range(s.n_pages):
        L.put_bounds(raw, s.kv, s.D, p, L.page_bounds(cache, p))
    return raw


def selection(torch, dg, rows, kv, take):
    new = lambda *shape: torch.full(shape, -77, dtype=torch.int32, device="cuda")
    return dg.KvSelection(new(rows + 1), new(rows), new(rows, kv, take))


def queries(s, group, dtype, how="dense", gain=1.0):
    q = s.tensor(s.kv * group, dtype, how)
    if gain != 1.0:
        q.mul_(gain)
    return q


FILLS = [
    # kv, D, P, new, lens: a page filled by one token, none, several, pages that earlier tokens began, no new tokens
    (1, 64, 32, [1], [32]), (3, 64, 32, [1, 2, 1, 70, 0], [33, 64, 31, 100, 64]), (2, 128, 64, [128, 3], [128, 66]),
    (5, 128, 32, [65, 1, 1], [96, 96, 97]), (2, 256, 32, [33, 40], [64, 32]), (1, 256, 256, [260], [600]),
    (9, 64, 128, [1, 129], [256, 256]),
]


@pytest.mark.parametrize("case", FILLS, ids=lambda c: f"kv{c[0]}_D{c[1]}_P{c[2]}_n{sum(c[3])}")
def test_bounds_are_exact(torch, dg, case):
    kv, D, P, new, lens = case
    say("bounds", case)
    s = Setup(torch, dg, kv, D, P, new, lens, 5 + sum(new), before=2, after=3).fill()
    cache = R.Cache(s.image, kv, D, P)
    want = np.full((s.n_pages, L.bounds_bytes(kv, D)), 0xA5, np.uint8)
    for i in range(len(lens)):
        pos = max(lens[i] - new[i], 0)
        for j in range(pos // P, lens[i] // P if new[i] else 0):
            L.put_bounds(want, kv, D, s.table[i, j], L.page_bounds(cache, s.table[i, j]))
    bounds = torch.full((s.n_pages, L.bounds_bytes(kv, D)), 0xA5, dtype=torch.uint8, device="cuda")
    dg.lw_kv_bounds(s.cache, s.batch, s.rows, bounds)
    assert np.array_equal(host(bounds), want)


def test_bounds_of_keys_that_are_special(torch, dg):
    # zeros, one that is not finite, pairs of the smallest and the largest size, and codes at random under any pair
    kv, D, P = 2, 64, 32
    s = Setup(torch, dg, kv, D, P, [6 * P], [6 * P], 8).fill()
    raw = s.image.reshape(s.n_pages, kv, P * (D + 8))
    page = lambda j: raw[s.table[0, j]]
    pair = lambda b, t, d, m: b[:, P * D + 4 * t:P * D + 4 * t + 4].__setitem__(Ellipsis, np.array([d, m], np.float16).view(np.uint8))
    for t in range(P):
        pair(page(0), t, 0.0, 0.0)
        pair(page(2), t, 6e-8, 0.0)
        pair(page(3), t, 65504.0, 65504.0)
        pair(page(4), t, 2.0 ** -8, 127.0 / 64 if t else -127.0 / 64)
    pair(page(1), 7, np.nan, 1.0)
    pair(page(5), 31, 1.0, -np.inf)
    s.pages.copy_(torch.from_numpy(s.image))
    bounds = torch.zeros((s.n_pages, L.bounds_bytes(kv, D)), dtype=torch.uint8, device="cuda")
    dg.lw_kv_bounds(s.cache, s.batch, s.rows, bounds)
    want, got = all_bounds(s, 0), host(bounds)
    for j in range(6):
        assert np.array_equal(got[s.table[0, j]], want[s.table[0, j]]), j


def test_bounds_skip_absent_pages(torch, dg):
    kv, D, P = 1, 64, 32
    s = Setup(torch, dg, kv, D, P, [200, 64], [200, 64], 3, table=[[0, -1, 99, 2, 3, -5], [2 ** 31 - 1, 4, -1, -1, -1, -1]],
              n_pages=5).fill()
    bounds = torch.full((5, L.bounds_bytes(kv, D)), 0x5A, dtype=torch.uint8, device="cuda")
    dg.lw_kv_bounds(s.cache, s.batch, s.rows, bounds)
    want = all_bounds(s, 0x5A)
    want[1] = 0x5A
    got = host(bounds)
    assert np.array_equal(got, want)


SELECTS = [
    # kv, group, D, P, new, lens, first, last, take, dtype, how
    (1, 1, 64, 32, [1], [1], 0, 0, 1, "fp16", "dense"), (2, 4, 128, 32, [1, 1, 1], [500, 33, 900], 1, 1, 6, "fp16", "fused"),
    (2, 5, 64, 32, [3, 0, 7], [1700, 64, 700], 0, 0, 9, "bf16", "misaligned"), (1, 16, 128, 64, [2], [1900], 2, 3, 8, "bf16", "dense"),
    (1, 20, 64, 32, [2], [1100], 0, 2, 5, "fp16", "heads first"), (1, 40, 256, 32, [1], [700], 1, 0, 4, "bf16", "fused"),
    (2, 2, 256, 32, [4], [1030], 0, 0, 2, "fp16", "dense"), (3, 3, 64, 32, [1, 9], [130, 2000], 1, 1, 70, "fp16", "dense"),
    (1, 8, 128, 256, [2], [1100], 0, 1, 3, "bf16", "dense"),
]


@pytest.mark.parametrize("case", SELECTS, ids=lambda c: f"kv{c[0]}x{c[1]}_D{c[2]}_P{c[3]}_take{c[8]}_{c[9]}")
def test_selections_are_exact_and_attention_over_them(torch, dg, case):
    kv, group, D, P, new, lens, first, last, take, dtype, how = case
    say("select", case)
    s = Setup(torch, dg, kv, D, P, new, lens, 17 + take, before=1, after=2).fill()
    raw = all_bounds(s)
    bounds = torch.from_numpy(raw).cuda()
    q = queries(s, group, dtype, how)
    sel = selection(torch, dg, s.rows, kv, take)
    dg.lw_kv_select(s.cache, s.batch, q, bounds, sel, first, last)
    want_lens, want = L.select(raw, kv, D, P, s.n_pages, s.table, s.start, s.lens, host(q), first, last, take)
    assert np.array_equal(host(sel.lens), want_lens)
    assert np.array_equal(host(sel.table), want)
    start = host(sel.start)
    assert np.array_equal(start, np.clip(np.arange(s.rows + 1), s.start[0], s.start[-1]))
    attend_over(torch, dg, s, sel, q, dtype, how)


@pytest.mark.parametrize("case", [(1, 1024, 64, 32, [1], [300], 0, 1, 3, "bf16", "dense"),
                                  (2, 70, 128, 64, [1, 2], [640, 129], 1, 0, 4, "fp16", "heads first"),
                                  (1024, 1, 64, 32, [1], [200], 0, 0, 4, "fp16", "dense")],
                         ids=["group1024", "group70", "kv1024"])
def test_as_many_heads_as_there_may_be(torch, dg, case):
    test_selections_are_exact_and_attention_over_them(torch, dg, case)


def attend_over(torch, dg, s, sel, q, dtype, how, lse=True):
    """Attention over a selection, with work and without, against fp64; rows of no sequence keep what they have."""
    kv, D, P, heads = s.kv, s.D, s.P, q.shape[1]
    group = heads // kv
    need = dg.lw_kv_attend_selected_scratch_bytes(s.cache, sel, heads)
    scale = 1.3 * D ** -0.5
    table, lens = host(sel.table), host(sel.lens)
    a, b = int(s.start[0]), int(s.start[-1])
    for room in (0, need):
        out = s.tensor(heads, dtype, how)
        out.fill_(5.0)
        logs = torch.full((s.rows, heads), 5.0, device="cuda")
        work = torch.full((room,), 0xFF, dtype=torch.uint8, device="cuda") if room else None
        dg.lw_kv_attend_selected(s.cache, sel, q, out, scale=scale, lse=logs if lse else None, work=work)
        got, got_lse = host(out), host(logs)
        for rows in (slice(0, a), slice(b, s.rows)):
            assert np.all(got[rows] == 5) and np.all(got_lse[rows] == 5)
        for g in range(kv):
            one = R.Cache(np.ascontiguousarray(s.image.reshape(s.n_pages, kv, -1)[:, g]), 1, D, P)
            mine = slice(g * group, (g + 1) * group)
            ref, ref_lse, by = R.attend(one, table[a:b, g], np.arange(b - a + 1), lens[a:b], host(q)[a:b, mine], scale)
            err, err_lse = R.bounds(ref, ref_lse, by, D, dtype == "bf16")
            off = np.abs(got[a:b, mine] - ref)
            assert np.all(off <= err), (g, room, float(np.max(off - err)))
            if lse:
                x = got_lse[a:b, mine]
                assert np.array_equal(np.isinf(x), np.isinf(ref_lse))
                fine = np.isfinite(ref_lse)
                assert np.all(np.abs(x[fine] - ref_lse[fine]) <= err_lse[fine])


def test_many_pages_chosen_alone_and_shared_out(torch, dg):
    """One long sequence: scores by workgroups of their own with work, and in one workgroup without."""
    kv, group, D, P, take = 1, 4, 64, 32, 40
    s = Setup(torch, dg, kv, D, P, [2], [32 * 1300 + 5], 4).fill()
    raw = all_bounds(s)
    bounds, q = torch.from_numpy(raw).cuda(), queries(s, group, "fp16")
    need = dg.lw_kv_select_scratch_bytes(s.cache, s.batch, s.rows, kv * group)
    assert need > 0
    want_lens, want = L.select(raw, kv, D, P, s.n_pages, s.table, s.start, s.lens, host(q), 1, 2, take)
    for room in (need, need - 4, 0):
        sel = selection(torch, dg, s.rows, kv, take)
        work = torch.full((room,), 0xFF, dtype=torch.uint8, device="cuda") if room else None
        dg.lw_kv_select(s.cache, s.batch, q, bounds, sel, 1, 2, work=work)
        say("room", room)
        assert np.array_equal(host(sel.lens), want_lens) and np.array_equal(host(sel.table), want)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("take", [17, 12000])
def test_the_longest_table(torch, dg, take, shared):
    """32768 pages a sequence (a few, again and again), of which the host knows nothing: planned for one token."""
    kv, group, D, P, n = 1, 2, 64, 32, 32768
    rng = np.random.default_rng(7)
    s = Setup(torch, dg, kv, D, P, [2], [n * P - 40], 4, table=rng.integers(0, 90, (1, n)), n_pages=90).fill()
    raw = all_bounds(s)
    bounds, q = torch.from_numpy(raw).cuda(), queries(s, group, "bf16")
    short = dg.KvBatch(s.batch.start, s.batch.lens, s.batch.table, max_len=1)
    b = s.batch if shared else short
    need = dg.lw_kv_select_scratch_bytes(s.cache, b, 2, 2)
    assert bool(need) == shared
    sel = selection(torch, dg, 2, kv, take)
    work = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    dg.lw_kv_select(s.cache, b, q, bounds, sel, 2, 3, work=work)
    one = [L.scores(raw, kv, D, np.arange(90), 0, x) for x in host(q)]
    for i in range(2):
        pos = n * P - 42 + i
        own = pos // P
        key = np.array(one[i])[s.table[0, :own]]
        key[:2] = key[own - 3:] = np.inf
        mine = np.sort(np.argsort(-key, kind="stable")[:take - 1])
        assert np.array_equal(host(sel.table)[i, 0], np.append(s.table[0, mine], s.table[0, own]))
        assert host(sel.lens)[i] == (take - 1) * P + pos % P + 1


@pytest.mark.parametrize("shared", [False, True])
def test_equal_scores_take_the_first(torch, dg, shared):
    """Every page the same: the scores are equal, and the first are taken, also where as many are as a cut can have."""
    kv, D, P = 2, 64, 32
    n = 700
    s = Setup(torch, dg, kv, D, P, [1], [n * P + 1], 6, table=[[0] * (n + 1)], n_pages=1).fill()
    bounds, q = torch.from_numpy(all_bounds(s)).cuda(), queries(s, 2, "bf16")
    # pages by their place: the same page again and again, but for the row's own, which is absent
    s.batch.table[0, n] = -1
    for take, first, last in ((1, 0, 0), (2, 0, 0), (50, 0, 3), (n, 0, 1), (n + 1, 2, 2), (n + 9, 0, 0)):
        sel = selection(torch, dg, 1, kv, take)
        work = torch.empty(dg.lw_kv_select_scratch_bytes(s.cache, s.batch, 1, 4), dtype=torch.uint8, device="cuda") if shared else None
        dg.lw_kv_select(s.cache, s.batch, q, bounds, sel, first, last, work=work)
        got = host(sel.table)[0]
        k = min(take - 1, n)
        assert np.all(got[:, :k] == 0) and np.all(got[:, k:] == -1)
        assert host(sel.lens)[0] == k * P + 1


def test_places_of_equal_scores(torch, dg):
    # two kinds of pages with equal scores within a kind: which places are taken shows in the table
    kv, D, P, n = 1, 64, 32, 40
    s = Setup(torch, dg, kv, D, P, [1], [n * P + 3], 6).fill()
    raw = all_bounds(s)
    for j in range(n):
        raw[s.table[0, j]] = raw[s.table[0, j % 2]]
    bounds, q = torch.from_numpy(raw).cuda(), queries(s, 3, "fp16")
    for take in (3, 11, 21, 22, 30, 40):
        sel = selection(torch, dg, 1, kv, take)
        dg.lw_kv_select(s.cache, s.batch, q, bounds, sel, 0, 0)
        _, want = L.select(raw, kv, D, P, s.n_pages, s.table, s.start, s.lens, host(q), 0, 0, take)
        assert np.array_equal(host(sel.table), want), take


def test_queries_that_are_special(torch, dg):
    """Zeros, NaN, infinities, the largest and smallest numbers, and heads 2^100 apart."""
    kv, group, D, P, n = 1, 6, 64, 32, 30
    s = Setup(torch, dg, kv, D, P, [8], [n * P + 8], 12).fill()
    raw = all_bounds(s)
    bounds = torch.from_numpy(raw).cuda()
    q = queries(s, group, "bf16")
    q[0].zero_()
    q[1, 2, 5] = float("nan")
    q[2, :, 1] = float("inf")
    q[3].mul_(2.0 ** 120)
    q[4].mul_(2.0 ** -120)
    q[5, 0].mul_(2.0 ** 100)
    q[6, :5].zero_()
    q[7, 0].fill_(127.0), q[7, 1].fill_(127.5), q[7, 2].fill_(2.0 ** -133)
    sel = selection(torch, dg, 8, kv, 7)
    dg.lw_kv_select(s.cache, s.batch, q, bounds, sel, 1, 1)
    _, want = L.select(raw, kv, D, P, s.n_pages, s.table, s.start, s.lens, host(q), 1, 1, 7)
    assert np.array_equal(host(sel.table), want)


def test_pages_that_are_not_finite_come_first_and_make_their_rows_nan(torch, dg):
    kv, group, D, P, n = 1, 2, 64, 32, 25
    s = Setup(torch, dg, kv, D, P, [1], [n * P + 1], 2).fill()
    image = s.image.reshape(s.n_pages, kv, -1)
    image[s.table[0, 17], 0, P * D:P * D + 2] = np.array([np.nan], np.float16).view(np.uint8)
    s.pages.copy_(torch.from_numpy(s.image))
    raw = all_bounds(s)
    bounds, q = torch.from_numpy(raw).cuda(), queries(s, group, "fp16")
    sel = selection(torch, dg, 1, kv, 4)
    dg.lw_kv_select(s.cache, s.batch, q, bounds, sel, 0, 0)
    _, want = L.select(raw, kv, D, P, s.n_pages, s.table, s.start, s.lens, host(q), 0, 0, 4)
    assert np.array_equal(host(sel.table), want) and s.table[0, 17] in host(sel.table)[0, 0]
    out = torch.zeros_like(q)
    dg.lw_kv_attend_selected(s.cache, sel, q, out)
    assert torch.isnan(out).all()


def test_absent_pages_and_rows_that_see_nothing(torch, dg):
    kv, group, D, P = 2, 2, 64, 32
    table = [[3, -1, 5, 99, 0, 7, -1, 1], [-1] * 8, [2, 4, -1, -1, -1, -1, -1, -1], [6, 2, 1, 0, 3, 4, 5, 7]]
    # the second sequence has no page at all, the third's own is absent, the fourth is shorter than its new tokens and
    # the fifth longer than the table
    s = Setup(torch, dg, kv, D, P, [2, 1, 1, 3, 1], [250, 200, 70, 2, 700], 3, table=table + [[1, 2, 3, 4, 5, 6, 7, 0]], n_pages=8).fill()
    raw = all_bounds(s)
    bounds, q = torch.from_numpy(raw).cuda(), queries(s, group, "fp16")
    for first, last, take in ((0, 0, 1), (1, 1, 4), (0, 5, 6), (3, 0, 20)):
        sel = selection(torch, dg, s.rows, kv, take)
        dg.lw_kv_select(s.cache, s.batch, q, bounds, sel, first, last)
        want_lens, want = L.select(raw, kv, D, P, s.n_pages, s.table, s.start, s.lens, host(q), first, last, take)
        assert np.array_equal(host(sel.lens), want_lens) and np.array_equal(host(sel.table), want)
        attend_over(torch, dg, s, sel, q, "fp16", "dense")


def test_no_sequences_select_nothing(torch, dg):
    kv, D, P = 1, 64, 32
    s = Setup(torch, dg, kv, D, P, [2], [100], 3).fill()
    empty = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
    b = dg.KvBatch(empty(1), empty(0), empty(0, 4))
    sel = selection(torch, dg, 3, kv, 2)
    bounds = torch.zeros((s.n_pages, L.bounds_bytes(kv, D)), dtype=torch.uint8, device="cuda")
    q = torch.zeros((3, 1, D), dtype=torch.float16, device="cuda")
    dg.lw_kv_select(s.cache, b, q, bounds, sel, 0, 0)
    out = torch.full_like(q, 3.0)
    dg.lw_kv_attend_selected(s.cache, sel, q, out)
    assert np.all(host(sel.table) == -1) and not host(sel.lens).any() and torch.all(out == 3)


def test_all_pages_taken_is_attention_over_all(torch, dg):
    """With as many pages as there are the call is lw_kv_attend's, up to the order of sums."""
    kv, group, D, P = 2, 4, 128, 32
    s = Setup(torch, dg, kv, D, P, [1, 3], [900, 400], 3).fill()
    bounds, q = torch.from_numpy(all_bounds(s)).cuda(), queries(s, group, "fp16")
    sel = selection(torch, dg, s.rows, kv, 29)
    dg.lw_kv_select(s.cache, s.batch, q, bounds, sel, 1, 1)
    a, b = torch.empty_like(q), torch.empty_like(q)
    la, lb = (torch.empty((s.rows, kv * group), device="cuda") for _ in range(2))
    dg.lw_kv_attend_selected(s.cache, sel, q, a, lse=la)
    dg.lw_kv_attend(s.cache, s.batch, q, b, lse=lb)
    # both are within half a step of fp16 of nearly the same number
    assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -10 * b.float().abs() + 2.0 ** -16)
    assert torch.all((la - lb).abs() <= 2.0 ** -18)


def test_pages_past_four_gigabytes(torch, dg):
    """Pages whose place in the cache passes 32 bits."""
    kv, group, D, P = 8, 2, 128, 64
    size = R.page_bytes(kv, D, P)
    far = (1 << 32) // size + 1000
    pages = torch.empty((far + 8) * size, dtype=torch.uint8, device="cuda")
    s = Setup(torch, dg, kv, D, P, [1], [5 * P + 7], 3, table=[[0, 1, 2, 3, 4, 5]], n_pages=6).fill()
    pages[far * size:(far + 6) * size].copy_(s.pages)
    big = dg.KvCache(pages, kv, D, P)
    table = torch.arange(far, far + 6, dtype=torch.int32, device="cuda").view(1, 6)
    b = dg.KvBatch(s.batch.start, s.batch.lens, table)
    each = L.bounds_bytes(kv, D)
    q, near, there = queries(s, group, "fp16"), torch.zeros((6, each), dtype=torch.uint8, device="cuda"), None
    there = torch.zeros((far + 8, each), dtype=torch.uint8, device="cuda")
    prompt = torch.tensor([0, 5 * P], dtype=torch.int32, device="cuda"), torch.tensor([5 * P], dtype=torch.int32, device="cuda")
    results = []
    for cache, batch, bounds in ((s.cache, s.batch, near), (big, b, there)):
        dg.lw_kv_bounds(cache, dg.KvBatch(*prompt, batch.table), 5 * P, bounds)
        sel = selection(torch, dg, 1, kv, 3)
        dg.lw_kv_select(cache, batch, q, bounds, sel, 0, 0)
        out, lse = torch.empty_like(q), torch.empty((1, kv * group), device="cuda")
        dg.lw_kv_attend_selected(cache, sel, q, out, lse=lse)
        w = torch.zeros((1, kv, 6), device="cuda")
        dg.lw_kv_weigh(cache, batch, q, lse, w)
        many = torch.zeros((1, kv, 6), device="cuda")
        rows = 40
        wide = dg.KvBatch(torch.tensor([0, rows], dtype=torch.int32, device="cuda"), batch.lens, batch.table)
        dg.lw_kv_weigh(cache, wide, q.expand(rows, -1, -1).contiguous(), lse.expand(rows, -1).contiguous(), many)
        results.append((sel.table, out, lse, w, many))
    assert torch.equal(near, there[far:far + 6])
    assert torch.equal(results[0][0] + far, results[1][0])
    for x, y in zip(results[0][1:], results[1][1:]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("args", [["--pages", "2"], ["--prompt", "97", "--steps", "5", "--batch", "3", "--pages", "1"],
                                  ["--prompt", "40", "--steps", "30", "--batch", "1", "--pages", "64"]])
def test_example_over_chosen_pages(torch, dg, args):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import cached_decode
    # fp16 outputs (2^-11 of each) of fp32 scores
    assert cached_decode.main(args) < 1e-3


@pytest.mark.parametrize("args", [["--prompt", "5", "--steps", "3", "--batch", "9", "--pages", "1"],
                                  ["--prompt", "97", "--steps", "3", "--pages", "2"]], ids=["pieces", "the last piece"])
def test_example_attends_over_all_pages_for_pieces_of_one_token(torch, dg, monkeypatch, args):
    """Pieces of the prompt have as many rows as a step there, and are none: pages are chosen in the step alone, once as it
    is and once as it is captured."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import cached_decode
    calls, select = [], dg.lw_kv_select
    monkeypatch.setattr(dg, "lw_kv_select", lambda *a, **kw: (calls.append(1), select(*a, **kw)))
    assert cached_decode.main(args) < 1e-3
    assert len(calls) == 2


def test_example_makes_no_bounds_that_nothing_reads(torch, dg, monkeypatch):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import cached_decode
    calls, bounds = [], dg.lw_kv_bounds
    monkeypatch.setattr(dg, "lw_kv_bounds", lambda *a, **kw: (calls.append(1), bounds(*a, **kw)))
    assert cached_decode.main(["--prompt", "33", "--steps", "2"]) < 1e-3
    assert not calls
    assert cached_decode.main(["--prompt", "33", "--steps", "2", "--pages", "1"]) < 1e-3
    assert len(calls) == 5 + 2                               # (pieces of 8 tokens, the step and its capture)


def test_bindings_refusals(torch, dg):
    kv, D, P = 2, 64, 32
    s = Setup(torch, dg, kv, D, P, [3], [100], 3)
    q = s.tensor(4, "fp16")
    bounds = torch.zeros(s.n_pages * L.bounds_bytes(kv, D), dtype=torch.uint8, device="cuda")
    good = selection(torch, dg, 3, kv, 3)
    for call in (lambda: dg.lw_kv_bounds(s.cache, s.batch, 3, bounds[:-16]),
                 lambda: dg.lw_kv_select(s.cache, s.batch, q, bounds[:-16], good),
                 lambda: dg.lw_kv_select(s.cache, s.batch, q, bounds, selection(torch, dg, 2, kv, 3)),
                 lambda: dg.lw_kv_select(s.cache, s.batch, q, bounds, selection(torch, dg, 3, 1, 3)),
                 lambda: dg.lw_kv_select(s.cache, s.batch, q[:, :3], bounds, good),
                 lambda: dg.lw_kv_select(s.cache, s.batch, q.float(), bounds, good),
                 lambda: dg.lw_kv_attend_selected(s.cache, good, q, q[:, :2]),
                 lambda: dg.lw_kv_attend_selected(s.cache, good, q, q.clone(), lse=torch.zeros((3, 3), device="cuda")),
                 lambda: dg.KvSelection(good.start[:-1], good.lens, good.table),
                 lambda: dg.KvSelection(good.start.long(), good.lens, good.table),
                 lambda: dg.KvSelection(good.start, good.lens, good.table[0])):
        with pytest.raises(dg.LwError):
            call()
