"""GPU: attention weights of pages and the pages given up, through the C ABI, and the operators around a long sequence
together.  Weights lie within bounds derived from the arithmetic (kv_long_ref.weigh) of those in fp64; what is given up is
equal to the reference's."""
import numpy as np
import pytest

import kv_long_ref as L
import kv_ref as R
from test_gpu_kv import Setup, host, say
from test_gpu_kv_select import all_bounds, queries, selection

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


WEIGHS = [
    # kv, group, D, P, new, lens, causal, window, dtype, how: few rows and many (more than 16 a sequence on average),
    # groups past a tile, pages larger than a block of tokens, several blocks, pages that end inside one
    (1, 1, 64, 32, [1], [1], True, 0, "fp16", "dense"), (2, 4, 128, 32, [1, 1, 0, 1], [500, 33, 64, 300], True, 0, "bf16", "fused"),
    (2, 8, 128, 64, [1, 2], [700, 130], True, 100, "fp16", "misaligned"), (1, 20, 64, 32, [1], [333], True, 0, "fp16", "dense"),
    (2, 1, 256, 128, [3, 1], [400, 129], True, 0, "bf16", "heads first"), (3, 2, 64, 256, [1, 1], [600, 255], False, 0, "fp16", "dense"),
    (1, 4, 64, 32, [70], [70], True, 0, "fp16", "dense"), (2, 3, 128, 64, [40, 1, 9], [300, 500, 9], True, 0, "bf16", "fused"),
    (1, 5, 128, 256, [33], [700], True, 90, "fp16", "misaligned"), (2, 2, 256, 64, [50, 30], [310, 30], True, 0, "bf16", "dense"),
    (1, 1, 64, 128, [300], [310], False, 0, "fp16", "dense"), (1, 2, 256, 256, [24, 17], [520, 257], False, 30, "fp16", "dense"),
    (1, 30, 64, 32, [2, 3], [200, 90], True, 0, "bf16", "heads first"),
]


@pytest.mark.parametrize("case", WEIGHS, ids=lambda c: f"kv{c[0]}x{c[1]}_D{c[2]}_P{c[3]}_n{sum(c[4])}_w{c[7]}_{c[8]}")
def test_weights(torch, dg, case):
    kv, group, D, P, new, lens, causal, window, dtype, how = case
    say("weigh", case)
    s = Setup(torch, dg, kv, D, P, new, lens, 23 + sum(new), before=1, after=2).fill()
    q = queries(s, group, dtype, how)
    scale = 1.3 * D ** -0.5
    out, lse = torch.empty((s.rows, kv * group, D), dtype=q.dtype, device="cuda"), torch.zeros((s.rows, kv * group), device="cuda")
    dg.lw_kv_attend(s.cache, s.batch, q, out, scale=scale, causal=causal, window=window, lse=lse)
    pages = s.table.shape[1]
    rng = np.random.default_rng(1)
    for stride, decay, aliased in ((pages, 1.0, False), (pages + 3, 0.75, True), (max(pages - 1, 1), 0.0, False)):
        w, used, err = L.weigh(R.Cache(s.image, kv, D, P), s.table, s.start, s.lens, host(q), host(lse), scale, causal, window, stride)
        before = rng.random((len(lens), kv, stride)).astype(np.float32) * 3
        weights = torch.from_numpy(before.copy() if aliased else np.full_like(before, 9.0)).cuda()
        prior = None if decay == 0.0 else weights if aliased else torch.from_numpy(before).cuda()
        dg.lw_kv_weigh(s.cache, s.batch, q, lse, weights, before=prior, decay=decay, scale=scale, causal=causal, window=window)
        got = host(weights)
        ref = w + decay * before
        mask = np.broadcast_to(used[:, None], got.shape)
        off, bound = np.abs(got - ref), err + 2.0 ** -22 * (ref + before)
        assert np.all(off[mask] <= bound[mask]), (stride, float((off - bound)[mask].max()))
        assert np.array_equal(got[~mask], (before if aliased else np.full_like(before, 9.0))[~mask])
        # the rows' weights are one a head
        if decay == 0.0 and stride >= pages:
            assert abs(got.sum() - sum(new) * kv * group) < 1e-3 * sum(new) * kv * group


@pytest.mark.parametrize("case", [
    # as many heads as there may be, row tiles that end inside a token, more blocks than the chip has wavefronts for, many
    # sequences of many rows, one with few among them
    (1, 1024, 64, 32, [1], [70], True, 0, "fp16", "dense"), (1, 70, 128, 64, [1, 2], [140, 70], True, 0, "bf16", "heads first"),
    (1000, 1, 64, 32, [1], [40], True, 0, "bf16", "dense"), (300, 1, 64, 32, [20], [100], True, 0, "bf16", "dense"),
    (32, 1, 64, 32, [40], [6000], True, 0, "fp16", "dense"), (16, 2, 128, 256, [33], [5000], True, 3000, "bf16", "fused"),
    (2, 4, 64, 32, [9] * 30 + [0, 60, 1], [40] * 30 + [5, 400, 333], True, 25, "fp16", "misaligned"),
    (8, 2, 256, 64, [40], [2500], False, 0, "bf16", "dense")],
    ids=["group1024", "group70", "kv1000", "kv300", "kv32_long", "P256_long", "mixed", "D256_long"])
def test_weights_at_the_ends_of_the_ranges(torch, dg, case):
    test_weights(torch, dg, case)


@pytest.mark.parametrize("new", [[1, 1], [30, 30]], ids=["few", "many"])
def test_weights_of_absent_pages_and_rows_without_a_log_sum(torch, dg, new):
    kv, group, D, P = 1, 2, 64, 32
    table = [[0, -1, 2, 99, 4, 5], [-1, -1, -1, -1, -1, -1]]
    s = Setup(torch, dg, kv, D, P, new, [190, 150], 3, table=table, n_pages=6).fill()
    image = s.image.reshape(6, kv, -1)
    # behind the sequence's last token, and where no page is looked at, anything may lie
    image[5, 0, P * D + 4 * 30:P * D + 4 * 32] = np.array([np.nan] * 4, np.float16).view(np.uint8)
    image[1:4:2] = 0xFF
    s.pages.copy_(torch.from_numpy(s.image))
    q = queries(s, group, "fp16")
    out, lse = torch.empty_like(q), torch.zeros((s.rows, kv * group), device="cuda")
    dg.lw_kv_attend(s.cache, s.batch, q, out, lse=lse)
    assert torch.isinf(lse[new[0]:]).all()
    for value in (None, float("nan"), float("inf"), -float("inf")):
        if value is not None:
            lse[0, 1] = value
        w, used, err = L.weigh(R.Cache(s.image, kv, D, P), s.table, s.start, s.lens, host(q), host(lse), D ** -0.5, True, 0, 6)
        weights = torch.full((2, kv, 6), 9.0, device="cuda")
        dg.lw_kv_weigh(s.cache, s.batch, q, lse, weights)
        got = host(weights)
        assert np.all(np.abs(got - w)[used[:, None]] <= err[used[:, None]])
        assert not got[0, 0, [1, 3]].any() and not got[1, 0, :5].any() and got[1, 0, 5] == 9


def test_weights_are_the_same_again(torch, dg):
    for new in ([1, 1, 1], [33, 40, 50]):
        s = Setup(torch, dg, 2, 128, 64, new, [900, 400, 77], 3).fill()
        q = queries(s, 4, "bf16")
        out, lse = torch.empty_like(q), torch.empty((s.rows, 8), device="cuda")
        dg.lw_kv_attend(s.cache, s.batch, q, out, lse=lse)
        got = []
        for _ in range(3):
            w = torch.zeros((3, 2, s.table.shape[1]), device="cuda")
            dg.lw_kv_weigh(s.cache, s.batch, q, lse, w)
            got.append(w)
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_weights_of_many_sequences(torch, dg):
    """More than a wavefront looks at in a step, most of one page, some without new tokens."""
    n = 150
    rng = np.random.default_rng(4)
    new = [int(rng.integers(0, 2)) for _ in range(n)]
    new[0] = new[149] = 1
    lens = [int(rng.integers(max(x, 0), 100)) + x for x in new]
    for times in (1, 40):
        s = Setup(torch, dg, 2, 64, 32, [x * times for x in new], [x + 40 * times for x in lens], 3).fill()
        q = queries(s, 1, "fp16")
        out, lse = torch.empty_like(q), torch.empty((s.rows, 2), device="cuda")
        dg.lw_kv_attend(s.cache, s.batch, q, out, lse=lse)
        pages = s.table.shape[1]
        w, used, err = L.weigh(R.Cache(s.image, 2, 64, 32), s.table, s.start, s.lens, host(q), host(lse), 64 ** -0.5, True, 0, pages)
        weights = torch.full((n, 2, pages), 9.0, device="cuda")
        dg.lw_kv_weigh(s.cache, s.batch, q, lse, weights)
        got, mask = host(weights), np.broadcast_to(used[:, None], w.shape)
        assert np.all(np.abs(got - w)[mask] <= err[mask]) and np.all(got[~mask] == 9)


# ------------------------------------------------------------------ giving up

def give_up(torch, dg, kv, P, table, lens, weights, n_pages, keep, first, last, in_place=False):
    pages = torch.empty(n_pages * R.page_bytes(kv, 64, P), dtype=torch.uint8, device="cuda")
    cache = dg.KvCache(pages, kv, 64, P)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    lens = np.asarray(lens, np.int32)
    b = dg.KvBatch(torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda"), dev(lens), dev(table))
    left = b.table if in_place else torch.full_like(b.table, -9)
    gone, count = torch.full_like(b.table, -9), torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    dg.lw_kv_evict(cache, b, dev(weights), keep, left, gone, count, first=first, last=last)
    want = L.evict(table, lens, weights, P, n_pages, keep, first, last)
    assert np.array_equal(host(left), want[0]) and np.array_equal(host(gone), want[1]) and np.array_equal(host(count), want[2])
    if not in_place:
        assert np.array_equal(host(b.table), table)


@pytest.mark.parametrize("seed", range(6))
def test_pages_given_up(torch, dg, seed):
    rng = np.random.default_rng(seed)
    kv, P, n, stride = int(rng.integers(1, 9)), int(rng.choice([32, 64, 128, 256])), int(rng.integers(1, 7)), int(rng.integers(1, 90))
    n_pages = 2 * stride
    table = rng.integers(0, n_pages, (n, stride)).astype(np.int32)
    table[rng.random((n, stride)) < 0.2] = -1
    table[0, 0] = n_pages + 5
    lens = rng.integers(0, (stride + 3) * P, n)
    weights = np.exp(rng.standard_normal((n, kv, stride)) * 3).astype(np.float32)
    weights[rng.random(weights.shape) < 0.3] = 1.0                 # (equal sums, where kv is 1)
    for keep in (0, 1, stride // 3, stride, 10 ** 12):
        for first, last in ((0, 1), (2, 3), (stride, 1), (0, stride + 5)):
            for in_place in (False, True):
                say("evict", seed, keep, first, last)
                give_up(torch, dg, kv, P, table, lens, weights, n_pages, keep, first, last, in_place)


def test_weights_that_are_special(torch, dg):
    w = np.array([[[3.0, np.nan, -np.inf, 0.0, -0.0, np.inf, 1e-45, -1.0, 3e38, -np.nan, 5.0, 2.0]]], np.float32)
    table = np.arange(12, dtype=np.int32)[None]
    for keep in range(12):
        give_up(torch, dg, 1, 32, table, [12 * 32], w, 12, keep, 0, 1)
        give_up(torch, dg, 2, 32, table, [12 * 32], np.repeat(w, 2, 1)[:, :, :9].copy(), 12, keep, 1, 1)      # fewer weights than pages
    # heads' sums in 64 bits: 2^30 + 1 - 2^30 is 1
    w = np.zeros((1, 3, 4), np.float32)
    w[0, :, 0], w[0, :, 1], w[0, :, 2] = (2.0 ** 30, 1.0, -2.0 ** 30), (0.5, 0, 0), (1.5, 0, 0)
    give_up(torch, dg, 3, 32, table[:, :4], [4 * 32], w, 12, 3, 0, 1)


@pytest.mark.parametrize("new", [[2], [50]], ids=["few", "many"])
@pytest.mark.parametrize("D,power", [(64, 60), (128, -60), (128, 100), (256, -100), (64, 45), (256, 38)])
def test_weights_of_queries_and_scales_far_from_one(torch, dg, new, D, power):
    """Products that leave fp32's range unless a power of two goes from the queries to the scale or back; among them rows of
    other sizes, whose scores are all but nothing, and rows of zeros."""
    kv, group, P = 1, 3, 64
    s = Setup(torch, dg, kv, D, P, new, [200], 11).fill()
    q = queries(s, group, "bf16") * 2.0 ** power
    q[0, 1] *= 2.0 ** -70 if power > 0 else 2.0 ** -20
    q[new[0] // 2, 0] = 0
    q[-1, 2] *= 2.0 ** -30
    scale = 1.3 * D ** -0.5 * 2.0 ** -power
    out, lse = torch.empty_like(q), torch.empty((s.rows, kv * group), device="cuda")
    dg.lw_kv_attend(s.cache, s.batch, q, out, scale=scale, lse=lse)
    weights = torch.full((1, kv, s.table.shape[1]), 9.0, device="cuda")
    dg.lw_kv_weigh(s.cache, s.batch, q, lse, weights, scale=scale)
    w, used, err = L.weigh(R.Cache(s.image, kv, D, P), s.table, s.start, s.lens, host(q), host(lse), scale, True, 0, weights.shape[2])
    got = host(weights)
    assert np.all(np.abs(got - w)[used[:, None]] <= err[used[:, None]] + 2.0 ** -22 * w[used[:, None]])
    assert abs(got[0, 0][used[0]].sum() - new[0] * group) < 1e-3 * new[0] * group


@pytest.mark.parametrize("new", [[1], [30]], ids=["few", "many"])
def test_weights_of_half_precision_queries_under_a_small_scale(torch, dg, new):
    """Scores of all but nothing: every token that a row sees has the same weight."""
    s = Setup(torch, dg, 2, 128, 64, new, [180], 5).fill()
    q = queries(s, 2, "fp16")
    q[0, 0] = 65504
    q[-1, 3] = 0
    n = new[0]
    lse = torch.log(torch.arange(180 - n + 1, 181, device="cuda").float())[:, None].expand(n, 4).contiguous()
    weights = torch.empty((1, 2, 3), device="cuda")
    dg.lw_kv_weigh(s.cache, s.batch, q, lse, weights, scale=2.0 ** -70)
    seen = np.arange(180 - n + 1, 181)
    want = [2 * (np.clip(seen - 64 * j, 0, 64) / seen).sum() for j in range(3)]
    assert np.allclose(host(weights)[0], [want, want], rtol=2.0 ** -16, atol=0)


def test_equal_weights_give_up_the_first(torch, dg):
    n = 3000
    table = np.random.default_rng(2).permutation(n).astype(np.int32)[None]
    for keep in (0, 1, 1500, 2998, 2999):
        give_up(torch, dg, 2, 32, table, [n * 32 - 5], np.full((1, 2, n), 0.25, np.float32), n, keep, 0, 1)


def test_the_longest_table(torch, dg):
    n = 32768
    rng = np.random.default_rng(2)
    table = rng.permutation(n).astype(np.int32)[None]
    give_up(torch, dg, 1, 32, table, [n * 32], rng.random((1, 1, n)).astype(np.float32), n, 10000, 1, 2)


def test_as_many_sequences_as_there_may_be(torch, dg):
    """2^22 sequences of tables past 1024 pages: more threads than a launch takes along one dimension.  Pages without a
    weight are equal: the first go."""
    n, wide, keep = 1 << 22, 1025, 600
    cache = dg.KvCache(torch.empty(wide * R.page_bytes(1, 64, 32), dtype=torch.uint8, device="cuda"), 1, 64, 32)
    table = torch.arange(wide, dtype=torch.int32, device="cuda").repeat(n, 1)
    used = torch.arange(n, dtype=torch.int32, device="cuda") % 1000 + 2
    b = dg.KvBatch(torch.zeros(n + 1, dtype=torch.int32, device="cuda"), used * 32 - 5, table)
    gone, count = torch.full_like(table, -9), torch.full((n,), -9, dtype=torch.int32, device="cuda")
    dg.lw_kv_evict(cache, b, torch.empty((n, 1, 0), device="cuda"), keep, table, gone, count)
    drop = (used - keep).clamp(min=0).minimum(used - 2)
    assert torch.equal(count, drop)
    j = torch.arange(wide, dtype=torch.int32, device="cuda")
    for i in range(0, n, 1 << 18):
        d = drop[i:i + (1 << 18), None]
        assert torch.equal(table[i:i + (1 << 18)], torch.where((j >= 1) & (j <= d), -1, j))
        assert torch.equal(gone[i:i + (1 << 18)], torch.where(j < d, j + 1, -1))


def test_a_long_table_in_a_graph(torch, dg):
    """More shared memory than a kernel has without asking for it, asked for while a graph is captured."""
    n = 20000
    rng = np.random.default_rng(3)
    cache = dg.KvCache(torch.empty(n * R.page_bytes(1, 64, 32), dtype=torch.uint8, device="cuda"), 1, 64, 32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    table, lens = rng.permutation(n).astype(np.int32)[None], np.array([n * 32], np.int32)
    b = dg.KvBatch(torch.zeros(2, dtype=torch.int32, device="cuda"), dev(lens), dev(table))
    weights = torch.zeros((1, 1, n), device="cuda")
    left, gone, count = torch.empty_like(b.table), torch.empty_like(b.table), torch.empty_like(b.lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.lw_kv_evict(cache, b, weights, 12000, left, gone, count)
    for seed in range(3):
        w = np.random.default_rng(seed).random((1, 1, n)).astype(np.float32)
        weights.copy_(torch.from_numpy(w))
        graph.replay()
        want = L.evict(table, lens, w, 32, n, 12000, 1, 1)
        assert np.array_equal(host(left), want[0]) and np.array_equal(host(gone), want[1]) and np.array_equal(host(count), want[2])


def test_log_sums_past_the_largest_power_of_two(torch, dg):
    """3e38 is a number, its logarithm to base two is not one here: the row adds nothing, and no NaN."""
    for rows in (1, 40):
        s = Setup(torch, dg, 1, 64, 32, [rows], [100], 3).fill()
        q, w = queries(s, 2, "bf16"), torch.zeros((1, 1, 4), device="cuda")
        lse = torch.full((rows, 2), 3e38, device="cuda")
        dg.lw_kv_weigh(s.cache, s.batch, q, lse, w)
        assert not host(w).any()


def rounded_logs(far):
    """Eight log sums from `far` on, and what fp32 rounds off their products with the logarithm of e, of either sign."""
    l = [np.float32(far)]
    while len(l) < 8:
        l.append(np.nextafter(l[-1], np.float32(np.inf)))
    l, e = np.array(l), np.float32(1.44269504088896341)
    rest = l.astype(np.float64) * float(e) - (l * e).astype(np.float64)
    assert (rest > 0).any() and (rest < 0).any()
    return l


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 40], ids=["few", "many"])
@pytest.mark.parametrize("far", [7e4, 3e9, 1e10, 1e12, 1e20, 1e30])
def test_log_sums_far_above_and_below_the_scores(torch, dg, rows, far, D):
    """Ordinary scores are nothing beside the one, and past fp32 beside the other: 0 and infinity, no NaN; rows beside such
    a one keep what they give."""
    kv, group, P = 1, 8, 32
    s = Setup(torch, dg, kv, D, P, [rows], [100], 3).fill()
    q, w = queries(s, group, "bf16"), torch.zeros((1, kv, 4), device="cuda")
    logs = torch.from_numpy(rounded_logs(far)).cuda().expand(rows, group).contiguous()
    dg.lw_kv_weigh(s.cache, s.batch, q, logs, w)
    assert np.array_equal(host(w), np.zeros((1, kv, 4)))
    dg.lw_kv_weigh(s.cache, s.batch, q, -logs, w)
    assert np.all(np.isposinf(host(w)[0, 0]))
    out, lse = torch.empty_like(q), torch.empty((rows, group), device="cuda")
    dg.lw_kv_attend(s.cache, s.batch, q, out, lse=lse)
    lse[0, ::2] = logs[0, ::2]
    dg.lw_kv_weigh(s.cache, s.batch, q, lse, w)
    want, used, err = L.weigh(R.Cache(s.image, kv, D, P), s.table, s.start, s.lens, host(q), host(lse), D ** -0.5, True, 0, 4)
    assert used.all() and np.all(np.abs(host(w) - want) <= err)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 40], ids=["few", "many"])
@pytest.mark.parametrize("power", [17, 20, 24, 28])
def test_log_sums_beside_scores_as_large(torch, dg, rows, power, D):
    """Scores of 2^power, exactly, under log sums a step above and below: exp of the difference.  Off by an exponential's
    last place, by 2^-25 of the difference (up to 2^5) for the logarithm of e in fp32, and by the additions (kv_long_ref.weigh)."""
    kv, group, P = 1, 4, 32
    s = Setup(torch, dg, kv, D, P, [rows], [100], 3).fill()
    image = s.image.reshape(s.n_pages, kv, -1)
    image[:, :, P * D:P * (D + 4)] = np.tile(np.array([0.0, -1.0], np.float16).view(np.uint8), P)          # keys of ones
    s.pages.copy_(torch.from_numpy(s.image))
    q = torch.zeros((rows, group, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 5] = 2.0 ** power
    one = np.float32(2.0 ** power)
    logs = np.array([one, np.nextafter(one, np.float32(np.inf)), np.nextafter(one, np.float32(0)), one], np.float32)
    w = torch.zeros((1, kv, 4), device="cuda")
    dg.lw_kv_weigh(s.cache, s.batch, q, torch.from_numpy(logs).cuda().expand(rows, group).contiguous(), w, scale=1.0)
    seen = np.arange(100 - rows + 1, 101)
    tokens = np.array([np.clip(seen - P * j, 0, P).sum() for j in range(4)])
    want = tokens * np.exp(2.0 ** power - logs.astype(np.float64)).sum()
    chain = (rows * group + 16) * (P // 16 + 1) // 4 + 64
    assert np.all(np.abs(host(w)[0, 0] - want) <= want * (chain * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22))


def test_log_sums_up_to_the_largest_power_of_two_count(torch, dg):
    """2^127 is the last that does, on either side of zero; what lies past it adds nothing, also where its product with the
    logarithm of e is still a number."""
    past = float(np.nextafter(np.float32(2.0 ** 127), np.float32(np.inf)))
    for rows in (1, 40):
        s = Setup(torch, dg, 1, 64, 32, [rows], [100], 3).fill()
        q, w = queries(s, 2, "bf16"), torch.zeros((1, 1, 4), device="cuda")
        for value, want in ((2.0 ** 127, 0.0), (-2.0 ** 127, np.inf), (-past, 0.0), (past, 0.0), (-2.3e38, 0.0), (-3e38, 0.0)):
            dg.lw_kv_weigh(s.cache, s.batch, q, torch.full((rows, 2), value, device="cuda"), w)
            assert np.array_equal(host(w), np.full((1, 1, 4), want)), (rows, value)


def test_refusals_of_the_binding(torch, dg):
    kv, D, P = 2, 64, 32
    s = Setup(torch, dg, kv, D, P, [3], [100], 3)
    q, lse, w = s.tensor(4, "fp16"), torch.zeros((3, 4), device="cuda"), torch.zeros((1, kv, 4), device="cuda")
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
    for call in (lambda: dg.lw_kv_weigh(s.cache, s.batch, q, lse[:2], w), lambda: dg.lw_kv_weigh(s.cache, s.batch, q, lse, w[0]),
                 lambda: dg.lw_kv_weigh(s.cache, s.batch, q, lse, w.double()), lambda: dg.lw_kv_weigh(s.cache, s.batch, q, lse, w[:, :1].contiguous()),
                 lambda: dg.lw_kv_weigh(s.cache, s.batch, q, lse, w, before=w[:, :, :2].contiguous()),
                 lambda: dg.lw_kv_evict(s.cache, s.batch, w, 2, ints(1, 3), ints(1, 4), ints(1)),
                 lambda: dg.lw_kv_evict(s.cache, s.batch, w, 2, ints(1, 4), ints(1, 5), ints(1)),
                 lambda: dg.lw_kv_evict(s.cache, s.batch, w, 2, ints(1, 4), ints(1, 4), ints(2)),
                 lambda: dg.lw_kv_evict(s.cache, s.batch, w, 2, ints(1, 4).long(), ints(1, 4), ints(1))):
        with pytest.raises(dg.LwError):
            call()


# ------------------------------------------------------------------ together

class Loop:
    """A few sequences served token by token over a cache with a budget of pages: positions, append, bounds, a choice of
    pages, attention over it, and every few steps the weights that attention over everything gives, and pages given up."""

    def __init__(self, torch, dg, n=3, longest=400, take=4):
        self.torch, self.dg, self.n, self.take = torch, dg, n, take
        self.kv, self.group, self.D, self.P = 2, 3, 64, 32
        self.heads, wide = self.kv * self.group, -(-longest // self.P)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        rng = np.random.default_rng(11)
        pages = torch.zeros(n * wide * R.page_bytes(self.kv, self.D, self.P), dtype=torch.uint8, device="cuda")
        self.cache = dg.KvCache(pages, self.kv, self.D, self.P)
        self.table, self.lens = dev(rng.permutation(n * wide).reshape(n, wide).astype(np.int32)), dev(np.zeros(n, np.int32))
        self.bounds = torch.zeros((n * wide, dg.lw_kv_bounds_bytes(self.kv, self.D)), dtype=torch.uint8, device="cuda")
        self.weights = torch.zeros((n, self.kv, wide), device="cuda")
        self.gone, self.count = torch.zeros_like(self.table), torch.zeros_like(self.lens)
        self.plan = dg.lw_rope_make(self.D // 2, scaling=dg.LW_ROPE_LINEAR, factor=4.0)
        self.keep = {}

    def batch(self, new):
        start = self.torch.arange(0, (self.n + 1) * new, new, dtype=self.torch.int32, device="cuda")
        return self.dg.KvBatch(start, self.lens, self.table)

    def step(self, x, b, keep, sparse):
        """x [rows][heads + 2 kv][D], what a projection gives; lens count these tokens."""
        torch, dg, rows = self.torch, self.dg, x.shape[0]
        get = lambda name, *shape, dtype=torch.float16: keep.setdefault(name, torch.empty(shape, dtype=dtype, device="cuda"))
        qk = get("qk", rows, self.heads + self.kv, self.D)
        dg.lw_rope(self.plan, x[:, :self.heads + self.kv], qk, batch=b)
        q, k = qk[:, :self.heads], qk[:, self.heads:]
        dg.lw_kv_append(self.cache, b, k, x[:, self.heads + self.kv:].half() if x.dtype != torch.float16 else x[:, self.heads + self.kv:])
        dg.lw_kv_bounds(self.cache, b, rows, self.bounds)
        out, lse = get("out", rows, self.heads, self.D), get("lse", rows, self.heads, dtype=torch.float32)
        if sparse:
            if "sel" not in keep:
                i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")
                keep["sel"] = dg.KvSelection(i32(rows + 1), i32(rows), i32(rows, self.kv, self.take))
            dg.lw_kv_select(self.cache, b, q, self.bounds, keep["sel"])
            dg.lw_kv_attend_selected(self.cache, keep["sel"], q, out, lse=lse)
        else:
            dg.lw_kv_attend(self.cache, b, q, out, lse=lse)
            dg.lw_kv_weigh(self.cache, b, q, lse, self.weights, before=self.weights, decay=0.9)
        return q, out, lse


def test_served_together(torch, dg):
    m = Loop(torch, dg)
    rng = np.random.default_rng(8)
    turn = L.turns(m.D // 2, 10000.0, "linear", 4.0)
    new_x = lambda rows: torch.from_numpy(rng.standard_normal((rows, m.heads + 2 * m.kv, m.D)).astype(np.float32)).cuda()
    done = 0
    for at, (new, sparse) in enumerate([(130, False), (1, False), (1, True), (61, True), (1, True), (5, False), (1, True)]):
        m.lens.add_(new)
        x, keep = new_x(m.n * new), {}
        b = m.batch(new)
        table = host(m.table).copy()
        before = host(m.weights).astype(np.float64)
        q, out, lse = m.step(x, b, keep, sparse)
        say("step", at, new, sparse)
        image = host(m.cache.pages)
        cache, start, lens = R.Cache(image, m.kv, m.D, m.P), host(b.start), host(m.lens)
        pos = np.repeat(lens - new, new) + np.tile(np.arange(new), m.n)
        # queries: turned and rounded once (test_gpu_rope has the bounds; here half a step and a little)
        ref = L.rope(host(x)[:, :m.heads], pos, turn, True)
        assert np.all(np.abs(host(q) - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -18)
        if sparse:
            raw = host(m.bounds)
            want_lens, want = L.select(raw, m.kv, m.D, m.P, len(raw), table, start, lens, host(q), 1, 1, m.take)
            assert np.array_equal(host(keep["sel"].table), want) and np.array_equal(host(keep["sel"].lens), want_lens)
            for g in range(m.kv):
                one = R.Cache(np.ascontiguousarray(image.reshape(len(raw), m.kv, -1)[:, g]), 1, m.D, m.P)
                mine = slice(g * m.group, (g + 1) * m.group)
                o, l, by = R.attend(one, want[:, g], np.arange(len(want) + 1), want_lens, host(q)[:, mine], m.D ** -0.5)
                err, err_l = R.bounds(o, l, by, m.D, False)
                assert np.all(np.abs(host(out)[:, mine] - o) <= err) and np.all(np.abs(host(lse)[:, mine] - l) <= err_l)
        else:
            w, used, err = L.weigh(cache, table, start, lens, host(q), host(lse), m.D ** -0.5, True, 0, table.shape[1])
            present = (table >= 0)[:, None]
            ref = np.where(present, w + np.float64(np.float32(0.9)) * before, 0)
            mask = np.broadcast_to(used[:, None], w.shape)
            assert np.all(np.abs(host(m.weights) - ref)[mask] <= (err + 2.0 ** -22 * (ref + before))[mask])
            weights, keep_pages = host(m.weights), 6
            dg.lw_kv_evict(m.cache, b, m.weights, keep_pages, m.table, m.gone, m.count, first=1, last=2)
            want = L.evict(table, lens, weights, m.P, m.cache.n_pages, keep_pages, 1, 2)
            assert np.array_equal(host(m.table), want[0]) and np.array_equal(host(m.gone), want[1]) and np.array_equal(host(m.count), want[2])
        done += new
        for s in range(m.n):                                       # every full page that is there has its bounds
            for j in range(done // m.P):
                p = host(m.table)[s, j]
                if p >= 0 and at in (0, 3):
                    check = np.zeros((1, host(m.bounds).shape[1]), np.uint8)
                    hi, lo, es = L.page_bounds(cache, p)
                    L.put_bounds(check, m.kv, m.D, 0, (hi, lo, es))
                    assert np.array_equal(host(m.bounds)[p], check[0])
    assert host(m.count).max() >= 0 and (host(m.table)[:, :done // m.P] < 0).any()


@pytest.mark.parametrize("sparse", [True, False])
def test_captured_steps_follow_the_batch(torch, dg, sparse):
    """The same steps eager and replayed from a graph, which has to follow lens, table and what the buffers hold."""
    results = []
    for graphed in (False, True):
        m = Loop(torch, dg)
        rng = np.random.default_rng(8)
        first = torch.from_numpy(rng.standard_normal((m.n * 94, m.heads + 2 * m.kv, m.D)).astype(np.float32)).cuda()
        m.lens.add_(94)
        m.step(first, m.batch(94), {}, False)
        x, keep, b, got = torch.empty((m.n, m.heads + 2 * m.kv, m.D), device="cuda"), {}, m.batch(1), []
        steps = [torch.from_numpy(rng.standard_normal(x.shape).astype(np.float32)).cuda() for _ in range(8)]

        def one():
            _, out, lse = m.step(x, b, keep, sparse)
            if not sparse:
                dg.lw_kv_evict(m.cache, b, m.weights, 3, m.table, m.gone, m.count)
            return out, lse

        graph = None
        for i, values in enumerate(steps):
            x.copy_(values)
            m.lens.add_(1)
            if graphed and i == 1:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    out, lse = one()
            if graph is not None:
                graph.replay()
            else:
                out, lse = one()
            torch.cuda.synchronize()
            got += [out.clone(), lse.clone(), m.table.clone(), m.bounds.clone(), m.weights.clone(), m.gone.clone()]
        results.append(got)
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.equal(a, b), i


def test_on_a_stream_of_its_own(torch, dg):
    s = Setup(torch, dg, 2, 64, 32, [1, 1], [500, 300], 3).fill()
    bounds, q = torch.from_numpy(all_bounds(s)).cuda(), queries(s, 2, "fp16")

    def run(stream):
        sel, out, lse = selection(torch, dg, 2, 2, 4), torch.empty_like(q), torch.empty((2, 4), device="cuda")
        w, y = torch.zeros((2, 2, s.table.shape[1]), device="cuda"), torch.empty_like(q)
        left, gone, count = torch.empty_like(s.batch.table), torch.empty_like(s.batch.table), torch.empty_like(s.batch.lens)
        torch.cuda.synchronize()
        dg.lw_rope(dg.lw_rope_make(32), q, y, batch=s.batch, stream=stream)
        dg.lw_kv_bounds(s.cache, s.batch, 2, bounds, stream=stream)
        dg.lw_kv_select(s.cache, s.batch, y, bounds, sel, stream=stream)
        dg.lw_kv_attend_selected(s.cache, sel, y, out, lse=lse, stream=stream)
        dg.lw_kv_weigh(s.cache, s.batch, y, lse, w, stream=stream)
        dg.lw_kv_evict(s.cache, s.batch, w, 5, left, gone, count, stream=stream)
        torch.cuda.synchronize()
        return y, sel.table, out, lse, w, left, gone, count

    for a, b in zip(run(None), run(torch.cuda.Stream())):
        assert torch.equal(a, b)
