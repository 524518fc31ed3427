"""GPU: rotary positions through the C ABI against the formula in fp64 (kv_long_ref.rope)."""
import numpy as np
import pytest

import kv_long_ref as L
from test_gpu_kv import TYPES, host, say

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


HALF = dict(fp16=2.0 ** -11, bf16=2.0 ** -8, fp32=2.0 ** -24)      # half a step, relative
TINY = dict(fp16=2.0 ** -25, bf16=0.0, fp32=0.0)                   # and among fp16's subnormal numbers


def tensor(torch, n, heads, dim, dtype, how, values=None):
    kind = getattr(torch, TYPES[dtype])
    if how == "fused":
        t = torch.full((n, heads + 3, dim), 7.0, dtype=kind, device="cuda")[:, 1:1 + heads]
    elif how == "heads first":
        t = torch.full((heads, n, dim), 7.0, dtype=kind, device="cuda").transpose(0, 1)
    elif how == "misaligned":
        flat = torch.full((1 + n * (heads * (dim + 1) + 5) + dim,), 7.0, dtype=kind, device="cuda")
        t = flat[1:].as_strided((n, heads, dim), (heads * (dim + 1) + 5, dim + 1, 1))
    else:
        t = torch.full((n, heads, dim), 7.0, dtype=kind, device="cuda")
    if values is not None:
        t.copy_(torch.from_numpy(values).cuda())
    return t


def check(got, x, pos, turn, halves, g, dtype):
    """A sine or cosine is off by at most 4 * 2^-24: the angle's 32 bits of a turn and its two roundings at up to pi/4,
    the sums' last three roundings, g's.  Two products, of which one is rounded, and their sum: 2^-23 more."""
    ref = L.rope(x, pos, turn, halves, g)
    n = len(turn)
    size = np.zeros_like(ref)
    for i in range(n):
        u, v = (i, i + n) if halves else (2 * i, 2 * i + 1)
        size[..., u] = size[..., v] = abs(g) * (np.abs(x[..., u]) + np.abs(x[..., v]))
    err = size * (2.0 ** -22 + 2.0 ** -23)
    bound = err * (1 + HALF[dtype]) + HALF[dtype] * np.abs(ref) + TINY[dtype]
    off = np.abs(got.astype(np.float64) - ref)
    assert np.all(off <= bound), (float(off.max()), float((off - bound).max()))


SHAPES = [
    # dim, pairs, heads, rows: whole heads, parts, odd numbers of pairs, more than a wavefront's 64 units, one of each
    (128, 64, 8, 5), (64, 32, 3, 70), (256, 128, 1, 2), (128, 32, 9, 3), (96, 24, 5, 4), (80, 40, 2, 3), (66, 33, 7, 5),
    (64, 1, 2, 3), (2, 1, 1, 1), (512, 256, 2, 2), (515, 256, 2, 2), (1024, 100, 1, 3), (77, 7, 70, 2), (8, 4, 40, 3),
    (1024, 256, 2, 2),
]


@pytest.mark.parametrize("halves", [True, False], ids=["halves", "pairs"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes_and_types(torch, dg, shape, halves):
    dim, pairs, heads, rows = shape
    rng = np.random.default_rng(sum(shape))
    turn = L.turns(pairs, 10000.0)
    plan = dg.lw_rope_make(pairs, dg.LW_ROPE_HALVES if halves else dg.LW_ROPE_PAIRS)
    pos = rng.integers(0, 200000, rows).astype(np.int32)
    dpos = torch.from_numpy(pos).cuda()
    for xt in TYPES:
        for yt in TYPES:
            for how in ("dense", "fused", "heads first", "misaligned"):
                say("rope", shape, halves, xt, yt, how)
                x = tensor(torch, rows, heads, dim, xt, how, rng.standard_normal((rows, heads, dim)).astype(np.float32) * 3)
                y = tensor(torch, rows, heads, dim, yt, "dense" if how == "heads first" else how)
                dg.lw_rope(plan, x, y, pos=dpos)
                check(host(y), host(x), pos, turn, halves, 1.0, yt)


@pytest.mark.parametrize("scaling,kw", [
    ("linear", dict(base=500000.0, factor=8.0)), ("base", dict(base=10000.0, factor=4.0)),
    ("index", dict(base=10000.0, factor=16.0, original=4096.0, low=1.0, high=32.0)),
    ("turns", dict(base=500000.0, factor=8.0, original=8192.0, low=1.0, high=4.0))])
def test_scalings_far_positions_and_amplitude(torch, dg, scaling, kw):
    rng = np.random.default_rng(5)
    number = dict(linear=1, base=2, index=3, turns=4)[scaling]
    pos = np.array([0, 1, -1, 4095, 131071, -131072, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 1000003], np.int32)
    for g in (1.0, 1.2772588729858398, -0.5):
        plan = dg.lw_rope_make(48, dg.LW_ROPE_HALVES, scaling=number, amplitude=g, **kw)
        x = tensor(torch, len(pos), 3, 128, "fp32", "dense", rng.standard_normal((len(pos), 3, 128)).astype(np.float32))
        y = torch.empty_like(x)
        dg.lw_rope(plan, x, y, pos=torch.from_numpy(pos).cuda())
        say("scaling", scaling, g)
        check(host(y), host(x), pos, L.turns(48, scaling=scaling, **kw), True, float(np.float32(g)), "fp32")


def batch(torch, dg, start, lens):
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    return dg.KvBatch(dev(start), dev(lens), torch.zeros((len(lens), 1), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dim,pairs", [(128, 64), (66, 20)])
def test_positions_of_a_batch(torch, dg, dim, pairs):
    # rows before and after the sequences, empty ones, one with more new tokens than it is long (negative positions)
    start, lens = [2, 5, 5, 6, 13], [1000, 7, 2 ** 31 - 1, 4]
    rows, rng = 15, np.random.default_rng(3)
    pos = np.zeros(rows, np.int64)
    for s in range(len(lens)):
        for i in range(start[s], start[s + 1]):
            pos[i] = lens[s] - start[s + 1] + i
    plan, b = dg.lw_rope_make(pairs), batch(torch, dg, start, lens)
    x = tensor(torch, rows, 6, dim, "fp16", "fused", rng.standard_normal((rows, 6, dim)).astype(np.float32))
    y = tensor(torch, rows, 6, dim, "bf16", "fused")
    dg.lw_rope(plan, x, y, batch=b)
    got = host(y)
    check(got[2:13], host(x)[2:13], pos[2:13], L.turns(pairs, 10000.0), True, 1.0, "bf16")
    assert np.all(got[:2] == 7) and np.all(got[13:] == 7)
    # many sequences: more than a wavefront looks at in a step
    n = 300
    lens = rng.integers(1, 5000, n).tolist()
    b = batch(torch, dg, list(range(n + 1)), lens)
    x = tensor(torch, n, 2, dim, "fp32", "dense", rng.standard_normal((n, 2, dim)).astype(np.float32))
    y = torch.empty_like(x)
    dg.lw_rope(plan, x, y, batch=b)
    check(host(y), host(x), np.array(lens) - 1, L.turns(pairs, 10000.0), True, 1.0, "fp32")


@pytest.mark.parametrize("halves", [True, False], ids=["halves", "pairs"])
@pytest.mark.parametrize("heads,dim,pairs", [(1, 128, 64), (2, 80, 40), (3, 64, 32), (1, 16, 8), (1, 2, 1), (5, 34, 3), (7, 64, 20)])
def test_rows_of_few_heads(torch, dg, heads, dim, pairs, halves):
    """Rows that share a wavefront: of one sequence, of several, of none, before the first sequence and behind the last."""
    rng = np.random.default_rng(heads * dim)
    news = [3, 0, 1, 1, 1, 0, 70, 2, 129, 1]
    start = (5 + np.concatenate(([0], np.cumsum(news)))).tolist()
    lens = [int(n + rng.integers(0, 5000)) for n in news]
    rows = start[-1] + 9
    pos = np.zeros(rows, np.int32)
    for s, n in enumerate(news):
        pos[start[s]:start[s + 1]] = lens[s] - n + np.arange(n)
    plan = dg.lw_rope_make(pairs, layout=dg.LW_ROPE_HALVES if halves else dg.LW_ROPE_PAIRS)
    x = tensor(torch, rows, heads, dim, "fp32", "dense", rng.standard_normal((rows, heads, dim)).astype(np.float32))
    for given in (False, True):
        y = tensor(torch, rows, heads, dim, "fp16", "fused")
        if given:
            dg.lw_rope(plan, x, y, pos=torch.from_numpy(pos).cuda())
        else:
            dg.lw_rope(plan, x, y, batch=batch(torch, dg, start, lens))
        got, mine = host(y), slice(0, rows) if given else slice(start[0], start[-1])
        check(got[mine], host(x)[mine], pos[mine], L.turns(pairs, 10000.0), halves, 1.0, "fp16")
        if not given:
            assert np.all(got[:start[0]] == 7) and np.all(got[start[-1]:] == 7)


@pytest.mark.parametrize("halves", [True, False], ids=["halves", "pairs"])
@pytest.mark.parametrize("dim,pairs", [(128, 64), (128, 24), (70, 33)])
def test_in_place_and_back(torch, dg, dim, pairs, halves):
    rng = np.random.default_rng(9)
    plan = dg.lw_rope_make(pairs, dg.LW_ROPE_HALVES if halves else dg.LW_ROPE_PAIRS)
    for dtype in TYPES:
        pos = torch.from_numpy(rng.integers(0, 100000, 33).astype(np.int32)).cuda()
        x = tensor(torch, 33, 11, dim, dtype, "fused", rng.standard_normal((33, 11, dim)).astype(np.float32))
        y = torch.empty((33, 11, dim), dtype=x.dtype, device="cuda")
        before = host(x.clone())
        dg.lw_rope(plan, x, y, pos=pos)
        dg.lw_rope(plan, x, x, pos=pos)
        assert torch.equal(x, y)
        back = torch.empty((33, 11, dim), device="cuda")
        dg.lw_rope(plan, y, back, pos=-pos)
        # two rotations' errors and the rounding between them, of a vector as long as x's pair
        size = np.abs(before).max() * 2
        assert np.abs(host(back) - before).max() <= size * (2 * HALF[dtype] + 2.0 ** -20)


def test_values_that_are_not_numbers_stay_in_their_pair(torch, dg):
    x = torch.ones((2, 2, 64), device="cuda")
    x[0, 1, 3], x[1, 0, 40] = float("nan"), float("inf")
    y = torch.empty_like(x)
    dg.lw_rope(dg.lw_rope_make(16), x, y, pos=torch.tensor([5, 6], dtype=torch.int32, device="cuda"))
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 1, 3] = want[0, 1, 19] = want[1, 0, 40] = True
    assert torch.equal(bad, want)


def test_positions_follow_a_captured_call(torch, dg):
    rng = np.random.default_rng(2)
    plan, b = dg.lw_rope_make(32), batch(torch, dg, [0, 1, 3], [10, 20])
    x = tensor(torch, 3, 4, 64, "fp32", "dense", rng.standard_normal((3, 4, 64)).astype(np.float32))
    y, z = torch.empty((3, 4, 64), dtype=torch.float16, device="cuda"), torch.empty((3, 4, 64), dtype=torch.float16, device="cuda")
    dg.lw_rope(plan, x, y, batch=b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.lw_rope(plan, x, y, batch=b)
    for _ in range(4):
        b.lens.add_(1000)
        x.mul_(1.25)
        graph.replay()
        dg.lw_rope(plan, x, z, batch=b)
        torch.cuda.synchronize()
        assert torch.equal(y, z)


def test_refusals_of_the_binding(torch, dg):
    plan = dg.lw_rope_make(32)
    x = torch.zeros((3, 2, 64), device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    b = batch(torch, dg, [0, 3], [3])
    for args in ((x.cpu(), x), (x, x.cpu()), (x[0], x), (x, x[:2]), (x.transpose(1, 2), x.transpose(1, 2)), (x, x.double())):
        with pytest.raises(dg.LwError):
            dg.lw_rope(plan, *args, pos=pos)
    for kw in (dict(), dict(pos=pos[:2]), dict(pos=pos.long()), dict(pos=pos, batch=b)):
        with pytest.raises(dg.LwError):
            dg.lw_rope(plan, x, x.clone(), **kw)


def test_as_many_rows_as_there_may_be(torch, dg):
    """2^26 rows, a wavefront each: more threads than a launch takes along one dimension.  Every row is turned, once."""
    n, dim = 1 << 26, 34
    x = torch.empty((n, 1, dim), dtype=torch.float16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    y, pos = x.clone(), torch.arange(n, dtype=torch.int32, device="cuda")
    dg.lw_rope(dg.lw_rope_make(1), y, y, pos=pos)
    assert torch.equal(y[:, :, 2:], x[:, :, 2:])
    for i in range(0, n, 1 << 22):
        a, b = (x[i:i + (1 << 22), 0, j].double() for j in (0, 1))
        angle = pos[i:i + (1 << 22)].double()                # (the plan is off by 2^-65 turns a position: 2^-36 in all)
        c, s = angle.cos(), angle.sin()
        err = (a.abs() + b.abs()) * (2.0 ** -22 + 2.0 ** -23)
        for j, want in ((0, a * c - b * s), (1, a * s + b * c)):
            off = (y[i:i + (1 << 22), 0, j].double() - want).abs()
            assert bool((off <= err + (want.abs() + err) * HALF["fp16"] + TINY["fp16"]).all()), (i, j)
