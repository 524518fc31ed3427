"""Rotary positions and the operators around long sequences without a GPU: plans against 60 digits, sizes, and the
refusals of every entry point (all before anything is enqueued)."""
import ctypes as C

import numpy as np
import pytest

import kv_long_ref as L

import decode_gemv_amd as dg
from decode_gemv_amd import lw

SCALINGS = dict(plain=0, linear=1, base=2, index=3, turns=4)


@pytest.mark.parametrize("pairs", [1, 2, 3, 24, 64, 128, 256])
@pytest.mark.parametrize("scaling,kw", [
    ("plain", dict(base=10000.0)), ("plain", dict(base=1.0)), ("linear", dict(base=500000.0, factor=8.0)),
    ("base", dict(base=10000.0, factor=4.0)), ("index", dict(base=10000.0, factor=16.0, original=4096.0, low=1.0, high=32.0)),
    ("index", dict(base=500000.0, factor=2.5, original=100.0, low=50.0, high=60.0)),
    ("turns", dict(base=500000.0, factor=8.0, original=8192.0, low=1.0, high=4.0)),
    ("linear", dict(base=3.0, factor=2.0 ** -40))])
def test_plans_against_60_digits(pairs, scaling, kw):
    if scaling == "base" and pairs == 1:
        with pytest.raises(dg.LwError):
            dg.lw_rope_make(pairs, scaling=SCALINGS[scaling], **kw)
        return
    p = dg.lw_rope_make(pairs, scaling=SCALINGS[scaling], amplitude=1.25, **kw).desc
    assert (p.pairs, p.layout, p.amplitude) == (pairs, 0, 1.25)
    want = L.turns(pairs, scaling=scaling, **kw)
    for i in range(dg.LW_ROPE_MOST):
        if i >= pairs:
            assert p.step[i] == 0
            continue
        # up to eight roundings to 64 bits of what may be up to a few turns (scaled up: many, of which the whole ones go)
        size = max(float(want[i]), 1.0 / 8) * 2.0 ** 64
        off = (int(p.step[i]) - int((want[i] % 1) * 2 ** 64)) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1 + 8 * size * 2.0 ** -64 * 2, i


@pytest.mark.parametrize("kw", [
    dict(pairs=0), dict(pairs=257), dict(layout=2), dict(layout=-1), dict(scaling=5), dict(scaling=-1), dict(base=0.5),
    dict(base=float("nan")), dict(base=float("inf")), dict(amplitude=float("inf")), dict(amplitude=float("nan")),
    dict(scaling=1, factor=0.0), dict(scaling=1, factor=-2.0), dict(scaling=1, factor=float("nan")), dict(pairs=1, scaling=2),
    dict(scaling=3, factor=2.0, original=0.0), dict(scaling=3, factor=2.0, original=4096.0, low=0.0),
    dict(scaling=3, factor=2.0, original=4096.0, base=1.0), dict(scaling=4, factor=2.0, original=4096.0, low=4.0, high=4.0),
    dict(scaling=4, factor=2.0, original=4096.0, low=-1.0), dict(scaling=4, factor=2.0, original=float("nan"))])
def test_refuses_plans(kw):
    with pytest.raises(dg.LwError) as e:
        dg.lw_rope_make(**{"pairs": 32, **kw})
    assert e.value.status == dg.LW_E_ARG
    assert dg.lib().lw_rope_make(None, None) == dg.LW_E_ARG


def test_refuses_plans_whose_turns_leave_64_bits():
    """original / (2 pi high) overflows: there is no pair that turns `high` times.  An overflow with low only keeps every
    pair on the ramp, which its last one ends."""
    kw = dict(scaling=3, factor=4.0, original=2.0 ** 64)
    for high in (1e-300, 5e-324):
        for low in (1.0, 1e-300):
            with pytest.raises(dg.LwError) as e:
                dg.lw_rope_make(32, low=low, high=high, **kw)
            assert e.value.status == dg.LW_E_ARG
    fine = dg.lw_rope_make(32, low=1e-300, high=32.0, **kw).desc
    assert list(fine.step) == list(dg.lw_rope_make(32, low=1e-200, high=32.0, **kw).desc.step)


@pytest.mark.parametrize("pairs,kw,takes", [
    # all pairs turn more than `high` times over the original context: lo = 10, hi = 13 kept to 7
    (4, dict(base=10.0, factor=4.0, original=8192.0, low=1.0, high=4.0), 4.0),
    (8, dict(base=10.0, factor=4.0, original=32768.0, low=1.0, high=32.0), 4.0),
    # all turn fewer than `low` times: hi = -2, lo kept to 0
    (32, dict(base=500000.0, factor=4.0, original=100.0, low=50.0, high=60.0), 1.0)])
def test_plans_whose_ramp_runs_the_other_way(pairs, kw, takes):
    """The ends that lw.h states, each kept on one side.  A step is a whole number of 2^-64 turns, off by half of one; `want`
    is in 64 bits, off by a few 2^-53 of itself, the power by its exponent of up to 13 times that."""
    got = dg.lw_rope_make(pairs, scaling=SCALINGS["index"], **kw).desc
    for i in range(pairs):
        want = kw["base"] ** (-i / pairs) / takes / (2 * np.pi)
        assert abs(got.step[i] * 2.0 ** -64 - want) <= 2.0 ** -48 * want + 2.0 ** -65


def test_sizes():
    assert dg.lw_kv_bounds_bytes(8, 128) == 8 * 260 and dg.lw_kv_bounds_bytes(1, 64) == 144
    for bad in ((0, 128), (1025, 128), (8, 96)):
        assert dg.lw_kv_bounds_bytes(*bad) == 0


# ------------------------------------------------------------------ refusals

class Args:
    """A valid call's structures over host memory (nothing is enqueued by a call that is refused)."""

    def __init__(self):
        self.mem = np.zeros(1 << 20, np.uint8)
        self.p = p = (self.mem.ctypes.data + 255) & ~255
        self.cache = lw.lw_kv_cache(p, 4, 2, 64, 32)
        self.batch = lw.lw_kv_batch(2, p, p, p, 3, 0)
        self.t = lw.lw_kv_tensor(p, 128, 64)
        self.sel = lw.lw_kv_selection(3, p, p, p, 5)
        self.plan = dg.lw_rope_make(32).desc


def changed(s, **kw):
    new = type(s).from_buffer_copy(bytes(s))
    for k, v in kw.items():
        setattr(new, k, v)
    return new


def ref(x):
    return C.byref(x) if x is not None else None


def rope(a, **kw):
    v = dict(plan=a.plan, batch=a.batch, pos=None, n=3, heads=2, dim=64, x=a.t, xt=0, y=a.t, yt=0)
    v.update(kw)
    return dg.lib().lw_rope(ref(v["plan"]), ref(v["batch"]), v["pos"], v["n"], v["heads"], v["dim"], ref(v["x"]), v["xt"],
                            ref(v["y"]), v["yt"], None)


def bounds(a, **kw):
    v = dict(cache=a.cache, batch=a.batch, n=3, bounds=a.p)
    v.update(kw)
    return dg.lib().lw_kv_bounds(ref(v["cache"]), ref(v["batch"]), v["n"], v["bounds"], None)


def select(a, **kw):
    v = dict(cache=a.cache, batch=a.batch, q=a.t, dtype=0, heads=4, bounds=a.p, first=1, last=1, sel=a.sel, work=None, wb=0)
    v.update(kw)
    return dg.lib().lw_kv_select(ref(v["cache"]), ref(v["batch"]), ref(v["q"]), v["dtype"], v["heads"], v["bounds"], v["first"],
                                 v["last"], ref(v["sel"]), v["work"], v["wb"], None)


def attend(a, **kw):
    v = dict(cache=a.cache, sel=a.sel, q=a.t, out=a.t, dtype=0, heads=4, scale=0.125, lse=None, work=None, wb=0)
    v.update(kw)
    return dg.lib().lw_kv_attend_selected(ref(v["cache"]), ref(v["sel"]), ref(v["q"]), ref(v["out"]), v["dtype"], v["heads"],
                                          v["scale"], v["lse"], v["work"], v["wb"], None)


def weigh(a, **kw):
    v = dict(cache=a.cache, batch=a.batch, n=3, q=a.t, dtype=0, heads=4, scale=0.125, causal=1, window=0, lse=a.p, before=None,
             decay=1.0, weights=a.p, stride=3)
    v.update(kw)
    return dg.lib().lw_kv_weigh(ref(v["cache"]), ref(v["batch"]), v["n"], ref(v["q"]), v["dtype"], v["heads"], v["scale"],
                                v["causal"], v["window"], v["lse"], v["before"], v["decay"], v["weights"], v["stride"], None)


def evict(a, **kw):
    v = dict(cache=a.cache, batch=a.batch, weights=a.p, stride=3, keep=2, first=1, last=1, table=a.p, gone=a.p, count=a.p)
    v.update(kw)
    return dg.lib().lw_kv_evict(ref(v["cache"]), ref(v["batch"]), v["weights"], v["stride"], v["keep"], v["first"], v["last"],
                                v["table"], v["gone"], v["count"], None)


CACHES = [(None, dg.LW_E_ARG), (dict(kv_heads=0), dg.LW_E_ARG), (dict(kv_heads=1025), dg.LW_E_ARG),
          (dict(head_dim=96), dg.LW_E_UNSUPPORTED), (dict(page_tokens=16), dg.LW_E_UNSUPPORTED), (dict(n_pages=-1), dg.LW_E_ARG)]
PAGES = [(dict(pages=None), dg.LW_E_ARG), (dict(pages=264), dg.LW_E_ARG)]


@pytest.mark.parametrize("change,status", CACHES + PAGES)
def test_refuses_caches(change, status):
    a = Args()
    bad = changed(a.cache, **change) if change else None
    for call in (bounds, select, attend, weigh) + ((evict,) if (change, status) in CACHES else ()):
        assert call(a, cache=bad) == status, call.__name__
        assert dg.lw_last_error()


@pytest.mark.parametrize("change", [dict(n_seqs=-1), dict(n_seqs=1 << 23), dict(start=None), dict(lens=None), dict(table=None),
                                    dict(table_stride=-1), dict(table_stride=1 << 27), dict(max_len=-1), dict(start=258),
                                    dict(lens=257), dict(table=259)])
def test_refuses_batches(change):
    a = Args()
    bad = changed(a.batch, **change)
    for call in (bounds, select, weigh):
        assert call(a, batch=bad) == dg.LW_E_ARG, call.__name__
    if "table" not in change:
        assert rope(a, batch=bad) == dg.LW_E_ARG
    if "start" not in change:
        assert evict(a, batch=bad) == dg.LW_E_ARG
    for call in (bounds, select, weigh, evict):
        assert call(a, batch=None) == dg.LW_E_ARG


@pytest.mark.parametrize("change", [dict(data=None), dict(data=257), dict(token_stride=-1), dict(head_stride=-8),
                                    dict(token_stride=1 << 33)])
def test_refuses_tensors(change):
    a = Args()
    bad = changed(a.t, **change)
    for call, names in ((rope, "xy"), (select, "q"), (attend, ("q", "out")), (weigh, "q")):
        for name in names:
            assert call(a, **{name: bad}) == dg.LW_E_ARG, (call.__name__, name)
            assert call(a, **{name: None}) == dg.LW_E_ARG


@pytest.mark.parametrize("kw", [
    dict(plan=None), dict(pos=1 << 12), dict(batch=None), dict(batch=None, pos=4098), dict(n=-1), dict(n=(1 << 26) + 1),
    dict(heads=0), dict(heads=65537), dict(dim=63), dict(dim=1025), dict(xt=3), dict(yt=-1), dict(yt=1)])
def test_refuses_rope(kw):
    assert rope(Args(), **kw) == dg.LW_E_ARG


def test_refuses_rope_in_place_with_other_strides_and_outputs_that_overlap():
    a = Args()
    assert rope(a, y=changed(a.t, token_stride=256)) == dg.LW_E_ARG
    assert rope(a, y=changed(a.t, head_stride=128)) == dg.LW_E_ARG
    other = changed(a.t, data=a.p + 4096)
    assert rope(a, y=changed(other, token_stride=0)) == dg.LW_E_ARG
    assert rope(a, y=changed(other, head_stride=0)) == dg.LW_E_ARG
    assert rope(a, plan=changed(a.plan, pairs=0)) == dg.LW_E_ARG
    assert rope(a, plan=changed(a.plan, layout=7)) == dg.LW_E_ARG


def test_refuses_selections():
    a = Args()
    for change in (dict(n_tokens=-1), dict(n_tokens=(1 << 26) + 1), dict(pages=0), dict(pages=32769), dict(start=None),
                   dict(lens=None), dict(table=None), dict(start=258), dict(lens=257), dict(table=259)):
        bad = changed(a.sel, **change)
        assert select(a, sel=bad) == dg.LW_E_ARG, change
        assert attend(a, sel=bad) == dg.LW_E_ARG, change
    assert select(a, sel=None) == attend(a, sel=None) == dg.LW_E_ARG


def test_refuses_the_rest():
    a = Args()
    for kw in (dict(bounds=None), dict(bounds=a.p + 8)):
        assert bounds(a, **kw) == select(a, **kw) == dg.LW_E_ARG
    for kw in (dict(first=-1), dict(last=-1), dict(first=4), dict(first=2, last=3), dict(work=a.p + 2, wb=64), dict(heads=3),
               dict(heads=0), dict(heads=4096)):
        assert select(a, **kw) == dg.LW_E_ARG, kw
    for kw in (dict(heads=3), dict(heads=0), dict(scale=0.0), dict(scale=float("nan")), dict(lse=a.p + 2),
               dict(work=a.p + 8, wb=64)):
        assert attend(a, **kw) == dg.LW_E_ARG, kw
    for kw in (dict(heads=3), dict(scale=-1.0), dict(window=-1), dict(lse=None), dict(lse=a.p + 1), dict(before=a.p + 2),
               dict(decay=-0.5), dict(decay=1.5), dict(decay=float("nan")), dict(weights=None), dict(weights=a.p + 2),
               dict(stride=-1), dict(stride=(1 << 24) + 1), dict(n=-1)):
        assert weigh(a, **kw) == dg.LW_E_ARG, kw
    assert weigh(a, batch=changed(a.batch, n_seqs=1 << 20), stride=1 << 12) == dg.LW_E_ARG
    for kw in (dict(keep=-1), dict(first=-1), dict(last=0), dict(stride=-1), dict(weights=None), dict(table=None), dict(gone=None),
               dict(count=None), dict(weights=a.p + 2), dict(table=a.p + 2), dict(gone=a.p + 1), dict(count=a.p + 3)):
        assert evict(a, **kw) == dg.LW_E_ARG, kw
    for call in (select, attend, weigh):
        assert call(a, dtype=dg.LW_F32) == dg.LW_E_UNSUPPORTED, call.__name__
    wide = changed(a.batch, table_stride=32769)
    assert select(a, batch=wide) == evict(a, batch=wide) == dg.LW_E_UNSUPPORTED


def test_refuses_pages_given_up_into_a_table():
    a = Args()
    q = a.p + 256
    other = changed(a.batch, table=q)
    for batch, table, gone in ((a.batch, a.p, a.p), (a.batch, q, a.p), (other, a.p, a.p), (other, q, q)):
        assert evict(a, batch=batch, table=table, gone=gone) == dg.LW_E_ARG
        assert "gone" in dg.lw_last_error()


def test_empty_calls_do_nothing():
    a = Args()
    none = lw.lw_kv_tensor(None, 0, 0)
    empty = changed(a.batch, n_seqs=0, start=None, lens=None, table=None)
    for kw in (dict(n=0, x=none, y=none), dict(batch=empty, x=none, y=none)):
        assert rope(a, **kw) == dg.LW_OK
    assert bounds(a, n=0, bounds=None) == bounds(a, batch=empty, bounds=None) == dg.LW_OK
    nobody = changed(a.sel, n_tokens=0, start=None, lens=None, table=None)
    assert select(a, sel=nobody, q=none, bounds=None) == attend(a, sel=nobody, q=none, out=none) == dg.LW_OK
    assert weigh(a, n=0, q=none, lse=None, weights=None) == weigh(a, batch=empty, q=none, lse=None, weights=None) == dg.LW_OK
    assert weigh(a, stride=0, q=none, lse=None, weights=None) == dg.LW_OK
    assert evict(a, batch=empty, weights=None, table=None, gone=None, count=None) == dg.LW_OK


def test_scratch():
    a = Args()
    attends = lambda sel, heads=4: dg.lib().lw_kv_attend_selected_scratch_bytes(ref(a.cache), ref(sel), heads)
    selects = lambda batch, n, heads=4: dg.lib().lw_kv_select_scratch_bytes(ref(a.cache), ref(batch), n, heads)
    assert attends(changed(a.sel, pages=1)) == 0 and attends(a.sel, 3) == 0 and attends(changed(a.sel, pages=0)) == 0
    assert 0 < attends(changed(a.sel, n_tokens=1, pages=128)) < 64 << 20
    assert attends(changed(a.sel, n_tokens=0)) == 0
    long_ = changed(a.batch, table_stride=8192)
    assert selects(a.batch, 1) == 0 and 0 < selects(long_, 1) < 1 << 20
    assert selects(long_, 1, 3) == 0 and selects(changed(long_, table_stride=-1), 1) == 0
    assert selects(changed(long_, max_len=64), 1) == 0


@pytest.mark.parametrize("kv,heads,D,P", [(8, 32, 128, 64), (4, 16, 256, 128), (1, 20, 64, 32), (16, 16, 64, 256)])
def test_scratch_of_the_largest_call_does_for_smaller_ones(kv, heads, D, P):
    cache = lw.lw_kv_cache(1 << 20, 1 << 20, kv, D, P)
    attends = lambda n, pages: dg.lib().lw_kv_attend_selected_scratch_bytes(C.byref(cache), C.byref(lw.lw_kv_selection(n, 16, 16, 16, pages)), heads)
    selects = lambda n, stride: dg.lib().lw_kv_select_scratch_bytes(C.byref(cache), C.byref(lw.lw_kv_batch(1, 16, 16, 16, stride, 0)), n, heads)
    for f, sizes in ((attends, (1, 2, 4, 7, 9, 16, 33, 64, 100, 129, 500)), (selects, (1, 100, 255, 256, 300, 1024, 32768))):
        counts = (1, 2, 3, 7, 16, 31, 32, 33, 64, 65, 127, 128, 300, 513, 2000)
        for i, n in enumerate(counts):
            for k, size in enumerate(sizes):
                if i:
                    assert f(n, size) >= f(counts[i - 1], size)
                if k:
                    assert f(n, size) >= f(n, sizes[k - 1])


def test_tensors_of_another_device_are_refused(monkeypatch):
    """(Without one: what the binding asks a tensor is answered for it.)"""
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    class There:
        dtype, shape = torch.int32, torch.Size([3, 2, 64])
        device = 0
        get_device = lambda self: self.device
        is_contiguous = lambda self: True
        data_ptr = lambda self: 256
        stride = lambda self: (128, 64, 1)

    t = There()
    assert lw._addr(t, "t") == 256 and lw._vectors(t, "t")[0].data == 256
    for device in (1, -1):
        t.device = device
        for call in (lw._addr, lw._vectors):
            with pytest.raises(dg.LwError, match="current device"):
                call(t, "t")
    for call in (lw._addr, lw._vectors):
        with pytest.raises(dg.LwError):
            call(None, "t")


def test_caches_batches_and_selections_of_another_device_are_refused(monkeypatch):
    """The tensors of a call may lie on the current device, and what they are used with on another: as above, without one."""
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    mem = np.zeros(1 << 16, np.uint8)

    class There:
        is_cuda = True

        def __init__(self, *shape, dtype=torch.float32, device=0):
            self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
            self.nbytes = self.numel() * dtype.itemsize

        numel = lambda self: int(np.prod(self.shape))
        element_size = lambda self: self.dtype.itemsize
        dim = lambda self: len(self.shape)
        get_device = lambda self: self.device
        is_contiguous = lambda self: True
        data_ptr = lambda self: (mem.ctypes.data + 255) & ~255
        stride = lambda self: tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    monkeypatch.setattr(lw, "_dptr", lambda t, what: C.c_void_p(t.data_ptr()))
    i32 = lambda *shape, device=0: There(*shape, dtype=torch.int32, device=device)
    cache = lambda device: dg.KvCache(There(4 * dg.lw_kv_page_bytes(2, 64, 32), dtype=torch.uint8, device=device), 2, 64, 32)
    batch = lambda *on: dg.KvBatch(*(i32(*shape, device=d) for shape, d in zip(((2,), (1,), (1, 3)), on)))
    here, sel = (cache(0), batch(0, 0, 0)), dg.KvSelection(i32(4), i32(3), i32(3, 2, 5))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    far = dg.KvSelection(i32(4, device=1), i32(3, device=1), i32(3, 2, 5, device=1))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    q, lse, weights = There(3, 4, 64, dtype=torch.float16), There(3, 4), There(1, 2, 3)
    bounds = There(4 * dg.lw_kv_bounds_bytes(2, 64), dtype=torch.uint8)
    plan = dg.lw_rope_make(32)
    for c, b, s in ((cache(1), here[1], sel), (here[0], batch(1, 1, 1), sel), (here[0], batch(0, 0, 1), sel),
                    (here[0], batch(1, 0, 0), sel), (*here, far)):
        calls = []
        if s is sel:
            calls += [lambda: dg.lw_kv_bounds(c, b, 3, bounds), lambda: dg.lw_kv_weigh(c, b, q, lse, weights),
                      lambda: dg.lw_kv_evict(c, b, weights, 2, i32(1, 3), i32(1, 3), i32(1))]
        if b is not here[1]:
            calls.append(lambda: dg.lw_rope(plan, q, There(3, 4, 64, dtype=torch.float16), batch=b))
        else:
            calls.append(lambda: dg.lw_kv_attend_selected(c, s, q, There(3, 4, 64, dtype=torch.float16)))
        for call in calls + [lambda: dg.lw_kv_select(c, b, q, bounds, s)]:
            with pytest.raises(dg.LwError, match="the cache, the batch and the selection") as e:
                call()
            assert e.value.status == dg.LW_E_ARG
