"""The 4-bit key/value cache without a GPU: the reference of the GPU tests against itself, sizes, and the refusals of
every entry point (all before anything is enqueued)."""
import ctypes as C

import numpy as np
import pytest

import kv_ref as R

import decode_gemv_amd as dg
from decode_gemv_amd import lw


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [32, 64])
def test_reference_places_fill_a_block_once(D, P):
    # every byte of a head block belongs to exactly one pair of codes or one pair (d, m)
    seen = np.zeros(P * (D + 8), int)
    for t in range(P):
        for byte, shift, at in R.places(D, P, t):
            np.add.at(seen, byte, 1)
            seen[at:at + 4] += 2
    assert np.all(seen == 2)


def test_reference_round_trip_and_quantiser():
    rng = np.random.default_rng(1)
    D, P = 64, 32
    block = np.zeros(P * (D + 8), np.uint8)
    x = rng.standard_normal((P, 2, D)).astype(np.float32)
    q, d, m = R.quantise(x)
    for t in range(P):
        for side in range(2):
            R.write(block, D, P, t, side, q[t, side], d[t, side], m[t, side])
    for t in range(P):
        for side in range(2):
            got, dd, mm = R.read(block, D, P, t, side)
            assert dd == d[t, side] and mm == m[t, side]
            assert np.array_equal(got, float(dd) * q[t, side] - float(mm))
            # half a step, and what the rounding of the pair to fp16 moves (15 steps of 2^-11 d, 2^-11 m)
            assert np.all(np.abs(got - x[t, side]) <= dd * (0.5 + 15 * 2.0 ** -11) + abs(mm) * 2.0 ** -11)


def test_quantiser_special_vectors():
    x = np.zeros((6, 64), np.float32)
    x[0] = 3.25                                    # constant: d = 0, worth -m
    x[1, 5] = np.nan
    x[2, 6] = -np.inf
    x[3, :2] = 3e38, -3e38                         # past fp16: the pair is kept within it
    x[4, :2] = 1e-7, -1e-7
    q, d, m = R.quantise(x)
    assert d[0] == 0 and m[0] == -3.25 and not q[0].any()
    assert np.isnan(d[1:3]).all() and np.isnan(m[1:3]).all()
    assert d[3] == 65504 and m[3] == 65504 and np.isfinite(d[4])
    assert d[5] == 0 and m[5] == 0


def test_page_bytes():
    assert dg.lw_kv_page_bytes(8, 128, 64) == 8 * 64 * 136
    for bad in ((0, 128, 64), (1025, 128, 64), (8, 96, 64), (8, 128, 16), (8, 128, 48), (8, 128, 512)):
        assert dg.lw_kv_page_bytes(*bad) == 0


# ------------------------------------------------------------------ refusals

def _args():
    """A valid call's structures over host memory (nothing is enqueued by a call that is refused)."""
    mem = np.zeros(1 << 20, np.uint8)
    p = (mem.ctypes.data + 255) & ~255
    cache = lw.lw_kv_cache(p, 4, 2, 64, 32)
    batch = lw.lw_kv_batch(2, p, p, p, 3, 0)
    t = lw.lw_kv_tensor(p, 128, 64)
    return mem, p, cache, batch, t


def _append(cache, batch, n, k, v, dtype):
    return dg.lib().lw_kv_append(cache and C.byref(cache), batch and C.byref(batch), n, k and C.byref(k), v and C.byref(v),
                                 dtype, None)


def _attend(cache, batch, n, q, out, dtype=0, heads=2, scale=0.125, causal=1, window=0, lse=None, work=None, nb=0):
    return dg.lib().lw_kv_attend(cache and C.byref(cache), batch and C.byref(batch), n, q and C.byref(q),
                                 out and C.byref(out), dtype, heads, scale, causal, window, lse, work, nb, None)


def _changed(s, **kw):
    new = type(s).from_buffer_copy(bytes(s))
    for k, v in kw.items():
        setattr(new, k, v)
    return new


CACHES = [(dict(kv_heads=0), dg.LW_E_ARG), (dict(kv_heads=1025), dg.LW_E_ARG), (dict(head_dim=96), dg.LW_E_UNSUPPORTED),
          (dict(page_tokens=16), dg.LW_E_UNSUPPORTED), (dict(page_tokens=96), dg.LW_E_UNSUPPORTED),
          (dict(n_pages=-1), dg.LW_E_ARG), (dict(pages=None), dg.LW_E_ARG), (dict(pages=264), dg.LW_E_ARG)]
BATCHES = [dict(n_seqs=-1), dict(n_seqs=1 << 23), dict(start=None), dict(lens=None), dict(table=None),
           dict(table_stride=-1), dict(table_stride=1 << 27), dict(max_len=-1), dict(start=258), dict(lens=257),
           dict(table=259)]
TENSORS = [dict(data=None), dict(data=257), dict(token_stride=-1), dict(head_stride=-8), dict(token_stride=1 << 33)]


@pytest.mark.parametrize("change,status", CACHES)
def test_refuses_caches(change, status):
    mem, p, cache, batch, t = _args()
    bad = _changed(cache, **change)
    assert _append(bad, batch, 3, t, t, 0) == status
    assert _attend(bad, batch, 3, t, t) == status
    assert dg.lw_last_error()


@pytest.mark.parametrize("change", BATCHES)
def test_refuses_batches(change):
    mem, p, cache, batch, t = _args()
    bad = _changed(batch, **change)
    assert _append(cache, bad, 3, t, t, 0) == dg.LW_E_ARG
    assert _attend(cache, bad, 3, t, t) == dg.LW_E_ARG
    assert dg.lib().lw_kv_read(C.byref(cache), C.byref(bad), 3, C.byref(t), C.byref(t), 0, None) == dg.LW_E_ARG


@pytest.mark.parametrize("change", TENSORS)
def test_refuses_tensors(change):
    mem, p, cache, batch, t = _args()
    bad = _changed(t, **change)
    for a, b in ((bad, t), (t, bad)):
        assert _append(cache, batch, 3, a, b, 0) == dg.LW_E_ARG
        assert _attend(cache, batch, 3, a, b) == dg.LW_E_ARG


def test_refuses_the_rest():
    mem, p, cache, batch, t = _args()
    assert _append(None, batch, 3, t, t, 0) == dg.LW_E_ARG
    assert _append(cache, None, 3, t, t, 0) == dg.LW_E_ARG
    assert _append(cache, batch, 3, None, t, 0) == dg.LW_E_ARG
    assert _append(cache, batch, 3, t, t, 3) == dg.LW_E_ARG
    assert _append(cache, batch, -1, t, t, 0) == dg.LW_E_ARG
    assert _append(cache, batch, (1 << 26) + 1, t, t, 0) == dg.LW_E_ARG
    assert _attend(cache, batch, 3, t, t, dtype=dg.LW_F32) == dg.LW_E_UNSUPPORTED
    for kw in (dict(heads=0), dict(heads=3), dict(heads=4096), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(lse=p + 2),
               dict(work=p + 8, nb=1 << 16)):
        assert _attend(cache, batch, 3, t, t, **kw) == dg.LW_E_ARG, kw
    assert _attend(cache, batch, (1 << 26) - 1, t, t, heads=64) == dg.LW_E_ARG        # 2^31 rows per kv head
    assert _attend(cache, batch, 1 << 23, t, t) == dg.LW_E_UNSUPPORTED               # more than 65535 tiles


def test_empty_calls_do_nothing():
    mem, p, cache, batch, t = _args()
    none = lw.lw_kv_tensor(None, 0, 0)
    empty = _changed(batch, n_seqs=0, start=None, lens=None, table=None)
    assert _append(cache, empty, 3, none, none, 0) == dg.LW_OK
    assert _append(cache, batch, 0, none, none, 0) == dg.LW_OK
    assert _attend(cache, batch, 0, none, none) == dg.LW_OK
    assert _attend(cache, empty, 3, none, none) == dg.LW_OK


def _scratch(cache, batch, n, heads):
    return dg.lib().lw_kv_attend_scratch_bytes(C.byref(cache), C.byref(batch), n, heads)


def test_scratch_grows_with_the_context_and_not_with_prompts():
    mem, p, cache, batch, t = _args()
    one = _changed(batch, n_seqs=1, table_stride=1 << 12)           # up to 131072 tokens
    short, long_ = _changed(one, max_len=100), _changed(one, max_len=100000)
    assert _scratch(cache, short, 1, 2) == 0
    assert 0 < _scratch(cache, long_, 1, 2) < 64 << 20
    assert _scratch(cache, one, 1, 2) >= _scratch(cache, long_, 1, 2)
    assert _scratch(cache, _changed(one, max_len=4096), 4096, 64) < 64 << 20
    assert _scratch(cache, _changed(one, table_stride=-1), 1, 2) == 0
    assert _scratch(cache, one, 1, 3) == 0
