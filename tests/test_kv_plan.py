"""How lw_kv_attend cuts a call up (lw_kv_plan), on the host: the library's own function, called by its C++ name."""
import ctypes as C

import numpy as np
import pytest

import decode_gemv_amd as dg
from decode_gemv_amd import lw

ANY = (1 << 64) - 1                                           # bytes of work without a limit
TOKENS = 0x7FFF0000                                           # of a sequence, at most, for the kernels


class Plan(C.Structure):
    _fields_ = [("tile", C.c_int), ("tiles", C.c_int64), ("target", C.c_int), ("splits", C.c_int), ("chunk", C.c_int),
                ("pieces", C.c_int64), ("first_at", C.c_size_t), ("work_bytes", C.c_size_t)]


def plan(D, kv, group, seqs, tokens, longest, window=0, room=ANY):
    f = dg.lib()._Z10lw_kv_planiiilllim                      # (int, int, int, long, long, long, int, unsigned long)
    f.restype, f.argtypes = Plan, [C.c_int] * 3 + [C.c_int64] * 3 + [C.c_int, C.c_size_t]
    return f(D, kv, group, seqs, tokens, longest, window, room)


def result(p, D, kv):
    return kv * p.tile * (D + 2) * 4


@pytest.mark.parametrize("shift", range(23, 27))
@pytest.mark.parametrize("kv,seqs,rows", [(1, 1, 128), (8, 1, 4096), (64, 1, 128), (1, 64, 8192), (8, 600, 76800)])
@pytest.mark.parametrize("room", [0, ANY], ids=["no_room", "room"])
def test_tables_of_more_tokens_than_the_kernels_count(shift, kv, seqs, rows, room):
    """2^23 to 2^26 pages of 256 tokens a sequence: sizes of chunks and their number stay what they are taken for."""
    p = plan(128, kv, 1, seqs, rows, (1 << shift) * 256, 0, room)
    assert p.tile == 128
    assert 1 <= p.splits <= 512 and (p.splits == 1 or room)
    assert p.chunk > 0 and p.chunk % 128 == 0
    assert (p.splits - 1) * p.chunk < TOKENS <= p.splits * p.chunk
    assert p.work_bytes == (p.tiles * p.splits * result(p, 128, kv) if p.splits > 1 else 0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_a_tile(D):
    """Which kernel takes how many rows: 8, 16 and 32 a sequence on average, 16 up to the work at which 128 rows are worth it,
    and 32 from there on for sequences of not more than 64.  Heads of 256 have no tiles of more than 16."""
    wide = lambda tile: min(tile, 16) if D == 256 else tile
    work = 1 << 19                                            # tokens at which one tile of 128 rows is work enough
    for seqs in (1, 3, 150):
        for rows, tile in ((1, 8), (8, 8), (9, 16), (16, 16), (17, 32), (32, 32), (33, 16), (64, 16), (400, 16)):
            assert plan(D, 1, 1, seqs, seqs * rows, 500).tile == wide(tile), (seqs, rows)
    for rows, tile in ((32, 32), (33, 32), (64, 32), (65, 128), (400, 128)):
        assert plan(D, 1, 1, 1, rows, work).tile == wide(tile), rows
    for rows in (33, 64, 65, 128):
        assert plan(D, 1, 1, 1, rows, work - 1).tile == 16
        assert plan(D, 4, 1, 1, rows, work // 4).tile == plan(D, 1, 1, 1, rows, work).tile


def test_one_long_sequence_among_many_is_cut():
    """However many sequences there are, up to where looking at all of them costs a fifteenth of walking the long one; not where
    the longest is short, and not prompts, which have workgroups enough."""
    for seqs in (127, 128, 129, 256, 500):
        assert plan(128, 8, 4, seqs, seqs, 131072).target > 0, seqs
    assert plan(128, 8, 4, 256, 256, 16384).target and not plan(128, 8, 4, 256, 256, 8000).target
    assert not plan(128, 8, 4, 4096, 4096, 131072).target
    assert not plan(128, 8, 4, 128, 128, 1024).target
    assert not plan(256, 4, 4, 1, 1024, 4096).target and plan(256, 4, 4, 1, 1024, 4096).tile == 16
    for seqs in (128, 256):                                   # and if only because there is no room for it
        p = plan(128, 8, 4, seqs, seqs, 131072, 0, 1 << 20)
        assert not p.target and p.pieces == p.tiles and not p.work_bytes


def scratch(D, kv, group, seqs, tokens, longest):
    cache = lw.lw_kv_cache(1 << 20, 4, kv, D, 32)
    batch = lw.lw_kv_batch(seqs, 1 << 20, 1 << 20, 1 << 20, 1 << 26, longest)
    return dg.lib().lw_kv_attend_scratch_bytes(C.byref(cache), C.byref(batch), tokens, kv * group)


@pytest.mark.parametrize("seed", range(40))
def test_work_for_the_largest_batch_does_for_smaller_ones(seed):
    """lw_kv_attend_scratch_bytes of a shape is what no smaller one (sequences, rows, longest sequence, with any window)
    wants more of, and does not fall as the shape grows; nor is it far more than the largest of them wants."""
    rng = np.random.default_rng(seed)
    log = lambda lo, hi: int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))
    D, kv, group = int(rng.choice([64, 128, 256])), log(1, 1024), log(1, 64)
    seqs, longest = log(1, 4000), log(1, 200000)
    tokens = log(1, 20000)
    have, want = scratch(D, kv, group, seqs, tokens, longest), 0
    for _ in range(3000):
        n, t, l = log(1, seqs), log(1, tokens), log(1, longest)
        want = max(want, plan(D, kv, group, n, t, l, int(rng.choice([0, log(1, 100000)]))).work_bytes)
        if rng.random() < 0.02:
            assert scratch(D, kv, group, n, t, l) <= have
    edges = [n for n in (seqs, 1023 // kv, 1024 // kv, 511 // kv, 1) if 1 <= n <= seqs]
    rows = [r * n for n in edges for r in (8, 9, 16, 17, 32, 33, 64, 65, 128)] + [128 * n for n in edges]
    for n in edges:
        for t in {min(tokens, max(1, r // group)) for r in rows} | {tokens}:
            want = max(want, plan(D, kv, group, n, t, longest).work_bytes)
    assert want <= have <= 2.5 * want + (1 << 12), (D, kv, group, seqs, tokens, longest, want, have)


def test_work_across_the_thresholds():
    for seqs in range(1, 400):
        assert scratch(128, 8, 4, seqs, seqs, 131072) <= scratch(128, 8, 4, seqs + 1, seqs + 1, 131072)
    assert scratch(128, 8, 4, 4096, 4096, 131072) > 0
    for tokens in range(1, 300):
        assert scratch(128, 2, 4, 3, tokens, 16384) <= scratch(128, 2, 4, 3, tokens + 1, 16384)
    for longest in range(900, 1100):
        assert scratch(64, 4, 4, 9, 9, longest) <= scratch(64, 4, 4, 9, 9, longest + 1)
