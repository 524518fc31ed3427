// kv_attend.hip -- attention of new tokens over the 4-bit key/value cache: how
// a call is cut up, and the launches of the kernel of up to 32 query rows
// (kv_rows.hpp).
#include <algorithm>
#include <cmath>

#include "kv_rows.hpp"

namespace {

template <int D, int ROWS, class T>
hipError_t launch(const KvAttend &a, const KvPlan &p, hipStream_t s)
{
    const unsigned y = (unsigned)std::min<int64_t>(p.pieces, 1 << 15), z = (unsigned)((p.pieces + y - 1) / y);
    hipLaunchKernelGGL((k_kv_attend<D, ROWS, T>), dim3(a.g.kv_heads, y, z), dim3(NW * 64), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.target) return e;
    return launch_join<D, ROWS, T>(a, p, s);
}

template <int D>
hipError_t launch_dim(const KvAttend &a, int dtype, const KvPlan &p, hipStream_t s)
{
    if (p.tile == 8) return dtype == LW_F16 ? launch<D, 8, _Float16>(a, p, s) : launch<D, 8, __bf16>(a, p, s);
    if constexpr (D <= 128)                                  // (lw_kv_plan)
        if (p.tile == 32) return dtype == LW_F16 ? launch<D, 32, _Float16>(a, p, s) : launch<D, 32, __bf16>(a, p, s);
    return dtype == LW_F16 ? launch<D, 16, _Float16>(a, p, s) : launch<D, 16, __bf16>(a, p, s);
}

}  // namespace

namespace {

// Whether sequences are cut into chunks.  Not up to 1024 tokens; from there on
// where there are fewer workgroups than the chip has places for: heads of 128,
// 32 on 8 (replays of a graph), 8 sequences of 1000 tokens 18.0 us cut and 17.8
// not, 8 of 1300 18.8 and 20.3, one of 1500 17.3 and 20.3, 48 of 500 to 8190 65
// and 87, 100 of 100 to 4000 70 and 68.  And where one sequence may be
// far longer than the others, whose workgroups would leave it alone on the
// chip: 128 sequences of 500 tokens and one of 131071, 57 us and not 786 (256:
// 76 and 893, 512: 128 and 934).  That has a price, as each workgroup looks at
// all sequences (n^2 kv looks): 128, 256, 512 and 1024 of 500 tokens and none
// longer, 27, 44, 100 and 232 us and not 26, 42, 75 and 143.  So it is done
// where the looks, 12 ps n^2 kv, come to a fifteenth at most of the time that a
// sequence of `span` tokens would be left alone, 5.8 ns a token.  (Sequences of
// more than one row tile have workgroups enough.)
bool cut(int64_t kv_heads, int64_t n_seqs, int64_t rows, int tile, int64_t span)
{
    if (span <= 1024) return false;
    if (std::max(n_seqs, (rows + tile - 1) / tile) * kv_heads < 1024) return true;
    return rows <= tile * n_seqs && n_seqs * n_seqs * kv_heads <= 32 * span;
}

}  // namespace

KvPlan lw_kv_plan(int head_dim, int kv_heads, int group, int64_t n_seqs, int64_t n_tokens, int64_t max_len, int window,
                  size_t room)
{
    KvPlan p = {};
    const int64_t rows = n_tokens * group;
    // tokens a row tile may see
    int64_t span = std::min<int64_t>(max_len, KV_MOST_TOKENS);
    if (window) span = std::min<int64_t>(span, (int64_t)window + 128 + STEP);
    // Query rows of a tile.  Up to 8, 16 or 32 a sequence on average: all of
    // them (8 sequences of 20 rows on 4000 tokens, heads of 128: 28.0 us with
    // 32 and 30.2 with 16, heads of 64 23.9 and 25.0; 32 sequences 63 and 75,
    // 45 and 57).  More: 128 (kv_prompt.hip) where there is work enough, by the
    // products of 128 rows with a token, as that kernel needs many workgroups
    // to be fast and others to follow them.  With tiles of 16, 32 and 128 rows,
    // 32 heads on 8, heads of 128 and (heads of 64), us:
    //   1024 on themselves, 2^18   41, 43, 51        (31, 28, 40)
    //   1024 on 2048, 2^19         76, 71, 83        (56, 54, 63)
    //   512 on 4096, 2^19          87, 108, 78       (63, 80, 63)
    //   256 on 8192, 2^19          121, 88, 77       (88, 63, 72)
    //   2048 on themselves, 2^20   100, 97, 89       (73, 68, 78)
    //   512 on 8192, 2^20          162, 182, 130     (116, 135, 112)
    //   4096 on 8192, 2^23         875, 770, 639     (601, 523, 487)
    // 33 to 64 rows with that work: 32, of which 128 would be half empty (8
    // sequences of 64 on 16384: 101, 94, 185 and 73, 66, 99); with less, 16 (8
    // of 64 on 4000: 39, 44, 63 and 31, 32, 39).  Heads of 256 have registers
    // for 16 rows and a second wavefront, but not for more: 1024 on 4096, 16
    // heads on 4, 131 us (32 rows and 128 rows took half as long again and a
    // fifth more).
    const bool much = (rows + 127) / 128 * kv_heads * std::min<int64_t>(span, 1 << 20) >= 1 << 19;
    p.tile = rows <= 8 * n_seqs                       ? 8
             : rows <= 16 * n_seqs || head_dim > 128 ? 16
             : rows <= 32 * n_seqs                   ? 32
             : !much                                 ? 16
             : rows <= 64 * n_seqs                   ? 32
                                                     : 128;
    p.tiles = p.pieces = rows / p.tile + n_seqs;
    p.splits = 1;
    const size_t result = (size_t)kv_heads * p.tile * (head_dim + 2) * sizeof(float);
    if (p.tile == 128) {
        // Chunks for two workgroups a CU: more cost their results' way through
        // memory (2048 new tokens on themselves: 101 us with twice as many, 89
        // so), fewer leave CUs idle (512 on 16384: 385 us with half, 235 so)
        const int64_t base = std::max(n_seqs, (rows + p.tile - 1) / p.tile) * kv_heads;
        int64_t splits = std::min((512 + base - 1) / base, (span + LEAST - 1) / LEAST);
        splits = std::max<int64_t>(std::min(splits, (int64_t)(room / result) / p.tiles), 1);
        p.chunk = (int)(((span + splits - 1) / splits + CHUNK - 1) / CHUNK * CHUNK);
        p.splits = (int)std::max<int64_t>((span + p.chunk - 1) / std::max(p.chunk, 1), 1);
        p.work_bytes = p.splits > 1 ? p.tiles * p.splits * result : 0;
        return p;
    }
    if (!cut(kv_heads, n_seqs, rows, p.tile, span)) return p;
    // Into about 768 pieces, three for a CU (replays of a graph): 16 sequences
    // of 501 to 8190 tokens take 28.5 us, with 512 32.7, with 1024 30.1 and with
    // 1536 31.7; one of 131071 42.7, 41.7, 42.9 and 45.8; 32 of 16384 119, 118,
    // 120 and 124.
    const size_t notes = p.tiles * sizeof(int2);
    int64_t pieces = std::max(768 / kv_heads, 1) + p.tiles;
    if (room < notes || (room - notes) / result < (size_t)pieces) pieces = room < notes ? 0 : (room - notes) / result;
    if (pieces <= p.tiles) return p;
    p.target = (int)(pieces - p.tiles);
    p.pieces = pieces;
    p.first_at = pieces * result;
    p.work_bytes = p.first_at + notes;
    return p;
}

size_t lw_kv_most_work(int head_dim, int kv_heads, int group, int64_t n_seqs, int64_t n_tokens, int64_t max_len)
{
    const int64_t rows = n_tokens * group, span = std::min<int64_t>(max_len, KV_MOST_TOKENS);
    auto result = [&](int tile) { return (size_t)kv_heads * tile * (head_dim + 2) * sizeof(float); };
    size_t most = 0;
    // cut(): sequences that are cut whatever their rows, and those that are for
    // the sake of a long one (the root as n (n kv) <= 32 span has it, or one more)
    const int64_t few = (1023 / kv_heads), many = (int64_t)std::sqrt(32.0 * (double)span / kv_heads) + 1;
    for (int tile = 8; span > 1024 && tile <= (head_dim > 128 ? 16 : 32); tile *= 2) {
        if (rows <= (tile == 8 ? 0 : tile / 2)) break;       // (one sequence of that many takes smaller tiles)
        const int64_t full = rows / tile;
        const int64_t tiles = std::max(few ? std::min(full, few) + std::min(n_seqs, few) : 0,
                                       std::min(full, std::min(n_seqs, many)) + std::min(n_seqs, many));
        most = std::max(most, (std::max(768 / kv_heads, 1) + tiles) * result(tile) + tiles * sizeof(int2));
    }
    // tiles of 128: by the larger of sequences and full tiles, x, as the plan
    // counts workgroups
    const KvPlan all = lw_kv_plan(head_dim, kv_heads, group, 1, n_tokens, max_len, 0, 0);
    if (all.tile == 128)
        for (int64_t x = 1; x * kv_heads < 512 && x <= std::max(n_seqs, (rows + 127) / 128); x++) {
            const int64_t splits = std::min((512 + x * kv_heads - 1) / (x * kv_heads), (span + LEAST - 1) / LEAST);
            if (splits > 1) most = std::max(most, (std::min(x, rows / 128) + std::min(x, n_seqs)) * splits * result(128));
        }
    return most;
}

hipError_t lw_launch_kv_attend(const KvAttend &a, int head_dim, int dtype, const KvPlan &p, hipStream_t s)
{
    if (p.tile == 128) return lw_launch_kv_prompt(a, head_dim, dtype, p, s);
    if (head_dim == 64) return launch_dim<64>(a, dtype, p, s);
    if (head_dim == 128) return launch_dim<128>(a, dtype, p, s);
    if (head_dim == 256) return launch_dim<256>(a, dtype, p, s);
    return hipErrorInvalidValue;
}
