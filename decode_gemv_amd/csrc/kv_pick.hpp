// kv_pick.hpp -- the largest m of a workgroup's keys in LDS, of equal ones the
// first, and the places of those taken in ascending order.  Internal to the
// library.
//
// The key that divides them is found from its highest 11 bits on: a histogram of
// the keys that share the bits found so far, and the counter in which the count
// from above passes m.  Keys count from the smallest on and are moved up as far
// as the largest allows: they then spread over the counters (64 lanes that reach
// for one of them take turns), and the first 11 bits mostly do.  Counts are whole
// numbers, so that the order in which lanes add does not matter.
#ifndef LW_KV_PICK_HPP
#define LW_KV_PICK_HPP

#include "kv_attend.hpp"

namespace {

constexpr int PICK_MOST = 32768;       // keys (their counts fit 16 bits)

// Keys are 0 (never taken), MUST (always) or between.
constexpr uint32_t MUST = ~0u;

// What a workgroup's keys are, of the last two those between.
struct Keys {
    uint32_t there, must, least, most;
};

// Taken are those between whose place y = (key - least) << up has
// (y & mask) > value, and of those where it is value the first `ties`.
struct Cut {
    uint32_t least, up, mask, value;
    int ties;

    __device__ __forceinline__ uint32_t place(uint32_t key) const { return (key - least) << up & mask; }
};

// fp32 numbers as whole numbers in the same order; above 0 for all but NaN with
// its sign bit set.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    return u >> 31 ? ~u : u | 0x80000000u;
}

// The bits of lanes before this one.
__device__ __forceinline__ int below(uint64_t x)
{
    return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(x >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)x, 0));
}

// The largest of x over the lanes up to this one (prefix() has the steps).
__device__ __forceinline__ uint32_t prefix_max(uint32_t x)
{
    auto with = [&](auto ctrl, auto rows) {
        x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl.value, rows.value, 0xF, true));
    };
    using std::integral_constant;
    with(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});
    with(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
    with(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
    with(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
    with(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});
    with(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});
    return x;
}

// What a thread has put: its keys' counts (there, and << 16 those that must be), and
// the smallest and largest of the others.
struct Tally {
    uint32_t counts = 0, least = ~0u, most = 0;

    __device__ __forceinline__ void add(uint32_t k)
    {
        counts += k == 0 ? 0u : k == MUST ? 0x10001u : 1u;
        least = k == 0 ? least : min(least, k);
        most = k == MUST ? most : max(most, k);
    }

    // The workgroup's, and the sum of x (at most 2^16).  sums: T / 16 words of LDS.
    // Ends with a barrier: the keys are there.
    template <int T>
    __device__ __forceinline__ Keys meet(uint32_t *sums, uint32_t &x) const
    {
        const uint32_t n = prefix(counts), low = prefix_max(~least), high = prefix_max(most);
        x = prefix(x);
        if ((threadIdx.x & 63) == 63) *reinterpret_cast<uint4 *>(sums + 4 * (threadIdx.x >> 6)) = make_uint4(n, ~low, high, x);
        __syncthreads();
        Keys r = {0, 0, ~0u, 0};
        x = 0;
#pragma unroll
        for (int w = 0; w < T / 64; w++) {
            const uint4 y = *reinterpret_cast<const uint4 *>(sums + 4 * w);
            r.there += y.x & 0xFFFFu;
            r.must += y.x >> 16;
            r.least = min(r.least, y.y);
            r.most = max(r.most, y.z);
            x += y.w;
        }
        return r;
    }
};

// Histograms have 2048 counters, 32 and four words of padding in a row (64 lanes
// that read a row each then meet no bank twice).  There are two, used in turn,
// and two numbers that a wavefront leaves for the others.
constexpr int PICK_ROW = 36, PICK_HIST = 64 * PICK_ROW, PICK_WORDS = 2 * PICK_HIST + 4;

// Keys whose loads are under way at once.
constexpr int PICK_AT_ONCE = 2;

// The cut that takes all that must be and so many of the others that they are m
// (fewer than there are).  hist: PICK_WORDS of LDS, 16-byte aligned.  One wavefront
// looks for the counter (all of a large workgroup doing so took longer than the
// barrier after it).
template <int T>
__device__ __forceinline__ Cut pick_cut(const uint32_t *key, int n, Keys all, int m, uint32_t *hist)
{
    constexpr int BITS[3] = {11, 11, 10}, SHIFT[3] = {21, 10, 0};
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Cut c = {all.least, 0, 0, 0, m - (int)all.must};
    if (c.ties <= 0) return {0, 0, ~0u, ~0u, 0};             // (none of them)
    c.up = __builtin_clz(max(all.most - all.least, 1u));
    for (int i = threadIdx.x; i < PICK_HIST / 4; i += T) reinterpret_cast<uint4 *>(hist)[i] = uint4{};
#pragma unroll
    for (int pass = 0; pass < 3; pass++) {
        uint32_t *h = hist + pass % 2 * PICK_HIST, *next = hist + (pass + 1) % 2 * PICK_HIST;
        uint2 *found = reinterpret_cast<uint2 *>(hist + 2 * PICK_HIST);
        __syncthreads();
        for (int i0 = wave * 64; i0 < n; i0 += PICK_AT_ONCE * T) {
            uint32_t k[PICK_AT_ONCE];
#pragma unroll
            for (int i = 0; i < PICK_AT_ONCE; i++) k[i] = key[min(i0 + i * T + lane, n - 1)];
#pragma unroll
            for (int i = 0; i < PICK_AT_ONCE; i++) {
                if (i0 + i * T >= n) break;
                const uint32_t x = (k[i] - c.least) << c.up >> SHIFT[pass] & ((1u << BITS[pass]) - 1);
                if (i0 + i * T + lane < n && k[i] - 1 < MUST - 1 && c.place(k[i]) == c.value)
                    atomicAdd(&h[x / 32 * PICK_ROW + x % 32], 1u);
            }
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            // rows from the last on, one a lane, then the counters of one row
            const uint4 *row = reinterpret_cast<const uint4 *>(h + (63 - lane) * PICK_ROW);
            int own = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) own += (int)(row[i].x + row[i].y + row[i].z + row[i].w);
            const int sum = prefix(own), r = __popcll(__ballot(sum < c.ties));
            const int above = r ? __builtin_amdgcn_readlane(sum, r - 1) : 0;
            const int in = lane < 32 ? (int)h[(63 - r) * PICK_ROW + 31 - lane] : 0, upto = above + prefix(in);
            const int i = __popcll(__ballot(upto < c.ties));
            // what the counter has, and what is taken of it; the counter
            if (lane == i) *found = make_uint2((uint32_t)in << 16 | (uint32_t)(c.ties - (upto - in)), (63 - r) * 32 + 31 - i);
        } else {
            for (int i = threadIdx.x - 64; i < PICK_HIST / 4; i += T - 64)         // (last read before the barrier above)
                reinterpret_cast<uint4 *>(next)[i] = uint4{};
        }
        __syncthreads();
        const uint2 f = *found;
        c.ties = (int)(f.x & 0xFFFFu);
        c.mask |= ((1u << BITS[pass]) - 1) << SHIFT[pass];
        c.value |= f.y << SHIFT[pass];
        if (f.x >> 16 == (uint32_t)c.ties) break;            // all that share the bits are taken
    }
    return c;
}

// put(place, rank) for each key taken (all that are there where `every`), rank by
// rank; returns their number.  sums: T / 64 words of LDS.  A wavefront has its share
// of the keys 64 at a time, whose ranks are counts of bits: what this takes is how
// many instructions wait for the one before.
template <int T, class F>
__device__ __forceinline__ int pick_each(const uint32_t *key, int n, bool every, Cut c, uint32_t *sums, F put)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int share = ((n + 63) / 64 + T / 64 - 1) / (T / 64) * 64, i0 = min(wave * share, n), i1 = min(i0 + share, n);
    // f(key's place, whether it is taken for sure, whether it is on the cut)
    auto each = [&](auto f) {
        for (int i = i0; i < i1; i += PICK_AT_ONCE * 64) {
            uint32_t k[PICK_AT_ONCE];
#pragma unroll
            for (int j = 0; j < PICK_AT_ONCE; j++) k[j] = key[min(i + j * 64 + lane, n - 1)];
#pragma unroll
            for (int j = 0; j < PICK_AT_ONCE; j++) {
                const int at = i + j * 64 + lane;
                if (at - lane >= i1) break;
                const uint32_t y = c.place(k[j]);
                const bool there = at < i1 && k[j] != 0, is = there && (every || k[j] == MUST || y > c.value);
                f(at, is, there && !is && y == c.value);
            }
        }
    };
    uint32_t mine = 0;                                       // taken for sure, and on the cut << 16
    each([&](int, bool is, bool tie) { mine += is ? 1u : tie ? 0x10000u : 0u; });
    mine = prefix(mine);
    if (lane == 63) sums[wave] = mine;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < T / 64; w++) {
        if (w < wave) before += sums[w];
        all += sums[w];
    }
    before = __builtin_amdgcn_readfirstlane(before);
    int above = before & 0xFFFFu, on = before >> 16;
    if ((int)(all >> 16) <= c.ties) {                        // (mostly: all on the cut are taken)
        above += on;
        each([&](int place, bool is, bool tie) {
            const uint64_t taken = __ballot(is || tie);
            if (is || tie) put(place, above + below(taken));
            above += __popcll(taken);
        });
    } else {
        each([&](int place, bool is, bool tie) {
            const uint64_t sure = __ballot(is), ties = __ballot(tie);
            const int rank = on + below(ties);
            if (is || (tie && rank < c.ties)) put(place, above + below(sure) + min(rank, c.ties));
            above += __popcll(sure);
            on += __popcll(ties);
        });
    }
    return (int)(all & 0xFFFFu) + min((int)(all >> 16), c.ties);
}

}  // namespace

#endif
