// kv_pick.hpp -- the largest m of a workgroup's keys in LDS, of equal ones the
// first, and the places of those taken in ascending order.  Internal to the
// library.
//
// The key that divides them is found from its highest byte on: a histogram of
// the keys that share the bytes found so far, and the byte in which the count
// from above passes m.  Sums and counts are whole numbers, so that the order in
// which the counters are reached does not matter.
#ifndef LW_KV_PICK_HPP
#define LW_KV_PICK_HPP

#include "kv_attend.hpp"

namespace {

constexpr int PICK_MOST = 32768;       // keys (their counts fit 16 bits)

// Taken are keys with (key & mask) > value, and of those where it is value the
// first `ties`.
struct Cut {
    uint32_t mask, value;
    int ties;
};

// fp32 numbers as whole numbers in the same order; above 0 for all but NaN with
// its sign bit set.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    return u >> 31 ? ~u : u | 0x80000000u;
}

// The cut that takes m of n keys, 1 <= m <= n.  hist: 512 counters in LDS.
// Begins with a barrier: the keys are then there.
template <int T>
__device__ __forceinline__ Cut pick_cut(const uint32_t *key, int n, int m, uint32_t *hist)
{
    const int lane = threadIdx.x & 63;
    Cut c = {0, 0, m};
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
#pragma unroll
    for (int pass = 0; pass < 4; pass++) {
        const int shift = 24 - 8 * pass;
        uint32_t *h = hist + pass % 2 * 256, *next = hist + (pass + 1) % 2 * 256;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += T) {
            const uint32_t k = key[i];
            if ((k & c.mask) == c.value) atomicAdd(&h[k >> shift & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 256) next[threadIdx.x] = 0;        // (last read before the barrier above)
        // bins 255 - 4 lane and the three below it
        const uint4 b = *reinterpret_cast<const uint4 *>(h + 252 - 4 * lane);
        const int own[4] = {(int)b.w, (int)b.z, (int)b.y, (int)b.x};
        const int sum = prefix(own[0] + own[1] + own[2] + own[3]);
        const int at = __popcll(__ballot(sum < c.ties));     // the lane whose bins the count passes in
        int above = at ? __builtin_amdgcn_readlane(sum, at - 1) : 0, bin = 255 - 4 * at, in = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            in = __builtin_amdgcn_readlane(own[i], at);
            if (above + in >= c.ties) break;
            above += in;
            bin--;
        }
        c.ties -= above;
        c.mask |= 0xFFu << shift;
        c.value |= (uint32_t)bin << shift;
        if (in == c.ties) break;                             // all that share the bytes are taken
    }
    return c;
}

// put(place, rank) for each key taken, rank by rank; returns their number.
// sums: T / 64 counters in LDS.
template <int T, class F>
__device__ __forceinline__ int pick_each(const uint32_t *key, int n, Cut c, uint32_t *sums, F put)
{
    const int each = (n + T - 1) / T, i0 = min((int)threadIdx.x * each, n), i1 = min(i0 + each, n);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t mine = 0;                                       // above the cut, and on it << 16
    for (int i = i0; i < i1; i++) {
        const uint32_t k = key[i] & c.mask;
        mine += k > c.value ? 1u : k == c.value ? 0x10000u : 0u;
    }
    const uint32_t upto = prefix(mine);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    uint32_t before = upto - mine, all = 0;
#pragma unroll
    for (int w = 0; w < T / 64; w++) {
        if (w < wave) before += sums[w];
        all += sums[w];
    }
    int above = before & 0xFFFFu, on = before >> 16;
    for (int i = i0; i < i1; i++) {
        const uint32_t k = key[i] & c.mask;
        const bool is = k > c.value, tie = k == c.value;
        if (is || (tie && on < c.ties)) put(i, above + min(on, c.ties));
        above += is;
        on += tie;
    }
    return (int)(all & 0xFFFFu) + min((int)(all >> 16), c.ties);
}

}  // namespace

#endif
