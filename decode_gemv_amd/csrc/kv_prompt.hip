// kv_prompt.hip -- attention of many new tokens over the 4-bit key/value cache,
// for heads of 64 and 128 (lw_kv_plan in kv_attend.hip says when).
//
// The mathematics is kv_attend.hip's.  There each wavefront unpacks the codes
// that it uses, which for many query rows is most of its work: 152 of some 440
// instructions for 32 tokens and 32 rows.  Here a workgroup has 128 rows of a
// sequence, 32 for each wavefront, and goes through the tokens in tiles of 64:
// each wavefront unpacks a quarter of a tile's keys and values into LDS, laid
// out as the matrix operands that all four then read in whole 16-byte lanes,
// and turns their pairs into the factors of scores and values, once per token
// instead of once per lane.  Two buffers: a tile is unpacked, and the one after
// it loaded, while the one before is used, with one barrier a tile.  No tokens
// are shared out between wavefronts, so nothing has to be joined at the end,
// and two workgroups stand on a CU whose phases (unpacking, products,
// exponentials) fill each other's gaps.
//
// What bounds it: issue.  For 32 tokens and 32 rows of 128 dimensions a
// wavefront has 768 cycles of matrix instructions and some 900 of others, at
// what they were measured to take (4 to 4.6 a multiply-add, a conversion or an
// operation on packed halves, 2.6 a multiplication or addition, 8.5 an
// exponential), and a SIMD does one such part in some 1800: with two wavefronts
// the two kinds hardly overlap, and the times of the parts add up (4096 tokens
// on 16384, 1467 us: unpacking takes 320, the values' products 250 for p dv and
// 250 for what its rounding leaves, the keys' 200, the factors' reads 200, the
// exponentials 130).  A wavefront alone on its SIMD issues one instruction in
// 5.4 cycles and takes as long for a part as two side by side, so the calls
// that leave the longest rows' workgroups alone at the end (prompts of up to
// 2048 tokens, where all are there from the start) are bound by those.
//
// Measured, bf16, 32 heads on 8 (replays of a graph; in brackets tiles of 32
// rows of kv_attend.hip): heads of 128, 16384 tokens on themselves 3.28 ms, 670
// TFLOP/s (4.03 ms), 2048 on 16384 814 us, 633 (943), 2048 on themselves 89 us,
// 386 (97); heads of 64, 2.15 ms, 511 (2.73), 614 us, 420 (645), and 78 us (68).
//
// Rounding: as in kv_attend.hip.  The second operand of p dv costs 24 % of the
// longest calls (3.28 ms and not 2.65) and 11 % of 2048 on themselves; without
// it fp16 results lie 3.0e-4 of their size from 64 bits, with it 2.1e-4, which
// is their own rounding.
#include <stddef.h>

#include <algorithm>
#include <type_traits>

#include "kv_attend.hpp"

namespace {

constexpr int WV = 4, WIDE = 32, ROWS = WV * WIDE;

template <int D>
struct Tile {
    static constexpr int TT = 64, SUBS = TT / 32;            // tokens of a tile
    static constexpr int DW = D / 8, PER = DW / 2;           // words of a token, and of a half of the lanes
    static constexpr int W = D >= 128 ? 4 : 2, U = DW / W;   // words of a key unit, units of a token
    static constexpr int NT = D / 32;                        // output tiles along the head
    static constexpr int TPW = TT / WV;                      // tokens of a wavefront's value words and pairs
    static constexpr int VS = 64 * WV / (TT / 4 * DW);       // threads that share a value unit, by halves of its words
    static_assert(TT * U == 64 * WV, "a thread has one key unit");
    uint4 k[SUBS][PER][64];                                  // operands of K Q^T
    uint2 v[SUBS][2][NT][64][2];                             // operands of V^T P^T
    float2 kf[TT], vf[TT];                                   // dk, 8 dk - mk; dv, 8 dv - mv
    float dmax[WV];                                          // largest dv of the tokens that a wavefront unpacked,
    uint32_t odd[WV];                                        // infinity where the pairs of some (these bits) are not finite
};

// What a wavefront has loaded of a tile.
template <int D>
struct Raw {
    uint32_t k[Tile<D>::W];
    uint4 v;
    uint32_t dm;                 // lanes below TPW: a key's pair, the others: a value's
};

// Where a thread's operands go in a tile, in bytes: its first key word's, its
// first code's of the value words' halves, and its pair's; what follows lies at
// fixed distances (kept in registers as they are, not as what they are made of).
template <int D>
struct Put {
    static constexpr int HALVES = 2 / Tile<D>::VS;
    uint32_t k, v[HALVES];
    __device__ __forceinline__ Put(int thread)
    {
        using L = Tile<D>;
        const int t = thread / (L::U * 16) * 16 + thread % 16, w = thread / 16 % L::U * L::W;
        k = ((t / 32 * L::PER + w % L::PER) * 64 + t % 32 + w / L::PER * 32) * 16;
        asm("" : "+v"(k));
        // token group g of the tile: half g % 2 of the lanes, place g / 2 % 2 of the operand
        const int vu = thread / L::VS, g = vu / L::DW, c = vu % L::DW;
#pragma unroll
        for (int i = 0; i < HALVES; i++) {
            const int n = 4 * (L::VS == 2 ? thread % 2 : i);
            v[i] = offsetof(Tile<D>, v) +
                   ((g / 4 * L::NT + n % L::NT) * 64 + c + L::DW * (n / L::NT) + g % 2 * 32) * 16 + g / 2 % 2 * 8;
            asm("" : "+v"(v[i]));
        }
    }
};

template <int D>
__device__ __forceinline__ void unpack(Tile<D> &o, const Raw<D> &r, const Put<D> &at, Masks mk, int wave, int lane)
{
    using L = Tile<D>;
    char *base = reinterpret_cast<char *>(&o);
#pragma unroll
    for (int i = 0; i < L::W; i++) *reinterpret_cast<h8 *>(base + at.k + i * 1024) = spread8(r.k[i], mk);
    const uint32_t *x = reinterpret_cast<const uint32_t *>(&r.v);
#pragma unroll
    for (int i = 0; i < Put<D>::HALVES; i++) {
        const uint32_t sel = (L::VS == 2 ? lane % 2 : i) ? 0x07060302u : 0x05040100u;
        const uint32_t a = __builtin_amdgcn_perm(x[1], x[0], sel), b = __builtin_amdgcn_perm(x[3], x[2], sel);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t p = j >= 2 ? a >> 8 : a, q = j >= 2 ? b >> 8 : b;
            const h2 lo = j % 2 ? centred<true>(p, mk) : centred<false>(p, mk);
            const h2 hi = j % 2 ? centred<true>(q, mk) : centred<false>(q, mk);
            *reinterpret_cast<uint2 *>(base + at.v[i] + j % L::NT * 1024 + j / L::NT * L::DW * 16) =
                make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
        }
    }
    // A value's pair that is not finite counts as (0, 0), so that it is nothing
    // to the rows that do not see it; step() makes the others' outputs NaN
    float d = half_lo(r.dm), c = fmaf(d, 8.0f, -half_hi(r.dm));
    const bool odd = !(fabsf(c) < __builtin_inff());
    const uint32_t odds = (uint32_t)(__ballot(odd) >> L::TPW) & ((1u << L::TPW) - 1);       // the values'
    if (lane < L::TPW) {
        o.kf[wave * L::TPW + lane] = make_float2(d, c);
    } else if (lane < 2 * L::TPW) {
        o.vf[wave * L::TPW + lane % L::TPW] = make_float2(odd ? 0.0f : d, odd ? 0.0f : c);
    }
    d = odd ? 0.0f : d;
    auto most = [&](auto ctrl) {
        d = fmaxf(d, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, d), ctrl.value, 0xF, 0xF, false)));
    };
    most(std::integral_constant<int, 0xB1>{});               // lane ^ 1
    most(std::integral_constant<int, 0x4E>{});               // lane ^ 2
    most(std::integral_constant<int, 0x141>{});              // 7 - lane of eight
    most(std::integral_constant<int, 0x140>{});              // 15 - lane of sixteen
    if (lane == L::TPW) {
        o.dmax[wave] = odds ? __builtin_inff() : d;
        o.odd[wave] = odds;
    }
}

template <int D>
struct Rows {
    static constexpr int NT = Tile<D>::NT;
    h8 q[Tile<D>::PER];
    f16v o[NT];
    float qs, qsum;
    float mo, ref, thr, dlim;    // offset, its reference, and what calls for a new one (kv_attend.hip)
    float l, z;

    __device__ __forceinline__ float k() const { return (float)(7 + 127 - (int)(__builtin_bit_cast(uint32_t, dlim) >> 23)); }
    __device__ __forceinline__ Offset offset() const { return offset_of(ref, qs, mo, k()); }
};

__device__ __forceinline__ f16v product(uint4 v, const h2 (&p)[4], f16v o)
{
    const h8 x = {p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, v), x, o, 0, 0, 0);
}

// 32 tokens of a tile, the first being t0.  masked: some of them may be hidden
// from some rows; a hidden token's score is -infinity.
template <int D>
__device__ __forceinline__ void step(Rows<D> &st, const Tile<D> &tile, int sub, int t0, bool masked, Span seen, Masks mk, int lane)
{
    using L = Tile<D>;
    constexpr int PIECES = 32 / L::TPW;
    const int g = lane / WIDE;
    f16v acc;
#pragma unroll
    for (int i = 0; i < 16; i++) acc[i] = 0.0f;
    auto values = [&](int kk, int n) { return *reinterpret_cast<const uint4 *>(&tile.v[sub][kk][n][lane][0]); };
    const float4 *kf = reinterpret_cast<const float4 *>(&tile.kf[sub * 32 + 4 * g]);
    const float4 *vf = reinterpret_cast<const float4 *>(&tile.vf[sub * 32 + 4 * g]);
    uint4 kw[L::PER];
#pragma unroll
    for (int j = 0; j < L::PER; j++) kw[j] = tile.k[sub][j][lane];
    float dm[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; i++) dm[i] = tile.dmax[sub * PIECES + i];
#pragma unroll
    for (int j = 0; j < L::PER; j++)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, kw[j]), st.q[j], acc, 0, 0, 0);
    // a lane's tokens: 8 a + 4 g + b, its four of every eight
    float s[4][4], top = -__builtin_inff(), dtop = 0.0f;
#pragma unroll
    for (int a = 0; a < 4; a++) {
        const float4 x = kf[4 * a], y = kf[4 * a + 1];
        s[a][0] = fmaf(acc[4 * a], x.x, x.y * st.qsum);
        s[a][1] = fmaf(acc[4 * a + 1], x.z, x.w * st.qsum);
        s[a][2] = fmaf(acc[4 * a + 2], y.x, y.y * st.qsum);
        s[a][3] = fmaf(acc[4 * a + 3], y.z, y.w * st.qsum);
    }
#pragma unroll
    for (int i = 0; i < PIECES; i++) dtop = fmaxf(dtop, dm[i]);
    if (masked) {
        int first = t0 + 4 * g - seen.lo;
        asm volatile("" : "+v"(first));                      // (kept from being worked out ahead of the loop)
        dtop = 0.0f;                                         // of what the row sees
#pragma unroll
        for (int a = 0; a < 4; a++) {
            const float4 x = vf[4 * a], y = vf[4 * a + 1];
            const float dv[4] = {x.x, x.z, y.x, y.z};
#pragma unroll
            for (int b = 0; b < 4; b++) {
                const bool out = (unsigned)(first + 8 * a + b) >= (unsigned)(seen.hi - seen.lo);
                s[a][b] = out ? -__builtin_inff() : s[a][b];
                dtop = fmaxf(dtop, out ? 0.0f : dv[b]);
            }
        }
        uint32_t bits = 0;                                   // tokens that count as (0, 0), and that the row sees
#pragma unroll
        for (int i = 0; i < PIECES; i++) bits |= tile.odd[sub * PIECES + i] << i * L::TPW;
        bits &= (uint32_t)((1ull << min(max(seen.hi - t0, 0), 32)) - 1) & ~(uint32_t)((1ull << min(max(seen.lo - t0, 0), 32)) - 1);
        dtop = bits ? __builtin_inff() : dtop;
    }
#pragma unroll
    for (int a = 0; a < 4; a++)
#pragma unroll
        for (int b = 0; b < 4; b++) top = fmaxf(top, s[a][b]);
    if (__any(top > st.thr || dtop > st.dlim)) {             // rare: a new offset, as in kv_attend.hip
        top = fmaxf(top, __shfl_xor(top, 32));
        dtop = fmaxf(dtop, __shfl_xor(dtop, 32));
        const bool need = top > st.thr || dtop > st.dlim;
        const Offset old = st.offset();
        if (need) {
            const uint32_t up = __builtin_bit_cast(uint32_t, fminf(fmaxf(dtop, 0x1p-24f), 65504.0f)) + 0x7FFFFFu;
            st.dlim = fmaxf(st.dlim, __builtin_bit_cast(float, up & 0xFF800000u));          // up to a power of two
            st.ref = fmaxf(st.ref, top);
            set_offset(st.ref, st.qs, st.k(), st.mo, st.thr);
        }
        const Offset now = st.offset();
#pragma unroll
        for (int a = 0; a < 4; a++)
#pragma unroll
            for (int b = 0; b < 4; b++) s[a][b] -= now.shift;
        const float f = between(old, now);
        st.l *= f;
        st.z = dtop > 65504.0f ? __builtin_nanf("") : st.z * f;
#pragma unroll
        for (int n = 0; n < L::NT; n++)
#pragma unroll
            for (int j = 0; j < 16; j++) st.o[n][j] *= f;
    }
#pragma unroll
    for (int kk = 0; kk < 2; kk++) {
        h2 e[4], rest[4];                                    // p dv, and what its rounding leaves
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const int a = 2 * kk + c / 2;
            const float4 x = vf[4 * a + c % 2];              // (dv, 8 dv - mv) of two tokens
            const float p = __builtin_amdgcn_exp2f(fmaf(s[a][c % 2 * 2], st.qs, -st.mo));
            const float r = __builtin_amdgcn_exp2f(fmaf(s[a][c % 2 * 2 + 1], st.qs, -st.mo));
            st.l += p;
            st.l += r;
            st.z = fmaf(r, x.w, fmaf(p, x.y, st.z));
            split2(p * x.x, r * x.z, mk, e[c], rest[c]);
        }
        uint4 vw[L::NT];
#pragma unroll
        for (int n = 0; n < L::NT; n++) {
            vw[n] = values(kk, n);
            st.o[n] = product(vw[n], e, st.o[n]);
        }
#pragma unroll
        for (int n = 0; n < L::NT; n++) st.o[n] = product(vw[n], rest, st.o[n]);
    }
}

// The row tile of workgroups y: the last first, as later rows see more tokens,
// every second four the other way round, as consecutive workgroups of an XCD
// go round its four shader engines and would give the first of them the
// longest of each four.  (Chunks come last in the grid for the same reason:
// with a tile's two chunks side by side, half of the engines get the short
// ones, which cost 2048 tokens on themselves a fifth.)
__device__ __forceinline__ int order_of(int tiles, int y)
{
    if ((y | 3) < tiles && y & 4) y ^= 3;
    return tiles - 1 - y;
}

template <int D, class T>
__global__ __launch_bounds__(WV * 64, (D > 64 ? 2 : 3)) void k_kv_prompt(KvAttend a)
{
    using L = Tile<D>;
    constexpr int PD = 64, ROWF = PD + 4;                    // dimensions of a pass of the end, and a row in LDS
    constexpr size_t BYTES = std::max(2 * sizeof(Tile<D>), sizeof(float) * ROWS * ROWF);
    __shared__ uint4 mem[BYTES / 16];
    __shared__ float sl[ROWS], sm[ROWS];
    Tile<D> *tiles = reinterpret_cast<Tile<D> *>(mem);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane % WIDE, g = lane / WIDE, head = blockIdx.x;
    const int split = blockIdx.z, x = order_of(gridDim.y, blockIdx.y);
    const RowTile t = row_tile<ROWS>(a, x);
    if (t.rows == 0) return;
    const Span mine = chunk_of(t, a.chunk, a.splits, split);
    if (split > 0 && mine.lo >= mine.hi) return;             // (chunk 0 always leaves a result)
    const int P = 1 << a.g.page_shift;

    const int32_t *pages = a.g.table + (int64_t)t.seq * a.g.stride;
    // 32 tokens lie in one page: the entries of a tile's (of a tile past the
    // end: the last one's), one a lane
    const int piece = wave * L::TPW;
    auto entries_at = [&](int t0) { return pages[min(t0 + lane % L::SUBS * 32, mine.hi - 1) >> a.g.page_shift]; };
    auto known = [&](int32_t entries) {                      // which of them name a page
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < L::SUBS; i++)
            bits |= (uint32_t)__builtin_amdgcn_readlane(entries, i) < a.g.n_pages ? 1u << i : 0u;
        return bits;
    };
    Raw<D> raw;
    auto load = [&](int t0, int32_t entries) {
        const uint32_t entry = (uint32_t)__builtin_amdgcn_readlane(entries, piece / 32);
        const bool here = entry < a.g.n_pages && t0 + piece < mine.hi;
        const auto block = __builtin_amdgcn_make_buffer_rsrc(
            a.g.pages + (uint64_t)(here ? entry : 0u) * (uint64_t)a.g.page_bytes + (uint32_t)head * (uint32_t)a.g.block_bytes,
            0, here ? a.g.block_bytes : 0, 0x00027000);
        const uint32_t at = (t0 + piece) & (P - 1), k = lane * L::W * 4;
        if constexpr (L::W == 4) {
            const uint4 w = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(block, k, at * (D / 2), 0));
            raw.k[0] = w.x, raw.k[1] = w.y, raw.k[2] = w.z, raw.k[3] = w.w;
        } else {
            const uint2 w = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(block, k, at * (D / 2), 0));
            raw.k[0] = w.x, raw.k[1] = w.y;
        }
        raw.v = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
            block, lane / L::VS * 16, P * (D / 2) + at * (D / 2), 0));
        raw.dm = __builtin_bit_cast(uint32_t, __builtin_amdgcn_raw_buffer_load_b32(
            block, lane % L::TPW * 4 + (lane < L::TPW ? 0 : P * 4), P * D + at * 4, 0));
    };

    Rows<D> st;
    Masks mk = masks();
    asm("v_mov_b32 %0, 1.0" : "=v"(mk.one));                 // (scalar registers are short here)
    asm("v_mov_b32 %0, 0x000f000f" : "=v"(mk.low));
    asm("v_mov_b32 %0, 0x00f000f0" : "=v"(mk.high));
    const Put<D> put(threadIdx.x);
    const bool any = mine.lo < mine.hi;
    uint32_t now = 0, next = 0;                              // the parts with a page of the tile in use, and of the one loaded;
    int32_t after = -1;                                      // the entries of the one after it
    {
        Query<D, WIDE, T> q;
        const int2 at = token_of(a, t, min(wave * WIDE + m, t.rows - 1));
        q.load(a.q, t.row0 + at.x, (int64_t)head * a.group + at.y, lane);
        if (any) {
            const int32_t entries = entries_at(mine.lo);
            load(mine.lo, entries);
            now = known(entries);
            after = entries_at(mine.lo + L::TT);
        }
        q.make(st.qs, st.qsum, a.scale, [&](int j, h8 y) { st.q[j] = y; });
    }
    st.mo = NONE;
    st.ref = st.thr = UNSEEN;
    st.l = st.z = st.dlim = 0.0f;
#pragma unroll
    for (int n = 0; n < L::NT; n++)
#pragma unroll
        for (int j = 0; j < 16; j++) st.o[n][j] = 0.0f;
    // what the lane's row sees, what any of the wavefront's rows do, and all
    const Span seen = span_of(a, t, wave * WIDE + m);
    const int rows = min(t.rows - wave * WIDE, WIDE);
    const Span first = span_of(a, t, wave * WIDE), last = span_of(a, t, wave * WIDE + max(rows, 1) - 1);
    const int some_hi = rows > 0 ? last.hi : 0, all_hi = rows < WIDE ? 0 : first.hi;
    if (any) {
        unpack<D>(tiles[0], raw, put, mk, wave, lane);
        load(mine.lo + L::TT, after);
        next = known(after);
        after = entries_at(mine.lo + 2 * L::TT);
        __syncthreads();
        int buf = 0;
        for (int t0 = mine.lo; t0 < mine.hi; t0 += L::TT) {
            // the next tile's other buffer was last read before the barrier
            if (t0 + L::TT < mine.hi) unpack<D>(tiles[buf ^ 1], raw, put, mk, wave, lane);
            load(t0 + 2 * L::TT, after);
            const uint32_t behind = known(after);
            after = entries_at(t0 + 3 * L::TT);
            const Tile<D> &tile = tiles[buf];
#pragma unroll
            for (int sub = 0; sub < L::SUBS; sub++) {
                const int ts = t0 + sub * 32;
                if (ts >= some_hi || ts + 32 <= first.lo || ts >= mine.hi) continue;
                if (!(now >> sub & 1u)) continue;                      // (32 absent tokens)
                step<D>(st, tile, sub, ts, ts < last.lo || ts + 32 > all_hi, seen, mk, lane);
            }
            now = next;
            next = behind;
            __syncthreads();
            buf ^= 1;
        }
    }

    const Offset offset = st.offset();
    const float own = __builtin_amdgcn_exp2f(-offset.part);  // (1, or a power of two)
    st.l *= own;
    st.z *= own;
    st.l += __shfl_xor(st.l, 32);
    st.z += __shfl_xor(st.z, 32);
    if (g == 0) {
        sl[wave * WIDE + m] = st.l;
        sm[wave * WIDE + m] = offset.whole;
    }
    float *part = chunks_of(t, a.chunk, a.splits) > 1 ? part_of<D, ROWS>(a, (int64_t)x * a.splits + split, head) : nullptr;
    float *so = reinterpret_cast<float *>(mem) + wave * (WIDE * ROWF);
#pragma unroll
    for (int pass = 0; pass < D / PD; pass++) {
        if (pass) __syncthreads();
#pragma unroll
        for (int n = 0; n < L::NT; n++)
#pragma unroll
            for (int j = 0; j < 16; j++) {
                const int r = 8 * (j / 4) + 4 * g + j % 4, d = 8 * (r % L::DW) + r / L::DW * L::NT + n;
                if (D > 64 && j / 4 % (D / PD) != pass) continue;             // (d / 64 is that)
                so[m * ROWF + d % PD] = fmaf(st.o[n][j], n % 2 ? 0x1p-4f * own : own, st.z);
            }
        __syncthreads();
#pragma unroll
        for (int i = lane; i < WIDE * PD / 8; i += 64) {
            const int r = wave * WIDE + i / (PD / 8), d0 = i % (PD / 8) * 8, d = pass * PD + d0;
            if (r >= t.rows) break;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<float4 *>(y + j) = *reinterpret_cast<const float4 *>(so + i / (PD / 8) * ROWF + d0 + j);
            if (part) {
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    *reinterpret_cast<float4 *>(part + r * D + d + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                if (d == 0) *reinterpret_cast<float2 *>(part + ROWS * D + 2 * r) = make_float2(sm[r], sl[r]);
            } else {
                write_row<D, T>(a, t, head, r, d, y, sl[r], sm[r]);
            }
        }
    }
}

template <int D, class T>
hipError_t launch(const KvAttend &a, const KvPlan &p, hipStream_t s)
{
    hipLaunchKernelGGL((k_kv_prompt<D, T>), dim3(a.g.kv_heads, (unsigned)p.tiles, p.splits), dim3(WV * 64), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || p.splits == 1 ? e : launch_join<D, ROWS, T>(a, p, s);
}

}  // namespace

hipError_t lw_launch_kv_prompt(const KvAttend &a, int head_dim, int dtype, const KvPlan &p, hipStream_t s)
{
    const bool half = dtype == LW_F16;
    if (head_dim == 64) return half ? launch<64, _Float16>(a, p, s) : launch<64, __bf16>(a, p, s);
    if (head_dim == 128) return half ? launch<128, _Float16>(a, p, s) : launch<128, __bf16>(a, p, s);
    return hipErrorInvalidValue;
}
