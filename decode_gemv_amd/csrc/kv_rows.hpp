// kv_rows.hpp -- attention of new tokens over the 4-bit key/value cache, on
// the matrix cores.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t),  over visible t
//
// with k_t = dk (ck - 8) + (8 dk - mk) and v_t alike from the codes c.  The
// matrix cores contract the codes themselves, and the pairs are applied to
// what comes out, where there is one value per token instead of one per
// element:
//   q.k_t  = dk_t q.(ck_t - 8) + (8 dk_t - mk_t) sum(q)
//   sum_t p_t v_t = sum_t (p_t dv_t)(cv_t - 8) + sum_t p_t (8 dv_t - mv_t)
// A pair of codes becomes a matrix operand by one AND-OR that puts them under
// fp16's exponent of 1024, and one packed subtraction that centres them (those
// at bits 4..7 as 16 (c - 8); the 16 goes into q and into the output).
// Without the centring the sums carry 8 sum(q) and 8 sum(p dv), which cancel
// only afterwards.  The codes' own bits, as fp16 denormals, would save the
// subtraction, but the matrix cores align products by the operands' exponents
// and cut off what is far below the largest: measured over 131071 tokens, the
// logarithm of the sum is then off by 1e-5, and so by 6e-8.
//
// The scores are formed transposed, S^T = K Q^T: a lane then owns one query
// row and a few tokens, four in a row, and these are at once the operand of
// O^T = V^T P^T (a contraction may take its tokens in any order, if both
// operands agree), so the probabilities never leave their lane, the running
// maximum, the sums and the rescaling are per lane, and the loop has no
// exchange between lanes, no shared memory and no barrier.
//
// A workgroup has one tile of 8, 16 or 32 query rows of a sequence (row = token
// * group + head, all on one kv head) and a chunk of the sequence's tokens;
// its wavefronts take 32-token tiles in turn and meet in LDS at the end.
// Where row tiles are few, sequences are cut into chunks of one size for the
// whole batch (piece_of) and k_kv_join adds the chunks' partial results, in
// order: results do not depend on timing.  (Much work: kv_prompt.hip.)
//
// Rounding: q is scaled by a power of two per row and held in fp16 (exact for
// fp16 and bf16 inputs but for elements 2^29 below the row's largest); p dv
// is scaled to lie high in fp16's range and held in two fp16 operands, rounded
// and what that left (2^-21 in all).  Scores, maxima, sums and outputs are fp32.
#ifndef LW_KV_ROWS_HPP
#define LW_KV_ROWS_HPP

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_attend.hpp"

namespace {

// Wavefronts of a workgroup.  16 sequences of 501 to 8190 tokens (replays of a
// graph, with the join; a call among others takes some 6 us less) take 28.5 us
// with 4, 31.6 with 2 and 32.3 with 8, one of 131071 42.7, 46.0 and 44.1, 96 in
// a window of 1024 35.5, 40.4 and 41.4.
constexpr int NW = 4;

// A row tile has 8, 16 or 32 rows.  16 and 32 are the columns of a matrix
// instruction; 8 rows take both halves of the 16, with the same queries, and
// each half keeps its own half of the tokens: the work on scores and
// probabilities, which goes by columns, is then done once and not twice.
template <int ROWS> struct Mma {       // 16 x 16 x 32: lane = row/column l % 16, 8 of the 32 at 8 * (l / 16)
    using Acc = f4;
    static constexpr int WIDE = 16, ACC = 4;
    static __device__ __forceinline__ Acc go(h8 a, h8 b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mma<32> {           // 32 x 32 x 16: lane = row/column l % 32, 8 of the 16 at 8 * (l / 32)
    using Acc = f16v;
    static constexpr int WIDE = 32, ACC = 16;
    static __device__ __forceinline__ Acc go(h8 a, h8 b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// Wavefronts a SIMD is to hold (the registers that leaves).  Six of 8 rows of
// 64 dimensions take 36.5 us in bf16 and 35.5 in fp16 for 96 sequences of 16
// heads in a window of 1024 tokens (replays of a graph), five 39.2 and 38.6;
// 200 sequences of 600 tokens 29.0 and 29.8.
template <int D, int ROWS>
constexpr int WAVES = D * ROWS <= 512 ? 6 : D * ROWS <= 1024 ? 4 : D * ROWS <= 2048 ? 3 : 2;

// What a lane holds of 32 tokens: key words and value words, and the pairs of
// the tokens whose scores it will have (groups of four).
template <int D, int ROWS>
struct Shape {
    static constexpr int WIDE = Mma<ROWS>::WIDE;
    static constexpr int COPIES = WIDE / ROWS;               // columns of a row
    static constexpr int G = 64 / WIDE;                      // lanes that share a column
    static constexpr int SUB = STEP / WIDE;                  // token tiles of a step (2 or 1)
    static constexpr int VG = STEP / 4 / G;                  // token groups of a lane's value words
    static constexpr int TG = VG / COPIES;                   // and of its scores
    static constexpr int DW = D / 8;                         // words of a token
    static constexpr int PER = DW / G;                       // of them, those of a lane's part
    static constexpr int REPS = DW > WIDE ? DW / WIDE : 1;   // value words of a lane in each token group
    static constexpr int PARTS = DW < WIDE ? WIDE / DW : 1;  // lanes that share a value word
    static constexpr int NT = 8 / PARTS;                     // output tiles of a value word
    // Up to 16 rows keep their query operands in registers.  32 rows keep them in
    // LDS, one copy for the workgroup: D/4 registers fewer, which is a second
    // wavefront per SIMD, for D/16 reads a step
    static constexpr bool QREG = ROWS <= 16;
    static constexpr int ROWF = D + 4;                       // a row in LDS where the wavefronts' results meet, spread over the banks
};

// A lane's tokens of a step: scores, and probabilities in pairs.
template <int D, int ROWS> using Scores = float[Shape<D, ROWS>::TG][4];
template <int D, int ROWS> using Probs = h2[Shape<D, ROWS>::TG][2];

template <int D, int ROWS>
struct Keys {
    uint32_t w[Shape<D, ROWS>::SUB][Shape<D, ROWS>::PER];
    uint4 dm[Shape<D, ROWS>::TG];
};

template <int D, int ROWS>
struct Values {
    uint4 w[Shape<D, ROWS>::VG][Shape<D, ROWS>::REPS];
    uint4 dm[Shape<D, ROWS>::TG];
};

// First token of group i of a lane's scores.
template <int D, int ROWS>
__device__ __forceinline__ int group_token(int i, int lane)
{
    using H = Shape<D, ROWS>;
    return 4 * ((H::COPIES > 1 ? lane % H::WIDE / ROWS : i) * H::G + lane / H::WIDE);
}

// One head's part of a page as a buffer: its loads take a uniform offset (t0
// is a multiple of 32, so a step's part of each array starts at one) and a
// lane's own, which is the same for all steps; those of a buffer of no bytes
// (absent pages, steps past the end) give zeros and cost no traffic, and need
// no branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *block, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(block), 0, bytes, 0x00027000);
}

template <class T>
__device__ __forceinline__ T load_part(__amdgpu_buffer_rsrc_t b, uint32_t lane, uint32_t uniform)
{
    if constexpr (sizeof(T) == 16)
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b128(b, lane, uniform, 0));
    else
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b64(b, lane, uniform, 0));
}

template <int D, int ROWS>
__device__ __forceinline__ void load_keys(Keys<D, ROWS> &o, __amdgpu_buffer_rsrc_t block, int P, int t0, int lane)
{
    using H = Shape<D, ROWS>;
    constexpr int W = D >= 128 ? 4 : 2;
    const int m = lane % H::WIDE, g = lane / H::WIDE;
#pragma unroll
    for (int u = 0; u < H::SUB; u++)
#pragma unroll
        for (int j = 0; j < H::PER; j += W) {
            const uint32_t at = 4 * (kv_kword<D>(m, g * H::PER) + kv_kword<D>(u * H::WIDE, j));
            uint32_t *q = &o.w[u][j];
            if constexpr (W == 4) {
                const uint4 x = load_part<uint4>(block, at, t0 * (D / 2));
                q[0] = x.x, q[1] = x.y, q[2] = x.z, q[3] = x.w;
            } else {
                const uint2 x = load_part<uint2>(block, at, t0 * (D / 2));
                q[0] = x.x, q[1] = x.y;
            }
        }
#pragma unroll
    for (int i = 0; i < H::TG; i++)
        o.dm[i] = load_part<uint4>(block, 4 * group_token<D, ROWS>(0, lane) + 16 * i * H::G, P * D + t0 * 4);
}

template <int D, int ROWS>
__device__ __forceinline__ void load_values(Values<D, ROWS> &o, __amdgpu_buffer_rsrc_t block, int P, int t0, int lane)
{
    using H = Shape<D, ROWS>;
    const int m = lane % H::WIDE, g = lane / H::WIDE;
#pragma unroll
    for (int i = 0; i < H::VG; i++)
#pragma unroll
        for (int r = 0; r < H::REPS; r++)
            o.w[i][r] = load_part<uint4>(block, (g * H::DW + m % H::DW) * 16 + (i * H::G * H::DW + r * H::WIDE) * 16,
                                         P * (D / 2) + t0 * (D / 2));
#pragma unroll
    for (int i = 0; i < H::TG; i++)
        o.dm[i] = load_part<uint4>(block, 4 * group_token<D, ROWS>(0, lane) + 16 * i * H::G, P * D + P * 4 + t0 * 4);
}

// One wavefront's running state for its row tile.  Sums are relative to 2^mo
// of their row, where mo lies so far below the row's largest score that
// p dv is high in fp16's range.
template <int D, int ROWS>
struct State {
    static constexpr int TILES = D / Mma<ROWS>::WIDE;        // output tiles along the head
    h8 q[Shape<D, ROWS>::QREG ? Shape<D, ROWS>::PER : 1];    // query operands, where registers hold them
    typename Mma<ROWS>::Acc o[TILES];
    float qs, qsum;              // score = qs * (acc dk + (8 dk - mk) qsum), log2 units
    float mo, ref;               // the offset, and the row's largest raw score when it was set (kv_attend.hpp)
    float thr;                   // the raw score that calls for a new offset,
    uint32_t dlim;               // and the dv (fp16 bits) that does
    float l, z;                  // sum p, sum p (8 dv - mv)

    __device__ __forceinline__ Offset offset() const { return offset_of(ref, qs, mo, (float)(6 + 15 - (int)(dlim >> 10))); }
};

// Raw scores of 32 tokens.
template <int D, int ROWS>
__device__ __forceinline__ void scores(Scores<D, ROWS> &s, const State<D, ROWS> &st, const h8 *q,
                                       const Keys<D, ROWS> &k, Masks mk, int lane)
{
    using M = Mma<ROWS>;
    using H = Shape<D, ROWS>;
    typename M::Acc acc[H::SUB];
#pragma unroll
    for (int u = 0; u < H::SUB; u++) {
#pragma unroll
        for (int i = 0; i < M::ACC; i++) acc[u][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < H::PER; j++) acc[u] = M::go(spread8(k.w[u][j], mk), H::QREG ? st.q[j] : q[j * 64], acc[u]);
    }
    const bool second = lane % H::WIDE / ROWS != 0;
#pragma unroll
    for (int n = 0; n < H::TG; n++)
#pragma unroll
        for (int b = 0; b < 4; b++) {
            float x = acc[n * 4 / M::ACC][n * 4 % M::ACC + b];
            if constexpr (H::COPIES == 2) x = second ? acc[H::SUB - 1][b] : x;
            const uint32_t dm = reinterpret_cast<const uint32_t *>(&k.dm[n])[b];
            s[n][b] = fmaf(x, half_lo(dm), fmaf(half_lo(dm), 8.0f, -half_hi(dm)) * st.qsum);
        }
}

// Hides the tokens of t0..t0+31 that the lane's row does not see.
template <int D, int ROWS>
__device__ __forceinline__ void hide(Scores<D, ROWS> &s, Values<D, ROWS> &v, int t0, Span seen, int lane)
{
    using H = Shape<D, ROWS>;
    int first = t0 + group_token<D, ROWS>(0, lane) - seen.lo;
    asm volatile("" : "+v"(first));                          // (kept from being worked out ahead of the loop)
#pragma unroll
    for (int i = 0; i < H::TG; i++) {
        uint32_t *dv = reinterpret_cast<uint32_t *>(&v.dm[i]);
#pragma unroll
        for (int b = 0; b < 4; b++) {
            const bool out = (unsigned)(first + 4 * i * H::G + b) >= (unsigned)(seen.hi - seen.lo);
            s[i][b] = out ? -__builtin_inff() : s[i][b];
            dv[b] = out ? 0u : dv[b];                        // what lies there may be NaN
        }
    }
}

// Sees to it that the tokens' p dv fit fp16: where a score or a pair of a row
// has outgrown its offset (rarely, after the first steps), sets a new one, for
// which p dv is below 2^7 for all seen so far, and brings the sums to it.
// Scores may then exceed the reference 2^7 times before the next.  A row's
// offset depends on what the row sees and on nothing else.
template <int D, int ROWS>
__device__ __forceinline__ void fit(State<D, ROWS> &st, Scores<D, ROWS> &s, const Values<D, ROWS> &v)
{
    using H = Shape<D, ROWS>;
    float top = -__builtin_inff();
    h2 pair = {(_Float16)0.0f, (_Float16)0.0f};
#pragma unroll
    for (int i = 0; i < H::TG; i++) {
        const uint32_t *dv = reinterpret_cast<const uint32_t *>(&v.dm[i]);
#pragma unroll
        for (int b = 0; b < 4; b++) {
            top = fmaxf(top, s[i][b]);
            pair = __builtin_elementwise_max(pair, halves(dv[b]));  // (a NaN asks for nothing)
        }
    }
    uint32_t dtop = __builtin_bit_cast(uint32_t, pair) & 0xFFFFu;  // d >= 0: its bits are in order
    if (!__any(top > st.thr || dtop > st.dlim)) return;
#pragma unroll
    for (int o = H::WIDE; o < 64; o *= 2) {
        top = fmaxf(top, __shfl_xor(top, o));
        dtop = max(dtop, (uint32_t)__shfl_xor((int)dtop, o));
    }
    const bool need = top > st.thr || dtop > st.dlim;
    const Offset old = st.offset();
    if (need) {
        st.dlim = max(st.dlim, min(dtop, 0x7BFFu) | 0x03FFu);       // up to the next power of two
        st.ref = fmaxf(st.ref, top);
        set_offset(st.ref, st.qs, (float)(6 + 15 - (int)(st.dlim >> 10)), st.mo, st.thr);
    }
    const Offset now = st.offset();
#pragma unroll
    for (int i = 0; i < H::TG; i++)
#pragma unroll
        for (int b = 0; b < 4; b++) s[i][b] -= now.shift;
    const float f = between(old, now);
    st.l *= f;
    st.z *= f;
#pragma unroll
    for (int i = 0; i < State<D, ROWS>::TILES; i++)
#pragma unroll
        for (int j = 0; j < Mma<ROWS>::ACC; j++) st.o[i][j] *= f;
}

// From scores to probabilities p dv, as matrix operand, what the rounding to
// fp16 leaves of them as a second operand, and the sums of p.
template <int D, int ROWS>
__device__ __forceinline__ void probabilities(Probs<D, ROWS> &hi, Probs<D, ROWS> &lo, State<D, ROWS> &st,
                                              const Scores<D, ROWS> &s, const Values<D, ROWS> &v, Masks mk)
{
    using H = Shape<D, ROWS>;
#pragma unroll
    for (int i = 0; i < H::TG; i++) {
        const uint32_t *dv = reinterpret_cast<const uint32_t *>(&v.dm[i]);
        float e[4];
#pragma unroll
        for (int b = 0; b < 4; b++) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[i][b], st.qs, -st.mo));
            st.l += p;
            st.z = fmaf(p, fmaf(half_lo(dv[b]), 8.0f, -half_hi(dv[b])), st.z);
            e[b] = fmaf(p, half_lo(dv[b]), 0.0f);            // (takes dv as it is)
        }
#pragma unroll
        for (int c = 0; c < 2; c++) split2(e[2 * c], e[2 * c + 1], mk, hi[i][c], lo[i][c]);
    }
}

// O^T += V^T P^T, eight tokens of a lane a time: the codes of two tokens meet
// in one word, from which pairs of codes are taken as operands.
template <int D, int ROWS>
__device__ __forceinline__ void gather(State<D, ROWS> &st, const Probs<D, ROWS> &hi,
                                       const Probs<D, ROWS> &lo, const Values<D, ROWS> &v, Masks mk, int lane)
{
    using M = Mma<ROWS>;
    using H = Shape<D, ROWS>;
    const int m = lane % H::WIDE, part = m / H::DW;
    const uint32_t keep = m < ROWS ? ~0u : 0u;               // COPIES 2: whether the first half of the tokens is the column's
    auto other = [&](uint32_t x) {                           // x & ~keep
        uint32_t y;
        asm("v_bfi_b32 %0, %1, 0, %2" : "=v"(y) : "v"(keep), "v"(x));
        return y;
    };
#pragma unroll
    for (int i = 0; i < H::VG; i += 2) {
        auto operand = [&](const Probs<D, ROWS> &x) {
            uint4 w;
            if constexpr (H::COPIES == 2) {
                const uint32_t a = __builtin_bit_cast(uint32_t, x[0][0]), b = __builtin_bit_cast(uint32_t, x[0][1]);
                w = make_uint4(a & keep, b & keep, other(a), other(b));
            } else {
                w = make_uint4(__builtin_bit_cast(uint32_t, x[i][0]), __builtin_bit_cast(uint32_t, x[i][1]),
                               __builtin_bit_cast(uint32_t, x[i + 1][0]), __builtin_bit_cast(uint32_t, x[i + 1][1]));
            }
            return __builtin_bit_cast(h8, w);
        };
        const h8 p = operand(hi), rest = operand(lo);
#pragma unroll
        for (int r = 0; r < H::REPS; r++) {
            uint32_t w[2][4];                                // [halves of a word][pairs of tokens]
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const uint32_t *x = reinterpret_cast<const uint32_t *>(&v.w[i + c / 2][r]);
                const uint32_t a = x[2 * (c % 2)], b = x[2 * (c % 2) + 1];
                if constexpr (H::PARTS == 1) {
                    w[0][c] = __builtin_amdgcn_perm(b, a, 0x05040100u);
                    w[1][c] = __builtin_amdgcn_perm(b, a, 0x07060302u);
                } else if constexpr (H::PARTS == 2) {
                    w[0][c] = __builtin_amdgcn_perm(b, a, part ? 0x07060302u : 0x05040100u);
                } else {
                    w[0][c] = __builtin_amdgcn_perm(b, a, 0x0C040C00u + 0x00010001u * (uint32_t)part);
                }
            }
#pragma unroll
            for (int n = 0; n < H::NT; n++) {
                h8 x;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const uint32_t y = n % 4 >= 2 ? w[n / 4][c] >> 8 : w[n / 4][c];
                    const h2 z = n % 2 ? centred<true>(y, mk) : centred<false>(y, mk);
                    x[2 * c] = z[0];
                    x[2 * c + 1] = z[1];
                }
                st.o[r * H::NT + n] = M::go(x, p, st.o[r * H::NT + n]);
                st.o[r * H::NT + n] = M::go(x, rest, st.o[r * H::NT + n]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// SELECTED: a row's tokens lie in pages of its own for each head, and rows are cut
// as the host says (kv_selected.hip).
template <int D, int ROWS, class T, bool SELECTED = false>
__global__ __launch_bounds__(NW * 64, (WAVES<D, ROWS>)) void k_kv_attend(KvAttend a)
{
    using M = Mma<ROWS>;
    using S = State<D, ROWS>;
    using H = Shape<D, ROWS>;
    __shared__ __align__(16) float so[NW * H::WIDE * H::ROWF];
    __shared__ float sl[NW * H::WIDE], sm[NW * H::WIDE];     // by wavefront and column
    h8 *sq = reinterpret_cast<h8 *>(so);                     // the loop's; so is the end's
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane % H::WIDE, g = lane / H::WIDE, head = blockIdx.x;
    Piece piece = {0, INT_MAX, 0};
    const int y = blockIdx.z * gridDim.y + blockIdx.y;
    if (y >= a.pieces) return;
    RowTile t;
    if constexpr (SELECTED) {
        t = selected_tile<ROWS>(a, y / a.splits);
        piece = {y % a.splits, a.chunk, y};
    } else {
        t = a.target ? piece_of<ROWS>(a, y, piece) : row_tile<ROWS>(a, tile_at(a.pieces, y));
    }
    if (t.rows == 0) return;
    const Span mine = chunk_of(t, piece.chunk, INT_MAX, piece.split);
    if (piece.split > 0 && mine.lo >= mine.hi) return;       // (chunk 0 always leaves a result)

    // (what the loop seldom or never needs is worked out anew from the thread's
    // number where it is needed: registers)
    auto thread = [&]() {
        unsigned i = threadIdx.x;
        asm volatile("" : "+v"(i));
        return i;
    };
    auto seen = [&]() { return span_of(a, t, (int)(thread() % ROWS)); };
    const Span head_row = span_of(a, t, 0), last_row = span_of(a, t, t.rows - 1);
    const int all_lo = last_row.lo, all_hi = head_row.hi;     // tokens every row sees
    const int P = 1 << a.g.page_shift;
    // (the table's entry of a step past the end is the last one's again)
    const int32_t *pages = a.g.table + (SELECTED ? (int64_t)t.seq * a.g.kv_heads + head : (int64_t)t.seq) * a.g.stride;
    auto entry_at = [&](int t0) { return pages[min(t0, mine.hi - 1) >> a.g.page_shift]; };
    auto present = [&](int32_t entry) { return (uint32_t)entry < a.g.n_pages; };
    auto block_of = [&](int32_t entry, int t0) {
        const bool there = present(entry) && t0 < mine.hi;
        return buffer_of(a.g.pages + (uint64_t)(there ? (uint32_t)entry : 0u) * (uint64_t)a.g.page_bytes +
                             (uint32_t)head * (uint32_t)a.g.block_bytes,
                         there ? a.g.block_bytes : 0);
    };
    constexpr int HOP = NW * STEP;
    const Masks mk = masks();
    // A step's key registers are loaded anew once the
    // scores have used them, its value registers after the second product, so
    // both are under way nearly all the time.
    State<D, ROWS> st;
    Keys<D, ROWS> k;
    Values<D, ROWS> v;
    int32_t page = -1, after = -1;
    int t0 = mine.lo + wave * STEP;
    const bool any = t0 < mine.hi;
    {
        Query<D, H::WIDE, T> q;
        const int2 at = token_of(a, t, min(m % ROWS, t.rows - 1));
        q.load(a.q, t.row0 + at.x, (int64_t)head * a.group + at.y, lane);
        if (any) {
            // (the loads' order is the loop's, or its waits would fit neither)
            page = __builtin_amdgcn_readfirstlane(entry_at(t0));
            after = entry_at(t0 + HOP);
            load_keys<D, ROWS>(k, block_of(page, t0), P, t0 & (P - 1), lane);
            asm volatile("" ::: "memory");
            load_values<D, ROWS>(v, block_of(page, t0), P, t0 & (P - 1), lane);
            asm volatile("" ::: "memory");
        }
        q.make(st.qs, st.qsum, a.scale, [&](int j, h8 y) {
            if constexpr (H::QREG)
                st.q[j] = y;
            else if (wave == j % NW)
                sq[j * 64 + lane] = y;
        });
    }
    if (!H::QREG) __syncthreads();
    st.mo = NONE;
    st.ref = st.thr = UNSEEN;
    st.dlim = 0;
    st.l = st.z = 0.0f;
#pragma unroll
    for (int i = 0; i < S::TILES; i++)
#pragma unroll
        for (int j = 0; j < M::ACC; j++) st.o[i][j] = 0.0f;
    if (any) {
        do {
            const int32_t ahead = __builtin_amdgcn_readfirstlane(after);
            after = entry_at(t0 + 2 * HOP);
            const auto block = block_of(ahead, t0 + HOP);
            const int tn = (t0 + HOP) & (P - 1);
            Scores<D, ROWS> s;
            Probs<D, ROWS> hi, lo;
            scores<D, ROWS>(s, st, sq + lane, k, mk, lane);
            // the scores are done here, not where they are used, so that the
            // keys' registers are free
#pragma unroll
            for (int n = 0; n < H::TG; n++)
#pragma unroll
                for (int b = 0; b < 4; b++) asm volatile("" : "+v"(s[n][b]));
            load_keys<D, ROWS>(k, block, P, tn, lane);
            if (!present(page))
                hide<D, ROWS>(s, v, t0, Span{0, 0}, lane);
            else if (t0 < all_lo || t0 + STEP > all_hi || t.rows < ROWS)
                hide<D, ROWS>(s, v, t0, seen(), lane);
            fit<D, ROWS>(st, s, v);
            probabilities<D, ROWS>(hi, lo, st, s, v, mk);
            // the values are unpacked here, not above the branch in fit()
#pragma unroll
            for (int n = 0; n < H::VG; n++)
#pragma unroll
                for (int r = 0; r < H::REPS; r++)
                    asm volatile("" : "+v"(v.w[n][r].x), "+v"(v.w[n][r].y), "+v"(v.w[n][r].z), "+v"(v.w[n][r].w));
            gather<D, ROWS>(st, hi, lo, v, mk, lane);
            load_values<D, ROWS>(v, block, P, tn, lane);
            asm volatile("" ::: "memory");                   // (or they are moved to the next step's start)
            t0 += HOP;
            page = ahead;
        } while (t0 < mine.hi);
    }

    // the lanes that share a row, then the wavefronts
    const unsigned last = thread();
    const int m_ = last % H::WIDE, g_ = last % 64 / H::WIDE;
    const Offset offset = st.offset();
    const float own = __builtin_amdgcn_exp2f(-offset.part);  // (1, or a power of two)
    st.l *= own;
    st.z *= own;
#pragma unroll
    for (int o = Mma<ROWS>::WIDE; o < 64; o *= 2) {
        st.l += __shfl_xor(st.l, o);
        st.z += __shfl_xor(st.z, o);
    }
    if (g_ == 0) {
        sl[wave * H::WIDE + m_] = st.l;
        sm[wave * H::WIDE + m_] = offset.whole;
    }
    __syncthreads();
    constexpr int MEET = NW * H::COPIES;                     // results of a row, at every ROWS entries
    float mo = sm[m_ % ROWS];
#pragma unroll
    for (int w = 1; w < MEET; w++) mo = fmaxf(mo, sm[w * ROWS + m_ % ROWS]);
    float *part = chunks_of(t, piece.chunk, INT_MAX) > 1 ? part_of<D, ROWS>(a, piece.n, head) : nullptr;
    const float meet = __builtin_amdgcn_exp2f(offset.whole - mo), f = own * meet, fixed = st.z * meet;
#pragma unroll
    for (int i = 0; i < S::TILES; i++)
#pragma unroll
        for (int j = 0; j < M::ACC; j++) {
            const int r = i / H::NT, n = i % H::NT;
            const int row = H::WIDE == 16 ? 4 * g_ + j : 8 * (j / 4) + 4 * g_ + j % 4;  // along the head
            const int d = 8 * (row % H::DW + r * H::WIDE) + (row / H::DW) * H::NT + n;
            so[(wave * H::WIDE + m_) * H::ROWF + d] = fmaf(st.o[i][j], n % 2 ? 0x1p-4f * f : f, fixed);
        }
    __syncthreads();
    for (int i = last; i < t.rows * (D / 8); i += NW * 64) {
        const int r = i / (D / 8), d = i % (D / 8) * 8;
        float y[8], top = sm[r], l = 0.0f;
#pragma unroll
        for (int w = 1; w < MEET; w++) top = fmaxf(top, sm[w * ROWS + r]);
#pragma unroll
        for (int w = 0; w < MEET; w++) l += sl[w * ROWS + r] * __builtin_amdgcn_exp2f(sm[w * ROWS + r] - top);
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = 0.0f;
#pragma unroll
        for (int w = 0; w < MEET; w++)
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] += so[(w * ROWS + r) * H::ROWF + d + j];
        if (part) {
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<float4 *>(part + r * D + d + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
            if (d == 0) *reinterpret_cast<float2 *>(part + ROWS * D + 2 * r) = make_float2(top, l);
        } else {
            write_row<D, T>(a, t, head, r, d, y, l, top);
        }
    }
}

}  // namespace

#endif
