// kv_attend.hip -- attention of new tokens over the 4-bit key/value cache, on
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
// output's error against 64 bits is then 7e-4 and not 3e-4.
//
// The scores are formed transposed, S^T = K Q^T: a lane then owns one query
// row and a few tokens, four in a row, and these are at once the operand of
// O^T = V^T P^T (a contraction may take its tokens in any order, if both
// operands agree), so the probabilities never leave their lane, the running
// maximum, the sums and the rescaling are per lane, and the loop has no
// exchange between lanes, no shared memory and no barrier.
//
// A workgroup has one tile of 16 or 32 query rows of a sequence (row = token
// * group + head, all on one kv head) and a chunk of the sequence's tokens;
// its wavefronts take 32-token tiles in turn and meet in LDS at the end.
// Where row tiles are few, a sequence is cut into several chunks and
// k_kv_join adds the chunks' partial results, in order: results do not
// depend on timing.
//
// Rounding: q is scaled by a power of two per row and held in fp16 (exact for
// fp16 and bf16 inputs but for elements 2^29 below the row's largest);
// p dv is rounded to fp16 once, scaled to lie high in fp16's range, and
// multiplies the centred code, so the output's error from it is a random
// 2^-12 of the centred part; scores, maxima, sums and outputs are fp32.
#include <algorithm>

#include "kv.h"

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int NW = 4;                  // wavefronts of a workgroup
constexpr int STEP = 32;               // tokens of a wavefront's step
constexpr float NONE = -1e30f;         // log2 of "nothing seen yet"
constexpr float SLACK = 6.0f;          // log2 of how far p may exceed the reference before rescaling

// Wavefronts a SIMD is to hold (the registers that leaves).
template <int D, int TILE> constexpr int WAVES = D * TILE <= 2048 ? 2 : 1;

template <int TILE> struct Mma;
template <> struct Mma<16> {           // 16 x 16 x 32: lane = row/column l % 16, 8 of the 32 at 8 * (l / 16)
    using Acc = f4;
    static constexpr int ACC = 4, GROUPS = 4;
    static __device__ __forceinline__ Acc go(h8 a, h8 b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mma<32> {           // 32 x 32 x 16: lane = row/column l % 32, 8 of the 16 at 8 * (l / 32)
    using Acc = f16v;
    static constexpr int ACC = 16, GROUPS = 2;
    static __device__ __forceinline__ Acc go(h8 a, h8 b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

__device__ __forceinline__ float half_lo(uint32_t w) { return (float)__builtin_bit_cast(h2, w)[0]; }
__device__ __forceinline__ float half_hi(uint32_t w) { return (float)__builtin_bit_cast(h2, w)[1]; }

__device__ __forceinline__ h2 halves(uint32_t w) { return __builtin_bit_cast(h2, w); }

// Two codes, one in each half at bits 0..3 (shifted: 4..7), as fp16 c - 8
// (16 (c - 8)): under the exponent of 1024 they are 1024 + c, and one packed
// subtraction is exact.
template <bool SHIFTED>
__device__ __forceinline__ h2 centred(uint32_t w)
{
    return SHIFTED ? halves((w & 0x00F000F0u) | 0x64006400u) - h2{(_Float16)1152.0f, (_Float16)1152.0f}
                   : halves((w & 0x000F000Fu) | 0x64006400u) - h2{(_Float16)1032.0f, (_Float16)1032.0f};
}

// Eight codes of a word in the order 0 4 1 5 2 6 3 7, those of odd dimensions
// times 16.
__device__ __forceinline__ h8 spread8(uint32_t w)
{
    const h2 a = centred<false>(w), b = centred<true>(w), c = centred<false>(w >> 8), d = centred<true>(w >> 8);
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <class T> __device__ __forceinline__ float to_f(T x) { return (float)x; }

// The visible tokens of a packed row: first and one past the last.
struct Span {
    int lo, hi;
};

// Everything the parts of a call agree on about a row tile.
struct RowTile {
    int seq, r0, rows;           // first row (token * group + head) and rows in use (0: nothing to do)
    int row0, n_new, len;        // first packed row of the sequence, its new tokens, its length
    int lo, hi;                  // tokens any of the rows may see: [lo, hi), lo a multiple of STEP
};

template <int TILE>
__device__ __forceinline__ Span span_of(const KvAttend &a, const RowTile &t, int r)
{
    const int i = (t.r0 + r) / a.group, pos = t.len - t.n_new + i;
    Span s = {0, a.causal ? pos + 1 : t.len};
    if (a.window && pos >= a.window) s.lo = pos - a.window + 1;
    if (r >= t.rows || s.hi < s.lo) s.hi = s.lo;
    return s;
}

// Row tile x of the call.  Sequence s owns the tiles from
// floor(start[s] * group / TILE) + s on, as many as its rows need at most, so
// its tiles are found without a prefix sum (and one may find nothing to do).
template <int TILE>
__device__ __forceinline__ RowTile row_tile(const KvAttend &a, int x)
{
    const KvGeom &g = a.g;
    RowTile t = {};
    auto first = [&](int row, int s) {
        const int64_t rr = (int64_t)min(max(row, 0), g.n_tokens) * a.group;
        return (int)(rr / TILE) + s;
    };
    const int seq = kv_count_le(g.n_seqs, x, [&](int s) { return first(g.start[s + 1], s + 1); });
    t.seq = __builtin_amdgcn_readfirstlane(seq);
    if (t.seq >= g.n_seqs) return t;
    const int2 rows = kv_rows(g, t.seq);
    t.row0 = rows.x;
    t.n_new = rows.y - rows.x;
    t.len = max(g.lens[t.seq], 0);
    const int local = x - first(rows.x, t.seq);
    const int64_t r0 = (int64_t)local * TILE, all = (int64_t)t.n_new * a.group;
    if (local < 0 || r0 >= all) return t;
    t.r0 = (int)r0;
    t.rows = (int)min((int64_t)TILE, all - r0);
    const Span b = span_of<TILE>(a, t, 0), e = span_of<TILE>(a, t, t.rows - 1);
    t.lo = b.lo & ~(STEP - 1);
    const int64_t cap = min(g.stride << g.page_shift, (int64_t)0x7FFF0000);     // the table names no more
    t.hi = max((int)min((int64_t)e.hi, cap), t.lo);
    return t;
}

// Chunk z of a row tile's tokens; the last takes what is left.
__device__ __forceinline__ Span chunk_of(const KvAttend &a, const RowTile &t, int z)
{
    Span s = {t.lo + z * a.chunk, t.hi};
    if (z + 1 < a.splits && (int64_t)s.lo + a.chunk < t.hi) s.hi = s.lo + a.chunk;
    return s;
}

// What is loaded of 32 tokens: key words, value words, and the pairs of the
// tokens whose scores the lane will hold (groups of four).
template <int D, int TILE>
struct Tokens {
    static constexpr int KW = D * STEP / 8 / 64;             // key words a lane holds
    static constexpr int REPS = D / 8 > TILE ? D / 8 / TILE : 1;
    static constexpr int TG = STEP / 4 / Mma<TILE>::GROUPS;  // token groups of a lane
    uint32_t k[KW];
    uint4 v[TG][REPS];
    uint4 dk[TG], dv[TG];
};

template <int D, int TILE>
__device__ __forceinline__ void load_tokens(Tokens<D, TILE> &o, const uint8_t *block, int P, int t0, int lane)
{
    using K = Tokens<D, TILE>;
    constexpr int G = Mma<TILE>::GROUPS, W = D >= 128 ? 4 : 2, DW = D / 8;
    constexpr int SUB = STEP / TILE;                         // token tiles per step (2 or 1)
    constexpr int PER = DW / G;                              // words of a token that a lane holds
    const int m = lane % TILE, g = lane / TILE;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(block);
    const uint32_t *dm = w + P * (D / 4);
#pragma unroll
    for (int u = 0; u < SUB; u++)
#pragma unroll
        for (int j = 0; j < PER; j += W) {
            const uint32_t *p = w + kv_kword<D>(t0 + u * TILE + m, g * PER + j);
            uint32_t *q = &o.k[u * PER + j];
            if constexpr (W == 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p);
                q[0] = x.x, q[1] = x.y, q[2] = x.z, q[3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                q[0] = x.x, q[1] = x.y;
            }
        }
#pragma unroll
    for (int i = 0; i < K::TG; i++) {
        const int t = t0 + 4 * (i * G + g);
        o.dk[i] = *reinterpret_cast<const uint4 *>(dm + t);
        o.dv[i] = *reinterpret_cast<const uint4 *>(dm + P + t);
#pragma unroll
        for (int r = 0; r < K::REPS; r++)
            o.v[i][r] = *reinterpret_cast<const uint4 *>(w + P * DW + kv_vword<D>(t, (m + r * TILE) % DW));
    }
}

// One wavefront's running state for its row tile.  Values are relative to
// 2^mo of their row; mo = mrow - kd, mrow the row's reference score (log2)
// and kd a power that puts p dv high in fp16's range.
template <int D, int TILE>
struct State {
    static constexpr int TILES = D / TILE;                   // output tiles along the head
    static constexpr int QW = D / 8 / Mma<TILE>::GROUPS;     // query operands of a lane
    h8 q[QW];
    typename Mma<TILE>::Acc o[TILES];
    float qs, qsum;              // score = qs * (acc dk + (8 dk - mk) qsum), log2 units
    float mrow, mo, thr;         // reference, offset, and the raw score that calls for a new reference
    float l, z;                  // sum p, sum p (8 dv - mv)
    float dlim;                  // largest dv that kd allows for
    int kd;
};

// The 32 tokens t0..t0+31; masked: some of them may be hidden from some rows.
template <int D, int TILE>
__device__ __forceinline__ void step(State<D, TILE> &st, Tokens<D, TILE> &tk, int t0, Span seen, bool masked, int lane)
{
    using M = Mma<TILE>;
    using K = Tokens<D, TILE>;
    using S = State<D, TILE>;
    constexpr int G = M::GROUPS, SUB = STEP / TILE, DW = D / 8;
    const int m = lane % TILE, g = lane / TILE;

    float s[K::TG][4];
#pragma unroll
    for (int u = 0; u < SUB; u++) {
        typename M::Acc acc;
#pragma unroll
        for (int i = 0; i < M::ACC; i++) acc[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < S::QW; j++) acc = M::go(spread8(tk.k[u * S::QW + j]), st.q[j], acc);
#pragma unroll
        for (int i = 0; i < M::ACC; i++) s[u * (M::ACC / 4) + i / 4][i % 4] = acc[i];
    }
#pragma unroll
    for (int i = 0; i < K::TG; i++) {
        const uint32_t *dk = reinterpret_cast<const uint32_t *>(&tk.dk[i]);
#pragma unroll
        for (int b = 0; b < 4; b++) s[i][b] = fmaf(s[i][b], half_lo(dk[b]), fmaf(half_lo(dk[b]), 8.0f, -half_hi(dk[b])) * st.qsum);
    }
    if (masked) {
#pragma unroll
        for (int i = 0; i < K::TG; i++) {
            uint32_t *dv = reinterpret_cast<uint32_t *>(&tk.dv[i]);
#pragma unroll
            for (int b = 0; b < 4; b++) {
                const int t = t0 + 4 * (i * G + g) + b;
                const bool hide = (unsigned)(t - seen.lo) >= (unsigned)(seen.hi - seen.lo);
                s[i][b] = hide ? -__builtin_inff() : s[i][b];
                dv[b] = hide ? 0u : dv[b];                   // what lies there may be NaN
            }
        }
    }
    float top = -__builtin_inff(), dtop = 0.0f;
#pragma unroll
    for (int i = 0; i < K::TG; i++) {
        const uint32_t *dv = reinterpret_cast<const uint32_t *>(&tk.dv[i]);
#pragma unroll
        for (int b = 0; b < 4; b++) {
            top = fmaxf(top, s[i][b]);
            dtop = fmaxf(dtop, half_lo(dv[b]));
        }
    }
    if (__any(top > st.thr || dtop > st.dlim)) {             // rare: a new reference
#pragma unroll
        for (int o = TILE; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
#pragma unroll
        for (int o = 1; o < 64; o *= 2) dtop = fmaxf(dtop, __shfl_xor(dtop, o));
        const float old = st.mo;
        if (dtop > st.dlim) {
            const int e = (int)((__builtin_bit_cast(uint32_t, dtop) >> 23) & 255u) - 127;   // dtop > 0 here
            st.kd = 6 - e;
            st.dlim = ldexpf(1.0f, e + 1);
        }
        st.mrow = fmaxf(st.mrow, top * st.qs);
        st.mo = st.mrow - (float)st.kd;
        st.thr = (st.mrow + SLACK) / st.qs;
        const float f = __builtin_amdgcn_exp2f(old - st.mo);
        st.l *= f;
        st.z *= f;
#pragma unroll
        for (int i = 0; i < S::TILES; i++)
#pragma unroll
            for (int j = 0; j < M::ACC; j++) st.o[i][j] *= f;
    }
    // probabilities, and the operand p dv of the second product
    h2 pd[K::TG][2];
#pragma unroll
    for (int i = 0; i < K::TG; i++) {
        const uint32_t *dv = reinterpret_cast<const uint32_t *>(&tk.dv[i]);
        float e[4];
#pragma unroll
        for (int b = 0; b < 4; b++) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[i][b], st.qs, -st.mo));
            st.l += p;
            st.z = fmaf(p, fmaf(half_lo(dv[b]), 8.0f, -half_hi(dv[b])), st.z);
            e[b] = p * half_lo(dv[b]);
        }
        pd[i][0] = h2{(_Float16)e[0], (_Float16)e[1]};
        pd[i][1] = h2{(_Float16)e[2], (_Float16)e[3]};
    }
    // O^T += V^T P^T, two token groups of a lane a time: the codes of a pair
    // of tokens meet in one word, then one AND makes the pair an operand
    constexpr int PARTS = DW < TILE ? TILE / DW : 1;         // lanes that share a word of eight dimensions
    constexpr int NT = 8 / PARTS;                            // output tiles of a word
    const int part = m / DW;
#pragma unroll
    for (int i = 0; i < K::TG; i += 2) {
        const uint4 pw = make_uint4(__builtin_bit_cast(uint32_t, pd[i][0]), __builtin_bit_cast(uint32_t, pd[i][1]),
                                    __builtin_bit_cast(uint32_t, pd[i + 1][0]), __builtin_bit_cast(uint32_t, pd[i + 1][1]));
        const h8 p = __builtin_bit_cast(h8, pw);
#pragma unroll
        for (int r = 0; r < K::REPS; r++) {
            uint32_t w[2][4];                                // [halves of a word][pairs]
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const uint32_t *x = reinterpret_cast<const uint32_t *>(&tk.v[i + c / 2][r]);
                const uint32_t a = x[2 * (c % 2)], b = x[2 * (c % 2) + 1];
                if constexpr (PARTS == 1) {
                    w[0][c] = __builtin_amdgcn_perm(b, a, 0x05040100u);
                    w[1][c] = __builtin_amdgcn_perm(b, a, 0x07060302u);
                } else if constexpr (PARTS == 2) {
                    w[0][c] = __builtin_amdgcn_perm(b, a, part ? 0x07060302u : 0x05040100u);
                } else {
                    w[0][c] = __builtin_amdgcn_perm(b, a, 0x0C040C00u + 0x00010001u * (uint32_t)part);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
                h8 x;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const uint32_t y = n % 4 >= 2 ? w[n / 4][c] >> 8 : w[n / 4][c];
                    const h2 z = n % 2 ? centred<true>(y) : centred<false>(y);
                    x[2 * c] = z[0];
                    x[2 * c + 1] = z[1];
                }
                st.o[r * NT + n] = M::go(x, p, st.o[r * NT + n]);
            }
        }
    }
}

// The row's query as matrix operand, and the factors of its scores.
template <int D, int TILE, class T>
__device__ __forceinline__ void load_query(State<D, TILE> &st, const KvAttend &a, const RowTile &t, int head, int lane)
{
    using S = State<D, TILE>;
    const int m = lane % TILE, g = lane / TILE;
    const int r = t.r0 + min(m, t.rows - 1), tok = r / a.group, h = head * a.group + r % a.group;
    const T *p = static_cast<const T *>(a.q.data) + (int64_t)(t.row0 + tok) * a.q.token + (int64_t)h * a.q.head +
                 g * (S::QW * 8);
    float x[S::QW][8];
#pragma unroll
    for (int j = 0; j < S::QW; j++) {
        T e[8];
        if (a.q.wide) {
            *reinterpret_cast<uint4 *>(e) = *reinterpret_cast<const uint4 *>(p + 8 * j);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) e[i] = p[8 * j + i];
        }
#pragma unroll
        for (int i = 0; i < 8; i++) x[j][i] = to_f(e[i]);
    }
    float top = 0.0f;
    double sum = 0.0;            // its error would be common to all tokens of the row, times m
#pragma unroll
    for (int j = 0; j < S::QW; j++)
#pragma unroll
        for (int i = 0; i < 8; i++) {
            top = fmaxf(top, fabsf(x[j][i]));
            sum += x[j][i];
        }
#pragma unroll
    for (int o = TILE; o < 64; o *= 2) {
        top = fmaxf(top, __shfl_xor(top, o));
        sum += __shfl_xor(sum, o);
    }
    // the largest element goes to [2^14, 2^15); an infinity stays one and
    // makes the row NaN, as its scores are
    const int e = top > 0.0f ? (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127 : 0;
    st.qs = a.scale * 1.44269504088896341f * ldexpf(1.0f, e - 14);
    st.qsum = ldexpf((float)sum, 14 - e);
#pragma unroll
    for (int j = 0; j < S::QW; j++) {
        constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
        for (int i = 0; i < 8; i++)
            st.q[j][i] = (_Float16)ldexpf(x[j][order[i]], 14 - e - (order[i] % 2 ? 4 : 0));
    }
}

// Floats of a row in LDS: the row starts spread over the banks.
template <int D> constexpr int ROWF = D + 4;

// Partial results of the call's row tile (x, head) and chunk z: [TILE] rows of
// D values, then [TILE] of (mo, l).
template <int D, int TILE>
__device__ __forceinline__ float *part_of(const KvAttend &a, int64_t x, int head, int z)
{
    return a.part + (((x * a.g.kv_heads + head) * a.splits) + z) * (TILE * (D + 2));
}

template <int D, class T>
__device__ __forceinline__ void write_row(const KvAttend &a, const RowTile &t, int head, int r, int d0, const float *y,
                                          float l, float mo)
{
    const int row = t.r0 + r, tok = t.row0 + row / a.group, h = head * a.group + row % a.group;
    T *p = static_cast<T *>(a.out.data) + (int64_t)tok * a.out.token + (int64_t)h * a.out.head + d0;
    T e[8];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < 8; i++) e[i] = (T)(y[i] * inv);
    if (a.out.wide) {
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(e);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) p[i] = e[i];
    }
    if (a.lse && d0 == 0) {
        int e = 0;                                           // l's power of two joins mo exactly
        const float f = frexpf(l, &e);
        a.lse[(int64_t)tok * ((int64_t)a.g.kv_heads * a.group) + h] =
            l == 0.0f ? -__builtin_inff() : (__builtin_amdgcn_logf(f) + ((float)e + mo)) * 0.693147180559945309f;
    }
}

template <int D, int TILE, class T>
__global__ __launch_bounds__(NW * 64, (WAVES<D, TILE>)) void k_kv_attend(KvAttend a)
{
    using M = Mma<TILE>;
    using S = State<D, TILE>;
    using K = Tokens<D, TILE>;
    __shared__ float so[NW * TILE * ROWF<D>];
    __shared__ float sl[NW][TILE], sm[NW][TILE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane % TILE, g = lane / TILE, head = blockIdx.y;
    const int x = gridDim.x - 1 - blockIdx.x;                // later rows see more tokens: they go first
    const RowTile t = row_tile<TILE>(a, x);
    if (t.rows == 0) return;
    const Span mine = chunk_of(a, t, blockIdx.z);
    if (blockIdx.z > 0 && mine.lo >= mine.hi) return;        // (chunk 0 always leaves a result)

    State<D, TILE> st;
    load_query<D, TILE, T>(st, a, t, head, lane);
    st.mrow = st.mo = NONE;
    st.thr = NONE / fmaxf(st.qs, 1.0f);
    st.l = st.z = st.dlim = 0.0f;
    st.kd = 0;
#pragma unroll
    for (int i = 0; i < S::TILES; i++)
#pragma unroll
        for (int j = 0; j < M::ACC; j++) st.o[i][j] = 0.0f;

    const Span seen = span_of<TILE>(a, t, m);
    const Span head_row = span_of<TILE>(a, t, 0), last_row = span_of<TILE>(a, t, t.rows - 1);
    const int all_lo = last_row.lo, all_hi = head_row.hi;     // tokens every row sees
    const int P = 1 << a.g.page_shift;
    auto page_at = [&](int t0) -> int64_t {
        return t0 < mine.hi ? kv_page(a.g, t.seq, t0) : -1;
    };
    auto block_of = [&](int64_t page) { return a.g.pages + page * a.g.page_bytes + (int64_t)head * a.g.block_bytes; };
    constexpr int HOP = NW * STEP;
    int t0 = mine.lo + wave * STEP;
    int64_t page = page_at(t0);
    while (t0 < mine.hi) {
        const int64_t after = page_at(t0 + HOP);
        if (page >= 0) {
            K cur;
            load_tokens<D, TILE>(cur, block_of(page), P, t0 & (P - 1), lane);
            step<D, TILE>(st, cur, t0, seen, t0 < all_lo || t0 + STEP > all_hi || t.rows < TILE, lane);
        }
        t0 += HOP;
        page = after;
    }

    // the lanes that share a row, then the wavefronts
#pragma unroll
    for (int o = TILE; o < 64; o *= 2) {
        st.l += __shfl_xor(st.l, o);
        st.z += __shfl_xor(st.z, o);
    }
    if (g == 0) {
        sl[wave][m] = st.l;
        sm[wave][m] = st.mo;
    }
    __syncthreads();
    float mo = sm[0][m];
#pragma unroll
    for (int w = 1; w < NW; w++) mo = fmaxf(mo, sm[w][m]);
    {
        const float f = __builtin_amdgcn_exp2f(st.mo - mo);
        const float fixed = st.z * f;
        constexpr int DW = D / 8, PARTS = DW < TILE ? TILE / DW : 1, NT = 8 / PARTS;
#pragma unroll
        for (int i = 0; i < S::TILES; i++)
#pragma unroll
            for (int j = 0; j < M::ACC; j++) {
                const int r = i / NT, n = i % NT;
                const int row = TILE == 16 ? 4 * g + j : 8 * (j / 4) + 4 * g + j % 4;     // along the head
                const int d = 8 * (row % DW + r * TILE) + (row / DW) * NT + n;
                const float unit = n % 2 ? 0x1p-4f : 1.0f;
                so[(wave * TILE + m) * ROWF<D> + d] = fmaf(st.o[i][j], unit * f, fixed);
            }
    }
    __syncthreads();
    float *part = a.splits > 1 ? part_of<D, TILE>(a, x, head, blockIdx.z) : nullptr;
    for (int i = threadIdx.x; i < t.rows * (D / 8); i += NW * 64) {
        const int r = i / (D / 8), d0 = i % (D / 8) * 8;
        float y[8], top = sm[0][r], l = 0.0f;
#pragma unroll
        for (int w = 1; w < NW; w++) top = fmaxf(top, sm[w][r]);
#pragma unroll
        for (int w = 0; w < NW; w++) l += sl[w][r] * __builtin_amdgcn_exp2f(sm[w][r] - top);
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; w++)
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] += so[(w * TILE + r) * ROWF<D> + d0 + j];
        if (part) {
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<float4 *>(part + r * D + d0 + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
            if (d0 == 0) *reinterpret_cast<float2 *>(part + TILE * D + 2 * r) = make_float2(top, l);
        } else {
            write_row<D, T>(a, t, head, r, d0, y, l, top);
        }
    }
}

// Join the chunks of a row tile: eight dimensions of a row per thread.
template <int D, int TILE, class T>
__global__ __launch_bounds__(256) void k_kv_join(KvAttend a)
{
    const int64_t x = blockIdx.x;
    const int head = blockIdx.y;
    const RowTile t = row_tile<TILE>(a, (int)x);
    if (t.rows == 0) return;
    const int used = min((t.hi - t.lo + a.chunk - 1) / a.chunk, a.splits);
    for (int i = blockIdx.z * 256 + threadIdx.x; i < t.rows * (D / 8); i += gridDim.z * 256) {
        const int r = i / (D / 8), d0 = i % (D / 8) * 8;
        float y[8], top = NONE, l = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = 0.0f;
        for (int z = 0; z < max(used, 1); z++) {
            const float *p = part_of<D, TILE>(a, x, head, z);
            const float2 ml = *reinterpret_cast<const float2 *>(p + TILE * D + 2 * r);
            const float now = fmaxf(top, ml.x);
            const float fo = __builtin_amdgcn_exp2f(top - now), fn = __builtin_amdgcn_exp2f(ml.x - now);
            top = now;
            l = l * fo + ml.y * fn;
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(p + r * D + d0 + j);
                y[j] = y[j] * fo + v.x * fn;
                y[j + 1] = y[j + 1] * fo + v.y * fn;
                y[j + 2] = y[j + 2] * fo + v.z * fn;
                y[j + 3] = y[j + 3] * fo + v.w * fn;
            }
        }
        write_row<D, T>(a, t, head, r, d0, y, l, top);
    }
}

template <int D, int TILE, class T>
hipError_t launch(const KvAttend &a, const KvPlan &p, hipStream_t s)
{
    hipLaunchKernelGGL((k_kv_attend<D, TILE, T>), dim3((unsigned)p.tiles, a.g.kv_heads, p.splits), dim3(NW * 64), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL((k_kv_join<D, TILE, T>), dim3((unsigned)p.tiles, a.g.kv_heads, 1), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int D>
hipError_t launch_dim(const KvAttend &a, int dtype, const KvPlan &p, hipStream_t s)
{
    if (p.tile == 16)
        return dtype == LW_F16 ? launch<D, 16, _Float16>(a, p, s) : launch<D, 16, __bf16>(a, p, s);
    return dtype == LW_F16 ? launch<D, 32, _Float16>(a, p, s) : launch<D, 32, __bf16>(a, p, s);
}

}  // namespace

KvPlan lw_kv_plan(int head_dim, int kv_heads, int group, int64_t n_seqs, int64_t n_tokens, int64_t max_len, int window,
                  int most)
{
    KvPlan p;
    p.tile = n_tokens * group <= 16 * n_seqs ? 16 : 32;
    p.tiles = n_tokens * group / p.tile + n_seqs;
    // tokens a row tile may see
    int64_t span = max_len;
    if (window) span = std::min<int64_t>(span, (int64_t)window + (p.tile + group - 1) / group + STEP);
    span = std::max<int64_t>(span, 1);
    const int64_t base = std::max(std::min(n_seqs, n_tokens), (n_tokens * group + p.tile - 1) / p.tile) * kv_heads;
    int64_t splits = std::min((1024 + base - 1) / base, (span + 2 * NW * STEP - 1) / (2 * NW * STEP));
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, std::min(most, 1024)));
    p.chunk = (int)(((span + splits - 1) / splits + NW * STEP - 1) / (NW * STEP) * (NW * STEP));
    p.splits = (int)((span + p.chunk - 1) / p.chunk);
    p.work_bytes = p.splits > 1 ? (size_t)p.tiles * kv_heads * p.splits * p.tile * (head_dim + 2) * sizeof(float) : 0;
    return p;
}

hipError_t lw_launch_kv_attend(const KvAttend &a, int head_dim, int dtype, const KvPlan &p, hipStream_t s)
{
    if (head_dim == 64) return launch_dim<64>(a, dtype, p, s);
    if (head_dim == 128) return launch_dim<128>(a, dtype, p, s);
    if (head_dim == 256) return launch_dim<256>(a, dtype, p, s);
    return hipErrorInvalidValue;
}
