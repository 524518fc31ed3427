// kv_attend.hpp -- what the attention kernels of the 4-bit key/value cache
// share: the unpacking of codes, the cutting of a call into row tiles and
// chunks of tokens, the queries as matrix operands, and the writing of
// results.  Internal to the library.
#ifndef LW_KV_ATTEND_HPP
#define LW_KV_ATTEND_HPP

#include <limits.h>

#include <type_traits>

#include "kv.h"

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int STEP = 32;               // tokens of a wavefront's step
constexpr float NONE = -0x1.fffffep127f;  // log2 of "nothing seen yet"
constexpr float UNSEEN = -0x1p60f;     // and the raw score of it (what there is lies within 2^44)
constexpr int CHUNK = 128, LEAST = 512;  // chunks are multiples of the first, and from the second on

__device__ __forceinline__ float half_lo(uint32_t w) { return (float)__builtin_bit_cast(h2, w)[0]; }
__device__ __forceinline__ float half_hi(uint32_t w) { return (float)__builtin_bit_cast(h2, w)[1]; }

__device__ __forceinline__ h2 halves(uint32_t w) { return __builtin_bit_cast(h2, w); }

// Constants that the compiler is to keep in registers: an AND and an OR with
// two of them are one instruction, with two literals they are two.
struct Masks {
    uint32_t low, high, exp;     // codes at bits 0..3 and 4..7 of each half, fp16's exponent of 1024
    float one;                   // a product with it and a subtraction of an fp16 number are one instruction
};

__device__ __forceinline__ Masks masks()
{
    Masks k;
    asm("s_mov_b32 %0, 0x000f000f" : "=s"(k.low));
    asm("s_mov_b32 %0, 0x00f000f0" : "=s"(k.high));
    asm("v_mov_b32 %0, 0x64006400" : "=v"(k.exp));
    asm("s_mov_b32 %0, 1.0" : "=s"(k.one));
    return k;
}

// Two codes, one in each half at bits 0..3 (SHIFTED: 4..7), as fp16 c - 8
// (16 (c - 8)): under the exponent of 1024 they are 1024 + c, and one packed
// subtraction is exact.
template <bool SHIFTED>
__device__ __forceinline__ h2 centred(uint32_t w, Masks k)
{
    return SHIFTED ? halves((w & k.high) | k.exp) - h2{(_Float16)1152.0f, (_Float16)1152.0f}
                   : halves((w & k.low) | k.exp) - h2{(_Float16)1032.0f, (_Float16)1032.0f};
}

// x and y as fp16, and what their rounding leaves of them, as fp16 too
// (2^-21 of them is lost).  The two are held as they are: of a product the
// compiler may else make the rounded value from the product in 32 bits and the
// rest from one rounding of the product itself, and where the two round apart,
// once in some 2^13 times, the rest is off by a last place of the first.
__device__ __forceinline__ void split2(float x, float y, Masks k, h2 &hi, h2 &rest)
{
    asm("" : "+v"(x), "+v"(y));
    uint32_t w = __builtin_bit_cast(uint32_t, h2{(_Float16)x, (_Float16)y});
    asm("" : "+v"(w));                                       // (both from one conversion)
    hi = halves(w);
    rest = h2{(_Float16)fmaf(x, k.one, -(float)hi[0]), (_Float16)fmaf(y, k.one, -(float)hi[1])};
}

// Eight codes of a word in the order 0 4 1 5 2 6 3 7, those of odd dimensions
// times 16.
__device__ __forceinline__ h8 spread8(uint32_t w, Masks k)
{
    const h2 a = centred<false>(w, k), b = centred<true>(w, k);
    const h2 c = centred<false>(w >> 8, k), d = centred<true>(w >> 8, k);
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A row's sums are relative to 2^o, o = ref qs - k for a raw score ref and a
// small number k: p = exp2(s qs - mo), mo = o.  Where ref qs is large, o has no
// place for k, and the product of s and qs before the subtraction, which is
// exact in a fused one, differs from ref qs by more than p can bear: there
// (FAR) ref is taken from the raw scores, which is exact for those near it, and
// mo is -k.  For a step's scores: a row that is so asks for a look each step.
constexpr float FAR = 0x1p20f;

struct Offset {
    float whole, part;           // o = whole - part
    float shift;                 // to be taken from raw scores
};

__device__ __forceinline__ Offset offset_of(float ref, float qs, float mo, float k)
{
    const bool far = fabsf(ref * qs) >= FAR && ref > 0.5f * UNSEEN;
    return {far ? ref * qs : mo, far ? k : 0.0f, far ? ref : 0.0f};
}

__device__ __forceinline__ void set_offset(float ref, float qs, float k, float &mo, float &thr)
{
    const float x = ref * qs;
    const bool far = fabsf(x) >= FAR;
    asm volatile("" : "+v"(qs));                             // (the division is done here, not ahead of the loop)
    mo = far ? -k : x - k;
    thr = far ? -__builtin_inff() : ref + 7.0f / qs;
}

// What brings sums from one offset to another.
__device__ __forceinline__ float between(const Offset &old, const Offset &now)
{
    return __builtin_amdgcn_exp2f((old.whole - now.whole) - (old.part - now.part));
}

// The visible tokens of a packed row: first and one past the last.
struct Span {
    int lo, hi;
};

// Everything the parts of a call agree on about a row tile.
struct RowTile {
    int seq, rows;               // rows in use (0: nothing to do)
    int row0, n_new, len;        // the sequence's first packed row, new tokens and length
    int tok0, rem0;              // new token and head of the tile's first row
    int lo, hi;                  // tokens any of the rows may see: [lo, hi), lo a multiple of STEP
};

// New token (x) and head of the kv head's group (y) of row r of the tile.
__device__ __forceinline__ int2 token_of(const KvAttend &a, const RowTile &t, int r)
{
    const unsigned i = t.rem0 + r, q = (i * a.group_inv) >> 21;
    return make_int2(t.tok0 + (int)q, (int)(i - q * a.group));
}

__device__ __forceinline__ Span span_of(const KvAttend &a, const RowTile &t, int r)
{
    const int pos = t.len - t.n_new + token_of(a, t, r).x;
    Span s = {0, a.causal ? pos + 1 : t.len};
    if (a.window && pos >= a.window) s.lo = pos - a.window + 1;
    if (r >= t.rows || s.hi < s.lo) s.hi = s.lo;
    return s;
}

// Tokens that the table can name.
__device__ __forceinline__ int cap_of(const KvGeom &g)
{
    return (int)min(g.stride << g.page_shift, (int64_t)KV_MOST_TOKENS);
}

// Row tile `local` of a sequence.
template <int ROWS>
__device__ __forceinline__ RowTile tile_of(const KvAttend &a, const KvSeq &q, int local)
{
    RowTile t = {};
    t.seq = q.seq;
    if (q.seq < 0) return t;
    t.row0 = q.row0;
    t.n_new = q.n_new;
    t.len = q.len;
    const int r0 = local * ROWS, all = q.n_new * a.group;
    if (local < 0 || r0 >= all) return t;
    t.rows = min(ROWS, all - r0);
    t.tok0 = r0 / a.group;
    t.rem0 = r0 - t.tok0 * a.group;
    const Span b = span_of(a, t, 0), e = span_of(a, t, t.rows - 1);
    t.lo = b.lo & ~(STEP - 1);
    t.hi = max(min(e.hi, cap_of(a.g)), t.lo);
    return t;
}

// The number of a sequence's first row tile.  Sequence s owns those from
// floor(start[s] * group / ROWS) + s on, as many as its rows need at most, so
// its tiles are found without a prefix sum (and one may find nothing to do).
template <int ROWS>
__device__ __forceinline__ int first_tile(const KvAttend &a, int row, int s)
{
    return min(max(row, 0), a.g.n_tokens) * a.group / ROWS + s;      // < 2^31
}

template <int ROWS>
__device__ __forceinline__ RowTile row_tile(const KvAttend &a, int x)
{
    const KvSeq q = kv_find(a.g, x, [&](int next, int s) { return first_tile<ROWS>(a, next, s + 1); });
    return tile_of<ROWS>(a, q, x - first_tile<ROWS>(a, q.row0, q.seq));
}

// The row tile that workgroups of number z take: the last first, as later rows
// see more tokens, and those of one parity before the others.  Row tiles with
// nothing to do come at regular distances (every second where sequences fill
// one tile each), and workgroups go round the eight XCDs: in plain order all
// the work could fall to every second XCD.
__device__ __forceinline__ int tile_at(int tiles, int z)
{
    const int first = (tiles + 1) / 2;
    return z < first ? 2 * (first - 1 - z) : 2 * (tiles - first - 1 - (z - first)) + 1;
}

// Sum of x over the lanes up to this one: along rows of 16 lanes, then what
// the rows before have in their last lane.
template <class T>
__device__ __forceinline__ T prefix(T x)
{
    auto add = [&](auto ctrl, auto rows) {
        x += __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl.value, rows.value, 0xF, true));
    };
    using std::integral_constant;
    add(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});      // one lane on (0 comes in),
    add(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});      // two,
    add(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});      // four,
    add(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});      // eight
    add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});      // lane 15 of rows 0 and 2 to the next row
    add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});      // lane 31 to rows 2 and 3
    return x;
}

// What a workgroup has to do: chunk `split` of a row tile, of `chunk` tokens,
// whose results are number n of the kv head's.
struct Piece {
    int split, chunk, n;
};

// Piece y of a batch whose sequences are cut into chunks of one size, the
// same for all, for which the batch makes about a.target (at most that and
// one more per row tile): then workgroups have the same work however
// different the sequences are, and none has nothing to do.  The wavefront's
// lanes look at 64 sequences at a time, B times at once (what a look takes is
// its loads' latency: 512 sequences of 500 tokens in chunks take 100 us with
// four looks at once and 110 with one).
template <int ROWS, int B>
__device__ __forceinline__ KvSeq find_piece(const KvAttend &a, int y, Piece &o, int &local)
{
    const KvGeom &g = a.g;
    const int lane = threadIdx.x & 63, cap = cap_of(g);
    int row0[B], n_new[B], len[B], tiles[B], span[B];
    auto look = [&](int s) {
        int b[B], e[B], l[B];
#pragma unroll
        for (int i = 0; i < B; i++) {
            const int mine = min(s + 64 * i + lane, g.n_seqs - 1);
            b[i] = g.start[mine];
            e[i] = g.start[mine + 1];
            l[i] = g.lens[mine];
        }
#pragma unroll
        for (int i = 0; i < B; i++) {
            len[i] = max(l[i], 0);
            row0[i] = min(max(b[i], 0), g.n_tokens);
            n_new[i] = min(max(e[i], row0[i]), g.n_tokens) - row0[i];
            tiles[i] = s + 64 * i + lane < g.n_seqs ? (n_new[i] * a.group + ROWS - 1) / ROWS : 0;
            const int pos = len[i] - n_new[i];               // the first row's
            const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
            span[i] = max(min(len[i], cap) - (lo & ~(STEP - 1)), 0);
        }
    };
    float all = 0.0f;
    for (int s = 0; s < g.n_seqs; s += 64 * B) {
        look(s);
#pragma unroll
        for (int i = 0; i < B; i++) all += (float)tiles[i] * (float)span[i];
    }
    all = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, prefix(all)), 63));
    const float part = fminf(all / (float)a.target, 0x1p30f);
    o.chunk = max((__builtin_amdgcn_readfirstlane((int)ceilf(part)) + CHUNK - 1) / CHUNK * CHUNK, LEAST);
    int before = 0;
    for (int s = 0; s < g.n_seqs; s += 64 * B) {
        if (g.n_seqs > 64 * B) look(s);
#pragma unroll
        for (int i = 0; i < B; i++) {
            const int chunks = max((int)(((unsigned)span[i] + o.chunk - 1) / (unsigned)o.chunk), 1);
            const int sum = prefix(tiles[i] * chunks);
            const int c = __popcll(__ballot(before + sum <= y));
            if (c < 64) {
                const int each = __builtin_amdgcn_readlane(chunks, c);
                const int in = y - before - (c ? __builtin_amdgcn_readlane(sum, c - 1) : 0);
                local = in / each;
                // (else a start that decreases has taken the sums past 2^31)
                if (in < 0 || local >= __builtin_amdgcn_readlane(tiles[i], c)) return {-1, 0, 0, 0};
                o.split = in - local * each;
                return {s + 64 * i + c, __builtin_amdgcn_readlane(row0[i], c), __builtin_amdgcn_readlane(n_new[i], c),
                        __builtin_amdgcn_readlane(len[i], c)};
            }
            before += __builtin_amdgcn_readlane(sum, 63);
        }
    }
    return {-1, 0, 0, 0};
}

template <int ROWS>
__device__ __forceinline__ RowTile piece_of(const KvAttend &a, int y, Piece &o)
{
    int local = 0;
    const KvSeq q = a.g.n_seqs > 64 ? find_piece<ROWS, 4>(a, y, o, local) : find_piece<ROWS, 1>(a, y, o, local);
    o.n = y;
    const RowTile t = tile_of<ROWS>(a, q, local);
    if (t.rows && o.split == 0 && blockIdx.x == 0 && threadIdx.x == 0)
        a.first[first_tile<ROWS>(a, q.row0, q.seq) + local] = make_int2(y, o.chunk);
    return t;
}

// Chunks that a row tile's tokens fill, at least one and at most `most`.  A
// tile of one chunk writes its outputs itself, those of more are joined.
__device__ __forceinline__ int chunks_of(const RowTile &t, int chunk, int most)
{
    return min(max((int)(((unsigned)(t.hi - t.lo) + (unsigned)chunk - 1) / (unsigned)chunk), 1), most);
}

// Chunk z; the last of the most takes what is left.
__device__ __forceinline__ Span chunk_of(const RowTile &t, int chunk, int most, int z)
{
    const int64_t lo = t.lo + (int64_t)z * chunk, hi = z + 1 < most ? lo + chunk : t.hi;
    return {(int)min(lo, (int64_t)t.hi), (int)min(hi, (int64_t)t.hi)};
}

// A lane's part of its row's query, for matrix instructions of WIDE columns.
template <int D, int WIDE, class T>
struct Query {
    static constexpr int G = 64 / WIDE, PER = D / 8 / G;     // lanes that share a column, words of a lane's part
    T x[PER][8];

    // head vector of new token tok (of the sequence whose rows start at row0) and query head h
    __device__ __forceinline__ void load(const KvTensor &q, int64_t row, int64_t h, int lane)
    {
        const T *p = static_cast<const T *>(q.data) + row * q.token + h * q.head + lane / WIDE * (PER * 8);
#pragma unroll
        for (int j = 0; j < PER; j++) {
            if (q.wide) {
                *reinterpret_cast<uint4 *>(x[j]) = *reinterpret_cast<const uint4 *>(p + 8 * j);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) x[j][i] = p[8 * j + i];
            }
        }
    }

    // Factors of the row's scores (score = qs * (acc dk + (8 dk - mk) qsum),
    // in log2 units, for the accumulated products acc), and put(j, operand)
    // for each word.
    template <class F>
    __device__ __forceinline__ void make(float &qs, float &qsum, float scale, F put) const
    {
        float top = 0.0f, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; j++)
#pragma unroll
            for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf((float)x[j][i]));
#pragma unroll
        for (int o = WIDE; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
        // the largest element goes to [2^14, 2^15), also before they are summed;
        // an infinity stays one and makes the row NaN, as its scores are
        const int e = top > 0.0f ? (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127 : 0;
        // (at least a normal number: a hidden token's score is -infinity times
        // this; scores that small are zero either way)
        qs = fmaxf(scale * 1.44269504088896341f * ldexpf(1.0f, e - 14), 0x1p-126f);
#pragma unroll
        for (int j = 0; j < PER; j++) {
            constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
            h8 y;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float v = ldexpf((float)x[j][order[i]], 14 - e);
                sum += v;
                y[i] = (_Float16)(order[i] % 2 ? v * 0x1p-4f : v);
            }
            put(j, y);
        }
#pragma unroll
        for (int o = WIDE; o < 64; o *= 2) sum += __shfl_xor(sum, o);
        qsum = sum;
    }
};

// Partial results of the call's row tile (x, head) and chunk z: [ROWS] rows of
// D values, then [ROWS] of (mo, l).
template <int D, int ROWS>
__device__ __forceinline__ float *part_of(const KvAttend &a, int64_t n, int head)
{
    return a.part + (n * a.g.kv_heads + head) * (ROWS * (D + 2));
}

template <int D, class T>
__device__ __forceinline__ void write_row(const KvAttend &a, const RowTile &t, int head, int r, int d0, const float *y,
                                          float l, float mo)
{
    const int2 at = token_of(a, t, r);
    const int64_t tok = t.row0 + at.x, h = (int64_t)head * a.group + at.y;
    T *p = static_cast<T *>(a.out.data) + tok * a.out.token + h * a.out.head + d0;
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
        a.lse[tok * ((int64_t)a.g.kv_heads * a.group) + h] =
            l == 0.0f ? -__builtin_inff() : (__builtin_amdgcn_logf(f) + ((float)e + mo)) * 0.693147180559945309f;
    }
}

// Joins the chunks of rows: D/8 threads take eight dimensions each of a row,
// in a.slices slices (a power of two) that take the chunks in turn and meet
// in LDS.
template <int D, int ROWS, class T>
__global__ __launch_bounds__(256) void k_kv_join(KvAttend a)
{
    constexpr int C = D / 8;
    __shared__ __align__(16) float sy[256 / C][D];
    __shared__ float2 sml[256 / C];
    const int64_t x = blockIdx.x;
    const int head = blockIdx.y, part = threadIdx.x / C, slice = part % a.slices;
    const int r = blockIdx.z * (256 / C / a.slices) + part / a.slices;
    const int2 at = a.target ? a.first[x] : make_int2((int)x * a.splits, a.chunk);
    const RowTile t = row_tile<ROWS>(a, (int)x);
    if (t.rows == 0) return;                                 // (and the first chunk's number is nobody's)
    // (where start decreases, a tile's chunks may not all have had a workgroup,
    // and what its first one's number would be is anything)
    if (a.target && at.y < LEAST) return;
    const int used = chunks_of(t, at.y, a.target ? INT_MAX : a.splits);
    if (used == 1 || (a.target && (at.x < 0 || at.x > a.pieces - used))) return;
    const int d0 = threadIdx.x % C * 8;
    float y[8], top = NONE, l = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] = 0.0f;
    auto add = [&](float mo, float n, const float *v) {
        const float now = fmaxf(top, mo);
        const float fo = __builtin_amdgcn_exp2f(top - now), fn = __builtin_amdgcn_exp2f(mo - now);
        top = now;
        l = l * fo + n * fn;
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = y[j] * fo + v[j] * fn;
    };
    // (eight chunks' loads at once: their latency is what this takes)
    for (int z0 = slice; z0 < used && r < t.rows; z0 += 8 * a.slices) {
        float2 ml[8];
        float v[8][8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float *p = part_of<D, ROWS>(a, at.x + min(z0 + i * a.slices, used - 1), head);
            ml[i] = *reinterpret_cast<const float2 *>(p + ROWS * D + 2 * r);
            *reinterpret_cast<float4 *>(v[i]) = *reinterpret_cast<const float4 *>(p + r * D + d0);
            *reinterpret_cast<float4 *>(v[i] + 4) = *reinterpret_cast<const float4 *>(p + r * D + d0 + 4);
        }
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (z0 + i * a.slices < used) add(ml[i].x, ml[i].y, v[i]);
    }
    if (slice) {
        *reinterpret_cast<float4 *>(&sy[part][d0]) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4 *>(&sy[part][d0 + 4]) = make_float4(y[4], y[5], y[6], y[7]);
        if (d0 == 0) sml[part] = make_float2(top, l);
    }
    __syncthreads();
    if (slice || r >= t.rows) return;
    const int slices = min(a.slices, used);
    float most = top;
    for (int z = 1; z < slices; z++) most = fmaxf(most, sml[part + z].x);
    const float f = __builtin_amdgcn_exp2f(top - most);
    l *= f;
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] *= f;
    for (int z = 1; z < slices; z++) {
        const float2 ml = sml[part + z];
        const float g = __builtin_amdgcn_exp2f(ml.x - most);
        l = fmaf(ml.y, g, l);
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = fmaf(sy[part + z][d0 + j], g, y[j]);
    }
    write_row<D, T>(a, t, head, r, d0, y, l, most);
}

template <int D, int ROWS, class T>
hipError_t launch_join(const KvAttend &a, const KvPlan &p, hipStream_t s)
{
    constexpr int PARTS = 2048 / D;                          // rows times slices of a workgroup
    KvAttend b = a;
    b.slices = 1;
    const int64_t chunks = p.target ? 2 * p.pieces / p.tiles : p.splits;      // a row tile's, about
    while (8 * b.slices < chunks && b.slices < PARTS) b.slices *= 2;
    const unsigned z = (ROWS + PARTS / b.slices - 1) / (PARTS / b.slices);
    hipLaunchKernelGGL((k_kv_join<D, ROWS, T>), dim3((unsigned)p.tiles, b.g.kv_heads, z), dim3(256), 0, s, b);
    return hipGetLastError();
}

}  // namespace

#endif
