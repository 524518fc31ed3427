// kv_weigh.hip -- the attention weight that each page of a sequence gathered:
//
//   w_j = decay w_j + sum_{rows r, heads h} sum_{t in page j, seen by r} exp(scale q_rh.k_t - lse_rh)
//
// The scores are formed as in kv_rows.hpp, transposed, from the keys' codes: a
// lane then has one query row and four tokens of each 16, and what it sums up
// belongs to one page, so that the lanes meet once a page.
//
// Few rows a sequence (k_kv_weigh): the queries stay in registers and the keys
// go past them, in equal parts of all sequences' pages for each wavefront.
// Many (k_kv_weigh_rows): the keys stay in registers, unpacked once, and the
// queries go past them, through LDS.
//
// (Times here and below are replays of a graph, one call after the other.)  Few
// rows are bound by HBM: one token on 131071, 64 heads on 8 of 128 (71 MB of keys),
// 17.5 us, 4.1 TB/s; 16 sequences of 1 to 3 tokens on up to 8190, 32 heads (37 MB),
// 13.8: four pages or five a wavefront, so that the chain of loads to the first of
// them is half of that.  Many are bound by vector instructions and matrix ones
// after one another: 1024 new tokens of each of two sequences, 11 thousand tokens
// in all, 32 heads on 8 of 128, 115 us, 0.74 PFLOP/s (16 by 16 products of operands
// in fp16 that every workgroup made took 160).  Of the cycles in which a CU has
// work there its SIMDs are at vector instructions for 77 % and at products for 38,
// which do little beside each other; and a CU has work for four fifths of the time,
// as units are 240 for 256 CUs and end apart.
#include <algorithm>
#include <type_traits>

#include "kv_attend.hpp"

namespace {

// The kernel's arguments, read anew where this stands: what a loop or the
// beginning of one needs of them then holds no scalar registers elsewhere.
__device__ __forceinline__ const KvWeigh &arguments()
{
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const KvWeigh *)p;
}

// A row's log sum as log2, x, and what its rounding leaves of it, y: as a factor
// 2^-y of the row's sums, or, from 2^16 on (FAR_SUM), as a number that each score
// loses before the exponential.  y grows with x, by 2^-24 of it: far out the factor
// leaves fp32's range (from 2^31 on) while what it belongs to is nothing or
// infinite already, and their product would not be a number.  Scores that near such
// a log sum are products with the fp32 logarithm of e, too, so that its own rest
// (REST) is not for them: a score of l then weighs 1.
constexpr float FAR_SUM = 0x1p16f;

struct LogSum {
    float x, rest, factor;       // rest 0, or factor 1
};

// Those of log sums up to 2^127 (the next number's is another); false for NaN.
__device__ __forceinline__ bool counted(float x) { return fabsf(x) <= 1.44269504088896341f * 0x1p127f; }

__device__ __forceinline__ LogSum log2_of(float l)
{
    constexpr float L = 1.44269504088896341f, REST = (float)(1.44269504088896340736 - (double)L);
    const float x = l * L, y = fmaf(l, L, -x);
    const bool far = fabsf(x) >= FAR_SUM;
    return {x, far ? y : 0.0f, far ? 1.0f : __builtin_amdgcn_exp2f(-(y + l * REST))};
}

// A lane's part of its row's query (PER words of eight elements), for matrix
// instructions of 16 columns.
template <int D, class T>
struct Part {
    static constexpr int PER = D / 32;
    uint4 w[PER];

    // (16 bytes at any address of an element: the hardware takes them)
    __device__ __forceinline__ void load(const KvTensor &q, int64_t row, int64_t h, int lane)
    {
        typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
        const T *p = static_cast<const T *>(q.data) + row * q.token + h * q.head + lane / 16 * (PER * 8);
#pragma unroll
        for (int j = 0; j < PER; j++) w[j] = __builtin_bit_cast(uint4, *reinterpret_cast<const any4 *>(p + 8 * j));
    }

    static __device__ __forceinline__ float low(uint32_t w)
    {
        return std::is_same<T, __bf16>::value ? __builtin_bit_cast(float, w << 16) : half_lo(w);
    }
    static __device__ __forceinline__ float high(uint32_t w)
    {
        return std::is_same<T, __bf16>::value ? __builtin_bit_cast(float, w & 0xFFFF0000u) : half_hi(w);
    }

    // Operands in the order that spread8 has (those of odd dimensions by 1/16), the
    // row scaled by a power of two as Query::make does, and the factors of its
    // scores: score = qs * (acc dk + (8 dk - mk) qsum), in log2 units.  Conversions
    // cut off what they cannot hold: elements 2^28 below the row's largest.
    template <class F>
    __device__ __forceinline__ void make(float &qs, float &qsum, float scale, F put) const
    {
        typedef unsigned short us2 __attribute__((ext_vector_type(2)));
        us2 most = {0, 0};                                   // (bits of numbers above 0 are in their order)
#pragma unroll
        for (int j = 0; j < PER; j++)
            each(w[j], [&](uint32_t x) { most = __builtin_elementwise_max(most, __builtin_bit_cast(us2, x & 0x7FFF7FFFu)); });
        uint32_t top = max((uint32_t)most[0], (uint32_t)most[1]);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const float t = low(top);
        // (a row below 2^-112 stays below 2^14, so that its factor is a number)
        const int e = t > 0.0f ? max((int)(__builtin_bit_cast(uint32_t, t) >> 23) - 127, -112) : 0;
        const float even = __builtin_bit_cast(float, (uint32_t)(127 + 14 - e) << 23);
        qs = fmaxf(scale * 1.44269504088896341f * __builtin_bit_cast(float, (uint32_t)max(127 + e - 14, 0) << 23), 0x1p-126f);
        const float odd = even * 0x1p-4f;
        const h2 one = {(_Float16)1.0f, (_Float16)1.0f}, many = {(_Float16)16.0f, (_Float16)16.0f};
        float sum = 0.0f;
        auto pair = [&](float a, float b, bool second) {
            const float f = second ? odd : even;
            const h2 y = __builtin_bit_cast(h2, __builtin_amdgcn_cvt_pkrtz(a * f, b * f));
            sum = __builtin_amdgcn_fdot2(y, second ? many : one, sum, false);
            return y;
        };
#pragma unroll
        for (int j = 0; j < PER; j++) {
            const h2 a = pair(low(w[j].x), low(w[j].z), false), b = pair(high(w[j].x), high(w[j].z), true);
            const h2 c = pair(low(w[j].y), low(w[j].w), false), d = pair(high(w[j].y), high(w[j].w), true);
            put(j, h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]});
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        qsum = sum;
    }

    // The row times the power of two that makes its largest element 1 to 2 (0: of
    // zeros, and what is below 2^-112 grows by no more); returns its inverse's
    // exponent.
    __device__ __forceinline__ int to_one()
    {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; j++)
            each(w[j], [&](uint32_t x) { top = fmaxf(top, fmaxf(fabsf(low(x)), fabsf(high(x)))); });
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const int e = top > 0.0f ? max((int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127, -112) : 0;
#pragma unroll
        for (int j = 0; j < PER; j++)
            each(w[j], [&](uint32_t &x) {
                typedef T t2 __attribute__((ext_vector_type(2)));
                x = __builtin_bit_cast(uint32_t, t2{(T)ldexpf(low(x), -e), (T)ldexpf(high(x), -e)});
            });
        return e;
    }

    template <class X, class F>
    static __device__ __forceinline__ void each(X &x, F f)
    {
        f(x.x), f(x.y), f(x.z), f(x.w);
    }
};

__device__ __forceinline__ float all_lanes(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, prefix(x)), 63));
}

// A lane's sequence s of the 64 that a wavefront looks at.
struct Look {
    int row0, n_new, len, pages;         // pages: those that are weighed
};

__device__ __forceinline__ Look look_at(const KvWeigh &b, int s)
{
    const KvGeom &g = b.a.g;
    Look x = {0, 0, 0, 0};
    if (s >= g.n_seqs) return x;
    x.row0 = min(max(g.start[s], 0), g.n_tokens);
    x.n_new = min(max(g.start[s + 1], x.row0), g.n_tokens) - x.row0;
    x.len = max(g.lens[s], 0);
    if (x.n_new)
        x.pages = min((min(x.len, KV_MOST_TOKENS) + (1 << g.page_shift) - 1) >> g.page_shift, (int)b.stride);
    return x;
}

// The sequences in one row, of n pages units(n) units each.
struct Line {
    Look mine;                           // of the first 64 sequences
    int all;                             // units

    template <class F>
    __device__ __forceinline__ Line(const KvWeigh &b, F units)
    {
        const int lane = threadIdx.x & 63;
        mine = look_at(b, lane);
        all = __builtin_amdgcn_readlane(prefix(units(mine.pages)), 63);
        for (int s0 = 64; s0 < b.a.g.n_seqs; s0 += 64)
            all += __builtin_amdgcn_readlane(prefix(units(look_at(b, s0 + lane).pages)), 63);
    }
};

// Unit `number` of all: its sequence (-1: past the last), its number there, and
// the sequence's pages.  first: the line's, or null, where it has not been kept.
struct Unit {
    KvSeq q;
    int at, pages;
};

template <class F>
__device__ __forceinline__ Unit find_unit(const KvWeigh &b, const Look *first, int number, F units)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int s0 = 0; s0 < b.a.g.n_seqs; s0 += 64) {
        const Look x = s0 || !first ? look_at(b, s0 + lane) : *first;
        const int n = units(x.pages), upto = prefix(n);
        const int c = __popcll(__ballot(before + upto <= number));
        auto of = [&](int y) { return __builtin_amdgcn_readlane(y, c); };
        if (c < 64) return {{s0 + c, of(x.row0), of(x.n_new), of(x.len)}, number - before - (of(upto) - of(n)), of(x.pages)};
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return {{-1, 0, 0, 0}, 0, 0};
}

// ------------------------------------------------------------------ few rows

constexpr int NW = 4;

// A row tile has 16 rows, the columns of a matrix instruction, or 8, which take
// both halves of them with the same queries: each half then has the scores of half
// of the tokens, which are a third of the work.
template <int D, int ROWS>
struct Step {                          // a lane's key words of 32 tokens, and the pairs of those whose scores it has
    static constexpr int PER = D / 32, TG = ROWS / 8;
    uint32_t w[2][PER];
    uint4 dm[TG];
};

// (`bytes` 0: zeros, and no traffic)
template <int D, int ROWS>
__device__ __forceinline__ void load_step(Step<D, ROWS> &o, const uint8_t *block, uint32_t bytes, int P, int t0, int lane)
{
    constexpr int W = D >= 128 ? 4 : 2, PER = Step<D, ROWS>::PER;
    const auto from = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(block), 0, bytes, 0x00027000);
    const int m = lane % 16, g = lane / 16;
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
        for (int j = 0; j < PER; j += W) {
            const uint32_t at = 4 * (kv_kword<D>(m, g * PER) + kv_kword<D>(16 * u, j));
            if constexpr (W == 4)
                *reinterpret_cast<uint4 *>(&o.w[u][j]) =
                    __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(from, at, t0 * (D / 2), 0));
            else
                *reinterpret_cast<uint2 *>(&o.w[u][j]) =
                    __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(from, at, t0 * (D / 2), 0));
        }
#pragma unroll
    for (int u = 0; u < Step<D, ROWS>::TG; u++)
        o.dm[u] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                                from, 16 * g + 64 * (ROWS == 8 ? m / 8 : u), P * D + t0 * 4, 0));
}

// A tile's rows: loaded, then made into operands.
template <int D, int ROWS, class T>
struct Rows {
    Part<D, T> raw;
    h8 q[D / 32];
    float qs, qsum, log_sum;
    float most, left, factor;    // the log sum: what goes from raw scores, and from scores, and a factor of sums
    bool counts;
    Span seen;

    __device__ __forceinline__ void load(const KvWeigh &b, const RowTile &t, int head, int lane)
    {
        const KvAttend &a = b.a;
        const int r = lane % ROWS;
        const int2 at = token_of(a, t, min(r, t.rows - 1));
        const int64_t tok = t.row0 + at.x, h = (int64_t)head * a.group + at.y;
        raw.load(a.q, tok, h, lane);
        log_sum = b.lse[tok * ((int64_t)a.g.kv_heads * a.group) + h];
        counts = r < t.rows;
        seen = span_of(a, t, r);
    }

    __device__ __forceinline__ void make(float scale)
    {
        raw.make(qs, qsum, scale, [&](int j, h8 y) { q[j] = y; });
        const LogSum lse = log2_of(log_sum);
        counts = counts && counted(lse.x);
        // (a far log sum goes from the raw scores, where a fused product takes it for
        // nothing, but for what is left of it; raw scores lie within 2^44, and one that
        // is past all of them goes as it is)
        most = lse.x * __builtin_amdgcn_rcpf(qs);
        const bool far = fabsf(lse.x) >= FAR_SUM && fabsf(most) < 0x1p60f;
        left = far ? fmaf(-most, qs, lse.x) + lse.rest : lse.x;
        most = far ? most : 0.0f;
        factor = lse.factor;
    }

    // sum over the lane's tokens of t0 .. t0 + 31
    __device__ __forceinline__ float sum(const Step<D, ROWS> &k, int t0, bool all, Masks mk, int lane) const
    {
        f4 acc[2];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            acc[u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < D / 32; j++)
                acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(spread8(k.w[u][j], mk), q[j], acc[u], 0, 0, 0);
        }
        const bool second = lane % 16 >= ROWS;
        float p[ROWS / 8][4], total = 0.0f;
#pragma unroll
        for (int u = 0; u < ROWS / 8; u++) {
            const uint32_t dm[4] = {k.dm[u].x, k.dm[u].y, k.dm[u].z, k.dm[u].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float x = ROWS == 8 && second ? acc[1][i] : acc[u][i];
                const float s = fmaf(x, half_lo(dm[i]), fmaf(fmaf(half_lo(dm[i]), 8.0f, -half_hi(dm[i])), qsum, -most));
                p[u][i] = __builtin_amdgcn_exp2f(fmaf(s, qs, -left));
            }
        }
        if (!all) {
            const unsigned first = t0 + 4 * (lane / 16) + (second ? 16 : 0) - seen.lo, many = seen.hi - seen.lo;
#pragma unroll
            for (int u = 0; u < ROWS / 8; u++)
#pragma unroll
                for (int i = 0; i < 4; i++) p[u][i] = first + 16 * u + i < many ? p[u][i] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < ROWS / 8; u++)
#pragma unroll
            for (int i = 0; i < 4; i++) total += p[u][i];
        return total;
    }
};

// The pages of all sequences in one row, of which each wavefront takes an equal
// part of a head's.
template <int D, int ROWS, class T>
__global__ __launch_bounds__(NW * 64) void k_kv_weigh(KvWeigh args)
{
    const int lane = threadIdx.x & 63, head = blockIdx.x;
    auto pages = [](int n) { return n; };
    const Line line(args, pages);
    const int waves = gridDim.y * NW, part = (line.all + waves - 1) / waves;
    int at = (blockIdx.y * NW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * part;
    const int end = min(at + part, line.all);
    const Masks mk = masks();
    while (at < end) {
        const Unit unit = find_unit(arguments(), &line.mine, at, pages);
        if (unit.q.seq < 0) return;
        const KvWeigh &b = arguments();
        const KvAttend &a = b.a;
        const KvGeom &g = a.g;
        const KvSeq q = unit.q;
        const int P = 1 << g.page_shift, hops = g.page_shift - 5;        // (32 tokens a step)
        const int32_t *table = g.table + (int64_t)q.seq * g.stride;
        auto present = [&](int32_t entry) { return (uint32_t)entry < g.n_pages; };
        // up to 64 pages: a lane keeps the entry and the weight of one
        const int j0 = unit.at, n = min(min(unit.pages - j0, end - at), 64), steps = n << hops;
        at += n;
        const int32_t entries = lane < n && j0 + lane < g.stride ? table[j0 + lane] : -1;
        const int64_t own = ((int64_t)q.seq * g.kv_heads + head) * b.stride + j0;
        for (int i = 0; i * ROWS < q.n_new * a.group; i++) { // (mostly one)
            const RowTile t = tile_of<ROWS>(a, q, i);
            const Span e = span_of(a, t, 0), f = span_of(a, t, t.rows - 1);
            Rows<D, ROWS, T> r;
            r.load(arguments(), t, head, lane);
            const float *before = i ? b.weights : b.before;
            const float prior = before && lane < n ? before[own + lane] : 0.0f;
            Step<D, ROWS> k[2];                              // two steps' loads are under way
            auto load = [&](Step<D, ROWS> &k, int step) {
                const int32_t entry = __builtin_amdgcn_readlane(entries, step >> hops);
                const int t0 = (j0 << g.page_shift) + 32 * step;
                const bool here = step < steps && present(entry) && t0 < t.hi && t0 + 32 > t.lo;
                load_step<D, ROWS>(k, g.pages + (uint64_t)(here ? (uint32_t)entry : 0u) * (uint64_t)g.page_bytes +
                                          (uint32_t)head * (uint32_t)g.block_bytes,
                                   here ? g.block_bytes : 0, P, t0 & (P - 1), lane);
            };
            load(k[0], 0);
            load(k[1], 1);
            r.make(a.scale);
            float sum = 0.0f, mine = 0.0f;
            for (int s = 0; s < steps; s += 2) {
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const int step = s + x, t0 = (j0 << g.page_shift) + 32 * step;
                    if (step >= steps) break;
                    if (t0 < t.hi && t0 + 32 > t.lo) sum += r.sum(k[x], t0, t0 >= f.lo && t0 + 32 <= e.hi, mk, lane);
                    load(k[x], step + 2);
                    if (step + 1 & (1 << hops) - 1) continue;
                    const float total = all_lanes(r.counts ? sum * r.factor : 0.0f);
                    mine = lane == step >> hops ? total : mine;
                    sum = 0.0f;
                }
            }
            if (lane < n) {
                const KvWeigh &z = arguments();
                z.weights[((int64_t)q.seq * z.a.g.kv_heads + head) * z.stride + j0 + lane] =
                    present(entries) ? fmaf(i ? 1.0f : z.decay, prior, mine) : 0.0f;
            }
        }
    }
}

// ------------------------------------------------------------------ many rows

// A workgroup, one a CU, has some blocks of 32 tokens of a sequence, and takes half
// as many row tiles of 32 at a time as it has wavefronts: two wavefronts bring one
// of them into LDS for all (two buffers, one barrier a time; what comes after them
// is loaded before it is used).  A block is a wavefront's, or, where there are few,
// several wavefronts', which take the row tiles in turn.  How many blocks a
// workgroup has is worked out from the lengths: the fewest with which every CU has
// as many turns as another.
//
// The codes are unpacked once, into the queries' own type, which holds them
// exactly, and their pairs are multiplied by the scale, so that a row needs no more
// than the sum of its elements and a score is two fused products: vector
// instructions are most of the time, and matrix ones hardly go on beside them
// (those of 32 by 32 more than those of 16 by 16: 128 cycles of them and 32 fused
// products, four wavefronts a SIMD, take 81 ns a wavefront with the small ones and
// 70 with the large, 58 without the products).  Row tiles that see none of a unit's
// tokens are left out where they lie before it (causal), and not where it is behind
// their window: 1024 new tokens on 8192 take 90 us, in a window of 64 still 48.
constexpr int TB = 32;

typedef float f16x __attribute__((ext_vector_type(16)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

// What the types of a query have for themselves.
template <class T> struct Kind;
template <>
struct Kind<_Float16> {
    typedef h8 v8;
    static __device__ __forceinline__ f16x product(h8 a, h8 b, f16x c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ float dot(uint32_t a, uint32_t b, float c)
    {
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
    }
    static constexpr uint32_t ONES = 0x3C003C00u;
};
template <>
struct Kind<__bf16> {
    typedef bf8 v8;
    static __device__ __forceinline__ f16x product(bf8 a, bf8 b, f16x c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ float dot(uint32_t a, uint32_t b, float c)
    {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2, a), __builtin_bit_cast(bf2, b), c, false);
    }
    static constexpr uint32_t ONES = 0x3F803F80u;
};

template <int D>
struct Made {                          // a row tile
    uint4 q[D / 16][64];               // lane: row % 32, half the dimensions
    float4 row[32];                    // sum of q, factor of the scores, log sum and its factor (0: adds nothing)
    float rest[32];                    // and what the scores lose with it
    int factors[2];                    // whether any of 16 rows' scores have a factor or lose something
};

// The lane, found anew where this stands (as arguments()).
__device__ __forceinline__ int lane_again()
{
    unsigned all = ~0u;
    asm volatile("" : "+s"(all));
    return (int)__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0));
}

// A wavefront's priority by how much it has done of what lies between barriers, in
// quarters: those behind go first, as the last alone would leave its SIMD idle
// between dependent instructions (115 us, and 118 as the hardware chooses).
__device__ __forceinline__ void give_way(int done)
{
    if (done == 0) __builtin_amdgcn_s_setprio(3);
    else if (done == 1) __builtin_amdgcn_s_setprio(2);
    else if (done == 2) __builtin_amdgcn_s_setprio(1);
    else __builtin_amdgcn_s_setprio(0);
}

// What a row's token sees.
__device__ __forceinline__ Span span_at(const KvAttend &a, const KvSeq &q, int token)
{
    RowTile t = {};
    t.rows = 1;
    t.n_new = q.n_new;
    t.len = q.len;
    t.tok0 = token;
    return span_of(a, t, 0);
}

// Wavefronts of a workgroup (registers, LDS; heads of 128 with 16 115 us, with 12
// 118.5).
template <int D> constexpr int MANY = D == 256 ? 8 : 16;

template <int D, class T>
__global__ __launch_bounds__(MANY<D> * 64) void k_kv_weigh_rows(KvWeigh args)
{
    typedef typename Kind<T>::v8 v8;
    constexpr int PER = D / 32, WORDS = D / 16, W = D >= 128 ? 4 : 2;
    constexpr int waves = MANY<D>, side = waves / 2;         // row tiles at a time
    __shared__ Made<D> made[2 * side];
    __shared__ float sums[waves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), head = blockIdx.x;
    const int col = lane % 32, half = lane / 32;             // of a product: row, and tokens 8 i + 4 half + 0 .. 3
    const int shift = args.a.g.page_shift, P = 1 << shift, each = P / TB;    // a page's blocks
    const int all = Line(args, [&](int n) { return n * each; }).all, groups = gridDim.y;
    if (all == 0) return;
    const int turns = (all + groups * waves - 1) / (groups * waves), some = (all + turns * groups - 1) / (turns * groups);
    const int most = min((some + each - 1) / each * each, waves / each * each);        // whole pages
    for (int number = blockIdx.y;; number += groups) {
        const Unit unit = find_unit(arguments(), nullptr, number, [&](int n) { return (n * each + most - 1) / most; });
        if (unit.q.seq < 0) return;
        const KvWeigh &b = arguments();
        const KvAttend &a = b.a;
        const KvGeom &g = a.g;
        const KvSeq q = unit.q;
        // the unit's blocks, and wavefronts that share one
        const int blocks = min(unit.pages * each - unit.at * most, most), ways = min(waves / blocks, side);
        const int way = wave / blocks, base = unit.at * most * TB, t0 = base + (wave - way * blocks) * TB;
        // the scale, as a factor of the pairs and, where that could leave their range, a
        // power of two of each row's scores
        float times = a.scale;
        int power = 0;
        if (!(times >= 0x1p-40f && times <= 0x1p40f)) times = frexpf(times, &power);
        power = __builtin_amdgcn_readfirstlane(power);
        times *= 1.44269504088896341f;
        // the keys of t0 .. t0 + 31, as operands, and what makes scores of the lane's
        // tokens (four of each 8): score = acc dk + ck (sum of q), in log2 units
        v8 k[WORDS];
        float dk[16], ck[16];
        const int64_t page = t0 >> shift < unit.pages ? kv_page(g, q.seq, t0) : -1;
        {
            // (bytes 0: zeros, and no traffic)
            const auto from = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t *>(g.pages + max(page, (int64_t)0) * g.page_bytes + (int64_t)head * g.block_bytes), 0,
                page < 0 ? 0 : g.block_bytes, 0x00027000);
            const int at = t0 & (P - 1), lane = lane_again(), col = lane % 32, half = lane / 32;
            uint32_t w[WORDS];
#pragma unroll
            for (int j = 0; j < WORDS; j += W) {
                const uint32_t off = 4 * kv_kword<D>(col, half * WORDS + j);
                if constexpr (W == 4)
                    *reinterpret_cast<uint4 *>(w + j) =
                        __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(from, off, at * (D / 2), 0));
                else
                    *reinterpret_cast<uint2 *>(w + j) =
                        __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(from, off, at * (D / 2), 0));
            }
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const uint4 dm = __builtin_bit_cast(
                    uint4, __builtin_amdgcn_raw_buffer_load_b128(from, 32 * u + 16 * half, P * D + at * 4, 0));
                const uint32_t d[4] = {dm.x, dm.y, dm.z, dm.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    dk[4 * u + i] = half_lo(d[i]) * times;
                    ck[4 * u + i] = fmaf(half_lo(d[i]), 8.0f, -half_hi(d[i])) * times;
                }
            }
#pragma unroll
            for (int j = 0; j < WORDS; j++)
#pragma unroll
                for (int i = 0; i < 8; i++) k[j][i] = (T)((float)(w[j] >> 4 * i & 15u) - 8.0f);
        }
        // rows' tokens and heads, without a division each
        const int rows = q.n_new * a.group, tiles = (rows + 31) / 32, group = a.group;
        struct Place {
            int tok, head;
        };
        auto place = [&](int row) {
            const int tok = row / group;
            return Place{tok, row - tok * group};
        };
        const Place hop = place(32 * side);
        auto go_on = [&](Place &p) {
            p.tok += hop.tok;
            p.head += hop.head;
            if (p.head >= group) {
                p.head -= group;
                p.tok++;
            }
        };
        // (rows before the first that sees the block's first token see none of it)
        int i0 = 0;
        if (a.causal) {
            const int64_t before = (int64_t)base - (q.len - q.n_new);
            if (before > 0) i0 = (int)min(before * group / 32, (int64_t)tiles) / side * side;
        }
        // this wavefront's 16 rows of the row tile that is `coming`: loaded, and put
        // into LDS
        int coming = i0 + wave / 2;
        Place mine = place(32 * coming + wave % 2 * 16 + lane_again() % 16);
        Part<D, T> raw;
        float log_sum = 0.0f;
        auto load = [&] {
            if (coming >= tiles) return;
            const KvWeigh &b = arguments();
            const int lane = lane_again();
            const bool in = 32 * coming + wave % 2 * 16 + lane % 16 < rows;     // (past the last one: that one)
            const int64_t tok = q.row0 + (in ? mine.tok : q.n_new - 1);
            const int64_t h = (int64_t)head * group + (in ? mine.head : group - 1);
            raw.load(b.a.q, tok, h, lane);
            log_sum = b.lse[tok * ((int64_t)b.a.g.kv_heads * group) + h];
        };
        auto put = [&](Made<D> &o) {
            if (coming >= tiles) return;
            const int lane = lane_again(), own = wave % 2 * 16 + lane % 16, quarter = lane / 16;
            float sum = 0.0f, squares = 0.0f;
            auto count = [&] {
                sum = squares = 0.0f;
#pragma unroll
                for (int j = 0; j < PER; j++)
                    Part<D, T>::each(raw.w[j], [&](uint32_t x) {
                        sum = Kind<T>::dot(x, Kind<T>::ONES, sum);
                        squares = Kind<T>::dot(x, x, squares);
                    });
                sum += __shfl_xor(sum, 16);
                squares += __shfl_xor(squares, 16);
                sum += __shfl_xor(sum, 32);
                squares += __shfl_xor(squares, 32);
            };
            count();
            int by = power;
            // rows whose products could leave fp32's range: brought to 1 by a power of two
            if (__any(!(squares >= 0x1p-100f && squares < 0x1p100f))) {
                by += raw.to_one();
                count();
            }
#pragma unroll
            for (int j = 0; j < PER; j++) o.q[quarter % 2 * PER + j][quarter / 2 * 32 + own] = raw.w[j];
            const LogSum lse = log2_of(log_sum);
            const bool counts = 32 * coming + own < rows && counted(lse.x);
            if (quarter == 0) {
                o.row[own] = make_float4(sum, ldexpf(1.0f, min(max(by, -126), 127)), lse.x, counts ? lse.factor : 0.0f);
                o.rest[own] = lse.rest;
            }
            const int factors = __any(by != 0 || (counts && fabsf(lse.x) >= FAR_SUM));
            if (lane == 0) o.factors[wave % 2] = factors;
        };
        auto next = [&] {
            coming += side;
            go_on(mine);
        };
        float total = 0.0f;
        int turn = 0;
        Place first = place(32 * (i0 + min(lane_again(), side)));            // of row tile `lane` of those in LDS
        load();
        for (int i = i0 - side; i < tiles; i += side, turn ^= 1) {
            __syncthreads();
            put(made[turn * side + wave / 2]);
            next();
            load();
            // (nothing is there yet; or the wavefront brings tiles, and has no block)
            if (i < i0 || way >= ways) continue;
            const Made<D> *o = made + (turn ^ 1) * side;
            const int have = min(tiles - i, side);
            // of row tile `lane`: the tokens that some of its rows see, and that all do
            const int more = min(max(rows - 32 * (i + lane), 1), 32) - 1;
            const int last = first.tok + (int)((unsigned)(first.head + more) * a.group_inv >> 21);
            const Span e = span_at(arguments().a, q, first.tok), f = span_at(arguments().a, q, last);
            const int2 factor = *reinterpret_cast<const int2 *>(o[min(lane, have - 1)].factors);
            const uint64_t some = __ballot(e.lo < t0 + TB && f.hi > t0), every = __ballot(f.lo <= t0 && e.hi >= t0 + TB);
            const uint64_t plain = __ballot(!(factor.x | factor.y));
            for (int n = way; n < have; n += ways) {
                if (!(some >> n & 1)) continue;
                give_way(n / (side / 4));
                const float4 row = o[n].row[col];
                f16x acc = {};
#pragma unroll
                for (int j = 0; j < WORDS; j++) acc = Kind<T>::product(k[j], __builtin_bit_cast(v8, o[n].q[j][lane]), acc);
                if (plain >> n & 1) {
#pragma unroll
                    for (int x = 0; x < 16; x++) acc[x] = fmaf(acc[x], dk[x], fmaf(ck[x], row.x, -row.z));
                } else {
#pragma unroll
                    for (int x = 0; x < 16; x++) acc[x] = fmaf(fmaf(acc[x], dk[x], ck[x] * row.x), row.y, -row.z);
                    const float rest = o[n].rest[lane_again() % 32];
#pragma unroll
                    for (int x = 0; x < 16; x++) acc[x] -= rest;
                }
#pragma unroll
                for (int x = 0; x < 16; x++) acc[x] = __builtin_amdgcn_exp2f(acc[x]);
                if (!(every >> n & 1)) {
                    const KvAttend &a = arguments().a;
                    const unsigned row0 = __builtin_amdgcn_readlane(first.head, n) + col;
                    const Span seen = span_at(a, q, __builtin_amdgcn_readlane(first.tok, n) + (int)(row0 * a.group_inv >> 21));
                    const unsigned from = t0 + 4 * half - seen.lo, many = seen.hi - seen.lo;
#pragma unroll
                    for (int x = 0; x < 16; x++) acc[x] = from + x / 4 * 8 + x % 4 < many ? acc[x] : 0.0f;
                }
#pragma unroll
                for (int m = 8; m; m /= 2)
#pragma unroll
                    for (int x = 0; x < m; x++) acc[x] += acc[x + m];
                total += row.w != 0.0f ? acc[0] * row.w : 0.0f;
            }
            give_way(3);
            go_on(first);
        }
        total = all_lanes(total);
        if (lane == 0) sums[wave] = total;
        __syncthreads();
        const int at = wave * 64 + lane_again(), j = (base >> shift) + at;
        if (at * each < blocks) {
            const KvWeigh &b = arguments();
            const KvGeom &g = b.a.g;
            const int64_t own = ((int64_t)q.seq * g.kv_heads + head) * b.stride;
            float x = 0.0f;
            if (kv_page(g, q.seq, j << shift) >= 0) {
                for (int w = 0; w < ways; w++)
                    for (int n = 0; n < each; n++) x += sums[w * blocks + at * each + n];
                if (b.before) x = fmaf(b.decay, b.before[own + j], x);
            }
            b.weights[own + j] = x;
        }
        __syncthreads();                                     // (the next block's rows and sums)
    }
}

template <int D, class T>
hipError_t launch(const KvWeigh &b, hipStream_t s)
{
    const KvGeom &g = b.a.g;
    const int64_t rows = (int64_t)g.n_tokens * b.a.group;
    // By the average, which is all that the host knows.  It is dear for a batch of both
    // kinds: 63 sequences with one token on 2000, 32 heads on 8 of 128, 16.7 us, one
    // with 190 17.8 and with 500 30.5, alone; together the first are 254 us (the
    // prompt's keys are read once for each 16 rows), with the second 112 (the tokens'
    // rows fill an eighth of a tile of 32).
    if (rows <= 16 * (int64_t)g.n_seqs) {
        // Four wavefronts a SIMD: one token on 131071, 64 heads on 8, 17.5 us, with two
        // 18.6 and with eight 20.0; 16 sequences of up to 8190 13.8, 14.6 and 14.6.
        const dim3 grid(g.kv_heads, std::max(4096 / g.kv_heads / NW, 1));
        // Eight rows where no sequence has more, as far as the host can tell (the first
        // of those calls with 16: 18.6 us; the second has sequences of 4 to 12 rows, of
        // which 8 read the keys twice: 14.7 us, and 13.8 with 16).
        if (rows <= 8 || (b.a.group <= 8 && g.n_tokens <= g.n_seqs))
            hipLaunchKernelGGL((k_kv_weigh<D, 8, T>), grid, dim3(NW * 64), 0, s, b);
        else
            hipLaunchKernelGGL((k_kv_weigh<D, 16, T>), grid, dim3(NW * 64), 0, s, b);
    } else {
        hipLaunchKernelGGL((k_kv_weigh_rows<D, T>), dim3(g.kv_heads, std::max(256 / g.kv_heads, 1)), dim3(MANY<D> * 64), 0, s, b);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t lw_launch_kv_weigh(const KvWeigh &b, int head_dim, int dtype, hipStream_t s)
{
    const bool half = dtype == LW_F16;
    if (head_dim == 64) return half ? launch<64, _Float16>(b, s) : launch<64, __bf16>(b, s);
    if (head_dim == 128) return half ? launch<128, _Float16>(b, s) : launch<128, __bf16>(b, s);
    if (head_dim == 256) return half ? launch<256, _Float16>(b, s) : launch<256, __bf16>(b, s);
    return hipErrorInvalidValue;
}
