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
// queries go past them, made into operands once a workgroup.
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

// A row's log sum, as log2 and what its rounding leaves.
__device__ __forceinline__ float2 log2_of(float l)
{
    constexpr float L = 1.44269504088896341f, REST = (float)(1.44269504088896340736 - (double)L);
    const float x = l * L;
    return make_float2(x, fmaf(l, L, -x) + l * REST);
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

private:
    template <class F>
    static __device__ __forceinline__ void each(uint4 x, F f)
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
    float2 lse;
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
        lse = log2_of(log_sum);
        counts = counts && fabsf(lse.x) < __builtin_inff();
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
                const float s = fmaf(x, half_lo(dm[i]), fmaf(half_lo(dm[i]), 8.0f, -half_hi(dm[i])) * qsum);
                p[u][i] = __builtin_amdgcn_exp2f(fmaf(s, qs, -lse.x));
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
                    const float total = all_lanes(r.counts ? sum * __builtin_amdgcn_exp2f(-r.lse.y) : 0.0f);
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

// A workgroup, one a CU, has some blocks of 32 tokens of a sequence, and takes as
// many row tiles at a time as it has wavefronts: each makes one of them into
// operands in LDS for all (two buffers, one barrier a time; what comes after them
// is loaded before it is used).  A block is a wavefront's, or, where there are few,
// several wavefronts', which take the row tiles in turn.  How many blocks a
// workgroup has is worked out from the lengths: the fewest with which every CU has
// as many turns as another.
constexpr int TB = 32;

template <int D>
struct Made {                          // a row tile
    h8 q[D / 32][64];
    float4 row[16];                    // qs, qsum, log sum, 2^-what its rounding leaves (0: adds nothing)
    int2 seen[16];
    int4 tile;                         // tokens that some of its rows see, and that all do
};

// Wavefronts of a workgroup (registers, LDS).
template <int D> constexpr int MANY = D == 256 ? 8 : 16;

template <int D, class T>
__global__ __launch_bounds__(MANY<D> * 64) void k_kv_weigh_rows(KvWeigh args)
{
    constexpr int PER = D / 32;
    constexpr int waves = MANY<D>;
    __shared__ Made<D> made[2 * waves];
    __shared__ float sums[waves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), head = blockIdx.x;
    const int m = lane % 16, quarter = lane / 16;
    const Masks mk = masks();
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
        const int blocks = min(unit.pages * each - unit.at * most, most), ways = waves / blocks;
        const int way = wave / blocks, base = unit.at * most * TB, t0 = base + (wave - way * blocks) * TB;
        // the keys of t0 .. t0 + 31, as operands, and what makes scores of the lane's
        // tokens (four of each 16)
        h8 k[2][PER];
        h2 dk[2][2];
        float ck[2][4];
        const int64_t page = t0 >> shift < unit.pages ? kv_page(g, q.seq, t0) : -1;
        {
            Step<D, 16> x;
            load_step<D, 16>(x, g.pages + max(page, (int64_t)0) * g.page_bytes + (int64_t)head * g.block_bytes,
                         page < 0 ? 0 : g.block_bytes, P, t0 & (P - 1), lane);
#pragma unroll
            for (int u = 0; u < 2; u++) {
#pragma unroll
                for (int j = 0; j < PER; j++) k[u][j] = spread8(x.w[u][j], mk);
                const uint32_t d[4] = {x.dm[u].x, x.dm[u].y, x.dm[u].z, x.dm[u].w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    dk[u][i / 2][i % 2] = halves(d[i])[0];
                    ck[u][i] = fmaf(half_lo(d[i]), 8.0f, -half_hi(d[i]));
                }
            }
        }
        // 16 rows, row tile i of the sequence: loaded, and made into operands
        const int tiles = (q.n_new * a.group + 15) / 16;
        Part<D, T> raw;
        float log_sum = 0.0f;
        auto load = [&](int i) {
            if (i >= tiles) return;
            const KvWeigh &b = arguments();
            const KvAttend &a = b.a;
            const RowTile t = tile_of<16>(a, q, i);
            const int2 at = token_of(a, t, min(m, t.rows - 1));
            const int64_t tok = t.row0 + at.x, h = (int64_t)head * a.group + at.y;
            raw.load(a.q, tok, h, lane);
            log_sum = b.lse[tok * ((int64_t)a.g.kv_heads * a.group) + h];
        };
        auto put = [&](int i, Made<D> &o) {
            if (i >= tiles) return;
            const KvAttend &a = arguments().a;
            const RowTile t = tile_of<16>(a, q, i);
            float qs, qsum;
            raw.make(qs, qsum, a.scale, [&](int j, h8 y) { o.q[j][lane] = y; });
            const float2 lse = log2_of(log_sum);
            const bool counts = m < t.rows && fabsf(lse.x) < __builtin_inff();
            const Span seen = span_of(a, t, m), e = span_of(a, t, 0), f = span_of(a, t, t.rows - 1);
            if (quarter == 0) {
                o.row[m] = make_float4(qs, qsum, lse.x, counts ? __builtin_amdgcn_exp2f(-lse.y) : 0.0f);
                o.seen[m] = make_int2(seen.lo, seen.hi);
                // (a row past the last one adds nothing, whatever it sees)
                if (m == 0) o.tile = make_int4(e.lo, f.hi, f.lo, e.hi);
            }
        };
        float total = 0.0f;
        // (rows before the first that sees the block's first token see none of it)
        int i0 = 0;
        if (a.causal) {
            const int64_t before = (int64_t)base - (q.len - q.n_new);
            if (before > 0) i0 = (int)min(before * a.group / 16, (int64_t)tiles) / waves * waves;
        }
        int turn = 0;
        load(i0 + wave);
        put(i0 + wave, made[wave]);
        load(i0 + waves + wave);
        for (int i = i0; i < tiles; i += waves, turn ^= 1) {
            __syncthreads();
            put(i + waves + wave, made[(turn ^ 1) * waves + wave]);
            load(i + 2 * waves + wave);
            const Made<D> *o = made + turn * waves;
            const int have = min(tiles - i, waves);
            const int4 tile = o[min(lane, have - 1)].tile;
            h8 y[PER];
            float4 row;
            auto fetch = [&](int n) {
#pragma unroll
                for (int j = 0; j < PER; j++) y[j] = o[n].q[j][lane];
                row = o[n].row[m];
            };
            if (way >= ways) continue;                       // (makes tiles, and has no block)
            fetch(min(way, have - 1));
            for (int n = way; n < have; n += ways) {
                f4 acc[2];
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    acc[u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < PER; j++) acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[u][j], y[j], acc[u], 0, 0, 0);
                }
                const float4 now = row;
                fetch(min(n + ways, have - 1));             // the next one's, while this one's are worked on
                const int lo = __builtin_amdgcn_readlane(tile.x, n), hi = __builtin_amdgcn_readlane(tile.y, n);
                if (lo >= t0 + TB || hi <= t0) continue;
                const bool every = __builtin_amdgcn_readlane(tile.z, n) <= t0 && __builtin_amdgcn_readlane(tile.w, n) >= t0 + TB;
                float p[2][4], sum = 0.0f;
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int x = 0; x < 4; x++)
                        p[u][x] = __builtin_amdgcn_exp2f(fmaf(fmaf(acc[u][x], (float)dk[u][x / 2][x % 2], ck[u][x] * now.y), now.x, -now.z));
                if (!every) {
                    const int2 seen = o[n].seen[m];
                    const unsigned first = t0 + 4 * quarter - seen.x, many = seen.y - seen.x;
#pragma unroll
                    for (int u = 0; u < 2; u++)
#pragma unroll
                        for (int x = 0; x < 4; x++) p[u][x] = first + 16 * u + x < many ? p[u][x] : 0.0f;
                }
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int x = 0; x < 4; x++) sum += p[u][x];
                total += now.w != 0.0f ? sum * now.w : 0.0f;
            }
        }
        total = all_lanes(total);
        if (lane == 0) sums[wave] = total;
        __syncthreads();
        const int at = threadIdx.x, j = (base >> shift) + at;
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
    if (rows <= 16 * (int64_t)g.n_seqs) {
        // Four wavefronts a SIMD: one token on 131071, 64 heads on 8, 16.4 us, with two
        // 17.3 and with eight 18.8; 16 sequences of up to 8190 14.2, 15.6 and 14.4.
        const dim3 grid(g.kv_heads, std::max(4096 / g.kv_heads / NW, 1));
        // Eight rows where no sequence has more, as far as the host can tell (the first
        // of those calls with 16: 17.4 us; the second has sequences of 4 to 12 rows, of
        // which 8 would read the keys twice: 13.3 us with 16).
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
