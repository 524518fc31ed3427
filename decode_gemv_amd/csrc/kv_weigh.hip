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

__device__ __forceinline__ float all_lanes(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, prefix(x)), 63));
}

// Pages of sequence s that are weighed.
__device__ __forceinline__ int pages_of(const KvWeigh &b, int s)
{
    const KvGeom &g = b.a.g;
    const int row0 = min(max(g.start[s], 0), g.n_tokens), row1 = min(max(g.start[s + 1], row0), g.n_tokens);
    const int len = min(max(g.lens[s], 0), KV_MOST_TOKENS);
    return row1 == row0 ? 0 : min((len + (1 << g.page_shift) - 1) >> g.page_shift, (int)b.stride);
}

// Unit `number` of all sequences' in one row, where a sequence of n pages has
// units(n): its sequence (-1: past the last), its number there, the sequence's
// pages, and the number of all (to the end, or of those looked at).
struct Unit {
    int seq, at, pages, all;
};

template <class F>
__device__ __forceinline__ Unit find_unit(const KvWeigh &b, int number, F units)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int s0 = 0; s0 < b.a.g.n_seqs; s0 += 64) {
        const int pages = s0 + lane < b.a.g.n_seqs ? pages_of(b, s0 + lane) : 0;
        const int n = units(pages), upto = prefix(n);
        const int c = __popcll(__ballot(before + upto <= number));
        if (c < 64)
            return {s0 + c, number - before - (__builtin_amdgcn_readlane(upto, c) - __builtin_amdgcn_readlane(n, c)),
                    __builtin_amdgcn_readlane(pages, c), 0};
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return {-1, 0, 0, before};
}

__device__ __forceinline__ KvSeq sequence(const KvGeom &g, int s)
{
    KvSeq q = {s, min(max(g.start[s], 0), g.n_tokens), 0, max(g.lens[s], 0)};
    q.n_new = min(max(g.start[s + 1], q.row0), g.n_tokens) - q.row0;
    return q;
}

// ------------------------------------------------------------------ few rows

constexpr int NW = 4;

template <int D>
struct Step {                          // a lane's key words and pairs of 32 tokens
    static constexpr int PER = D / 32;
    uint32_t w[2][PER];
    uint4 dm[2];
};

// (`bytes` 0: zeros, and no traffic)
template <int D>
__device__ __forceinline__ void load_step(Step<D> &o, const uint8_t *block, uint32_t bytes, int P, int t0, int lane)
{
    constexpr int W = D >= 128 ? 4 : 2, PER = Step<D>::PER;
    const auto from = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(block), 0, bytes, 0x00027000);
    const int m = lane % 16, g = lane / 16;
#pragma unroll
    for (int u = 0; u < 2; u++) {
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
        o.dm[u] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(from, 16 * g + 64 * u, P * D + t0 * 4, 0));
    }
}

// 16 query rows.
template <int D, class T>
struct Rows {
    h8 q[D / 32];
    float qs, qsum;
    float2 lse;
    bool counts;
    Span seen;

    __device__ __forceinline__ void load(const KvWeigh &b, const RowTile &t, int head, int lane)
    {
        const KvAttend &a = b.a;
        const int m = lane % 16, r = min(m, t.rows - 1);
        const int2 at = token_of(a, t, r);
        const int64_t tok = t.row0 + at.x, h = (int64_t)head * a.group + at.y;
        Query<D, 16, T> x;
        x.load(a.q, tok, h, lane);
        const float l = b.lse[tok * ((int64_t)a.g.kv_heads * a.group) + h];
        x.make(qs, qsum, a.scale, [&](int j, h8 y) { q[j] = y; });
        counts = m < t.rows && fabsf(l) < __builtin_inff();
        lse = log2_of(l);
        seen = span_of(a, t, m);
    }

    // sum over the lane's tokens of t0 .. t0 + 31
    __device__ __forceinline__ float sum(const Step<D> &k, int t0, bool all, Masks mk, int lane) const
    {
        float total = 0.0f;
        const unsigned first = all ? 0 : t0 + 4 * (lane / 16) - seen.lo, many = all ? ~0u : seen.hi - seen.lo;
#pragma unroll
        for (int u = 0; u < 2; u++) {
            f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < D / 32; j++)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(spread8(k.w[u][j], mk), q[j], acc, 0, 0, 0);
            const uint32_t dm[4] = {k.dm[u].x, k.dm[u].y, k.dm[u].z, k.dm[u].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float s = fmaf(acc[i], half_lo(dm[i]), fmaf(half_lo(dm[i]), 8.0f, -half_hi(dm[i])) * qsum);
                const float p = __builtin_amdgcn_exp2f(fmaf(s, qs, -lse.x));
                total += first + 16 * u + i < many ? p : 0.0f;
            }
        }
        return total;
    }
};

// The pages of all sequences in one row, of which each wavefront takes an equal
// part of a head's.
template <int D, class T>
__global__ __launch_bounds__(NW * 64) void k_kv_weigh(KvWeigh args)
{
    const int lane = threadIdx.x & 63, head = blockIdx.x;
    auto pages = [](int n) { return n; };
    const int all = find_unit(args, INT_MAX, pages).all, waves = gridDim.y * NW, part = (all + waves - 1) / waves;
    int at = (blockIdx.y * NW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * part;
    const int end = min(at + part, all);
    const Masks mk = masks();
    while (at < end) {
        const Unit unit = find_unit(arguments(), at, pages);
        if (unit.seq < 0) return;
        const KvWeigh &b = arguments();
        const KvAttend &a = b.a;
        const KvGeom &g = a.g;
        const int P = 1 << g.page_shift;
        const KvSeq q = sequence(g, unit.seq);
        const int j0 = unit.at, j1 = min(unit.pages, j0 + end - at);
        at += j1 - j0;
        const int32_t *table = g.table + (int64_t)q.seq * g.stride;
        const int known = (int)min((int64_t)j1, g.stride);
        auto entry_at = [&](int j) { return j < known ? table[j] : -1; };
        auto present = [&](int32_t entry) { return (uint32_t)entry < g.n_pages; };
        for (int i = 0; i * 16 < q.n_new * a.group; i++) {   // (mostly one)
            const RowTile t = tile_of<16>(a, q, i);
            const Span e = span_of(a, t, 0), f = span_of(a, t, t.rows - 1);
            int32_t entry = __builtin_amdgcn_readfirstlane(entry_at(j0)), after = entry_at(j0 + 1);
            Step<D> k;
            auto load = [&](int32_t entry, int t0) {
                const bool here = present(entry) && t0 < t.hi && t0 + 32 > t.lo;
                load_step<D>(k, g.pages + (uint64_t)(here ? (uint32_t)entry : 0u) * (uint64_t)g.page_bytes +
                                    (uint32_t)head * (uint32_t)g.block_bytes,
                             here ? g.block_bytes : 0, P, t0 & (P - 1), lane);
            };
            load(entry, j0 << g.page_shift);
            Rows<D, T> r;
            r.load(arguments(), t, head, lane);
            for (int j = j0; j < j1; j++) {
                const int32_t next = __builtin_amdgcn_readfirstlane(after);
                after = entry_at(j + 2);
                float total = 0.0f;
                for (int s = 0; s < P; s += 32) {
                    const int t0 = (j << g.page_shift) + s;
                    const Step<D> now = k;
                    load(s + 32 < P ? entry : next, t0 + 32);
                    if (t0 < t.hi && t0 + 32 > t.lo) total += r.sum(now, t0, t0 >= f.lo && t0 + 32 <= e.hi, mk, lane);
                }
                total = all_lanes(r.counts ? total * __builtin_amdgcn_exp2f(-r.lse.y) : 0.0f);
                const KvWeigh &z = arguments();
                const int64_t to = ((int64_t)q.seq * z.a.g.kv_heads + head) * z.stride + j;
                if (!present(entry)) total = 0.0f;
                else if (i) total += z.weights[to];
                else if (z.before) total = fmaf(z.decay, z.before[to], total);
                if (lane == 0) z.weights[to] = total;
                entry = next;
            }
        }
    }
}

// ------------------------------------------------------------------ many rows

// A workgroup has WAVES blocks of TB tokens, one a wavefront, and takes the
// rows 16 * WAVES at a time: each wavefront makes 16 of them into operands in
// LDS for all (two buffers, one barrier a time).
template <int D>
struct Many {
    static constexpr int WAVES = 8, TB = 32, SUBS = TB / 16;
    static constexpr int TOKENS = WAVES * TB, ROWS = WAVES * 16;             // pages divide TOKENS
    struct Buffer {
        h8 q[WAVES][D / 32][64];
        float4 row[ROWS];                // qs, qsum, log sum, 2^-what its rounding leaves (0: adds nothing)
        int2 seen[ROWS];
    };
};

template <int D, class T>
__global__ __launch_bounds__(Many<D>::WAVES * 64) void k_kv_weigh_rows(KvWeigh args)
{
    using M = Many<D>;
    constexpr int W = D >= 128 ? 4 : 2, PER = D / 32;
    __shared__ typename M::Buffer buf[2];
    __shared__ float sums[M::TOKENS / 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), head = blockIdx.x;
    const int m = lane % 16, quarter = lane / 16;
    const Masks mk = masks();
    for (int number = blockIdx.y;; number += gridDim.y) {
        const int shift = args.a.g.page_shift, P = 1 << shift;
        const Unit unit = find_unit(arguments(), number, [&](int n) { return ((n << shift) + M::TOKENS - 1) / M::TOKENS; });
        if (unit.seq < 0) return;
        const KvWeigh &b = arguments();
        const KvAttend &a = b.a;
        const KvGeom &g = a.g;
        const KvSeq q = sequence(g, unit.seq);
        const int n_pages = unit.pages, block = unit.at;
        const int base = block * M::TOKENS, t0 = base + wave * M::TB;
        // the keys of t0 .. t0 + TB - 1, as operands, and what makes scores of
        // the lane's tokens (four of each 16)
        h8 k[M::SUBS][PER];
        float dk[M::SUBS][4], ck[M::SUBS][4];
#pragma unroll
        for (int u = 0; u < M::SUBS; u++) {
            const int t = t0 + 16 * u;
            const int64_t page = t >> g.page_shift < n_pages ? kv_page(g, q.seq, t) : -1;
            uint32_t w[PER];
            uint4 dm = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < PER; j++) w[j] = 0;
            if (page >= 0) {
                const uint32_t *words = reinterpret_cast<const uint32_t *>(g.pages + page * g.page_bytes + (int64_t)head * g.block_bytes);
#pragma unroll
                for (int j = 0; j < PER; j += W) {
                    const uint32_t *from = words + kv_kword<D>((t & (P - 1)) + m, quarter * PER + j);
                    if constexpr (W == 4)
                        *reinterpret_cast<uint4 *>(&w[j]) = *reinterpret_cast<const uint4 *>(from);
                    else
                        *reinterpret_cast<uint2 *>(&w[j]) = *reinterpret_cast<const uint2 *>(from);
                }
                dm = *reinterpret_cast<const uint4 *>(words + P * (D / 4) + (t & (P - 1)) + 4 * quarter);
            }
#pragma unroll
            for (int j = 0; j < PER; j++) k[u][j] = spread8(w[j], mk);
            const uint32_t d[4] = {dm.x, dm.y, dm.z, dm.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                dk[u][i] = half_lo(d[i]);
                ck[u][i] = fmaf(dk[u][i], 8.0f, -half_hi(d[i]));
            }
        }
        // 16 rows, row tile i of the sequence: loaded, and made into operands
        const int tiles = (q.n_new * a.group + 15) / 16;
        Query<D, 16, T> raw;
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
        auto put = [&](int i, typename M::Buffer &o) {
            if (i >= tiles) return;
            const KvAttend &a = arguments().a;
            const RowTile t = tile_of<16>(a, q, i);
            float qs, qsum;
            raw.make(qs, qsum, a.scale, [&](int j, h8 y) { o.q[wave][j][lane] = y; });
            const bool counts = m < t.rows && fabsf(log_sum) < __builtin_inff();
            const float2 lse = log2_of(log_sum);
            const Span seen = span_of(a, t, m);
            if (quarter == 0) {
                o.row[wave * 16 + m] = make_float4(qs, qsum, lse.x, counts ? __builtin_amdgcn_exp2f(-lse.y) : 0.0f);
                o.seen[wave * 16 + m] = make_int2(seen.lo, seen.hi);
            }
        };
        float total[M::SUBS];
#pragma unroll
        for (int u = 0; u < M::SUBS; u++) total[u] = 0.0f;
        // (rows before the first that sees the block's first token see none of it)
        int i0 = 0;
        if (a.causal) {
            const int64_t before = (int64_t)base - (q.len - q.n_new);
            if (before > 0) i0 = (int)min(before * a.group / 16, (int64_t)tiles) / M::WAVES * M::WAVES;
        }
        int turn = 0;
        load(i0 + wave);
        put(i0 + wave, buf[0]);
        load(i0 + M::WAVES + wave);
        for (int i = i0; i < tiles; i += M::WAVES, turn ^= 1) {
            __syncthreads();
            put(i + M::WAVES + wave, buf[turn ^ 1]);
            load(i + 2 * M::WAVES + wave);
            const typename M::Buffer &o = buf[turn];
            for (int n = 0; n < M::WAVES && i + n < tiles; n++) {
                const float4 row = o.row[n * 16 + m];
                const int2 seen = o.seen[n * 16 + m];
                const bool some = seen.x < t0 + M::TB && seen.y > t0;
                if (!__any(some)) continue;
                const bool every = __all(seen.x <= t0 && seen.y >= t0 + M::TB);
                h8 y[PER];
#pragma unroll
                for (int j = 0; j < PER; j++) y[j] = o.q[n][j][lane];
                const unsigned first = t0 + 4 * quarter - seen.x, many = seen.y - seen.x;
#pragma unroll
                for (int u = 0; u < M::SUBS; u++) {
                    f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < PER; j++) acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[u][j], y[j], acc, 0, 0, 0);
                    float sum = 0.0f;
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        const float s = fmaf(acc[x], dk[u][x], ck[u][x] * row.y);
                        const float p = __builtin_amdgcn_exp2f(fmaf(s, row.x, -row.z));
                        sum += every || first + 16 * u + x < many ? p : 0.0f;
                    }
                    total[u] += row.w != 0.0f ? sum * row.w : 0.0f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < M::SUBS; u++) {
            const float x = all_lanes(total[u]);
            if (lane == 0) sums[wave * M::SUBS + u] = x;
        }
        __syncthreads();
        const int page = threadIdx.x, j = (base >> shift) + page;
        if (page < M::TOKENS >> shift && j < n_pages) {
            const KvWeigh &b = arguments();
            const KvGeom &g = b.a.g;
            const int64_t own = ((int64_t)q.seq * g.kv_heads + head) * b.stride;
            float x = 0.0f;
            if (kv_page(g, q.seq, j << g.page_shift) >= 0) {
                for (int n = 0; n < P / 16; n++) x += sums[page * (P / 16) + n];
                if (b.before) x = fmaf(b.decay, b.before[own + j], x);
            }
            b.weights[own + j] = x;
        }
        __syncthreads();                                     // (the next block's rows and sums)
    }
}

template <int D, class T>
hipError_t launch(const KvWeigh &b, int64_t pages, hipStream_t s)
{
    const KvGeom &g = b.a.g;
    if ((int64_t)g.n_tokens * b.a.group <= 16 * (int64_t)g.n_seqs) {
        const unsigned y = std::max(4096 / g.kv_heads / NW, 1);
        hipLaunchKernelGGL((k_kv_weigh<D, T>), dim3(g.kv_heads, y), dim3(NW * 64), 0, s, b);
    } else {
        using M = Many<D>;
        const int64_t blocks = std::max<int64_t>(((pages << g.page_shift) + M::TOKENS - 1) / M::TOKENS, 1) * g.n_seqs;
        hipLaunchKernelGGL((k_kv_weigh_rows<D, T>), dim3(g.kv_heads, (unsigned)std::min<int64_t>(blocks, 4096)),
                           dim3(M::WAVES * 64), 0, s, b);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t lw_launch_kv_weigh(const KvWeigh &b, int head_dim, int dtype, int64_t pages, hipStream_t s)
{
    const bool half = dtype == LW_F16;
    if (head_dim == 64) return half ? launch<64, _Float16>(b, pages, s) : launch<64, __bf16>(b, pages, s);
    if (head_dim == 128) return half ? launch<128, _Float16>(b, pages, s) : launch<128, __bf16>(b, pages, s);
    if (head_dim == 256) return half ? launch<256, _Float16>(b, pages, s) : launch<256, __bf16>(b, pages, s);
    return hipErrorInvalidValue;
}
