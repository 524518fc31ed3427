// kv_select.hip -- the pages of a long sequence that matter: bounds of full
// pages' keys, the choice of pages for a row by its scores with them, and the
// giving up of those that gathered the least attention weight.
//
// A page's score bounds q.k over its keys: sum_d max(q_d hi_d, q_d lo_d) =
// sum_d (max(q_d, 0) hi_d + min(q_d, 0) lo_d), with q, hi and lo in 8 bits a
// product of 2 D whole numbers that the matrix cores form for 16 pages and 16
// query heads at once.  Scores are whole numbers times powers of two, so that
// neither the order of sums nor a fused product changes what is chosen.
#include <algorithm>
#include <type_traits>

#include "kv_pick.hpp"

namespace {

typedef int i4 __attribute__((ext_vector_type(4)));

constexpr int NOT_FINITE = 127;        // a page's e where a key is not finite

// The smallest e with top <= 127 * 2^e, for top > 0 and finite.
__device__ __forceinline__ int least_exponent(float top)
{
    int e;
    const float f = frexpf(top, &e);                         // in [0.5, 1)
    return e - 7 + (f > 127.0f / 128.0f);
}

// max over the 16 lanes of a row.
template <class X, class F>
__device__ __forceinline__ X over16(X x, F larger)
{
    auto with = [&](auto ctrl) {
        x = larger(x, __builtin_bit_cast(X, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl.value, 0xF, 0xF, true)));
    };
    with(std::integral_constant<int, 0xB1>{});               // lane ^ 1
    with(std::integral_constant<int, 0x4E>{});               // lane ^ 2
    with(std::integral_constant<int, 0x141>{});              // 7 - lane of eight
    with(std::integral_constant<int, 0x140>{});              // 15 - lane of sixteen
    return x;
}

// ------------------------------------------------------------------ bounds

constexpr int BOUND_WAVES = 4;

// A wavefront has one head of one page.  A lane takes every 16th token and D/4
// of the dimensions (all of a key unit's, or of two), in the units that
// kv_kword lays out: 1 KiB of the cache a load.
template <int D>
__global__ __launch_bounds__(BOUND_WAVES * 64) void k_kv_bounds(KvGeom g, uint8_t *bounds, int64_t bounds_bytes)
{
    constexpr int W = D >= 128 ? 4 : 2, U = D / 8 / W, REPS = U / 4;
    const int lane = threadIdx.x & 63, head = blockIdx.y * BOUND_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (head >= g.kv_heads) return;
    // sequence s owns numbers from floor(start[s] / P) + s on, as many as pages
    // its new tokens can fill
    auto first = [&](int row, int s) { return (min(max(row, 0), g.n_tokens) >> g.page_shift) + s; };
    const KvSeq q = kv_find(g, (int)blockIdx.x, [&](int next, int s) { return first(next, s + 1); });
    if (q.seq < 0 || q.n_new == 0) return;
    const int P = 1 << g.page_shift;
    const int local = (int)blockIdx.x - first(q.row0, q.seq);
    const int j = (max(q.len - q.n_new, 0) >> g.page_shift) + local;
    if (local < 0 || j >= q.len >> g.page_shift) return;
    const int64_t page = kv_page(g, q.seq, j << g.page_shift);
    if (page < 0) return;
    const uint8_t *block = g.pages + page * g.page_bytes + (int64_t)head * g.block_bytes;
    const uint32_t *pairs = reinterpret_cast<const uint32_t *>(block + P * D);
    float hi[REPS][W][8], lo[REPS][W][8];
#pragma unroll
    for (int r = 0; r < REPS; r++)
#pragma unroll
        for (int w = 0; w < W; w++)
#pragma unroll
            for (int i = 0; i < 8; i++) hi[r][w][i] = -__builtin_inff(), lo[r][w][i] = __builtin_inff();
    bool odd = false;
    for (int t = lane % 16; t < P; t += 16) {
        const uint32_t dm = pairs[t];
        const float d = half_lo(dm), m = half_hi(dm);
        odd |= !(fabsf(d) < __builtin_inff() && fabsf(m) < __builtin_inff());
#pragma unroll
        for (int r = 0; r < REPS; r++) {
            uint32_t word[W];
            const uint32_t *from = reinterpret_cast<const uint32_t *>(block) + kv_kword<D>(t, (lane / 16 + 4 * r) * W);
            if constexpr (W == 4)
                *reinterpret_cast<uint4 *>(word) = *reinterpret_cast<const uint4 *>(from);
            else
                *reinterpret_cast<uint2 *>(word) = *reinterpret_cast<const uint2 *>(from);
#pragma unroll
            for (int w = 0; w < W; w++)
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float v = fmaf((float)(word[w] >> 4 * i & 15u), d, -m);       // d q is exact
                    hi[r][w][i] = fmaxf(hi[r][w][i], v);
                    lo[r][w][i] = fminf(lo[r][w][i], v);
                }
        }
    }
    float top = 0.0f;
#pragma unroll
    for (int r = 0; r < REPS; r++)
#pragma unroll
        for (int w = 0; w < W; w++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                auto larger = [](float a, float b) { return fmaxf(a, b); };
                hi[r][w][i] = over16(hi[r][w][i], larger);
                lo[r][w][i] = -over16(-lo[r][w][i], larger);
                top = fmaxf(top, fmaxf(fabsf(hi[r][w][i]), fabsf(lo[r][w][i])));
            }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    odd = __any(odd);
    const int e = odd || top == 0.0f ? 0 : least_exponent(top);
    uint8_t *to = bounds + page * bounds_bytes;
    if (lane == 0) *reinterpret_cast<int32_t *>(to + g.kv_heads * (2 * D) + head * 4) = odd ? NOT_FINITE : e;
    if (lane % 16) return;
    to += head * (2 * D);
#pragma unroll
    for (int r = 0; r < REPS; r++)
#pragma unroll
        for (int side = 0; side < 2; side++) {
            uint32_t code[2 * W];
#pragma unroll
            for (int i = 0; i < 8 * W; i++) {
                const float x = ldexpf(side ? lo[r][i / 8][i % 8] : hi[r][i / 8][i % 8], -e);
                const int c = odd ? 0 : (int)(side ? floorf(x) : ceilf(x));
                code[i / 4] = (i % 4 ? code[i / 4] : 0) | (uint32_t)(c & 255) << i % 4 * 8;
            }
#pragma unroll
            for (int i = 0; i < 2 * W; i += 4)
                *reinterpret_cast<uint4 *>(to + side * D + (lane / 16 + 4 * r) * (W * 8) + 4 * i) =
                    make_uint4(code[i], code[i + 1], code[i + 2], code[i + 3]);
        }
}

// ------------------------------------------------------------------ selection

// The query heads of a kv head as operands: 16 of them in the columns, D/64
// groups of 64 dimensions; a lane has 16 dimensions of its column's head.
template <int D, class T>
struct Heads {
    static constexpr int C = D / 64;
    i4 pos[C], neg[C];           // max(x, 0) and min(x, 0) of the whole numbers
    int e;                       // and their power of two; NO_HEAD where they are zeros
    static constexpr int NO_HEAD = -1000;

    __device__ __forceinline__ void load(const KvSelect &a, int64_t row, int64_t kv, int h0, int lane)
    {
        const int h = min(h0 + lane % 16, a.group - 1);
        const T *p = static_cast<const T *>(a.q.data) + row * a.q.token + (kv * a.group + h) * a.q.head + lane / 16 * 16;
        T x[C][16];
#pragma unroll
        for (int c = 0; c < C; c++) {
            if (a.q.wide) {
                reinterpret_cast<uint4 *>(x[c])[0] = reinterpret_cast<const uint4 *>(p + c * 64)[0];
                reinterpret_cast<uint4 *>(x[c])[1] = reinterpret_cast<const uint4 *>(p + c * 64)[1];
            } else {
#pragma unroll
                for (int i = 0; i < 16; i++) x[c][i] = p[c * 64 + i];
            }
        }
        // (as bits, which for numbers above 0 are in order, with infinities and NaN
        // at the end)
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 16; i++) most = max(most, __builtin_bit_cast(uint32_t, fabsf((float)x[c][i])));
        most = max(most, (uint32_t)__shfl_xor((int)most, 16));
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        const bool none = most - 1 >= 0x7F7FFFFFu;
        const int k = none ? 0 : least_exponent(__builtin_bit_cast(float, most));
        e = none ? NO_HEAD : k;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int w = 0; w < 4; w++) {
                uint32_t up = 0, down = 0;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int v = none ? 0 : (int)rintf(ldexpf((float)x[c][4 * w + i], -k));
                    up |= (uint32_t)(max(v, 0) & 255) << 8 * i;
                    down |= (uint32_t)(min(v, 0) & 255) << 8 * i;
                }
                pos[c][w] = (int)up;
                neg[c][w] = (int)down;
            }
    }
};

// What a workgroup knows of its row.
struct Wanted {
    KvSeq q;
    int own;                     // the number of the row's page
    int n;                       // pages before it that the table has
    int tok;                     // the row's place in its page
    const int32_t *pages;        // the sequence's entries
};

__device__ __forceinline__ Wanted wanted(const KvSelect &a, int row)
{
    Wanted w = {};
    w.q = kv_find(a.g, row, [](int next, int) { return next; });
    if (w.q.seq >= 0 && (row < w.q.row0 || row >= w.q.row0 + w.q.n_new)) w.q.seq = -1;
    if (w.q.seq < 0) return w;
    const int pos = w.q.len - (w.q.row0 + w.q.n_new - row);
    w.own = pos < 0 ? -1 : pos >> a.g.page_shift;
    w.n = (int)min((int64_t)max(w.own, 0), a.g.stride);
    w.tok = pos & ((1 << a.g.page_shift) - 1);
    w.pages = a.g.table + (int64_t)w.q.seq * a.g.stride;
    return w;
}

// put(page, key, more) for the pages of tiles tile0, tile0 + hop, ... (of 16
// pages each) before `tiles`: a key's order is the pages', 0 means not to be
// had.  Groups of more than 16 query heads come 16 at a time, and of what they
// give the largest counts (more: not the first).
template <int D, class T, class F>
__device__ __forceinline__ void score_tiles(const KvSelect &a, const Wanted &w, int row, int kv, int tile0, int hop, int tiles,
                                            F put)
{
    constexpr int C = D / 64;
    const int lane = threadIdx.x & 63, col = lane % 16, quarter = lane / 16;
    const uint8_t *mine = a.bounds + kv * (2 * D) + quarter * 16;
    const uint8_t *power = a.bounds + a.g.kv_heads * (2 * D) + kv * 4;
    const int parts = (a.group + 15) / 16;
    int top = Heads<D, T>::NO_HEAD;
    for (int part = parts > 1 ? -parts : 0; part < parts; part++) {
        const int h0 = 16 * (part < 0 ? part + parts : part);
        Heads<D, T> q;
        q.load(a, row, kv, h0, lane);
        if (part < 0 || parts == 1) top = max(top, over16(q.e, [](int x, int y) { return max(x, y); }));
        if (part < 0) continue;                              // (first the largest power of all heads)
        const int by = q.e == Heads<D, T>::NO_HEAD ? 0 : max(q.e - top, -64);
        for (int tile = tile0; tile < tiles; tile += hop) {
            // the lane's page as an operand's row, and the one whose score it puts
            const int j = tile * 16 + col, k = tile * 16 + 4 * quarter + col % 4;
            const int32_t entry = j < w.n ? w.pages[j] : -1, other = k < w.n ? w.pages[k] : -1;
            const bool here = (uint32_t)entry < a.g.n_pages;
            const uint8_t *from = mine + (int64_t)(here ? entry : 0) * a.bounds_bytes;
            i4 hi[C], lo[C];
#pragma unroll
            for (int c = 0; c < C; c++) {
                hi[c] = lo[c] = i4{0, 0, 0, 0};
                if (here) {
                    hi[c] = *reinterpret_cast<const i4 *>(from + c * 64);
                    lo[c] = *reinterpret_cast<const i4 *>(from + D + c * 64);
                }
            }
            const bool there = (uint32_t)other < a.g.n_pages;
            const int e = there ? *reinterpret_cast<const int32_t *>(power + (int64_t)other * a.bounds_bytes) : 0;
            i4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < C; c++) {
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(hi[c], q.pos[c], acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(lo[c], q.neg[c], acc, 0, 0, 0);
            }
            float x = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float y = h0 + col < a.group ? ldexpf((float)acc[i], by) : -__builtin_inff();
                const float most = over16(y, [](float p, float r) { return fmaxf(p, r); });
                x = col == i ? most : x;
            }
            if (col < 4 && k < w.n) {
                const uint32_t key = ordered(e == NOT_FINITE ? __builtin_inff() : ldexpf(x, e));
                const bool must = k < a.first || k >= w.own - a.last;
                put(k, !there ? 0u : must ? ~0u : key, part > 0);
            }
        }
    }
}

// Keys into the workspace: where few rows have many pages, many workgroups share
// a row's.
template <int D, class T>
__global__ __launch_bounds__(256) void k_kv_score(KvSelect a)
{
    const int kv = blockIdx.y, row = blockIdx.z;
    const Wanted w = wanted(a, row);
    if (w.q.seq < 0) return;
    const int tiles = (w.n + 15) / 16;
    uint32_t *to = a.work + ((int64_t)row * a.g.kv_heads + kv) * a.g.stride;
    const int tile0 = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (tile0 >= tiles) return;
    score_tiles<D, T>(a, w, row, kv, tile0, gridDim.x * 4, tiles, [&](int k, uint32_t x, bool more) { to[k] = more ? max(to[k], x) : x; });
}

// The pages of a row and kv head.  THREADS a workgroup; the keys come from the
// workspace where there is one.
template <int D, class T, int THREADS>
__global__ __launch_bounds__(THREADS) void k_kv_select(KvSelect a)
{
    extern __shared__ __align__(16) uint32_t mem[];
    uint32_t *hist = mem, *sums = mem + 512, *key = mem + 512 + THREADS / 64;
    const int kv = blockIdx.x, row = blockIdx.y + blockIdx.z * gridDim.y;
    if (row >= a.g.n_tokens) return;
    const Wanted w = wanted(a, row);
    int32_t *to = a.table + ((int64_t)row * a.g.kv_heads + kv) * a.take;
    if (kv == 0 && threadIdx.x == 0) {
        const int b0 = a.g.n_seqs ? min(max(a.g.start[0], 0), a.g.n_tokens) : 0;
        const int b1 = a.g.n_seqs ? min(max(a.g.start[a.g.n_seqs], b0), a.g.n_tokens) : 0;
        a.start[row] = min(max(row, b0), b1);
        if (row + 1 == a.g.n_tokens) a.start[row + 1] = b1;
    }
    int n = w.q.seq < 0 ? 0 : w.n, got = 0;
    if (n > 0 && a.take > 1) {
        if (a.work) {
            const uint32_t *from = a.work + ((int64_t)row * a.g.kv_heads + kv) * a.g.stride;
            for (int j = threadIdx.x; j < n; j += THREADS) key[j] = from[j];
        } else if (n < a.take) {                             // all of them that are present
            for (int j = threadIdx.x; j < n; j += THREADS) key[j] = (uint32_t)w.pages[j] < a.g.n_pages;
        } else {
            score_tiles<D, T>(a, w, row, kv, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), THREADS / 64, (n + 15) / 16,
                              [&](int k, uint32_t x, bool more) { key[k] = more ? max(key[k], x) : x; });
        }
        __syncthreads();
        int have = 0;
        for (int j0 = 0; j0 < n; j0 += THREADS) {
            const int j = j0 + threadIdx.x;
            have += __syncthreads_count(j < n && key[j] != 0);
        }
        Cut c = {~0u, 0u, 0};                                // those that are there
        if (have >= a.take) c = pick_cut<THREADS>(key, n, a.take - 1, hist);
        got = pick_each<THREADS>(key, n, c, sums, [&](int j, int rank) { to[rank] = w.pages[j]; });
    }
    const bool none = w.q.seq < 0 || w.own < 0;
    for (int i = got + threadIdx.x; i < a.take; i += THREADS)
        to[i] = i == got && !none && w.own < a.g.stride ? w.pages[w.own] : -1;
    if (kv == 0 && threadIdx.x == 0) a.lens[row] = none ? 0 : (got << a.g.page_shift) + w.tok + 1;
}

// ------------------------------------------------------------------ giving up

template <int THREADS>
__global__ __launch_bounds__(THREADS) void k_kv_evict(KvEvict a)
{
    extern __shared__ __align__(16) uint32_t mem[];
    uint32_t *hist = mem, *sums = mem + 512, *key = mem + 512 + THREADS / 64;
    const int64_t s = blockIdx.x;
    const int stride = (int)a.g.stride;
    const int32_t *from = a.g.table + s * stride;
    int32_t *to = a.table + s * stride, *gone = a.gone + s * stride;
    const int len = max(a.g.lens[s], 0);
    const int used = (int)(((int64_t)len + (1 << a.g.page_shift) - 1) >> a.g.page_shift), n = min(used, stride);
    const float *w = a.weights + s * a.g.kv_heads * a.stride;
    int here = 0, may = 0;
    for (int j0 = 0; j0 < stride; j0 += THREADS) {
        const int j = j0 + threadIdx.x;
        const int32_t entry = j < stride ? from[j] : -1;
        const bool present = j < n && (uint32_t)entry < a.g.n_pages;
        const bool spare = present && j >= a.first && j < used - a.last;
        uint32_t k = 0;
        if (spare) {
            double sum = 0.0;
            if (j < a.stride)
                for (int h = 0; h < a.g.kv_heads; h++) sum += (double)w[h * a.stride + j];
            const float x = (float)sum + 0.0f;               // (-0 counts as 0)
            // the lowest weight has the largest key; at least 1
            k = j < a.stride && x == x ? ~ordered(x) : 1u;
        }
        if (j < n) key[j] = k;
        if (j < stride) to[j] = entry;
        here += __syncthreads_count(present);
        may += __syncthreads_count(spare);
    }
    const int drop = (int)min((int64_t)may, max((int64_t)here - a.keep, (int64_t)0));
    int got = 0;
    if (drop) {
        Cut c = {~0u, 0u, 0};
        if (drop < may) c = pick_cut<THREADS>(key, n, drop, hist);
        got = pick_each<THREADS>(key, n, c, sums, [&](int j, int rank) {
            gone[rank] = from[j];
            to[j] = -1;
        });
    }
    for (int i = got + threadIdx.x; i < stride; i += THREADS) gone[i] = -1;
    if (threadIdx.x == 0) a.count[s] = got;
}

template <class F>
hipError_t with_types(int head_dim, int dtype, F f)
{
    auto typed = [&](auto dim) { return dtype == LW_F16 ? f(dim, _Float16{}) : f(dim, __bf16{}); };
    if (head_dim == 64) return typed(std::integral_constant<int, 64>{});
    if (head_dim == 128) return typed(std::integral_constant<int, 128>{});
    if (head_dim == 256) return typed(std::integral_constant<int, 256>{});
    return hipErrorInvalidValue;
}

// LDS of a workgroup that picks from n keys.
size_t pick_bytes(int64_t n, int threads) { return (512 + threads / 64 + std::max<int64_t>(n, 1)) * sizeof(uint32_t); }

// A kernel's LDS beyond 64 KiB has to be asked for.
hipError_t allow(const void *f, size_t bytes)
{
    if (bytes <= 64 << 10) return hipSuccess;
    return hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

static_assert(KV_PICK_MOST == PICK_MOST, "");

hipError_t lw_launch_kv_bounds(const KvGeom &g, int head_dim, uint8_t *bounds, int64_t bounds_bytes, hipStream_t s)
{
    const int64_t x = (g.n_tokens >> g.page_shift) + (int64_t)g.n_seqs;
    const dim3 grid((unsigned)x, (unsigned)((g.kv_heads + BOUND_WAVES - 1) / BOUND_WAVES)), block(BOUND_WAVES * 64);
    if (head_dim == 64) hipLaunchKernelGGL((k_kv_bounds<64>), grid, block, 0, s, g, bounds, bounds_bytes);
    else if (head_dim == 128) hipLaunchKernelGGL((k_kv_bounds<128>), grid, block, 0, s, g, bounds, bounds_bytes);
    else if (head_dim == 256) hipLaunchKernelGGL((k_kv_bounds<256>), grid, block, 0, s, g, bounds, bounds_bytes);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

bool lw_kv_select_shared(int kv_heads, int64_t n_tokens, int64_t pages)
{
    return kv_heads * n_tokens <= 128 && pages >= 512;
}

hipError_t lw_launch_kv_select(const KvSelect &a, int head_dim, int dtype, int64_t pages, hipStream_t s)
{
    return with_types(head_dim, dtype, [&](auto dim, auto type) {
        constexpr int D = dim.value;
        using T = decltype(type);
        if (a.work) {
            const unsigned x = (unsigned)std::max<int64_t>((pages + 63) / 64, 1);
            hipLaunchKernelGGL((k_kv_score<D, T>), dim3(x, a.g.kv_heads, a.g.n_tokens), dim3(256), 0, s, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        const unsigned y = (unsigned)std::min(a.g.n_tokens, 1 << 15), z = (a.g.n_tokens + y - 1) / y;
        const dim3 grid(a.g.kv_heads, y, z);
        auto go = [&](auto f, int threads) {
            const size_t bytes = pick_bytes(a.g.stride, threads);
            const hipError_t e = allow(reinterpret_cast<const void *>(f), bytes);
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL(f, grid, dim3(threads), bytes, s, a);
            return hipGetLastError();
        };
        return pages > 1024 ? go(k_kv_select<D, T, 1024>, 1024) : go(k_kv_select<D, T, 256>, 256);
    });
}

hipError_t lw_launch_kv_evict(const KvEvict &a, hipStream_t s)
{
    auto go = [&](auto f, int threads) {
        const size_t bytes = pick_bytes(a.g.stride, threads);
        const hipError_t e = allow(reinterpret_cast<const void *>(f), bytes);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(f, dim3(a.g.n_seqs), dim3(threads), bytes, s, a);
        return hipGetLastError();
    };
    return a.g.stride > 1024 ? go(k_kv_evict<1024>, 1024) : go(k_kv_evict<256>, 256);
}
