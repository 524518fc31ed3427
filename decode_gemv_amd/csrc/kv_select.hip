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

// A step of a maximum over lanes that leaves each of two partners half of the
// numbers: of x[0 .. 2 N) those of its half (upper: the second) in x[0 .. N).
template <int CTRL, int N>
__device__ __forceinline__ void halve(float *x, bool upper)
{
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float keep = upper ? x[N + i] : x[i], give = upper ? x[i] : x[N + i];
        x[i] = fmaxf(keep, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, give), CTRL, 0xF, 0xF, true)));
    }
}

// A workgroup has one head of one page, its wavefronts take 16 tokens in turn.  A
// lane takes one of them and D/4 of the dimensions (all of a key unit's, or of
// two), in the units that kv_kword lays out: 1 KiB of the cache a load.  At the
// end the 16 lanes of a unit share its channels out, and the wavefronts meet.
// A page takes 4.2 us (kernel trace), most of it the latencies of the row's place,
// the table's entry and the keys (8.5 with one wavefront, and every lane all
// channels); where no page is full, as for most tokens, workgroups end after the
// first, 2.0 to 2.3.  Many pages at once are bound by those chains, too: 5 prompts
// of 8192 tokens (640 pages of 64, 8 heads of 128, 24 MB) 24 us, 16 of them 70,
// 1.1 TB/s (replays of a graph).
template <int D>
__global__ __launch_bounds__(BOUND_WAVES * 64) void k_kv_bounds(KvGeom g, uint8_t *bounds, int64_t bounds_bytes)
{
    constexpr int W = D >= 128 ? 4 : 2, U = D / 8 / W, REPS = U / 4, N = W * 8;
    constexpr int OWN = N / 16;                              // channels of a lane at the end, of each unit
    __shared__ float meet[BOUND_WAVES][REPS][2 * OWN][64];
    __shared__ int odds[BOUND_WAVES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), head = blockIdx.y;
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
    float x[REPS][2][N];                                     // largest, and largest of the negatives
#pragma unroll
    for (int r = 0; r < REPS; r++)
#pragma unroll
        for (int i = 0; i < N; i++) x[r][0][i] = x[r][1][i] = -__builtin_inff();
    bool odd = false;
    for (int t = wave * 16 + lane % 16; t < P; t += BOUND_WAVES * 16) {
        const uint32_t dm = pairs[t];
        uint32_t word[REPS][W];
#pragma unroll
        for (int r = 0; r < REPS; r++) {
            const uint32_t *from = reinterpret_cast<const uint32_t *>(block) + kv_kword<D>(t, (lane / 16 + 4 * r) * W);
            if constexpr (W == 4)
                *reinterpret_cast<uint4 *>(word[r]) = *reinterpret_cast<const uint4 *>(from);
            else
                *reinterpret_cast<uint2 *>(word[r]) = *reinterpret_cast<const uint2 *>(from);
        }
        const float d = half_lo(dm), m = half_hi(dm);
        odd |= !(fabsf(d) < __builtin_inff() && fabsf(m) < __builtin_inff());
#pragma unroll
        for (int r = 0; r < REPS; r++)
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float v = fmaf((float)(word[r][i / 8] >> 4 * (i % 8) & 15u), d, -m);       // d q is exact
                x[r][0][i] = fmaxf(x[r][0][i], v);
                x[r][1][i] = fmaxf(x[r][1][i], -v);
            }
    }
    odd = __any(odd);
    // 7 - lane of eight and 15 - lane of sixteen first: what lane ^ 1 and lane ^ 2
    // share out is then the same for all that have it
    const bool b8 = lane & 8, b4 = lane & 4, b2 = lane & 2, b1 = lane & 1;
#pragma unroll
    for (int r = 0; r < REPS; r++)
#pragma unroll
        for (int side = 0; side < 2; side++) {
            halve<0x140, N / 2>(x[r][side], b8);
            halve<0x141, N / 4>(x[r][side], b4);
            halve<0x4E, N / 8>(x[r][side], b2);
            halve<0xB1, N / 16>(x[r][side], b1);
#pragma unroll
            for (int i = 0; i < OWN; i++) meet[wave][r][side * OWN + i][lane] = x[r][side][i];
        }
    if (lane == 0) odds[wave] = odd;
    __syncthreads();
    if (wave) return;
    float top = 0.0f;
#pragma unroll
    for (int w = 0; w < BOUND_WAVES; w++) odd |= odds[w] != 0;
#pragma unroll
    for (int r = 0; r < REPS; r++)
#pragma unroll
        for (int i = 0; i < 2 * OWN; i++) {
            float &y = x[r][i / OWN][i % OWN];
#pragma unroll
            for (int w = 1; w < BOUND_WAVES; w++) y = fmaxf(y, meet[w][r][i][lane]);
            top = fmaxf(top, fabsf(y));
        }
    top = over16(top, [](float a, float b) { return fmaxf(a, b); });
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const int e = odd || top == 0.0f ? 0 : least_exponent(top);
    uint8_t *to = bounds + page * bounds_bytes;
    if (lane == 0) *reinterpret_cast<int32_t *>(to + g.kv_heads * (2 * D) + head * 4) = odd ? NOT_FINITE : e;
    to += head * (2 * D);
    // the lane's channels of a unit: from OWN * (its number of sixteen, the first
    // bit the highest) on
    const int c = (b8 ? N / 2 : 0) + (b4 ? N / 4 : 0) + (b2 ? N / 8 : 0) + (b1 ? N / 16 : 0);
#pragma unroll
    for (int r = 0; r < REPS; r++)
#pragma unroll
        for (int side = 0; side < 2; side++)
#pragma unroll
            for (int i = 0; i < OWN; i++) {
                const float y = side ? -x[r][1][i] : x[r][0][i], z = ldexpf(y, -e);
                const int code = odd ? 0 : (int)(side ? floorf(z) : ceilf(z));
                to[side * D + (lane / 16 + 4 * r) * N + c + i] = (uint8_t)code;
            }
}

// ------------------------------------------------------------------ selection

// The query heads of a kv head as operands: 16 of them in the columns, D/64
// groups of 64 dimensions; a lane has 16 dimensions of its column's head.
template <int D, class T>
struct Raw {
    static constexpr int C = D / 64;
    T x[C][16];

    __device__ __forceinline__ void load(const KvSelect &a, int64_t row, int64_t kv, int h0, int lane)
    {
        const int h = min(h0 + lane % 16, a.group - 1);
        const T *p = static_cast<const T *>(a.q.data) + row * a.q.token + (kv * a.group + h) * a.q.head + lane / 16 * 16;
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
    }
};

template <int D>
struct Heads {
    static constexpr int C = D / 64, NO_HEAD = -1000;
    i4 pos[C], neg[C];           // max(x, 0) and min(x, 0) of the whole numbers
    int e;                       // and their power of two; NO_HEAD where they are zeros

    // Each wavefront makes one group of 64 dimensions for all, as far as there are
    // groups.  Every wavefront of the workgroup comes here; mem is free again after
    // the next barrier.
    template <class T>
    __device__ __forceinline__ Heads(const Raw<D, T> &r, i4 (*mem)[2][64], int wave, int lane)
    {
        // (as bits, which for numbers above 0 are in order, with infinities and NaN
        // at the end)
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 16; i++) most = max(most, __builtin_bit_cast(uint32_t, fabsf((float)r.x[c][i])));
        most = max(most, (uint32_t)__shfl_xor((int)most, 16));
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        const bool none = most - 1 >= 0x7F7FFFFFu;
        const int k = none ? 0 : least_exponent(__builtin_bit_cast(float, most));
        e = none ? NO_HEAD : k;
#pragma unroll
        for (int c = 0; c < C; c++) {
            if (wave != c) continue;
            i4 up, down;
#pragma unroll
            for (int w = 0; w < 4; w++) {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; i++)                  // rounded to a whole number by the sum's last place: its low byte
                    v[i] = __builtin_bit_cast(uint32_t, ldexpf((float)r.x[c][4 * w + i], -k) + 0x1.8p23f);
                uint32_t all = __builtin_amdgcn_perm(__builtin_amdgcn_perm(v[3], v[2], 0x0C0C0400u),
                                                     __builtin_amdgcn_perm(v[1], v[0], 0x0C0C0400u), 0x05040100u);
                if (none) all = 0;
                const uint32_t below = (all >> 7 & 0x01010101u) * 255u;      // the bytes of negative ones
                up[w] = (int)(all & ~below);
                down[w] = (int)(all & below);
            }
            mem[c][0][lane] = up;
            mem[c][1][lane] = down;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; c++) {
            pos[c] = mem[c][0][lane];
            neg[c] = mem[c][1][lane];
        }
    }
};

// Tiles whose loads are under way at once (registers).
template <int D> constexpr int TILES = D == 256 ? 2 : 4;

// What a workgroup knows of its row.
struct Wanted {
    KvSeq q;
    int own;                     // the number of the row's page
    int n;                       // pages before it that the table has (0: where the cache has none)
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
    w.n = a.g.n_pages ? (int)min((int64_t)max(w.own, 0), a.g.stride) : 0;
    w.tok = pos & ((1 << a.g.page_shift) - 1);
    w.pages = a.g.table + (int64_t)w.q.seq * a.g.stride;
    return w;
}

// put(page, key, part) for the pages of tiles tile0, tile0 + hop, ... (of 16
// pages each) before `tiles`: a key's order is the pages', 0 means not to be
// had.  Groups of more than 16 query heads come 16 at a time, and of what they
// give the largest counts (part of `parts`).  raw: the first 16 heads'.
// N tiles' loads are under way at once, and the entries of the N after them:
// their latency is what this takes.  Every wavefront of the workgroup comes here.
template <int D, class T, int N, class F>
__device__ __forceinline__ void score_tiles(const KvSelect &a, const Wanted &w, int row, int kv, Raw<D, T> raw,
                                            i4 (*mem)[2][64], int tile0, int hop, int tiles, F put)
{
    constexpr int C = D / 64;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane % 16, quarter = lane / 16;
    const uint8_t *mine = a.bounds + kv * (2 * D) + quarter * 16;
    const uint8_t *power = a.bounds + a.g.kv_heads * (2 * D) + kv * 4;
    const int parts = (a.group + 15) / 16;
    // the lane's page as an operand's row, and the one whose score it puts
    int32_t entry[N], other[N];
    auto look = [&](int first) {
#pragma unroll
        for (int n = 0; n < N; n++) {
            const int j = (first + n * hop) * 16 + col, k = j - col + 4 * quarter + col % 4;
            entry[n] = j < w.n ? w.pages[j] : -1;
            other[n] = k < w.n ? w.pages[k] : -1;
        }
    };
    look(tile0);
    int top = Heads<D>::NO_HEAD;
    for (int part = parts > 1 ? -parts : 0; part < parts; part++) {
        const int h0 = 16 * (part < 0 ? part + parts : part);
        if (parts > 1) {
            raw.load(a, row, kv, h0, lane);
            __syncthreads();                                 // (the part before has been read)
        }
        const Heads<D> q(raw, mem, wave, lane);
        if (part < 0 || parts == 1) top = max(top, over16(q.e, [](int x, int y) { return max(x, y); }));
        if (part < 0) continue;                              // (first the largest power of all heads)
        const int by = q.e == Heads<D>::NO_HEAD ? 0 : max(q.e - top, -64);
        for (int first = tile0; first < tiles; first += N * hop) {
            i4 hi[N][C], lo[N][C];
            int e[N];
            bool there[N];
#pragma unroll
            for (int n = 0; n < N; n++) {
                there[n] = (uint32_t)other[n] < a.g.n_pages;
                if (n && first + n * hop >= tiles) continue;
                const uint8_t *from = mine + (int64_t)((uint32_t)entry[n] < a.g.n_pages ? entry[n] : 0) * a.bounds_bytes;
#pragma unroll
                for (int c = 0; c < C; c++) {
                    hi[n][c] = *reinterpret_cast<const i4 *>(from + c * 64);
                    lo[n][c] = *reinterpret_cast<const i4 *>(from + D + c * 64);
                }
                e[n] = *reinterpret_cast<const int32_t *>(power + (int64_t)(there[n] ? other[n] : 0) * a.bounds_bytes);
            }
            look(first + N * hop < tiles ? first + N * hop : tile0);
#pragma unroll
            for (int n = 0; n < N; n++) {
                if (n && first + n * hop >= tiles) continue;
                i4 acc = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < C; c++) {
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(hi[n][c], q.pos[c], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(lo[n][c], q.neg[c], acc, 0, 0, 0);
                }
                float x = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float y = h0 + col < a.group ? ldexpf((float)acc[i], by) : -__builtin_inff();
                    const float most = over16(y, [](float p, float r) { return fmaxf(p, r); });
                    x = col == i ? most : x;
                }
                const int k = (first + n * hop) * 16 + 4 * quarter + col;
                if (col < 4 && k < w.n) {
                    const uint32_t key = ordered(e[n] == NOT_FINITE ? __builtin_inff() : ldexpf(x, e[n]));
                    const bool must = k < a.first || k >= w.own - a.last;
                    put(k, !there[n] ? 0u : must ? MUST : key, part);
                }
            }
        }
    }
}

// Keys into the workspace: where few rows have many pages, many workgroups share
// a row's.  For 16 rows of 8 to 512 pages and 8 heads of 128 (7 MB of bounds) it
// takes 6.6 us (kernel trace), for one row of 4096 (8.5 MB) 5.9, 1.4 TB/s: with one
// tile or two a wavefront the chain of loads is what counts, from the row's place
// over the entries to the bounds.
template <int D, class T>
__global__ __launch_bounds__(256) void k_kv_score(KvSelect a)
{
    __shared__ i4 mem[D / 64][2][64];
    const int kv = blockIdx.y, row = blockIdx.z;
    Raw<D, T> raw;
    raw.load(a, row, kv, 0, threadIdx.x & 63);
    const Wanted w = wanted(a, row);
    const int tiles = w.q.seq < 0 ? 0 : (w.n + 15) / 16;
    if ((int)blockIdx.x * 4 >= tiles) return;
    uint32_t *to = a.work + ((int64_t)row * a.g.kv_heads + kv) * a.g.stride;
    score_tiles<D, T, TILES<D>>(a, w, row, kv, raw, mem, blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6),
                               gridDim.x * 4, tiles, [&](int k, uint32_t x, int part) { to[k] = part ? max(to[k], x) : x; });
}

// The pages of a row and kv head.  THREADS a workgroup; the keys come from the
// workspace where there is one.  With those it takes 6.0 us (kernel trace) for up to
// 512 pages and 9.2 for 4096: passes over the keys in LDS, for each a barrier or two
// and one wavefront's search for the counter; with the scores of 80 pages of its own
// 8.3, a third each for the row's place, the scores and the choice.
template <int D, class T, int THREADS>
__global__ __launch_bounds__(THREADS) void k_kv_select(KvSelect a)
{
    extern __shared__ __align__(16) uint32_t mem[];
    uint32_t *hist = mem, *sums = mem + PICK_WORDS, *key = mem + PICK_WORDS + 8 * (THREADS / 64);       // (all 16-byte aligned)
    const int kv = blockIdx.x, row = blockIdx.y + blockIdx.z * gridDim.y;
    if (row >= a.g.n_tokens) return;
    Raw<D, T> raw;
    if (!a.work) raw.load(a, row, kv, 0, threadIdx.x & 63);
    const Wanted w = wanted(a, row);
    const bool none = w.q.seq < 0 || w.own < 0;
    const int32_t last = !none && w.own < a.g.stride ? w.pages[w.own] : -1;
    int32_t *to = a.table + ((int64_t)row * a.g.kv_heads + kv) * a.take;
    if (kv == 0 && threadIdx.x == 0) {
        const int b0 = a.g.n_seqs ? min(max(a.g.start[0], 0), a.g.n_tokens) : 0;
        const int b1 = a.g.n_seqs ? min(max(a.g.start[a.g.n_seqs], b0), a.g.n_tokens) : 0;
        a.start[row] = min(max(row, b0), b1);
        if (row + 1 == a.g.n_tokens) a.start[row + 1] = b1;
    }
    const int n = w.q.seq < 0 ? 0 : w.n;
    int got = 0;
    if (n > 0 && a.take > 1) {
        Tally tally;
        if (n < a.take) {                                    // all of them that are present
            for (int j = threadIdx.x; j < n; j += THREADS) {
                key[j] = (uint32_t)w.pages[j] < a.g.n_pages;
                tally.add(key[j]);
            }
        } else if (a.work) {
            const uint32_t *from = a.work + ((int64_t)row * a.g.kv_heads + kv) * a.g.stride;
            for (int j0 = threadIdx.x; j0 < n; j0 += 8 * THREADS) {
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 8; i++) x[i] = from[min(j0 + i * THREADS, n - 1)];
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (j0 + i * THREADS < n) {
                        key[j0 + i * THREADS] = x[i];
                        tally.add(x[i]);
                    }
            }
        } else {
            const int parts = (a.group + 15) / 16;
            score_tiles<D, T, TILES<D>>(a, w, row, kv, raw, reinterpret_cast<i4 (*)[2][64]>(hist),
                                        __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), THREADS / 64, (n + 15) / 16,
                                        [&](int k, uint32_t x, int part) {
                                            if (part) x = max(key[k], x);
                                            key[k] = x;
                                            if (part == parts - 1) tally.add(x);
                                        });
        }
        uint32_t nothing = 0;
        const Keys all = tally.meet<THREADS>(sums + 4 * (THREADS / 64), nothing);
        const bool every = (int)all.there < a.take;
        Cut c = {};
        if (!every) c = pick_cut<THREADS>(key, n, all, a.take - 1, hist);
        // (their places first: one load's latency then for all of them)
        uint16_t *list = reinterpret_cast<uint16_t *>(hist);
        if (a.take <= 4 * PICK_HIST) {
            got = pick_each<THREADS>(key, n, every, c, sums, [&](int j, int rank) { list[rank] = (uint16_t)j; });
            __syncthreads();
            for (int i = threadIdx.x; i < got; i += THREADS) to[i] = w.pages[list[i]];
        } else {
            got = pick_each<THREADS>(key, n, every, c, sums, [&](int j, int rank) { to[rank] = w.pages[j]; });
        }
    }
    for (int i = got + threadIdx.x; i < a.take; i += THREADS) to[i] = i == got && !none ? last : -1;
    if (kv == 0 && threadIdx.x == 0) a.lens[row] = none ? 0 : (got << a.g.page_shift) + w.tok + 1;
}

// ------------------------------------------------------------------ giving up

// A workgroup has a sequence: its heads' weights are added in fp64 (their order is
// the heads', and what is rounded once to fp32 is compared as whole numbers).  94
// pages of 8 heads take 3.8 us (kernel trace); 64 sequences of 4 to 4096 pages 11.4:
// the longest's 131 KB of weights through one CU, then the passes over its keys.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void k_kv_evict(KvEvict a)
{
    extern __shared__ __align__(16) uint32_t mem[];
    uint32_t *hist = mem, *sums = mem + PICK_WORDS, *key = mem + PICK_WORDS + 8 * (THREADS / 64);       // (all 16-byte aligned)
    const int64_t s = blockIdx.x;
    const int stride = (int)a.g.stride;
    const int32_t *from = a.g.table + s * stride;
    int32_t *to = a.table + s * stride, *gone = a.gone + s * stride;
    const int len = max(a.g.lens[s], 0);
    const int used = (int)(((int64_t)len + (1 << a.g.page_shift) - 1) >> a.g.page_shift), n = min(used, stride);
    const float *w = a.weights + s * a.g.kv_heads * a.stride;
    const int known = (int)min((int64_t)n, a.stride);
    uint32_t here = 0;
    Tally tally;
    for (int j0 = threadIdx.x; j0 < stride; j0 += 2 * THREADS) {
        // (two pages and eight heads at once: their loads' latency is what this takes)
        double sum[2] = {0.0, 0.0};
        int32_t entry[2];
#pragma unroll
        for (int i = 0; i < 2; i++) entry[i] = j0 + i * THREADS < stride ? from[j0 + i * THREADS] : -1;
        for (int h0 = 0; h0 < (known ? a.g.kv_heads : 0); h0 += 8) {
            float x[2][8];
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int h = 0; h < 8; h++)
                    x[i][h] = w[min(h0 + h, a.g.kv_heads - 1) * a.stride + min(j0 + i * THREADS, known - 1)];
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int h = 0; h < 8; h++) sum[i] += h0 + h < a.g.kv_heads ? (double)x[i][h] : 0.0;
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int j = j0 + i * THREADS;
            const bool present = j < n && (uint32_t)entry[i] < a.g.n_pages;
            const bool spare = present && j >= a.first && j < used - a.last;
            const float total = (float)sum[i] + 0.0f;        // (-0 counts as 0)
            // the lowest weight has the largest key; at least 1
            const uint32_t k = !spare ? 0u : j < known && total == total ? ~ordered(total) : 1u;
            if (j < n) {
                key[j] = k;
                tally.add(k);
            }
            if (j < stride) to[j] = entry[i];
            here += present;
        }
    }
    const Keys all = tally.meet<THREADS>(sums + 4 * (THREADS / 64), here);
    const int drop = (int)min((int64_t)all.there, max((int64_t)here - a.keep, (int64_t)0));
    int got = 0;
    if (drop) {
        const bool every = drop == (int)all.there;
        Cut c = {};
        if (!every) c = pick_cut<THREADS>(key, n, all, drop, hist);
        got = pick_each<THREADS>(key, n, every, c, sums + THREADS / 64, [&](int j, int rank) {
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

// LDS of a workgroup that picks from n keys, which are as many as the table is wide:
// what a row has is known on the device only.  A wide table of few pages costs
// places on a CU: 128 rows of 80 pages take 20.5 us up to 4096 entries, 32.5 with
// 32768; one row 8.1 either way (replays of a graph).
size_t pick_bytes(int64_t n, int threads) { return (PICK_WORDS + 8 * (threads / 64) + (n + 3) / 4 * 4) * sizeof(uint32_t); }

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
    const dim3 grid((unsigned)x, (unsigned)g.kv_heads), block(BOUND_WAVES * 64);
    if (head_dim == 64) hipLaunchKernelGGL((k_kv_bounds<64>), grid, block, 0, s, g, bounds, bounds_bytes);
    else if (head_dim == 128) hipLaunchKernelGGL((k_kv_bounds<128>), grid, block, 0, s, g, bounds, bounds_bytes);
    else if (head_dim == 256) hipLaunchKernelGGL((k_kv_bounds<256>), grid, block, 0, s, g, bounds, bounds_bytes);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

bool lw_kv_select_shared(int kv_heads, int64_t n_tokens, int64_t pages)
{
    // Bounds, choice and attention with workgroups of their own for the scores, and
    // with the choice's: 128 pairs on up to 512 pages 30.5 us and 33.2, 100 on 391 of
    // heads of 256 35.4 and 38.7, 8 on 4096 27.9 and 61.3, 8 on 80 22.0 and 21.6.
    return n_tokens > 0 && kv_heads * n_tokens <= KV_SHARED_PAIRS && pages >= 256;
}

hipError_t lw_launch_kv_select(const KvSelect &a, int head_dim, int dtype, int64_t pages, hipStream_t s)
{
    return with_types(head_dim, dtype, [&](auto dim, auto type) {
        constexpr int D = dim.value;
        using T = decltype(type);
        if (a.work) {
            // (about 2048 wavefronts, of one tile at least)
            const int64_t most = 512 / std::max<int64_t>((int64_t)a.g.kv_heads * a.g.n_tokens, 1);
            const unsigned x = (unsigned)std::max<int64_t>(std::min((pages + 63) / 64, most), 1);
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
        // (with 512 and 256, bounds and attention with them: 4096 pages 27.9 us and 30.9,
        // 80 pages 23.1 and 21.6)
        return pages > 1024 ? go(k_kv_select<D, T, 512>, 512) : go(k_kv_select<D, T, 256>, 256);
    });
}

hipError_t lw_launch_kv_evict(const KvEvict &a, hipStream_t s)
{
    auto go = [&](auto f, int threads) {
        const size_t bytes = pick_bytes(a.g.stride, threads);
        const hipError_t e = allow(reinterpret_cast<const void *>(f), bytes);
        if (e != hipSuccess) return e;
        // (as many sequences at a time as a launch has threads for; a second dimension of
        // workgroups for the others took 11.9 us and not 11.6 for the 64 tables)
        KvEvict part = a;
        for (int left = a.g.n_seqs; left > 0; left -= 1 << KV_FOLD) {
            const int n = std::min(left, 1 << KV_FOLD);
            hipLaunchKernelGGL(f, dim3(n), dim3(threads), bytes, s, part);
            const hipError_t launched = hipGetLastError();
            if (launched != hipSuccess) return launched;
            part.g.lens += n;
            part.g.table += n * a.g.stride;
            part.weights += n * a.g.kv_heads * a.stride;
            part.table += n * a.g.stride;
            part.gone += n * a.g.stride;
            part.count += n;
        }
        return hipSuccess;
    };
    // (64 tables of 4096 pages, 1024 threads, 512 and 256: 11.6 us, 13.0 and 18.9; one
    // of 94: 5.6, 5.1 and 4.5)
    return a.g.stride > 1024 ? go(k_kv_evict<1024>, 1024) : go(k_kv_evict<256>, 256);
}
