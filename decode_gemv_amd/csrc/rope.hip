// rope.hip -- rotary positions: pairs of dimensions turned by pos * f_i,
//
//   (a, b) -> (a c - b s, a s + b c),  c = g cos(pos f_i), s = g sin(pos f_i)
//
// The angle is kept as a fraction of a turn in 64 bits: pos * step_i modulo
// 2^64 is exact in whole numbers, whatever the position, and its first 32 bits
// are the angle to 2^-33 turns.  They split into a quarter and a signed rest of
// at most an eighth, on which the sine and cosine are their Taylor sums (x^9
// and x^10: 2^-29 and 2^-31 of them are left out on pi/4).
//
// A wavefront has one row and some of its heads, or a few rows where they have
// few: a row's place in the batch is looked up once, a lane's sines and cosines
// serve all the heads it goes through.  Where the layout allows it a lane has
// eight elements (of the halves layout twice eight: both sides of eight pairs),
// else one pair or element.
//
// HBM bounds large calls: 22 thousand rows of 40 heads of 128, fp32 to bf16, 683 MB
// in 130 us, 5.3 TB/s, as fast as a copy.  Small ones take 4.0 us (kernel trace),
// the latencies of the row's place and its elements.
#include <algorithm>
#include <string>

#include "kv.h"

lw_status lw_fail(lw_status s, const std::string &msg);   // bundle.cpp

namespace {

constexpr int WAVES = 4;

struct Rope {
    KvGeom g;                    // start, lens, n_seqs, n_tokens
    const int32_t *pos;          // or null
    KvTensor x, y;
    int32_t heads, per;          // and a wavefront's
    int32_t rows;                // a wavefront's (1, or as many as have their heads side by side)
    int32_t dim;
    lw_rope_plan plan;
};

template <class T, int N> struct Vec { T v[N]; };

template <int N, class T>
__device__ __forceinline__ Vec<T, N> load(const T *p)
{
    Vec<T, N> e;
    if constexpr (N == 1) {
        e.v[0] = *p;
    } else {
#pragma unroll
        for (unsigned i = 0; i < sizeof(e) / 16; i++)
            reinterpret_cast<uint4 *>(&e)[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    return e;
}

template <int N, class T>
__device__ __forceinline__ void store(T *p, const Vec<T, N> &e)
{
    if constexpr (N == 1) {
        *p = e.v[0];
    } else {
#pragma unroll
        for (unsigned i = 0; i < sizeof(e) / 16; i++)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(&e)[i];
    }
}

// cos and sin of a 2^64th part of turns.
__device__ __forceinline__ float2 unit(uint64_t turns)
{
    const uint32_t t = (uint32_t)((turns + 0x80000000ull) >> 32);
    const uint32_t quarter = (t + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(t - (quarter << 30)) * (6.28318530717958648f * 0x1p-32f), z = x * x;
    float s = fmaf(z, 1.0f / 362880, -1.0f / 5040), c = fmaf(z, -1.0f / 3628800, 1.0f / 40320);
    s = fmaf(z, s, 1.0f / 120);
    c = fmaf(z, c, -1.0f / 720);
    s = fmaf(z, s, -1.0f / 6);
    c = fmaf(z, c, 1.0f / 24);
    c = fmaf(z, c, -0.5f);
    s = fmaf(x * z, s, x);
    c = fmaf(z, c, 1.0f);
    const float u = quarter & 1 ? s : c, v = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -u : u, quarter & 2 ? -v : v);
}

// N elements a lane (8 or 1).  What a head vector is made of, in the order that
// lanes take it: `turned` units of N pairs (HALVES) or N/2 of them (PAIRS), or
// of one pair (N = 1), then the rest in units of N elements.  SEVERAL: a.rows rows
// a wavefront.
template <int N, bool HALVES, bool SEVERAL, class X, class Y>
__global__ __launch_bounds__(WAVES * 64) void k_rope(Rope a)
{
    const int lane = threadIdx.x & 63;
    constexpr int PER = N == 1 ? 1 : HALVES ? N : N / 2;     // pairs of a unit
    constexpr bool TWO = N == 1 || HALVES;                   // a unit's sides lie apart
    const int pairs = a.plan.pairs, turned = pairs / PER, units = turned + (a.dim - 2 * pairs) / N;
    const int hop = units < 64 ? 64 / units : 1;             // heads side by side
    const int side = units < 64 ? lane / units : 0, sub = SEVERAL ? side / a.heads : 0;
    const int h0 = blockIdx.y * a.per + side - sub * a.heads, h1 = min((int)blockIdx.y * a.per + a.per, a.heads);
    const int group = (int)(blockIdx.z << KV_FOLD | blockIdx.x);
    const int row0 = (group * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * (SEVERAL ? a.rows : 1);
    if (row0 >= a.g.n_tokens) return;
    const int row = row0 + sub;
    bool mine = side < hop && (!SEVERAL || (sub < a.rows && row < a.g.n_tokens));
    auto find = [&](int row) { return kv_find(a.g, row, [](int next, int) { return next; }); };
    auto has = [&](const KvSeq &q) { return q.seq >= 0 && row >= q.row0 && row < q.row0 + q.n_new; };
    int32_t pos = 0;
    if (a.pos) {
        if (!SEVERAL || mine) pos = a.pos[row];
    } else if constexpr (SEVERAL) {
        // a sequence at a time, from the first row on (mostly one)
        bool found = false;
        for (uint64_t left = __ballot(mine); left;) {
            const int first = __builtin_amdgcn_readlane(row, __builtin_ctzll(left));
            const KvSeq q = find(first);
            const bool in = mine && !found && has(q);
            if (in) pos = q.len - (q.row0 + q.n_new - row);
            found = found || in;
            left &= ~__ballot(in || row == first);
        }
        mine = found;
    } else {
        const KvSeq q = find(row);
        if (!has(q)) return;
        pos = q.len - (q.row0 + q.n_new - row);
    }
    const X *px = static_cast<const X *>(a.x.data) + (int64_t)row * a.x.token;
    Y *py = static_cast<Y *>(a.y.data) + (int64_t)row * a.y.token;
    for (int u0 = 0; u0 < units; u0 += 64) {
        const int u = units < 64 ? lane - side * units : u0 + lane;
        if (!mine || u >= units) continue;
        if (u >= turned) {
            const int at = 2 * pairs + (u - turned) * N;
            for (int h = h0; h < h1; h += hop) {
                const Vec<X, N> x = load<N>(px + h * a.x.head + at);
                Vec<Y, N> y;
#pragma unroll
                for (int i = 0; i < N; i++) y.v[i] = (Y)(float)x.v[i];
                store(py + h * a.y.head + at, y);
            }
            continue;
        }
        float2 cs[PER];
#pragma unroll
        for (int i = 0; i < PER; i++) {
            cs[i] = unit((uint64_t)(int64_t)pos * a.plan.step[u * PER + i]);
            cs[i].x *= a.plan.amplitude;
            cs[i].y *= a.plan.amplitude;
        }
        const int at = HALVES ? u * PER : 2 * u * PER, other = at + (HALVES ? pairs : 1);
        for (int h = h0; h < h1; h += hop) {
            const Vec<X, N> x = load<N>(px + h * a.x.head + at);
            Vec<Y, N> y;
            auto turn = [&](int i, X p, X q, Y &yp, Y &yq) {
                const float u = (float)p, v = (float)q;
                yp = (Y)fmaf(u, cs[i].x, -(v * cs[i].y));
                yq = (Y)fmaf(u, cs[i].y, v * cs[i].x);
            };
            if constexpr (TWO) {
                const Vec<X, N> z = load<N>(px + h * a.x.head + other);
                Vec<Y, N> w;
#pragma unroll
                for (int i = 0; i < N; i++) turn(i, x.v[i], z.v[i], y.v[i], w.v[i]);
                store(py + h * a.y.head + at, y);
                store(py + h * a.y.head + other, w);
            } else {
#pragma unroll
                for (int i = 0; i < N / 2; i++) turn(i, x.v[2 * i], x.v[2 * i + 1], y.v[2 * i], y.v[2 * i + 1]);
                store(py + h * a.y.head + at, y);
            }
        }
    }
}

template <int N, bool HALVES, class X, class Y>
hipError_t launch(const Rope &a, dim3 grid, hipStream_t s)
{
    if (a.rows > 1) hipLaunchKernelGGL((k_rope<N, HALVES, true, X, Y>), grid, dim3(WAVES * 64), 0, s, a);
    else hipLaunchKernelGGL((k_rope<N, HALVES, false, X, Y>), grid, dim3(WAVES * 64), 0, s, a);
    return hipGetLastError();
}

template <class X, class Y>
hipError_t launch(const Rope &a, dim3 grid, bool wide, hipStream_t s)
{
    if (a.plan.layout == LW_ROPE_HALVES) return wide ? launch<8, true, X, Y>(a, grid, s) : launch<1, true, X, Y>(a, grid, s);
    return wide ? launch<8, false, X, Y>(a, grid, s) : launch<1, false, X, Y>(a, grid, s);
}

template <class X>
hipError_t launch_x(const Rope &a, int y_dtype, dim3 grid, bool wide, hipStream_t s)
{
    if (y_dtype == LW_F16) return launch<X, _Float16>(a, grid, wide, s);
    if (y_dtype == LW_BF16) return launch<X, __bf16>(a, grid, wide, s);
    return launch<X, float>(a, grid, wide, s);
}

}  // namespace

hipError_t lw_launch_rope(const lw_rope_plan &plan, const KvGeom &g, const int32_t *pos, int heads, int head_dim,
                          const KvTensor &x, int x_dtype, const KvTensor &y, int y_dtype, hipStream_t s)
{
    Rope a;
    a.g = g;
    a.pos = pos;
    a.x = x;
    a.y = y;
    a.heads = heads;
    a.dim = head_dim;
    a.plan = plan;
    // Eight elements a lane where every unit of eight is 16-byte aligned and lies
    // on one side of a pair (20000 rows of 40 heads of 128, fp32 to bf16, 116 us;
    // one off alignment 130).  One is dearer in 16 bits, by the instructions: fp16 to
    // fp16, 20000 rows of 40 heads of 128 with eight 82 us, 5.0 TB/s; of 66 with 33
    // pairs 53, 4.0; of 80 with 20 94, 2.7; of 96 with 12 179, 1.7.
    const int unit = plan.layout == LW_ROPE_HALVES ? 8 : 4;  // pairs
    const bool wide = x.wide && y.wide && head_dim % 8 == 0 && plan.pairs % unit == 0;
    // Heads a wavefront: as many as leave the chip 4096 wavefronts (those 20000 rows
    // with eight each: 122 us), in whole turns of those it takes side by side (one
    // row, 40 heads of 128, eight side by side: 2.9 us and 3.1 with one a wavefront;
    // 128 rows 3.3 and 5.6; off alignment one side by side: 2.5 and 3.2 with eight).
    const int64_t units = wide ? plan.pairs / unit + (head_dim - 2 * plan.pairs) / 8 : head_dim - plan.pairs;
    const int64_t hop = std::max<int64_t>(64 / units, 1), per = g.n_tokens * (int64_t)heads / 4096;
    a.per = (int)std::min<int64_t>(heads, std::max<int64_t>((per + hop - 1) / hop * hop, hop));
    // and rows, where they have fewer heads than that (20000 rows of one head of 128,
    // fp32 to bf16, 4.7 us and 15.0 with one a wavefront; 100000 of two of 80 17.8 and
    // 56, the rate of a copy)
    a.rows = (int)std::max<int64_t>(hop / heads, 1);
    const int64_t some = (int64_t)WAVES * a.rows;
    static_assert(kv_fold_fits(((int64_t)1 << 26) / WAVES, WAVES * 64), "as many rows as lw_rope takes");
    const KvFold f = kv_fold((g.n_tokens + some - 1) / some);
    const dim3 grid(f.a, (unsigned)((heads + a.per - 1) / a.per), f.b);
    if (x_dtype == LW_F16) return launch_x<_Float16>(a, y_dtype, grid, wide, s);
    if (x_dtype == LW_BF16) return launch_x<__bf16>(a, y_dtype, grid, wide, s);
    return launch_x<float>(a, y_dtype, grid, wide, s);
}
