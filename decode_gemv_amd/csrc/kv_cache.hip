// kv_cache.hip -- quantising new keys and values into the paged 4-bit cache,
// and reading cached tokens back.
//
// One key or value head vector x[0..D) is held as 4-bit codes q and an fp16
// pair (d, m), worth d q - m, the library's dequantisation rule ("Software-
// Defined Bandwidth Expansion", IV-A: grouped storage with a scale and an
// offset), with one group per vector:
//     m = fp16(-min x), d = fp16((max x - min x) / 15), within +-65504
//     q = clamp(rint((x + m) (1/d)), 0, 15),  0 where d = 0
// in fp32, each operation rounded once, with the pair that is stored (so the
// rounding of d and m is not an error of the codes).  A vector with a NaN or
// an infinity gets d = m = NaN: it reads back as NaN and is not lost.
//
// D/8 lanes hold a vector, eight elements each, so a lane makes one word of
// codes and the extremes meet in log2(D/8) lane exchanges.  A workgroup takes
// 2048/D consecutive rows and some of the heads, keys and values both: a row
// is looked up once for all of them, and the words of 16 tokens, 1 KiB of the
// cache in one piece at D = 128, come from one compute unit.  Both kernels
// are bound by memory, nothing is read twice: 22 thousand tokens of 8 heads of
// 128 in fp16 are appended in 24 us (4.8 TB/s) and read back in 20 (5.7), 72
// thousand read in 59 (6.3).  The quantising is not far behind: 13 vector
// instructions an element (extremes that carry a NaN along, in pairs for fp16)
// where 19 took 27.5 us.
#include <algorithm>
#include <type_traits>

#include "kv.h"

namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(_Float16 x) { return (float)x; }
__device__ __forceinline__ float to_f(__bf16 x) { return (float)x; }

// Eight consecutive elements: 16-byte accesses where the tensor allows them.
template <class T> struct Eight { T v[8]; };
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

template <class T>
__device__ __forceinline__ Eight<T> load8(const T *p, int wide)
{
    Eight<T> e;
    if (wide) {
#pragma unroll
        for (unsigned i = 0; i < sizeof(e) / 16; i++)
            reinterpret_cast<u4 *>(&e)[i] = __builtin_nontemporal_load(reinterpret_cast<const u4 *>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) e.v[i] = p[i];
    }
    return e;
}

// (Loads and stores are marked as passing the caches by: 64 us where plain
// stores take 206, 73 thousand tokens of 8 heads read back.)
template <class T>
__device__ __forceinline__ void store8(T *p, int wide, const Eight<T> &e)
{
    if (wide) {
#pragma unroll
        for (unsigned i = 0; i < sizeof(e) / 16; i++)
            __builtin_nontemporal_store(reinterpret_cast<const u4 *>(&e)[i], reinterpret_cast<u4 *>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) p[i] = e.v[i];
    }
}

typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// The larger of two, by element; NaN where one is.
template <class X>
__device__ __forceinline__ X larger(X a, X b) { return __builtin_elementwise_maximum(a, b); }

// The largest of x over the D/8 lanes that hold a vector.
template <int D, class X>
__device__ __forceinline__ X most(X x)
{
    auto with = [&](auto ctrl) {
        x = larger(x, __builtin_bit_cast(X, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl.value, 0xF, 0xF, true)));
    };
    with(std::integral_constant<int, 0xB1>{});                // lane ^ 1
    with(std::integral_constant<int, 0x4E>{});                // lane ^ 2
    with(std::integral_constant<int, 0x141>{});               // 7 - lane of eight
    if (D >= 128) with(std::integral_constant<int, 0x140>{}); // 15 - lane of sixteen
    if (D >= 256) x = larger(x, __builtin_bit_cast(X, __shfl_xor(__builtin_bit_cast(int, x), 16)));
    return x;
}

// The vector's largest element and minus its smallest, NaN where one is.
template <int D, class T>
__device__ __forceinline__ float2 extremes(const Eight<T> &e)
{
    if constexpr (std::is_same<T, _Float16>::value) {         // in pairs, and both at once
        const h2 *x = reinterpret_cast<const h2 *>(&e);
        const h2 hi = larger(larger(x[0], x[1]), larger(x[2], x[3]));
        const h2 low = larger(larger(-x[0], -x[1]), larger(-x[2], -x[3]));
        const h2 both = most<D>(larger(h2{hi[0], low[0]}, h2{hi[1], low[1]}));
        return make_float2((float)both[0], (float)both[1]);
    } else {
        float hi = to_f(e.v[0]), low = -hi;
#pragma unroll
        for (int i = 1; i < 8; i++) {
            hi = larger(hi, to_f(e.v[i]));
            low = larger(low, -to_f(e.v[i]));
        }
        return make_float2(most<D>(hi), most<D>(low));
    }
}

// The cached token of a lane's row.
struct Place {
    bool known;                  // the row belongs to a sequence
    int32_t tok;                 // place in its page
    uint8_t *page;               // null: the token is absent
};

// Where the row of each lane's vector lies.  The rows of a wavefront are
// consecutive, mostly of one sequence.
template <int D>
__device__ __forceinline__ Place place(const KvGeom &g, int row0)
{
    constexpr int LANES = D / 8, ROWS = 64 / LANES;
    const int mine = (threadIdx.x & 63) / LANES, row = row0 + mine;
    auto next_row = [](int next, int) { return next; };
    KvSeq q = kv_find(g, row0, next_row);
    if (q.seq >= 0 && row0 + ROWS > q.row0 + q.n_new) {
#pragma unroll
        for (int i = 1; i < ROWS; i++) {
            const KvSeq s = kv_find(g, row0 + i, next_row);
            if (i == mine) q = s;
        }
    }
    Place r = {q.seq >= 0 && row >= q.row0 && row < q.row0 + q.n_new, 0, nullptr};
    if (!r.known) return r;      // past the batch, or before its start
    const int pos = q.len - (q.row0 + q.n_new - row);
    const int64_t page = kv_page(g, q.seq, pos);
    r.tok = pos & ((1 << g.page_shift) - 1);
    if (page >= 0) r.page = g.pages + page * g.page_bytes;
    return r;
}

// Places in a head's block (words) of a token's word w and pair.
template <int D>
struct Slots {
    int k, v, kdm, vdm;
    __device__ __forceinline__ Slots(int P, int tok, int w)
        : k(kv_kword<D>(tok, w)), v(P * (D / 8) + kv_vword<D>(tok, w)), kdm(P * (D / 4) + tok), vdm(kdm + P)
    {
    }
};

// A lane's word of codes of its vector, and the vector's pair.
template <int D, class T>
__device__ __forceinline__ uint2 quantise(const Eight<T> &e)
{
    const float2 at = extremes<D>(e);
    const float hi = at.x, low = at.y;
    const bool bad = !(hi < __builtin_inff() && low < __builtin_inff());
    _Float16 m = (_Float16)__builtin_amdgcn_fmed3f(low, -65504.0f, 65504.0f);
    _Float16 d = (_Float16)fminf((hi + low) * (1.0f / 15.0f), 65504.0f);
    // 1/d, rounded once: one step from the approximation gives that for every
    // fp16 there is
    const float df = (float)d, r = __builtin_amdgcn_rcpf(df);
    const float inv = df == 0.0f ? 0.0f : fmaf(fmaf(-df, r, 1.0f), r, r);
    float half[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; j++) q[j] = __builtin_amdgcn_fmed3f(rintf((to_f(e.v[4 * i + j]) + (float)m) * inv), 0.0f, 15.0f);
        half[i] = fmaf(q[3], 4096.0f, fmaf(q[2], 256.0f, fmaf(q[1], 16.0f, q[0])));      // 16 bits, exact
    }
    if (bad) {
        d = m = (_Float16)__builtin_nanf("");
        half[0] = half[1] = 0.0f;
    }
    return make_uint2((uint32_t)half[0] | (uint32_t)half[1] << 16,
                      __builtin_bit_cast(uint16_t, d) | (uint32_t)__builtin_bit_cast(uint16_t, m) << 16);
}

// d q - m of a word's eight codes.
template <class T>
__device__ __forceinline__ Eight<T> dequantise(uint32_t word, uint32_t dm)
{
    const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)dm);
    const float m = (float)__builtin_bit_cast(_Float16, (uint16_t)(dm >> 16));
    const uint32_t q[2] = {word & 0x0F0F0F0Fu, word >> 4 & 0x0F0F0F0Fu};
    Eight<T> e;
#pragma unroll
    for (int i = 0; i < 8; i++) e.v[i] = (T)fmaf((float)(q[i % 2] >> (i / 2 * 8) & 0xFFu), d, -m);   // d q is exact
    return e;
}

template <int D, class T>
__global__ __launch_bounds__(THREADS) void k_kv_append(KvGeom g, KvTensor k, KvTensor v, int per)
{
    constexpr int LANES = D / 8, ROWS = 64 / LANES;
    const int w = threadIdx.x % LANES;
    const int row0 = blockIdx.x * (THREADS / LANES) + (threadIdx.x >> 6) * ROWS;
    if (row0 >= g.n_tokens) return;
    const int row = min(row0 + (int)(threadIdx.x & 63) / LANES, g.n_tokens - 1);
    const int h0 = blockIdx.y * per, h1 = min(h0 + per, g.kv_heads);
    const T *pk = static_cast<const T *>(k.data) + row * k.token + h0 * k.head + w * 8;
    const T *pv = static_cast<const T *>(v.data) + row * v.token + h0 * v.head + w * 8;
    Eight<T> xk = load8(pk, k.wide), xv = load8(pv, v.wide);
    const Place p = place<D>(g, row0);
    const Slots<D> at(1 << g.page_shift, p.tok, w);
    uint8_t *block = p.page + (int64_t)h0 * g.block_bytes;
    for (int h = h0; h < h1; h++) {
        const Eight<T> ck = xk, cv = xv;
        if (h + 1 < h1) {                                     // the next head's, while this one is worked on
            pk += k.head;
            pv += v.head;
            xk = load8(pk, k.wide);
            xv = load8(pv, v.wide);
        }
        const uint2 qk = quantise<D>(ck), qv = quantise<D>(cv);
        if (p.page) {
            uint32_t *to = reinterpret_cast<uint32_t *>(block);
            to[at.k] = qk.x;
            to[at.v] = qv.x;
            if (w == 0) {
                to[at.kdm] = qk.y;
                to[at.vdm] = qv.y;
            }
        }
        block += g.block_bytes;
    }
}

template <int D, class T>
__global__ __launch_bounds__(THREADS) void k_kv_read(KvGeom g, KvTensor k, KvTensor v, int per)
{
    constexpr int LANES = D / 8, ROWS = 64 / LANES;
    const int w = threadIdx.x % LANES;
    const int row0 = blockIdx.x * (THREADS / LANES) + (threadIdx.x >> 6) * ROWS;
    if (row0 >= g.n_tokens) return;
    const int row = row0 + (threadIdx.x & 63) / LANES;
    const int h0 = blockIdx.y * per, h1 = min(h0 + per, g.kv_heads);
    const Place p = place<D>(g, row0);
    if (!p.known) return;
    const Slots<D> at(1 << g.page_shift, p.tok, w);
    T *pk = static_cast<T *>(k.data) + row * k.token + h0 * k.head + w * 8;
    T *pv = static_cast<T *>(v.data) + row * v.token + h0 * v.head + w * 8;
    const uint8_t *block = p.page + (int64_t)h0 * g.block_bytes;
    uint4 x = make_uint4(0, 0, 0, 0);                         // an absent token's: zeros
    auto load = [&]() {
        const uint32_t *from = reinterpret_cast<const uint32_t *>(block);
        if (p.page) x = make_uint4(from[at.k], from[at.kdm], from[at.v], from[at.vdm]);
    };
    load();
    for (int h = h0; h < h1; h++) {
        const uint4 c = x;
        block += g.block_bytes;
        if (h + 1 < h1) load();                               // the next head's, while this one is worked on
        store8(pk, k.wide, dequantise<T>(c.x, c.y));
        store8(pv, v.wide, dequantise<T>(c.z, c.w));
        pk += k.head;
        pv += v.head;
    }
}

template <class F>
hipError_t with_types(int head_dim, int dtype, F f)
{
    auto typed = [&](auto dim) {
        if (dtype == LW_F16) return f(dim, _Float16{});
        if (dtype == LW_BF16) return f(dim, __bf16{});
        if (dtype == LW_F32) return f(dim, float{});
        return hipErrorInvalidValue;
    };
    if (head_dim == 64) return typed(std::integral_constant<int, 64>{});
    if (head_dim == 128) return typed(std::integral_constant<int, 128>{});
    if (head_dim == 256) return typed(std::integral_constant<int, 256>{});
    return hipErrorInvalidValue;
}

// Workgroups by rows and heads: as many heads each as leave the chip full.
struct Cut {
    dim3 grid;
    int per;
    Cut(const KvGeom &g, int head_dim)
    {
        const int rows = THREADS / (head_dim / 8);
        const int64_t blocks = (g.n_tokens + rows - 1) / rows;
        per = (int)std::min<int64_t>(g.kv_heads, std::max<int64_t>(1, blocks * g.kv_heads / 2048));
        grid = dim3((unsigned)blocks, (unsigned)((g.kv_heads + per - 1) / per));
    }
};

}  // namespace

hipError_t lw_launch_kv_append(const KvGeom &g, int head_dim, const KvTensor &k, const KvTensor &v, int dtype,
                               hipStream_t s)
{
    return with_types(head_dim, dtype, [&](auto dim, auto type) {
        const Cut c(g, head_dim);
        hipLaunchKernelGGL((k_kv_append<dim.value, decltype(type)>), c.grid, dim3(THREADS), 0, s, g, k, v, c.per);
        return hipGetLastError();
    });
}

hipError_t lw_launch_kv_read(const KvGeom &g, int head_dim, const KvTensor &k, const KvTensor &v, int dtype,
                             hipStream_t s)
{
    return with_types(head_dim, dtype, [&](auto dim, auto type) {
        const Cut c(g, head_dim);
        hipLaunchKernelGGL((k_kv_read<dim.value, decltype(type)>), c.grid, dim3(THREADS), 0, s, g, k, v, c.per);
        return hipGetLastError();
    });
}
