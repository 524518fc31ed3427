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
// 16 or 32 consecutive rows of one head and one side: the words of 16 tokens
// are 1 KiB of the cache in one piece (D = 128), written from one compute
// unit.  Both kernels are bound by memory: nothing is read twice.
#include "kv.h"

namespace {

constexpr int THREADS = 256;

template <class T> struct Eight { T v[8]; };

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(_Float16 x) { return (float)x; }
__device__ __forceinline__ float to_f(__bf16 x) { return (float)x; }

// Eight consecutive elements: 16-byte accesses where the tensor allows them.
template <class T>
__device__ __forceinline__ void load8(const T *p, int wide, float *x)
{
    Eight<T> e;
    if (wide) {
#pragma unroll
        for (unsigned i = 0; i < sizeof(e) / 16; i++)
            reinterpret_cast<uint4 *>(&e)[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) e.v[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = to_f(e.v[i]);
}

template <class T>
__device__ __forceinline__ void store8(T *p, int wide, const float *x)
{
    Eight<T> e;
#pragma unroll
    for (int i = 0; i < 8; i++) e.v[i] = (T)x[i];
    if (wide) {
#pragma unroll
        for (unsigned i = 0; i < sizeof(e) / 16; i++)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<uint4 *>(&e)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) p[i] = e.v[i];
    }
}

// The cached token of a packed row.
struct Place {
    bool known;                  // the row belongs to a sequence
    int32_t pos;
    int64_t page;                // < 0: the token is absent
};

// Where the row of each lane's vector lies.  The rows of a wavefront are
// consecutive; each is looked up by the whole wavefront.
template <int D>
__device__ __forceinline__ Place place(const KvGeom &g, int row0)
{
    constexpr int LANES = D / 8, ROWS = 64 / LANES;
    const int mine = (threadIdx.x & 63) / LANES, row = row0 + mine;
    KvSeq q = {-1, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < ROWS; i++) {
        const KvSeq s = kv_find(g, row0 + i, [](int next, int) { return next; });
        if (i == mine) q = s;
    }
    Place r = {q.seq >= 0 && row >= q.row0 && row < q.row0 + q.n_new, 0, -1};
    if (!r.known) return r;      // past the batch, or before its start
    r.pos = q.len - (q.row0 + q.n_new - row);
    r.page = kv_page(g, q.seq, r.pos);
    return r;
}

template <int D, class T>
__global__ __launch_bounds__(THREADS) void k_kv_append(KvGeom g, KvTensor k, KvTensor v)
{
    constexpr int LANES = D / 8, ROWS = 64 / LANES;
    const int w = threadIdx.x % LANES;
    const int row0 = blockIdx.x * (THREADS / LANES) + (threadIdx.x >> 6) * ROWS;
    if (row0 >= g.n_tokens) return;
    const int row = row0 + (threadIdx.x & 63) / LANES;
    const KvTensor &t = blockIdx.z ? v : k;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = 0.0f;
    if (row < g.n_tokens)
        load8(static_cast<const T *>(t.data) + row * t.token + blockIdx.y * t.head + w * 8, t.wide, x);
    const Place p = place<D>(g, row0);
    float lo = x[0], hi = x[0];
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        fine &= fabsf(x[i]) < __builtin_inff();
    }
    int bad = !fine;
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) {
        lo = fminf(lo, __shfl_xor(lo, o));
        hi = fmaxf(hi, __shfl_xor(hi, o));
        bad |= __shfl_xor(bad, o);
    }
    if (p.page < 0) return;
    _Float16 m = (_Float16)fminf(fmaxf(-lo, -65504.0f), 65504.0f);
    _Float16 d = (_Float16)fminf((hi - lo) * (1.0f / 15.0f), 65504.0f);
    if (bad) d = m = (_Float16)__builtin_nanf("");
    const float inv = (float)d == 0.0f ? 0.0f : 1.0f / (float)d;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float q = fminf(fmaxf(rintf((x[i] + (float)m) * inv), 0.0f), 15.0f);
        word |= (bad ? 0u : (uint32_t)q) << (4 * i);
    }
    const int P = 1 << g.page_shift, tok = p.pos & (P - 1);
    uint32_t *block = reinterpret_cast<uint32_t *>(g.pages + p.page * g.page_bytes +
                                                   (int64_t)blockIdx.y * g.block_bytes);
    block[blockIdx.z ? P * (D / 8) + kv_vword<D>(tok, w) : kv_kword<D>(tok, w)] = word;
    if (w == 0)
        block[P * (D / 4) + (blockIdx.z ? P : 0) + tok] =
            __builtin_bit_cast(uint16_t, d) | (uint32_t)__builtin_bit_cast(uint16_t, m) << 16;
}

template <int D, class T>
__global__ __launch_bounds__(THREADS) void k_kv_read(KvGeom g, KvTensor k, KvTensor v)
{
    constexpr int LANES = D / 8, ROWS = 64 / LANES;
    const int w = threadIdx.x % LANES;
    const int row0 = blockIdx.x * (THREADS / LANES) + (threadIdx.x >> 6) * ROWS;
    if (row0 >= g.n_tokens) return;
    const int row = row0 + (threadIdx.x & 63) / LANES;
    const KvTensor &t = blockIdx.z ? v : k;
    const Place p = place<D>(g, row0);
    if (!p.known) return;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = 0.0f;
    if (p.page >= 0) {
        const int P = 1 << g.page_shift, tok = p.pos & (P - 1);
        const uint32_t *block = reinterpret_cast<const uint32_t *>(g.pages + p.page * g.page_bytes +
                                                                   (int64_t)blockIdx.y * g.block_bytes);
        const uint32_t word = block[blockIdx.z ? P * (D / 8) + kv_vword<D>(tok, w) : kv_kword<D>(tok, w)];
        const uint32_t dm = block[P * (D / 4) + (blockIdx.z ? P : 0) + tok];
        const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)dm);
        const float m = (float)__builtin_bit_cast(_Float16, (uint16_t)(dm >> 16));
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = fmaf((float)(word >> (4 * i) & 15u), d, -m);   // d q is exact in fp32
    }
    store8(static_cast<T *>(t.data) + row * t.token + blockIdx.y * t.head + w * 8, t.wide, x);
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

dim3 grid_of(const KvGeom &g, int head_dim)
{
    const int rows = THREADS / (head_dim / 8);
    return dim3((unsigned)((g.n_tokens + rows - 1) / rows), (unsigned)g.kv_heads, 2);
}

}  // namespace

hipError_t lw_launch_kv_append(const KvGeom &g, int head_dim, const KvTensor &k, const KvTensor &v, int dtype,
                               hipStream_t s)
{
    return with_types(head_dim, dtype, [&](auto dim, auto type) {
        hipLaunchKernelGGL((k_kv_append<dim.value, decltype(type)>), grid_of(g, head_dim), dim3(THREADS), 0, s, g, k, v);
        return hipGetLastError();
    });
}

hipError_t lw_launch_kv_read(const KvGeom &g, int head_dim, const KvTensor &k, const KvTensor &v, int dtype,
                             hipStream_t s)
{
    return with_types(head_dim, dtype, [&](auto dim, auto type) {
        hipLaunchKernelGGL((k_kv_read<dim.value, decltype(type)>), grid_of(g, head_dim), dim3(THREADS), 0, s, g, k, v);
        return hipGetLastError();
    });
}
