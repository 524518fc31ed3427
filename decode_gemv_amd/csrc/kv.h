// kv.h -- launch interface between the entry points (kv_entry.hip) and the
// gfx950 kernels of the 4-bit key/value cache.  Internal to the library.
#ifndef LW_KV_H
#define LW_KV_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lw.h"

// Tokens of a sequence that are looked at, at most: positions and what lies a
// few steps past them fit 32 bits, chunks and pages divide it.
constexpr int32_t KV_MOST_TOKENS = 0x7FFF0000;

// A cache and a batch as the kernels see them: passed by value, so every
// field is uniform.
struct KvGeom {
    uint8_t *pages;
    const int32_t *start;        // [n_seqs + 1]
    const int32_t *lens;         // [n_seqs]
    const int32_t *table;        // [n_seqs][stride]
    int64_t stride;
    int64_t page_bytes;          // kv_heads * block_bytes
    uint32_t n_pages;            // (a table's entry reaches 2^31 - 1)
    int32_t block_bytes;         // one head's part of a page: page_tokens * (head_dim + 8)
    int32_t n_seqs, n_tokens, kv_heads;
    int32_t page_shift;          // log2(page_tokens)
};

// One packed tensor [n_tokens][heads][head_dim]; strides in elements.
struct KvTensor {
    void *data;
    int64_t token, head;
    int32_t wide;                // 1: every 8-element group is 16-byte aligned
};

struct KvAttend {
    KvGeom g;
    KvTensor q, out;
    float *lse;                  // [n_tokens][q_heads], or null
    float *part;                 // split partials (see kv_attend.hip), or null
    int32_t group;               // query heads per kv head
    uint32_t group_inv;          // ceil(2^21 / group): (x * group_inv) >> 21 = x / group for x < 2048
    int32_t causal, window;      // window 0: none
    int32_t target;              // chunks of tokens per kv head to cut the batch into (kv_attend.hpp), or 0:
    int32_t splits, chunk;       // every row tile into that many at most, of so many tokens (kv_prompt.hip)
    int32_t pieces;              // a kv head's workgroups, all with nothing to do included
    int2 *first;                 // target > 0: each row tile's first chunk's number, and the tokens of a chunk
    int32_t slices;              // of k_kv_join's workgroups
    float scale;                 // > 0
};

// How a call is cut up: rows per tile, row tiles, and chunks as in KvAttend;
// a kv head's pieces of work (chunks, or row tiles); the bytes of their results.
struct KvPlan {
    int tile;
    int64_t tiles;
    int target, splits, chunk;
    int64_t pieces;
    size_t first_at, work_bytes;
};

// `room`: bytes there are for results.
KvPlan lw_kv_plan(int head_dim, int kv_heads, int group, int64_t n_seqs, int64_t n_tokens, int64_t max_len,
                  int window, size_t room);

// Bytes that no plan of up to that many sequences, new tokens and max_len wants
// more of, with any window.
size_t lw_kv_most_work(int head_dim, int kv_heads, int group, int64_t n_seqs, int64_t n_tokens, int64_t max_len);

hipError_t lw_launch_kv_append(const KvGeom &g, int head_dim, const KvTensor &k, const KvTensor &v, int dtype,
                               hipStream_t s);
hipError_t lw_launch_kv_read(const KvGeom &g, int head_dim, const KvTensor &k, const KvTensor &v, int dtype,
                             hipStream_t s);
hipError_t lw_launch_kv_attend(const KvAttend &a, int head_dim, int dtype, const KvPlan &p, hipStream_t s);
hipError_t lw_launch_kv_prompt(const KvAttend &a, int head_dim, int dtype, const KvPlan &p, hipStream_t s);

#ifdef __HIPCC__
// ------------------------------------------------------------ device helpers

// A sequence of the batch, kept inside the tensors whatever the caller's
// arrays hold: its packed rows row0 .. row0 + n_new - 1, and its length.
struct KvSeq {
    int32_t seq;                 // -1: none
    int32_t row0, n_new, len;
};

// The sequence that x belongs to, for a bound(start[s + 1], s) that does not
// decrease with s: the first sequence whose bound is above x.  The
// wavefront's 64 lanes look at the ends of 64 parts of what is left, so 64
// sequences take one step and 4096 two, and what there is to know of the one
// found is then in a lane already (one load latency a step, where a binary
// search has one for each halving, and the loads after it).
template <class F>
__device__ __forceinline__ KvSeq kv_find(const KvGeom &g, int x, F bound)
{
    const int lane = threadIdx.x & 63;
    KvSeq r = {-1, 0, 0, 0};
    for (int lo = 0, n = g.n_seqs; n > 0;) {
        const int part = (n + 63) / 64;
        const int mine = lo + min(lane * part + part, n) - 1;
        const int a = g.start[mine], b = g.start[mine + 1], len = g.lens[mine];
        const int c = __popcll(__ballot(lane * part < n && bound(b, mine) <= x));
        if (c * part >= n) break;
        lo += c * part;
        n = min(part, n - c * part);
        if (part > 1) continue;
        r.seq = lo;
        r.row0 = min(max(__builtin_amdgcn_readlane(a, c), 0), g.n_tokens);
        r.n_new = min(max(__builtin_amdgcn_readlane(b, c), r.row0), g.n_tokens) - r.row0;
        r.len = max(__builtin_amdgcn_readlane(len, c), 0);
        break;
    }
    return r;
}

__device__ __forceinline__ int64_t kv_page(const KvGeom &g, int seq, int pos)
{
    const int64_t i = pos >> g.page_shift;
    if (pos < 0 || i >= g.stride) return -1;
    const int32_t p = g.table[(int64_t)seq * g.stride + i];
    return (uint32_t)p < g.n_pages ? p : -1;
}

// Word index, inside a head's block, of word w of token t's keys and values.
// Keys: tiles of 16 tokens, each a [unit][token] array of units of W words,
// so that the 64 lanes that hold a matrix instruction's 16 tokens x 4 parts
// read consecutive units.  Values: [token / 4][word][token % 4], so that one
// 16-byte load gives a lane four tokens of the same eight dimensions.
template <int D>
__device__ __forceinline__ int kv_kword(int t, int w)
{
    constexpr int W = D >= 128 ? 4 : D / 32, U = D / 8 / W;
    return (((t >> 4) * U + w / W) * 16 + (t & 15)) * W + w % W;
}

template <int D>
__device__ __forceinline__ int kv_vword(int t, int w)
{
    return ((t >> 2) * (D / 8) + w) * 4 + (t & 3);
}
#endif

#endif
