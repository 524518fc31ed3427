// kv_entry.hip -- the entry points of the 4-bit key/value cache: argument
// checks and launches.  Everything the kernels assume of the host's numbers
// is checked here; what lies in device memory (start, lens, table) the
// kernels check themselves.
#include <algorithm>
#include <climits>
#include <cmath>
#include <string>

#include "kv.h"

lw_status lw_fail(lw_status s, const std::string &msg);   // bundle.cpp

namespace {

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool kind_ok(int kv_heads, int head_dim, int page_tokens)
{
    return kv_heads >= 1 && kv_heads <= 1024 && (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
           (page_tokens == 32 || page_tokens == 64 || page_tokens == 128 || page_tokens == 256);
}

// The checks every entry point shares; g is what the kernels get.
lw_status geom(const lw_kv_cache *c, const lw_kv_batch *b, int64_t n_tokens, KvGeom &g)
{
    if (!c || !b) return lw_fail(LW_E_ARG, "null cache or batch");
    if (c->kv_heads < 1 || c->kv_heads > 1024) return lw_fail(LW_E_ARG, "kv_heads must be in 1..1024");
    if (!kind_ok(c->kv_heads, c->head_dim, c->page_tokens))
        return lw_fail(LW_E_UNSUPPORTED, "head_dim must be 64, 128 or 256 and page_tokens 32, 64, 128 or 256");
    if (c->n_pages < 0 || b->n_seqs < 0 || b->table_stride < 0 || b->max_len < 0 || n_tokens < 0)
        return lw_fail(LW_E_ARG, "negative size");
    if (b->n_seqs > (1 << 22) || n_tokens > (1 << 26))
        return lw_fail(LW_E_ARG, "more than 2^22 sequences or 2^26 new tokens");
    if (c->n_pages > ((int64_t)1 << 40)) return lw_fail(LW_E_ARG, "more than 2^40 pages");
    if (b->table_stride > ((int64_t)1 << 26)) return lw_fail(LW_E_ARG, "more than 2^26 pages per sequence");
    if (b->n_seqs && n_tokens) {
        if (!b->start || !b->lens || (!b->table && b->table_stride) || (!c->pages && c->n_pages))
            return lw_fail(LW_E_ARG, "null argument");
        if (!aligned(c->pages, 16) || !aligned(b->start, 4) || !aligned(b->lens, 4) || !aligned(b->table, 4))
            return lw_fail(LW_E_ARG, "pages must be 16-byte aligned, start, lens and table 4-byte aligned");
    }
    g.pages = static_cast<uint8_t *>(c->pages);
    g.start = b->start;
    g.lens = b->lens;
    g.table = b->table;
    g.n_pages = (uint32_t)std::min<int64_t>(c->n_pages, (int64_t)1 << 31);
    g.stride = b->table_stride;
    g.block_bytes = c->page_tokens * (c->head_dim + 8);
    g.page_bytes = (int64_t)g.block_bytes * c->kv_heads;
    g.n_seqs = (int32_t)b->n_seqs;
    g.n_tokens = (int32_t)n_tokens;
    g.kv_heads = c->kv_heads;
    g.page_shift = __builtin_ctz((unsigned)c->page_tokens);
    return LW_OK;
}

lw_status tensor(const lw_kv_tensor *t, const char *what, int dtype, KvTensor &out)
{
    if (!t || !t->data) return lw_fail(LW_E_ARG, std::string(what) + " is null");
    const int64_t most = (int64_t)1 << 32;     // keeps row * stride inside 64 bits
    if (t->token_stride < 0 || t->head_stride < 0 || t->token_stride > most || t->head_stride > most)
        return lw_fail(LW_E_ARG, std::string(what) + " has a stride outside 0..2^32");
    const size_t size = dtype == LW_F32 ? 4 : 2;
    if (!aligned(t->data, size)) return lw_fail(LW_E_ARG, std::string(what) + " is not aligned to its elements");
    out.data = t->data;
    out.token = t->token_stride;
    out.head = t->head_stride;
    out.wide = aligned(t->data, 16) && t->token_stride * size % 16 == 0 && t->head_stride * size % 16 == 0;
    return LW_OK;
}

lw_status device(hipError_t e, const char *what)
{
    if (e == hipSuccess) return LW_OK;
    return lw_fail(LW_E_DEVICE, std::string(what) + ": " + hipGetErrorString(e));
}

// Tokens of the longest sequence, as far as the host knows.
int64_t longest(const lw_kv_cache *c, const lw_kv_batch *b)
{
    const int64_t cap = b->table_stride * c->page_tokens;
    return b->max_len ? std::min(b->max_len, cap) : cap;
}

}  // namespace

extern "C" size_t lw_kv_page_bytes(int kv_heads, int head_dim, int page_tokens)
{
    if (!kind_ok(kv_heads, head_dim, page_tokens)) return 0;
    return (size_t)kv_heads * page_tokens * (head_dim + 8);
}

extern "C" lw_status lw_kv_append(const lw_kv_cache *cache, const lw_kv_batch *batch, int64_t n_tokens,
                                  const lw_kv_tensor *k, const lw_kv_tensor *v, int dtype, void *stream)
{
    KvGeom g;
    KvTensor tk, tv;
    lw_status st = geom(cache, batch, n_tokens, g);
    if (st) return st;
    if (dtype != LW_F16 && dtype != LW_BF16 && dtype != LW_F32) return lw_fail(LW_E_ARG, "unknown dtype");
    if (!batch->n_seqs || !n_tokens) return LW_OK;
    if ((st = tensor(k, "k", dtype, tk)) || (st = tensor(v, "v", dtype, tv))) return st;
    return device(lw_launch_kv_append(g, cache->head_dim, tk, tv, dtype, (hipStream_t)stream), "kv append launch");
}

extern "C" lw_status lw_kv_read(const lw_kv_cache *cache, const lw_kv_batch *batch, int64_t n_tokens,
                                const lw_kv_tensor *k, const lw_kv_tensor *v, int dtype, void *stream)
{
    KvGeom g;
    KvTensor tk, tv;
    lw_status st = geom(cache, batch, n_tokens, g);
    if (st) return st;
    if (dtype != LW_F16 && dtype != LW_BF16 && dtype != LW_F32) return lw_fail(LW_E_ARG, "unknown dtype");
    if (!batch->n_seqs || !n_tokens) return LW_OK;
    if ((st = tensor(k, "k", dtype, tk)) || (st = tensor(v, "v", dtype, tv))) return st;
    return device(lw_launch_kv_read(g, cache->head_dim, tk, tv, dtype, (hipStream_t)stream), "kv read launch");
}

extern "C" size_t lw_kv_attend_scratch_bytes(const lw_kv_cache *cache, const lw_kv_batch *batch, int64_t n_tokens,
                                             int q_heads)
{
    KvGeom g;
    if (geom(cache, batch, n_tokens, g) || !batch->n_seqs || !n_tokens) return 0;
    if (q_heads < 1 || q_heads % cache->kv_heads || q_heads / cache->kv_heads > 1024 ||
        n_tokens * (q_heads / cache->kv_heads) > (1 << 30))
        return 0;
    return lw_kv_most_work(cache->head_dim, cache->kv_heads, q_heads / cache->kv_heads, batch->n_seqs, n_tokens,
                           longest(cache, batch));
}

extern "C" lw_status lw_kv_attend(const lw_kv_cache *cache, const lw_kv_batch *batch, int64_t n_tokens,
                                  const lw_kv_tensor *q, const lw_kv_tensor *out, int dtype, int q_heads, float scale,
                                  int causal, int window, float *lse, void *work, size_t work_bytes, void *stream)
{
    KvAttend a;
    lw_status st = geom(cache, batch, n_tokens, a.g);
    if (st) return st;
    if (dtype != LW_F16 && dtype != LW_BF16) return lw_fail(LW_E_UNSUPPORTED, "q and out must be fp16 or bf16");
    if (q_heads < 1 || q_heads % cache->kv_heads)
        return lw_fail(LW_E_ARG, "q_heads must be a positive multiple of kv_heads");
    if (q_heads / cache->kv_heads > 1024) return lw_fail(LW_E_ARG, "more than 1024 query heads per kv head");
    if (n_tokens * (q_heads / cache->kv_heads) > (1 << 30))
        return lw_fail(LW_E_ARG, "more than 2^30 query rows per kv head");
    if (!(scale > 0.0f) || !std::isfinite(scale)) return lw_fail(LW_E_ARG, "scale must be positive and finite");
    if (window < 0) return lw_fail(LW_E_ARG, "negative window");
    if (!batch->n_seqs || !n_tokens) return LW_OK;
    if ((st = tensor(q, "q", dtype, a.q)) || (st = tensor(out, "out", dtype, a.out))) return st;
    if (!aligned(lse, 4)) return lw_fail(LW_E_ARG, "lse must be 4-byte aligned");
    if (!aligned(work, 16)) return lw_fail(LW_E_ARG, "work must be 16-byte aligned");
    const KvPlan p = lw_kv_plan(cache->head_dim, cache->kv_heads, q_heads / cache->kv_heads, batch->n_seqs, n_tokens,
                                longest(cache, batch), window, work ? work_bytes : 0);
    if (p.tile == 128 && p.tiles > 65535)
        return lw_fail(LW_E_UNSUPPORTED, "more than 65535 tiles of query rows (n_seqs + n_tokens * q_heads / kv_heads / 128)");
    a.lse = lse;
    a.part = static_cast<float *>(work);
    a.group = q_heads / cache->kv_heads;
    a.group_inv = ((1u << 21) + (unsigned)a.group - 1) / (unsigned)a.group;
    a.causal = causal != 0;
    a.window = window;
    a.target = p.target;
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.pieces = (int32_t)p.pieces;
    a.first = reinterpret_cast<int2 *>(static_cast<char *>(work) + p.first_at);
    a.slices = 1;
    a.scale = scale;
    return device(lw_launch_kv_attend(a, cache->head_dim, dtype, p, (hipStream_t)stream), "kv attend launch");
}
