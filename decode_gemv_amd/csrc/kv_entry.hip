// kv_entry.hip -- the entry points of the 4-bit key/value cache and of the
// rotary positions of what goes into it: argument checks and launches.
// Everything the kernels assume of the host's numbers is checked here; what lies
// in device memory (start, lens, table) the kernels check themselves.
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

// A batch's checks; what it gives of what the kernels get.
lw_status sequences(const lw_kv_batch *b, int64_t n_tokens, bool pages, KvGeom &g)
{
    if (b->n_seqs < 0 || b->table_stride < 0 || b->max_len < 0 || n_tokens < 0)
        return lw_fail(LW_E_ARG, "negative size");
    if (b->n_seqs > (1 << 22) || n_tokens > (1 << 26))
        return lw_fail(LW_E_ARG, "more than 2^22 sequences or 2^26 new tokens");
    if (b->table_stride > ((int64_t)1 << 26)) return lw_fail(LW_E_ARG, "more than 2^26 pages per sequence");
    if (b->n_seqs && n_tokens) {
        if (!b->start || !b->lens || (pages && !b->table && b->table_stride)) return lw_fail(LW_E_ARG, "null argument");
        if (!aligned(b->start, 4) || !aligned(b->lens, 4) || (pages && !aligned(b->table, 4)))
            return lw_fail(LW_E_ARG, "start, lens and table must be 4-byte aligned");
    }
    g.start = b->start;
    g.lens = b->lens;
    g.table = b->table;
    g.stride = b->table_stride;
    g.n_seqs = (int32_t)b->n_seqs;
    g.n_tokens = (int32_t)n_tokens;
    return LW_OK;
}

// A cache's, for a call that has something to do with its pages or not.
lw_status pages(const lw_kv_cache *c, bool busy, KvGeom &g)
{
    if (c->kv_heads < 1 || c->kv_heads > 1024) return lw_fail(LW_E_ARG, "kv_heads must be in 1..1024");
    if (!kind_ok(c->kv_heads, c->head_dim, c->page_tokens))
        return lw_fail(LW_E_UNSUPPORTED, "head_dim must be 64, 128 or 256 and page_tokens 32, 64, 128 or 256");
    if (c->n_pages < 0) return lw_fail(LW_E_ARG, "negative size");
    if (c->n_pages > ((int64_t)1 << 40)) return lw_fail(LW_E_ARG, "more than 2^40 pages");
    if (busy && !c->pages && c->n_pages) return lw_fail(LW_E_ARG, "null argument");
    if (busy && !aligned(c->pages, 16)) return lw_fail(LW_E_ARG, "pages must be 16-byte aligned");
    g.pages = static_cast<uint8_t *>(c->pages);
    g.n_pages = (uint32_t)std::min<int64_t>(c->n_pages, (int64_t)1 << 31);
    g.block_bytes = c->page_tokens * (c->head_dim + 8);
    g.page_bytes = (int64_t)g.block_bytes * c->kv_heads;
    g.kv_heads = c->kv_heads;
    g.page_shift = __builtin_ctz((unsigned)c->page_tokens);
    return LW_OK;
}

// The checks every entry point of the cache shares; g is what the kernels get.
lw_status geom(const lw_kv_cache *c, const lw_kv_batch *b, int64_t n_tokens, KvGeom &g)
{
    if (!c || !b) return lw_fail(LW_E_ARG, "null cache or batch");
    const lw_status st = pages(c, b->n_seqs > 0 && n_tokens > 0, g);
    return st ? st : sequences(b, n_tokens, true, g);
}

// Of query heads and what attention takes of them.
lw_status heads(const lw_kv_cache *c, int64_t n_tokens, int dtype, int q_heads)
{
    if (dtype != LW_F16 && dtype != LW_BF16) return lw_fail(LW_E_UNSUPPORTED, "queries and outputs must be fp16 or bf16");
    if (q_heads < 1 || q_heads % c->kv_heads)
        return lw_fail(LW_E_ARG, "q_heads must be a positive multiple of kv_heads");
    if (q_heads / c->kv_heads > 1024) return lw_fail(LW_E_ARG, "more than 1024 query heads per kv head");
    if (n_tokens * (q_heads / c->kv_heads) > (1 << 30))
        return lw_fail(LW_E_ARG, "more than 2^30 query rows per kv head");
    return LW_OK;
}

lw_status scaled(float scale)
{
    if (!(scale > 0.0f) || !std::isfinite(scale)) return lw_fail(LW_E_ARG, "scale must be positive and finite");
    return LW_OK;
}

void grouped(const lw_kv_cache *c, int q_heads, KvAttend &a)
{
    a.group = q_heads / c->kv_heads;
    a.group_inv = ((1u << 21) + (unsigned)a.group - 1) / (unsigned)a.group;
}

lw_status few_pages(const lw_kv_batch *b)
{
    if (b->table_stride > KV_PICK_MOST)
        return lw_fail(LW_E_UNSUPPORTED, "more than 32768 pages per sequence (table_stride)");
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
    if ((st = heads(cache, n_tokens, dtype, q_heads)) || (st = scaled(scale))) return st;
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
    grouped(cache, q_heads, a);
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

// ------------------------------------------------------------------ rotary positions

extern "C" lw_status lw_rope(const lw_rope_plan *plan, const lw_kv_batch *batch, const int32_t *pos, int64_t n_tokens,
                             int n_heads, int head_dim, const lw_kv_tensor *x, int x_dtype, const lw_kv_tensor *y,
                             int y_dtype, void *stream)
{
    if (!plan) return lw_fail(LW_E_ARG, "null plan");
    if (plan->pairs < 1 || plan->pairs > LW_ROPE_MOST || (plan->layout != LW_ROPE_HALVES && plan->layout != LW_ROPE_PAIRS))
        return lw_fail(LW_E_ARG, "not a plan of lw_rope_make");
    if (!batch == !pos) return lw_fail(LW_E_ARG, "either a batch or positions");
    if (n_heads < 1 || n_heads > 65536) return lw_fail(LW_E_ARG, "heads must be in 1..65536");
    if (head_dim < 2 * plan->pairs || head_dim > 1024) return lw_fail(LW_E_ARG, "head_dim must be in 2 * pairs..1024");
    for (const int t : {x_dtype, y_dtype})
        if (t != LW_F16 && t != LW_BF16 && t != LW_F32) return lw_fail(LW_E_ARG, "unknown dtype");
    if (n_tokens < 0 || n_tokens > (1 << 26)) return lw_fail(LW_E_ARG, "n_tokens must be in 0..2^26");
    KvGeom g = {};
    g.n_tokens = (int32_t)n_tokens;
    lw_status st;
    if (batch && (st = sequences(batch, n_tokens, false, g))) return st;
    if (!n_tokens || (batch && !batch->n_seqs)) return LW_OK;
    if (!aligned(pos, 4)) return lw_fail(LW_E_ARG, "pos must be 4-byte aligned");
    KvTensor tx, ty;
    if ((st = tensor(x, "x", x_dtype, tx)) || (st = tensor(y, "y", y_dtype, ty))) return st;
    if ((n_tokens > 1 && !ty.token) || (n_heads > 1 && !ty.head)) return lw_fail(LW_E_ARG, "y overlaps itself");
    if (tx.data == ty.data && (x_dtype != y_dtype || tx.token != ty.token || tx.head != ty.head))
        return lw_fail(LW_E_ARG, "in place, x and y must have the same type and strides");
    return device(lw_launch_rope(*plan, g, pos, n_heads, head_dim, tx, x_dtype, ty, y_dtype, (hipStream_t)stream),
                  "rope launch");
}

// ------------------------------------------------------------------ a few pages of a long cache

extern "C" size_t lw_kv_bounds_bytes(int kv_heads, int head_dim)
{
    if (!kind_ok(kv_heads, head_dim, 32)) return 0;
    return ((size_t)kv_heads * (2 * head_dim + 4) + 15) / 16 * 16;
}

extern "C" lw_status lw_kv_bounds(const lw_kv_cache *cache, const lw_kv_batch *batch, int64_t n_tokens, void *bounds,
                                  void *stream)
{
    KvGeom g;
    const lw_status st = geom(cache, batch, n_tokens, g);
    if (st) return st;
    if (!batch->n_seqs || !n_tokens) return LW_OK;
    if (!bounds || !aligned(bounds, 16)) return lw_fail(LW_E_ARG, "bounds must be 16-byte aligned and not null");
    return device(lw_launch_kv_bounds(g, cache->head_dim, static_cast<uint8_t *>(bounds),
                                      (int64_t)lw_kv_bounds_bytes(cache->kv_heads, cache->head_dim), (hipStream_t)stream),
                  "kv bounds launch");
}

namespace {

lw_status selection(const lw_kv_cache *c, const lw_kv_selection *sel)
{
    if (!sel) return lw_fail(LW_E_ARG, "null selection");
    if (sel->n_tokens < 0 || sel->n_tokens > (1 << 26)) return lw_fail(LW_E_ARG, "n_tokens must be in 0..2^26");
    if (sel->pages < 1 || sel->pages > KV_PICK_MOST) return lw_fail(LW_E_ARG, "pages must be in 1..32768");
    if (sel->n_tokens && (!sel->start || !sel->lens || !sel->table)) return lw_fail(LW_E_ARG, "null argument");
    if (!aligned(sel->start, 4) || !aligned(sel->lens, 4) || !aligned(sel->table, 4))
        return lw_fail(LW_E_ARG, "start, lens and table must be 4-byte aligned");
    return LW_OK;
}

int64_t pages_of(const lw_kv_cache *c, const lw_kv_batch *b)
{
    return (longest(c, b) + c->page_tokens - 1) / c->page_tokens;
}

}  // namespace

namespace {

size_t select_bytes(const lw_kv_cache *c, const lw_kv_batch *b, int64_t n_tokens)
{
    if (!b->n_seqs || !lw_kv_select_shared(c->kv_heads, n_tokens, pages_of(c, b))) return 0;
    return (size_t)n_tokens * c->kv_heads * b->table_stride * sizeof(uint32_t);
}

}  // namespace

extern "C" size_t lw_kv_select_scratch_bytes(const lw_kv_cache *cache, const lw_kv_batch *batch, int64_t n_tokens,
                                             int q_heads)
{
    KvGeom g;
    if (geom(cache, batch, n_tokens, g) || heads(cache, n_tokens, LW_F16, q_heads) || few_pages(batch)) return 0;
    // (calls of more rows than that need none)
    return select_bytes(cache, batch, std::min<int64_t>(n_tokens, KV_SHARED_PAIRS / cache->kv_heads));
}

extern "C" lw_status lw_kv_select(const lw_kv_cache *cache, const lw_kv_batch *batch, const lw_kv_tensor *q, int dtype,
                                  int q_heads, const void *bounds, int first, int last, const lw_kv_selection *sel,
                                  void *work, size_t work_bytes, void *stream)
{
    KvSelect a;
    if (!cache) return lw_fail(LW_E_ARG, "null cache or batch");
    lw_status st = selection(cache, sel);
    if (st || (st = geom(cache, batch, sel->n_tokens, a.g)) || (st = heads(cache, sel->n_tokens, dtype, q_heads)) ||
        (st = few_pages(batch)))
        return st;
    if (first < 0 || last < 0 || (int64_t)first + last >= sel->pages)
        return lw_fail(LW_E_ARG, "first and last must not be negative, and together below the selection's pages");
    if (!sel->n_tokens) return LW_OK;
    if ((st = tensor(q, "q", dtype, a.q))) return st;
    if (!bounds || !aligned(bounds, 16)) return lw_fail(LW_E_ARG, "bounds must be 16-byte aligned and not null");
    if (!aligned(work, 4)) return lw_fail(LW_E_ARG, "work must be 4-byte aligned");
    const size_t need = select_bytes(cache, batch, sel->n_tokens);
    a.bounds = static_cast<const uint8_t *>(bounds);
    a.bounds_bytes = (int64_t)lw_kv_bounds_bytes(cache->kv_heads, cache->head_dim);
    a.group = q_heads / cache->kv_heads;
    a.first = first;
    a.last = last;
    a.take = (int32_t)sel->pages;
    a.start = sel->start;
    a.lens = sel->lens;
    a.table = sel->table;
    a.work = need && work && work_bytes >= need ? static_cast<uint32_t *>(work) : nullptr;
    return device(lw_launch_kv_select(a, cache->head_dim, dtype, pages_of(cache, batch), (hipStream_t)stream),
                  "kv select launch");
}

namespace {

// How selected rows are cut: rows a tile, row tiles, and a tile's chunks.
struct Chunks {
    int tile;
    int64_t tiles;
    int splits, chunk;
    size_t result;               // bytes of one's
};

// Chunks that a row tile is wanted in, of `tiles`: as many as two workgroups a CU
// hold (heads of 256 have registers for one), of 256 tokens at least, two steps of
// each wavefront.  One more than that, which leaves some CUs more workgroups than
// others, where chunks of 2048 tokens outweigh it.  With the bounds and the choice,
// rounded up, down and so: heads of 128, 480 workgroups of 1024 tokens 45.0, 40.2
// and 40.2 us, 288 of 4096 65.8, 71.3 and 65.8; heads of 256, 26 of 2368 (with
// chunks of 1024 at least) 37.6, 32.1 and 32.1, 144 of 4096 74.0, 77.7 and 74.0.
int64_t wanted_chunks(const lw_kv_cache *c, int64_t tiles, int64_t span)
{
    const int64_t groups = c->head_dim == 256 ? 256 : 512, base = std::max<int64_t>(tiles * c->kv_heads, 1);
    return std::max(std::min(std::max<int64_t>(groups / base, 1), (span + 255) / 256),
                    std::min((groups + base - 1) / base, span / 2048));
}

Chunks chunks_of(const lw_kv_cache *c, const lw_kv_selection *sel, int q_heads, size_t room)
{
    Chunks p;
    const int group = q_heads / c->kv_heads;
    const int64_t span = sel->pages * c->page_tokens;
    p.tile = group <= 8 ? 8 : 16;
    p.tiles = sel->n_tokens * ((group + p.tile - 1) / p.tile);
    p.result = (size_t)c->kv_heads * p.tile * (c->head_dim + 2) * sizeof(float);
    const int64_t fit = (int64_t)(room / p.result / std::max<int64_t>(p.tiles, 1));
    const int64_t splits = std::max<int64_t>(std::min(wanted_chunks(c, p.tiles, span), fit), 1);
    p.chunk = (int)(((span + splits - 1) / splits + 127) / 128 * 128);
    p.splits = (int)((span + p.chunk - 1) / p.chunk);
    return p;
}

}  // namespace

extern "C" size_t lw_kv_attend_selected_scratch_bytes(const lw_kv_cache *cache, const lw_kv_selection *sel, int q_heads)
{
    KvGeom g;
    if (!cache || selection(cache, sel) || pages(cache, false, g) || heads(cache, sel->n_tokens, LW_F16, q_heads)) return 0;
    // the most that as many rows or fewer, on as many pages or fewer, want
    const Chunks p = chunks_of(cache, sel, q_heads, 0);
    const int64_t per = sel->n_tokens ? p.tiles / sel->n_tokens : 1, span = sel->pages * cache->page_tokens;
    int64_t most = 0;
    for (int64_t n = 1; n <= sel->n_tokens; n++) {
        const int64_t splits = wanted_chunks(cache, n * per, span);
        if (splits <= 1) break;
        most = std::max(most, n * per * splits);
    }
    return most * p.result;
}

extern "C" lw_status lw_kv_attend_selected(const lw_kv_cache *cache, const lw_kv_selection *sel, const lw_kv_tensor *q,
                                           const lw_kv_tensor *out, int dtype, int q_heads, float scale, float *lse,
                                           void *work, size_t work_bytes, void *stream)
{
    KvAttend a = {};
    if (!cache) return lw_fail(LW_E_ARG, "null cache or batch");
    lw_status st = selection(cache, sel);
    if (st || (st = pages(cache, sel->n_tokens > 0, a.g)) || (st = heads(cache, sel->n_tokens, dtype, q_heads)) ||
        (st = scaled(scale)))
        return st;
    if (!sel->n_tokens) return LW_OK;
    if ((st = tensor(q, "q", dtype, a.q)) || (st = tensor(out, "out", dtype, a.out))) return st;
    if (!aligned(lse, 4)) return lw_fail(LW_E_ARG, "lse must be 4-byte aligned");
    if (!aligned(work, 16)) return lw_fail(LW_E_ARG, "work must be 16-byte aligned");
    const Chunks p = chunks_of(cache, sel, q_heads, work ? work_bytes : 0);
    if (p.tiles * p.splits > (1 << 30)) return lw_fail(LW_E_UNSUPPORTED, "more than 2^30 tiles of query rows");
    a.g.start = sel->start;
    a.g.lens = sel->lens;
    a.g.table = sel->table;
    a.g.stride = sel->pages;
    a.g.n_seqs = a.g.n_tokens = (int32_t)sel->n_tokens;
    a.lse = lse;
    a.part = static_cast<float *>(work);
    grouped(cache, q_heads, a);
    a.causal = 1;
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.pieces = (int32_t)(p.tiles * p.splits);
    a.slices = 1;
    a.scale = scale;
    return device(lw_launch_kv_selected(a, cache->head_dim, dtype, p.tile, (hipStream_t)stream), "kv attend launch");
}

// ------------------------------------------------------------------ pages given up

extern "C" lw_status lw_kv_weigh(const lw_kv_cache *cache, const lw_kv_batch *batch, int64_t n_tokens,
                                 const lw_kv_tensor *q, int dtype, int q_heads, float scale, int causal, int window,
                                 const float *lse, const float *before, float decay, float *weights, int64_t stride,
                                 void *stream)
{
    KvWeigh b = {};
    lw_status st = geom(cache, batch, n_tokens, b.a.g);
    if (st || (st = heads(cache, n_tokens, dtype, q_heads)) || (st = scaled(scale))) return st;
    if (window < 0) return lw_fail(LW_E_ARG, "negative window");
    if (!(decay >= 0.0f && decay <= 1.0f)) return lw_fail(LW_E_ARG, "decay must be in 0..1");
    if (stride < 0 || stride > (1 << 24)) return lw_fail(LW_E_ARG, "stride must be in 0..2^24");
    if (batch->n_seqs * stride > (1 << 27)) return lw_fail(LW_E_ARG, "weights of more than 2^27 pages");
    if (!batch->n_seqs || !n_tokens || !stride) return LW_OK;
    if ((st = tensor(q, "q", dtype, b.a.q))) return st;
    if (!lse || !weights || !aligned(lse, 4) || !aligned(before, 4) || !aligned(weights, 4))
        return lw_fail(LW_E_ARG, "lse, before and weights must be 4-byte aligned, lse and weights not null");
    grouped(cache, q_heads, b.a);
    b.a.causal = causal != 0;
    b.a.window = window;
    b.a.scale = scale;
    b.lse = lse;
    b.before = decay == 0.0f ? nullptr : before;
    b.decay = decay;
    b.weights = weights;
    b.stride = stride;
    return device(lw_launch_kv_weigh(b, cache->head_dim, dtype, (hipStream_t)stream), "kv weigh launch");
}

extern "C" lw_status lw_kv_evict(const lw_kv_cache *cache, const lw_kv_batch *batch, const float *weights, int64_t stride,
                                 int64_t keep, int first, int last, int32_t *table, int32_t *gone, int32_t *count,
                                 void *stream)
{
    KvEvict a = {};
    if (!cache || !batch) return lw_fail(LW_E_ARG, "null cache or batch");
    lw_status st = pages(cache, false, a.g);
    if (st || (st = sequences(batch, 0, false, a.g)) || (st = few_pages(batch))) return st;
    if (keep < 0 || first < 0) return lw_fail(LW_E_ARG, "keep and first must not be negative");
    if (last < 1) return lw_fail(LW_E_ARG, "last must be at least 1");
    if (stride < 0 || stride > (1 << 24)) return lw_fail(LW_E_ARG, "stride must be in 0..2^24");
    if (!batch->n_seqs) return LW_OK;
    if (!batch->lens || !count || (batch->table_stride && (!batch->table || !table || !gone)) || (stride && !weights))
        return lw_fail(LW_E_ARG, "null argument");
    for (const void *p : {(const void *)batch->lens, (const void *)batch->table, (const void *)weights,
                          (const void *)table, (const void *)gone, (const void *)count})
        if (!aligned(p, 4)) return lw_fail(LW_E_ARG, "the arrays must be 4-byte aligned");
    if (batch->table_stride && (gone == table || gone == batch->table))
        return lw_fail(LW_E_ARG, "gone must not be one of the tables");
    a.weights = weights;
    a.stride = stride;
    a.keep = keep;
    a.first = first;
    a.last = last;
    a.table = table;
    a.gone = gone;
    a.count = count;
    return device(lw_launch_kv_evict(a, (hipStream_t)stream), "kv evict launch");
}
