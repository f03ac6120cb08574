// C ABI of the rotary positions, the paged key-value cache, the attention over it
// and the calls for long contexts (declared in include/w4.h): argument checks on the
// host, then the launches.  Nothing here allocates device or pinned memory.
#include <math.h>

#include <atomic>

#include "w4_kv.cuh"

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

w4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? W4_OK : W4_ERR_CUDA; }

// SM count of the current device, cached per device (see w4_api.cu).
int device_sms() {
    static std::atomic<int> cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev >= 0 && dev < 64) {
        const int c = cached[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return -1;
    if (dev >= 0 && dev < 64) cached[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

w4::Heads heads_of(const w4_heads *h) {
    if (!h) return {nullptr, 0, 0};
    return {static_cast<char *>(h->data), h->token_stride, h->head_stride};
}

// Rows of `size`-byte elements that start on 16-byte boundaries.
bool rows_aligned(const w4_heads *h, int size) {
    return aligned(h->data, 16) && h->token_stride * size % 16 == 0 &&
           h->head_stride * size % 16 == 0;
}

bool rotation_ok(const w4_rotation *r, int head_dim) {
    return r->table && aligned(r->table, 16) && r->rows >= 1 && r->rotary_dim >= 2 &&
           r->rotary_dim % 2 == 0 && r->rotary_dim <= head_dim &&
           (r->layout == W4_ROPE_HALF || r->layout == W4_ROPE_INTERLEAVED);
}

w4_status cache_ok(const w4_kv_cache *c, bool with_pool) {
    if (!c) return W4_ERR_INVALID_ARG;
    if (c->format != W4_KV_BF16 && c->format != W4_KV_INT8 && c->format != W4_KV_INT4)
        return W4_ERR_INVALID_ARG;
    if (c->kv_heads < 1 || c->kv_heads > 65535 || c->pages < 1 || c->page_tokens < 1 ||
        c->page_tokens % w4::kRecTokens || c->page_tokens > (1 << 20))
        return W4_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return W4_ERR_UNSUPPORTED;
    if (with_pool && (!c->pool || !aligned(c->pool, 128) || !aligned(c->error, 4)))
        return W4_ERR_INVALID_ARG;
    return W4_OK;
}

bool table_ok(const w4_block_table *t) {
    return t && t->pages && aligned(t->pages, 4) && t->seqs >= 1 && t->width >= 1 &&
           t->stride >= t->width;
}

w4::KvPool pool_of(const w4_kv_cache *c, const w4_block_table *t) {
    w4::KvPool p;
    p.records = static_cast<char *>(c->pool);
    p.kv_heads = c->kv_heads;
    p.page_records = c->page_tokens / w4::kRecTokens;
    p.page_shift = -1;
    for (int s = 0; s < 17; ++s)
        if (p.page_records == 1 << s) p.page_shift = s;
    p.page_tokens = c->page_tokens;
    p.pages = c->pages;
    p.error = c->error;
    p.table = t->pages;
    p.seqs = t->seqs;
    p.width = t->width;
    p.stride = t->stride;
    return p;
}

// The arguments that w4_kv_append and w4_kv_read share.
w4_status list_ok(const w4_kv_cache *cache, const w4_block_table *table, int tokens,
                  const int32_t *positions, const int32_t *seq_ids, int heads) {
    const w4_status st = cache_ok(cache, true);
    if (st != W4_OK) return st;
    if (!table_ok(table) || tokens < 0) return W4_ERR_INVALID_ARG;
    if (tokens > 0 && (!positions || !aligned(positions, 4) || !aligned(seq_ids, 4)))
        return W4_ERR_INVALID_ARG;
    if (!seq_ids && tokens % table->seqs) return W4_ERR_INVALID_ARG;
    // (query units, 16 a head at most, are counted in 32 bits)
    if ((long long)tokens * heads >= (1LL << 27)) return W4_ERR_UNSUPPORTED;
    return W4_OK;
}

// Queries that meet a cache: the new tokens of every sequence.
w4_status queries_ok(const w4_kv_cache *cache, const w4_heads *q, int q_heads, int tokens,
                     const w4_block_table *table) {
    if (!q || !q->data) return W4_ERR_INVALID_ARG;
    if (tokens < 1 || tokens > W4_MAX_TOKENS) return W4_ERR_UNSUPPORTED;
    if (q_heads < 1 || q_heads % cache->kv_heads) return W4_ERR_INVALID_ARG;
    if (q_heads / cache->kv_heads > 4096) return W4_ERR_UNSUPPORTED;
    if (!rows_aligned(q, 2)) return W4_ERR_INVALID_ARG;
    return (long long)table->seqs * q_heads * tokens < (1LL << 31) ? W4_OK : W4_ERR_UNSUPPORTED;
}

// The cache, its table and the lengths of a call that walks all sequences: what
// it counts in 32 bits are a sequence's tokens, to which kernels add a page (2^20
// tokens at most) or a unit of records, and records of all heads.
w4_status walk_ok(const w4_kv_cache *cache, const w4_block_table *table, const int32_t *lens) {
    const w4_status st = cache_ok(cache, true);
    if (st != W4_OK) return st;
    if (!table_ok(table) || !lens || !aligned(lens, 4)) return W4_ERR_INVALID_ARG;
    const long long room = (long long)table->width * cache->page_tokens;
    if (room > (1LL << 31) - (1 << 21) || (room / w4::kRecTokens * table->seqs) >= (1LL << 31) ||
        room / w4::kRecTokens * table->seqs * cache->kv_heads >= (1LL << 31))
        return W4_ERR_UNSUPPORTED;
    return W4_OK;
}

unsigned magic_of(int group) { return group > 1 ? 0xFFFFFFFFu / (unsigned)group + 1 : 0; }

w4_status paged_attn_common(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                            int q_heads, int tokens, const int32_t *lens,
                            const w4_block_table *table, const int32_t *blocks,
                            const int32_t *counts, int most, float scale, int window, float *lse,
                            void *workspace, size_t workspace_bytes, bool f32_out,
                            w4_stream_t stream) {
    const w4_status st = cache_ok(cache, true);
    if (st != W4_OK) return st;
    if (!table_ok(table) || !q || !out || !q->data || !out->data || !lens || !workspace)
        return W4_ERR_INVALID_ARG;
    if (tokens < 1 || tokens > W4_MAX_TOKENS) return W4_ERR_UNSUPPORTED;
    if (q_heads < 1 || q_heads % cache->kv_heads || window < 0 || !isfinite(scale))
        return W4_ERR_INVALID_ARG;
    if (q_heads / cache->kv_heads > 4096) return W4_ERR_UNSUPPORTED;
    if (!rows_aligned(q, 2) || !rows_aligned(out, f32_out ? 4 : 2) || !aligned(lens, 4) ||
        !aligned(lse, 4) || !aligned(workspace, 256))
        return W4_ERR_INVALID_ARG;
    if ((long long)table->width * cache->page_tokens > w4::kAbsent ||
        (long long)table->seqs * q_heads * tokens >= (1LL << 31))
        return W4_ERR_UNSUPPORTED;
    // records that the call could visit, counted in 32 bits (a head costs up to
    // 128 records more)
    const long long row_tiles = ((long long)tokens * (q_heads / cache->kv_heads) + 63) / 64;
    const long long longest =
        (long long)(blocks && most > table->width ? most : table->width) *
            (cache->page_tokens / w4::kRecTokens) + 128;
    if (longest * table->seqs >= (1LL << 31) ||
        longest * table->seqs * cache->kv_heads >= (1LL << 31) ||
        longest * table->seqs * cache->kv_heads * row_tiles >= (1LL << 31))
        return W4_ERR_UNSUPPORTED;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    if (workspace_bytes < w4::attn_workspace_bytes(cache->head_dim, sms))
        return W4_ERR_INVALID_ARG;
    w4::AttnArgs a;
    a.pool = pool_of(cache, table);
    a.q = heads_of(q);
    a.out = heads_of(out);
    a.lse = lse;
    a.f32_out = f32_out;
    a.lens = lens;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.group_magic = magic_of(a.group);
    a.tokens = tokens;
    a.scale = scale;
    // a window as wide as the longest sequence leaves nothing out (and so the
    // kernels may subtract one from a position of a token that is not there)
    a.window = window < table->width * cache->page_tokens ? window : 0;
    a.blocks = blocks;
    a.counts = counts;
    a.most = most;
    a.workspace = workspace;
    return cuda_status(w4::launch_paged_attn(a, cache->format, cache->head_dim, sms,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

w4_status sparse_attn_common(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                             int q_heads, int tokens, const int32_t *lens,
                             const w4_block_table *table, const int32_t *blocks,
                             const int32_t *counts, int most, float scale, float *lse,
                             void *workspace, size_t workspace_bytes, bool f32_out,
                             w4_stream_t stream) {
    if (!blocks || !counts || !aligned(blocks, 4) || !aligned(counts, 4) || most < 1)
        return W4_ERR_INVALID_ARG;
    return paged_attn_common(cache, q, out, q_heads, tokens, lens, table, blocks, counts, most,
                             scale, 0, lse, workspace, workspace_bytes, f32_out, stream);
}

}  // namespace

extern "C" {

w4_status w4_rope_table(const w4_rope_spec *spec, int rows, float *table, w4_stream_t stream) {
    if (!spec || !table || !aligned(table, 16) || rows < 1) return W4_ERR_INVALID_ARG;
    const int rot = spec->rotary_dim;
    if (rot < 2 || rot > 512 || rot % 2) return W4_ERR_INVALID_ARG;
    const double factor = spec->scaling == W4_ROPE_SCALE_NONE ? 1.0 : spec->factor;
    if (!(spec->base > 0) || !isfinite(spec->base) || !(factor > 0) || !isfinite(factor) ||
        !isfinite(spec->amplitude))
        return W4_ERR_INVALID_ARG;
    double base = spec->base;
    switch (spec->scaling) {
        case W4_ROPE_SCALE_NONE:
        case W4_ROPE_SCALE_LINEAR: break;
        case W4_ROPE_SCALE_BASE:
            if (rot > 2) base *= pow(factor, (double)rot / (rot - 2));
            break;
        case W4_ROPE_SCALE_PARTS:
            if (!(spec->original_context > 0) || !isfinite(spec->original_context) ||
                !(spec->low_turns < spec->high_turns) || !isfinite(spec->low_turns) ||
                !isfinite(spec->high_turns))
                return W4_ERR_INVALID_ARG;
            break;
        default: return W4_ERR_INVALID_ARG;
    }
    if (!isfinite(base)) return W4_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    unsigned long long turns[256];
    for (int i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * i / rot) / two_pi;    // turns per position
        if (spec->scaling == W4_ROPE_SCALE_LINEAR) {
            f /= factor;
        } else if (spec->scaling == W4_ROPE_SCALE_PARTS) {
            const double made = spec->original_context * f;
            double keep = (made - spec->low_turns) / (spec->high_turns - spec->low_turns);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f = f * (keep + (1 - keep) / factor);
        }
        if (!isfinite(f)) return W4_ERR_INVALID_ARG;
        f -= floor(f);                                    // whole turns change nothing
        const double scaled = ldexp(f, 64);
        turns[i] = scaled >= 18446744073709551615.0 ? 0ull : (unsigned long long)scaled;
    }
    return cuda_status(w4::launch_rope_table(turns, rot / 2, spec->amplitude, rows, table,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

w4_status w4_rope(const w4_heads *x, const w4_heads *y, int tokens, int heads, int head_dim,
                  const int32_t *positions, const w4_rotation *rotation, uint32_t *error,
                  w4_stream_t stream) {
    if (!x || !y || !rotation || tokens < 0 || heads < 1 || head_dim < 1 || head_dim > 1024)
        return W4_ERR_INVALID_ARG;
    if (!rotation_ok(rotation, head_dim) || !aligned(error, 4)) return W4_ERR_INVALID_ARG;
    if (tokens == 0) return W4_OK;
    if (!x->data || !y->data || !positions || !aligned(x->data, 2) || !aligned(y->data, 2) ||
        !aligned(positions, 4))
        return W4_ERR_INVALID_ARG;
    if ((long long)tokens * heads >= (1LL << 31)) return W4_ERR_UNSUPPORTED;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    const bool wide = rows_aligned(x, 2) && rows_aligned(y, 2) && head_dim % 8 == 0 &&
                      rotation->rotary_dim % 16 == 0;
    const w4::Rotation rot = {rotation->table, rotation->rows, rotation->rotary_dim / 2,
                              rotation->layout};
    return cuda_status(w4::launch_rope(heads_of(x), heads_of(y), tokens, heads, head_dim,
                                       positions, rot, error, wide, sms,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

w4_status w4_kv_pool_bytes(const w4_kv_cache *cache, size_t *bytes) {
    const w4_status st = cache_ok(cache, false);
    if (st != W4_OK) return st;
    if (!bytes) return W4_ERR_INVALID_ARG;
    *bytes = (size_t)cache->pages * cache->kv_heads * (cache->page_tokens / w4::kRecTokens) *
             w4::kv_record_bytes(cache->format, cache->head_dim);
    return W4_OK;
}

w4_status w4_kv_append(const w4_kv_cache *cache, const w4_heads *k, const w4_heads *v,
                       const w4_heads *q, const w4_heads *q_out, int q_heads, int tokens,
                       const int32_t *positions, const int32_t *seq_ids,
                       const w4_block_table *table, const w4_rotation *rotation,
                       w4_stream_t stream) {
    if (!q != !q_out || (q && q_heads < 1)) return W4_ERR_INVALID_ARG;
    // (in place and without a rotation there is nothing to do with q)
    if (!q || (!rotation && w4::same_place(heads_of(q), heads_of(q_out)))) q_heads = 0;
    const w4_status st = list_ok(cache, table, tokens, positions, seq_ids,
                                 2 * (cache ? cache->kv_heads : 0) + q_heads);
    if (st != W4_OK) return st;
    if (rotation &&
        (!rotation_ok(rotation, cache->head_dim) || rotation->rotary_dim % 16 != 0))
        return W4_ERR_INVALID_ARG;
    if (!k || !v) return W4_ERR_INVALID_ARG;
    if (tokens == 0) return W4_OK;
    if (!k->data || !v->data || !rows_aligned(k, 2) || !rows_aligned(v, 2))
        return W4_ERR_INVALID_ARG;
    if (q_heads > 0 && (!q->data || !q_out->data || !rows_aligned(q, 2) ||
                        !rows_aligned(q_out, 2)))
        return W4_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    w4::Rotation rot = {nullptr, 0, 0, W4_ROPE_HALF};
    if (rotation)
        rot = {rotation->table, rotation->rows, rotation->rotary_dim / 2, rotation->layout};
    const w4::TokenList list = {positions, seq_ids, tokens,
                                seq_ids ? tokens : tokens / table->seqs};
    return cuda_status(w4::launch_kv_append(
        pool_of(cache, table), cache->format, cache->head_dim, heads_of(k), heads_of(v),
        heads_of(q), heads_of(q_out), q_heads, list, rot, sms,
        reinterpret_cast<cudaStream_t>(stream)));
}

w4_status w4_kv_read(const w4_kv_cache *cache, const w4_heads *k_out, const w4_heads *v_out,
                     int tokens, const int32_t *positions, const int32_t *seq_ids,
                     const w4_block_table *table, w4_stream_t stream) {
    const w4_status st = list_ok(cache, table, tokens, positions, seq_ids,
                                 2 * (cache ? cache->kv_heads : 0));
    if (st != W4_OK) return st;
    if (!k_out && !v_out) return W4_ERR_INVALID_ARG;
    if (tokens == 0) return W4_OK;
    for (const w4_heads *h : {k_out, v_out})
        if (h && (!h->data || !rows_aligned(h, 2))) return W4_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    const w4::TokenList list = {positions, seq_ids, tokens,
                                seq_ids ? tokens : tokens / table->seqs};
    return cuda_status(w4::launch_kv_read(pool_of(cache, table), cache->format, cache->head_dim,
                                          heads_of(k_out), heads_of(v_out), list, sms,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

w4_status w4_paged_attn_workspace_bytes(const w4_kv_cache *cache, size_t *bytes) {
    const w4_status st = cache_ok(cache, false);
    if (st != W4_OK) return st;
    if (!bytes) return W4_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    *bytes = w4::attn_workspace_bytes(cache->head_dim, sms);
    return W4_OK;
}

w4_status w4_paged_attn(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                        int q_heads, int tokens, const int32_t *lens,
                        const w4_block_table *table, float scale, int window, float *lse,
                        void *workspace, size_t workspace_bytes, w4_stream_t stream) {
    return paged_attn_common(cache, q, out, q_heads, tokens, lens, table, nullptr, nullptr, 0,
                             scale, window, lse, workspace, workspace_bytes, false, stream);
}

w4_status w4_paged_attn_f32(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                            int q_heads, int tokens, const int32_t *lens,
                            const w4_block_table *table, float scale, int window, float *lse,
                            void *workspace, size_t workspace_bytes, w4_stream_t stream) {
    return paged_attn_common(cache, q, out, q_heads, tokens, lens, table, nullptr, nullptr, 0,
                             scale, window, lse, workspace, workspace_bytes, true, stream);
}

w4_status w4_key_bounds(const w4_kv_cache *cache, uint16_t *bounds, int tokens,
                        const int32_t *lens, const w4_block_table *table, w4_stream_t stream) {
    const w4_status st = walk_ok(cache, table, lens);
    if (st != W4_OK) return st;
    if (!bounds || !aligned(bounds, 16) || tokens < 1) return W4_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    return cuda_status(w4::launch_key_bounds(pool_of(cache, table), cache->format,
                                             cache->head_dim, bounds, tokens, lens, sms,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

w4_status w4_block_scores(const w4_kv_cache *cache, const uint16_t *bounds, const w4_heads *q,
                          int q_heads, int tokens, const int32_t *lens,
                          const w4_block_table *table, float *scores, int columns,
                          w4_stream_t stream) {
    w4_status st = walk_ok(cache, table, lens);
    if (st == W4_OK) st = queries_ok(cache, q, q_heads, tokens, table);
    if (st != W4_OK) return st;
    if (!bounds || !aligned(bounds, 16) || !scores || !aligned(scores, 4) ||
        columns < table->width)
        return W4_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    const int group = q_heads / cache->kv_heads;
    return cuda_status(w4::launch_block_scores(
        pool_of(cache, table), cache->head_dim, bounds, heads_of(q), group, magic_of(group),
        tokens, lens, scores, columns, sms, reinterpret_cast<cudaStream_t>(stream)));
}

w4_status w4_select(const float *scores, int seqs, int heads, int columns, const int32_t *lens,
                    int unit, int first, int last, int count, int32_t *index, int32_t *counts,
                    w4_stream_t stream) {
    if (seqs < 1 || heads < 1 || columns < 1 || unit < 1 || first < 0 || last < 0 || count < 1 ||
        (long long)first + last > count)
        return W4_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(scores), static_cast<const void *>(lens),
                          static_cast<const void *>(index), static_cast<const void *>(counts)})
        if (!p || !aligned(p, 4)) return W4_ERR_INVALID_ARG;
    if ((long long)seqs * heads >= (1LL << 27) || columns >= (1 << 30)) return W4_ERR_UNSUPPORTED;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    return cuda_status(w4::launch_select(scores, seqs, heads, columns, lens, unit, first, last,
                                         count, index, counts, sms,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

w4_status w4_sparse_attn(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                         int q_heads, int tokens, const int32_t *lens,
                         const w4_block_table *table, const int32_t *blocks,
                         const int32_t *counts, int most, float scale, float *lse,
                         void *workspace, size_t workspace_bytes, w4_stream_t stream) {
    return sparse_attn_common(cache, q, out, q_heads, tokens, lens, table, blocks, counts, most,
                              scale, lse, workspace, workspace_bytes, false, stream);
}

w4_status w4_sparse_attn_f32(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                             int q_heads, int tokens, const int32_t *lens,
                             const w4_block_table *table, const int32_t *blocks,
                             const int32_t *counts, int most, float scale, float *lse,
                             void *workspace, size_t workspace_bytes, w4_stream_t stream) {
    return sparse_attn_common(cache, q, out, q_heads, tokens, lens, table, blocks, counts, most,
                              scale, lse, workspace, workspace_bytes, true, stream);
}

w4_status w4_attn_weights(const w4_kv_cache *cache, const w4_heads *q, const float *lse,
                          int q_heads, int tokens, const int32_t *lens,
                          const w4_block_table *table, float scale, int window,
                          const float *before, float decay, float *weights, int columns,
                          w4_stream_t stream) {
    w4_status st = walk_ok(cache, table, lens);
    if (st == W4_OK) st = queries_ok(cache, q, q_heads, tokens, table);
    if (st != W4_OK) return st;
    if (!lse || !weights || !aligned(lse, 4) || !aligned(before, 4) || !aligned(weights, 4) ||
        !isfinite(scale) || !isfinite(decay) || window < 0 || columns < 1)
        return W4_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    const int room = table->width * cache->page_tokens;
    w4::AttnArgs a = {};
    a.pool = pool_of(cache, table);
    a.q = heads_of(q);
    a.lse = const_cast<float *>(lse);
    a.lens = lens;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.group_magic = magic_of(a.group);
    a.tokens = tokens;
    a.scale = scale;
    a.window = window < room ? window : 0;
    a.most = columns < room ? columns : room;
    return cuda_status(w4::launch_attn_weights(a, cache->format, cache->head_dim, before, decay,
                                               weights, columns, sms,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

w4_status w4_kv_gather(const w4_kv_cache *cache, const w4_block_table *table,
                       const int32_t *lens, const int32_t *index, const int32_t *counts, int most,
                       const w4_block_table *to, const float *weights, int columns,
                       float *weights_out, int columns_out, w4_stream_t stream) {
    w4_status st = walk_ok(cache, table, lens);
    if (st == W4_OK) st = walk_ok(cache, to, lens);
    if (st != W4_OK) return st;
    if (!index || !counts || !aligned(index, 4) || !aligned(counts, 4) || most < 1 ||
        to->seqs != table->seqs || to->pages == table->pages)
        return W4_ERR_INVALID_ARG;
    if (!weights != !weights_out || !aligned(weights, 4) || !aligned(weights_out, 4) ||
        (weights && (columns < 1 || columns_out < most || weights == weights_out)))
        return W4_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return W4_ERR_CUDA;
    return cuda_status(w4::launch_kv_gather(pool_of(cache, table), pool_of(cache, to),
                                            cache->format, cache->head_dim, lens, index, counts,
                                            most, weights, columns, weights_out, columns_out, sms,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
