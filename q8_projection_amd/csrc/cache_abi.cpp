// cache_abi.cpp -- the C ABI of the key/value cache and its attention
// (q8_cache.h): argument validation, then the launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/q8_cache.h"
#include "cache.h"
#include "launch.h"
#include "ranges.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 20;
constexpr int64_t kMaxSequences = int64_t(1) << 16;
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxLd = int64_t(1) << 40;
constexpr int64_t kMaxValues = int64_t(1) << 40;  // sequences * max_rows * heads * head_dim
constexpr int64_t kMaxHeads = 4096;

q8_status check_format(const q8_cache *c) {
    if (!c) return Q8_E_NULL;
    if (c->bits != 4 && c->bits != 8) return Q8_E_MODE;
    if (c->kv_heads < 1 || c->kv_heads > 256) return Q8_E_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return Q8_E_SHAPE;
    if (c->page_tokens < q8::kTileTokens || c->page_tokens > 4096 || (c->page_tokens & (c->page_tokens - 1)))
        return Q8_E_SHAPE;
    return Q8_OK;
}

// Sizes of a call of `heads` heads a row.
q8_status check_sizes(const q8_cache *c, const q8_cache_batch *b, int64_t heads) {
    if (q8_status s = check_format(c); s != Q8_OK) return s;
    if (!b) return Q8_E_NULL;
    if (c->pages < 1 || c->pages > INT32_MAX) return Q8_E_SHAPE;
    if (b->sequences < 0 || b->sequences > kMaxSequences || b->rows < 0 || b->rows > kMaxRows || b->max_rows < 1)
        return Q8_E_SHAPE;
    if (b->table_ld < 1 || b->table_ld > kMaxTokens / c->page_tokens) return Q8_E_SHAPE;
    if (!b->starts && b->rows != b->sequences) return Q8_E_SHAPE;
    if (heads < 1 || heads > kMaxHeads || heads % c->kv_heads) return Q8_E_SHAPE;
    const int64_t most = std::min(b->max_rows, b->rows);
    if (b->sequences * most > kMaxValues / (heads * c->head_dim)) return Q8_E_SHAPE;
    return Q8_OK;
}

q8_status check_pointers(const q8_cache *c, const q8_cache_batch *b) {
    if (!c->data || !b->table || !b->lens) return Q8_E_NULL;
    if (!q8::aligned_to(c->data, 16) || !q8::aligned_to(b->table, 4) || !q8::aligned_to(b->lens, 4) ||
        !q8::aligned_to(b->starts, 4))
        return Q8_E_ALIGN;
    return Q8_OK;
}

bool bad_ld(int64_t ld, int64_t row) { return ld < row || ld > kMaxLd || ld % 4; }

int log2_of(int v) {
    int n = 0;
    while ((1 << n) < v) ++n;
    return n;
}

q8::CacheArgs args_of(const q8_cache *c, const q8_cache_batch *b) {
    q8::CacheArgs a = {};
    a.data = static_cast<uint8_t *>(c->data);
    a.pages = c->pages;
    a.kv_heads = c->kv_heads;
    a.page_shift = log2_of(c->page_tokens);
    a.sequences = static_cast<int>(b->sequences);
    a.table_ld = b->table_ld;
    a.table = b->table;
    a.lens = b->lens;
    a.starts = b->starts;
    a.rows = static_cast<int>(b->rows);
    a.max_rows = static_cast<int>(std::min(b->max_rows, b->rows));
    return a;
}

bool few(const q8::AttentionArgs &a, int64_t dim) {
    return int64_t(a.c.max_rows) * a.group <= q8::few_rows(static_cast<int>(dim));
}

q8::Range pool_range(const q8_cache *c) { return {c->data, c->pages * q8_cache_page_bytes(c)}; }

// Whether `out` overlaps what a call reads beside its rows: the table, the lengths and the starts.
bool overlaps_batch(const q8::Range &out, const q8_cache_batch *b) {
    return q8::overlaps(out, {b->table, b->sequences * b->table_ld * 4}) ||
           q8::overlaps(out, {b->lens, b->sequences * 4}) || q8::overlaps(out, {b->starts, (b->sequences + 1) * 4});
}

}  // namespace

int64_t q8::attention_counter_bytes() { return (int64_t(kCountersPerCu) * device_info().cus * 4 + 255) / 256 * 256; }

extern "C" {

int64_t q8_cache_page_bytes(const q8_cache *cache) {
    if (check_format(cache) != Q8_OK) return 0;
    return q8::tile_bytes(cache->bits, cache->head_dim) * cache->kv_heads * (cache->page_tokens / q8::kTileTokens);
}

q8_status q8_cache_append(const q8_cache *cache, const q8_cache_batch *batch, const float *k, int64_t k_ld,
                          const float *v, int64_t v_ld, void *stream) {
    if (q8_status s = check_sizes(cache, batch, cache ? cache->kv_heads : 1); s != Q8_OK) return s;
    const int64_t row = int64_t(cache->kv_heads) * cache->head_dim, rows = batch->rows;
    if (bad_ld(k_ld, row) || bad_ld(v_ld, row)) return Q8_E_SHAPE;
    if (rows == 0 || batch->sequences == 0) return Q8_OK;
    if (!k || !v) return Q8_E_NULL;
    if (q8_status s = check_pointers(cache, batch); s != Q8_OK) return s;
    if (!q8::aligned_to(k, 16) || !q8::aligned_to(v, 16)) return Q8_E_ALIGN;
    const q8::Range pool = pool_range(cache);
    if (q8::overlaps(pool, {k, ((rows - 1) * k_ld + row) * 4}) || q8::overlaps(pool, {v, ((rows - 1) * v_ld + row) * 4}) ||
        overlaps_batch(pool, batch))
        return Q8_E_ALIAS;
    const q8::AppendArgs a = {args_of(cache, batch), k, v, k_ld, v_ld};
    return q8::launch_cache_append(cache->bits, cache->head_dim, a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Q8_OK
               : Q8_E_HIP;
}

q8_status q8_cache_read(const q8_cache *cache, const q8_cache_batch *batch, float *k, float *v, void *stream) {
    if (q8_status s = check_sizes(cache, batch, cache ? cache->kv_heads : 1); s != Q8_OK) return s;
    if (batch->rows == 0 || batch->sequences == 0) return Q8_OK;
    if (!k || !v) return Q8_E_NULL;
    if (q8_status s = check_pointers(cache, batch); s != Q8_OK) return s;
    if (!q8::aligned_to(k, 16) || !q8::aligned_to(v, 16)) return Q8_E_ALIGN;
    const int64_t bytes = batch->rows * cache->kv_heads * cache->head_dim * 4;
    const q8::Range pool = pool_range(cache), rk{k, bytes}, rv{v, bytes};
    if (q8::overlaps(rk, rv)) return Q8_E_ALIAS;
    for (const q8::Range &out : {rk, rv})
        if (q8::overlaps(out, pool) || overlaps_batch(out, batch)) return Q8_E_ALIAS;
    const q8::ReadArgs a = {args_of(cache, batch), k, v};
    return q8::launch_cache_read(cache->bits, cache->head_dim, a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Q8_OK
               : Q8_E_HIP;
}

int64_t q8_attention_workspace_bytes(const q8_cache *cache, const q8_cache_batch *batch, int64_t heads) {
    if (check_sizes(cache, batch, heads) != Q8_OK) return 0;
    q8::AttentionArgs a = {};
    a.c = args_of(cache, batch);
    a.heads = static_cast<int>(heads);
    a.group = a.heads / a.c.kv_heads;
    const int dim = cache->head_dim;
    if (few(a, dim)) return q8::few_workspace(dim, a);
    // as large as for any call of few rows, so that the largest call's serves them too
    a.c.max_rows = q8::few_rows(dim);
    a.group = 1;
    return std::max(q8::few_workspace(dim, a), q8::rows_workspace(dim));
}

q8_status q8_attention(const q8_cache *cache, const q8_cache_batch *batch, const float *q, int64_t q_ld,
                       int64_t heads, float scale, int64_t window, float *out, float *lse, void *workspace,
                       int64_t workspace_bytes, void *stream) {
    if (q8_status s = check_sizes(cache, batch, heads); s != Q8_OK) return s;
    const int64_t row = heads * cache->head_dim, rows = batch->rows;
    if (bad_ld(q_ld, row) || window < 0 || window > INT32_MAX) return Q8_E_SHAPE;
    if (rows == 0 || batch->sequences == 0) return Q8_OK;
    if (!q || !out || !workspace) return Q8_E_NULL;
    if (q8_status s = check_pointers(cache, batch); s != Q8_OK) return s;
    if (!q8::aligned_to(q, 16) || !q8::aligned_to(out, 16) || !q8::aligned_to(lse, 4) || !q8::aligned_to(workspace, 16))
        return Q8_E_ALIGN;
    const int64_t need = q8_attention_workspace_bytes(cache, batch, heads);
    if (workspace_bytes < need) return Q8_E_SHAPE;
    const q8::Range outs[] = {{out, rows * row * 4}, {lse, rows * heads * 4}, {workspace, need}};
    const q8::Range pool = pool_range(cache), rq{q, ((rows - 1) * q_ld + row) * 4};
    for (int i = 0; i < 3; ++i) {
        if (q8::overlaps(outs[i], pool) || q8::overlaps(outs[i], rq) || overlaps_batch(outs[i], batch)) return Q8_E_ALIAS;
        for (int j = 0; j < i; ++j)
            if (q8::overlaps(outs[i], outs[j])) return Q8_E_ALIAS;
    }
    q8::AttentionArgs a = {};
    a.c = args_of(cache, batch);
    a.q = q;
    a.q_ld = q_ld;
    a.heads = static_cast<int>(heads);
    a.group = a.heads / a.c.kv_heads;
    a.scale = scale;
    // (a window as long as a sequence can be hides nothing; the kernels' at - window, from at >= -kMaxRows on, keeps within 32 bits)
    a.window = window < kMaxTokens ? static_cast<int>(window) : 0;
    a.out = out;
    a.lse = lse;
    const auto launch = few(a, cache->head_dim) ? q8::launch_few : q8::launch_rows;
    return launch(cache->bits, cache->head_dim, a, workspace, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? Q8_OK
                                                                                                                 : Q8_E_HIP;
}

}  // extern "C"
