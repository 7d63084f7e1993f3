/*
 * q8_cache.h -- C ABI of libq8proj.so, the step of a decode step between the
 * Q8_0 projections of q8.h that make q, k and v and the one that takes the heads'
 * outputs: a paged cache of keys and values in 4 or 8 bits, written as it is
 * quantized and read back, and the attention that reads it (logicaffeine_compile,
 * codegen_cuda::lane page, Modules, kernels: a result written into the row of a
 * cache a position names; model::author page, Functions: attention over the cache
 * in decode, batch and prefill steps).
 *
 * The conventions are those of q8.h: caller-owned device memory, work enqueued
 * on `stream` and nothing else (no allocation, no synchronization, no device
 * read on the host), every argument checked before anything is enqueued, named
 * statuses.  Every call may be captured into a HIP graph; lengths, pages and rows
 * are read on the device, so a replayed call takes what is there then.
 */
#ifndef Q8PROJ_Q8_CACHE_H
#define Q8PROJ_Q8_CACHE_H

#include "q8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * The cache
 *
 * A pool of pages, each of page_tokens tokens of one layer: key and value of every
 * kv head.  A head's 32 consecutive dimensions of one token are a block, with one
 * 16-bit word and 32 codes.  What a block of values x_j stands for in the cache
 * (rint rounds half to even, every quotient is of the exact numbers):
 *
 *   4 bits: lo = min(0, min x), hi = max(0, max x)
 *           d  the smallest binary16 number with the low 5 bits of its pattern
 *              clear and 15 d >= hi - lo, at most 4352
 *           z  = min(15, rint(-lo / d)),  n_j = clamp(rint(x_j / d) + z, 0, 15)
 *           value d (n_j - z); the word is d's pattern with z in its low 4 bits
 *   8 bits: d  the smallest binary16 number with the low 7 bits of its pattern
 *              clear and 127 d >= max |x|, at most 512
 *           n_j = clamp(rint(x_j / d), -127, 127)
 *           value d n_j; the code is n_j + 128, the word is d's pattern
 *
 * A block of zeros has d = 0 and values 0.  Values are off by at most d/2, and
 * beyond 65280 (4 bits) or 65024 (8 bits) they saturate.  Every value is a binary16
 * number, exactly: the scales are kept that short for it, so that the matrix cores
 * take the cache's side of a product as it is.
 *
 * Layout of a page, page_tokens / 32 tiles of 32 tokens for each kv head,
 * [kv_heads][page_tokens / 32][tile].  With t the token in its tile, D = head_dim,
 * a = t / 8, b = t % 4, i = t % 8 / 4, a tile is, one after the other,
 *   key codes   [32 t][D], a byte each or two to a byte, the lower dimension in the
 *               low half
 *   key words   [4 a][4 b][D / 32][2 i], 16 bits each
 *   value codes 4 bits: [D / 64][4 a][16][4][8], code of dimension 64 u + 16 w + c at
 *               [u][a][c][w][t % 8], two to a byte, the lower token in the low half
 *               8 bits: [D / 32][4 a][16][2][4 b][2 i], dimension 32 u + 16 w + c at
 *               [u][a][c][w][b][i]
 *   value words [D / 32][4 a][4 b][2 i]
 * (what a lane of the attention's kernels takes lies together).  A pool needs no
 * initial contents.
 * ------------------------------------------------------------------------- */
typedef struct {
    int32_t bits;        /* 4 or 8 */
    int32_t kv_heads;    /* 1 .. 256 */
    int32_t head_dim;    /* 64, 128 or 256 */
    int32_t page_tokens; /* a power of two, 32 .. 4096 */
    int64_t pages;       /* 1 .. 2^31 - 1 */
    void *data;          /* pages * q8_cache_page_bytes bytes, 16-byte aligned */
} q8_cache;

/* Whose tokens a call means.  Sequence s has lens[s] tokens, those of this call's
 * rows included: its rows are starts[s] .. starts[s+1]-1 of the call's arrays, and
 * row i of n is token lens[s] - n + i.  Token t is in page table[s][t / page_tokens].
 *
 * Nothing in device memory that is out of range is followed: a token before the
 * first or past table_ld * page_tokens, or in a page that the pool does not have,
 * is no token.  It is not written, is read as zeros and not attended to.  Entries of
 * the table that no token needs are not read.  Lengths over 2^30 are taken as 2^30.  Rows that belong to no sequence
 * (behind the last one, or past a sequence's max_rows) are left as they were. */
typedef struct {
    int64_t sequences;      /* 0 .. 65536 */
    int64_t table_ld;       /* entries of a row of the table, 1 or more; at most 2^30 tokens */
    const int32_t *table;   /* [sequences][table_ld], 4-byte aligned */
    const int32_t *lens;    /* [sequences], 4-byte aligned */
    const int32_t *starts;  /* [sequences + 1], not decreasing, 4-byte aligned; or NULL: row s is sequence s's
                               (rows == sequences) */
    int64_t rows;           /* rows of the call's arrays, 0 .. 2^20 */
    int64_t max_rows;       /* rows of one sequence at most, 1 or more (sizes the launches and
                               chooses the kernels: best not far above the longest) */
} q8_cache_batch;

/* Bytes of a page (0 for sizes that are refused; pages and data are not looked at). */
int64_t q8_cache_page_bytes(const q8_cache *cache);

/* Write the rows' keys and values into the cache.
 *   k, v : f32 rows of [kv_heads][head_dim], k_ld and v_ld values apart (multiples
 *          of 4 from kv_heads * head_dim to 2^40), 16-byte aligned.
 * Tokens already in the cache stay as they were, those in the same bytes too.  Sequences
 * of one call may have the same pages (chunks of one prompt, say) and write to them, but two
 * rows must not be the same place of a page; nor may calls in flight at once write to one
 * page.  Inputs must be finite.  Rows that belong to no sequence are not written.
 * Limit: sequences * max_rows * kv_heads * head_dim <= 2^40 (else Q8_E_SHAPE).
 * Errors: Q8_E_NULL, Q8_E_MODE (bits), Q8_E_SHAPE, Q8_E_ALIGN, Q8_E_ALIAS, Q8_E_HIP. */
q8_status q8_cache_append(const q8_cache *cache, const q8_cache_batch *batch, const float *k, int64_t k_ld,
                          const float *v, int64_t v_ld, void *stream);

/* Read the rows' keys and values back: the values that the cache stands for.
 *   k, v : out, f32 [rows][kv_heads][head_dim], 16-byte aligned.
 * Limits and errors as q8_cache_append. */
q8_status q8_cache_read(const q8_cache *cache, const q8_cache_batch *batch, float *k, float *v, void *stream);

/* Attention of the rows' queries over the cache.  Query head h of kv head
 * h / (heads / kv_heads), at token p = lens[s] - n + i of its sequence, sees the
 * tokens t with p - window < t <= p (window 0: every t <= p):
 *
 *   z_t = scale * sum_j q_j k_tj,  out = sum_t exp(z_t) v_t / sum_t exp(z_t)
 *   lse = ln sum_t exp(z_t)
 *
 * A row that sees no token gives zeros, and -inf.  Sums are held in f32; products are of
 * the cache's exact values with two binary16 words of q and of exp(z):
 *   scale * q_j is off by 2^-22 of it, or 2^-39 of the largest of its row and head;
 *   exp(z_t) by 2^-22 of it, or 2^-24 of the largest among the 32 tokens of its tile (2^-36
 *   in the tile of the row's largest; for weights down to 2^-79 of that one).
 * scale * log2(e) * q_j and the scores must stay within f32's range.
 *   q     : f32 rows of [heads][head_dim], q_ld values apart (a multiple of 4 from
 *           heads * head_dim to 2^40), 16-byte aligned, finite.
 *   heads : a multiple of kv_heads up to 4096.
 *   scale : finite.
 *   window: 0 .. 2^31 - 1.
 *   out   : out, f32 [rows][heads][head_dim], 16-byte aligned.
 *   lse   : out, f32 [rows][heads], 4-byte aligned, or NULL.
 *   workspace : 16-byte aligned, at least q8_attention_workspace_bytes, zero-filled
 *           by the caller before its first use.  Every call leaves the counters at
 *           its head at zero again, so one workspace, as large as the largest call's,
 *           serves call after call.  Two calls in flight at once (two streams, or two
 *           captured graphs that may run at the same time) must not share one.
 * The same call gives the same bits every time.  How a sequence's tokens are divided
 * over workgroups depends on the whole batch, so between batches a row's sums are
 * added in another order.  For that every workgroup looks through all sequences, 64 a step:
 * one token each of 64, 256, 1024 and 4096 sequences of 500 tokens (32 heads of 8 kv heads,
 * 128 dimensions) takes 14, 50, 301 and 2470 us, so that batches of many hundreds of
 * sequences are faster as calls of some 256 each.
 * Limit: sequences * max_rows * heads * head_dim <= 2^40 (else Q8_E_SHAPE).
 * Errors: Q8_E_NULL, Q8_E_MODE (bits), Q8_E_SHAPE, Q8_E_ALIGN, Q8_E_ALIAS, Q8_E_HIP. */
q8_status q8_attention(const q8_cache *cache, const q8_cache_batch *batch, const float *q, int64_t q_ld,
                       int64_t heads, float scale, int64_t window, float *out, float *lse, void *workspace,
                       int64_t workspace_bytes, void *stream);

/* Bytes of the q8_attention workspace on the current device (0 for sizes it
 * refuses).  The lengths do not matter. */
int64_t q8_attention_workspace_bytes(const q8_cache *cache, const q8_cache_batch *batch, int64_t heads);

#ifdef __cplusplus
}
#endif

#endif /* Q8PROJ_Q8_CACHE_H */
