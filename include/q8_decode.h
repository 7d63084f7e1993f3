/*
 * q8_decode.h -- C ABI of libq8proj.so, the steps of a decode step around the
 * Q8_0 projections of q8.h: a mixture-of-experts layer whose experts are Q8_0
 * matrices, and the draw of the next token from the LM head's logits.
 *
 * The conventions are those of q8.h: caller-owned device memory, work enqueued
 * on `stream` and nothing else (no allocation, no synchronization, no device
 * read on the host), every argument checked before anything is enqueued, named
 * statuses.  Every call may be captured into a HIP graph.
 */
#ifndef Q8PROJ_Q8_DECODE_H
#define Q8PROJ_Q8_DECODE_H

#include "q8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Mixture of experts
 *
 * A layer of n_experts experts, each a gate, an up and a down projection of
 * Q8_0 weights, and a router of f32 weights.  Per token (a row x of k values):
 *
 *   z_e   = sum_k x_k R_ek            products and sums in f64, rounded to f32
 *   chosen: the top_k largest z, in descending order, the lowest e among equals
 *   gate_e = exp(z_e - max z) / S     in f64, rounded to f32; S sums the exps of
 *                                     the chosen (renormalize) or of all experts
 *   g, u  = W_gate,e a,  W_up,e a     as q8_matvec computes them (rounded to f32)
 *   h     = g / (1 + exp(-g)) * u     in f64, rounded to f32
 *   y     = residual + sum_chosen gate_e * (W_down,e a')
 *                                     every product and sum in f64, rounded once
 *
 * where a and a' are x and h in the layer's activation mode: quantized as
 * q8_quantize_act does (integer modes) or as they are (Q8_ACT_F32).  Finite inputs
 * may give an h that overflows f32: in Q8_ACT_F32 y is then the formula's with an
 * infinite h; in the integer modes that token's y is unspecified.
 *
 * A layer is for a few tokens: what it costs is reading the chosen experts' weights
 * (unchosen experts are not read).  Rows go in slices of 64, one after the other, each
 * of which reads its experts' weights again.  Within a slice a pass over an expert's
 * weights serves 4 of its tokens if the slice's rows * top_k is at most 2 * n_experts
 * (3 * n_experts in Q8_ACT_F32), else 16 in Q8_ACT_F32, 16 or 32 in Q8_ACT_I8 and 8 or
 * 16 in Q8_ACT_I8X2; an expert with more tokens takes several passes, which the caches
 * serve as far as they hold it.
 *
 * The same call gives the same bits every time.  The number of rows, and what the other
 * rows choose, decide the kernels and the order of the f64 sums: between batches a
 * token's g, u, h or y can round to the neighbouring f32, and in the integer modes a
 * quantized value of h can then differ by one.
 *
 * Limits (else Q8_E_SHAPE): those of the fields below, 0 <= rows <= 2^20, and at most
 * 2^31 blocks in each of the three matrices.
 * ------------------------------------------------------------------------- */
typedef struct {
    int32_t mode;        /* q8_act_mode of the three projections */
    int32_t n_experts;   /* 1 .. 512 */
    int32_t top_k;       /* choices per token, 1 .. min(n_experts, 16) */
    int32_t renormalize; /* gates of a token sum to one (non-zero), or the softmax over all experts (0) */
    int64_t k;           /* columns of x and y, a multiple of 64 up to 65536 */
    int64_t ff;          /* rows of gate and up, columns of down, a multiple of 64 up to 65536 */
    const float *router; /* f32 [n_experts][k], 16-byte aligned (q8_moe_route and q8_moe only) */
    const void *w_gate;  /* Q8_0 blocks [n_experts][ff][k/32], 4-byte aligned */
    const void *w_up;    /* Q8_0 blocks [n_experts][ff][k/32], 4-byte aligned */
    const void *w_down;  /* Q8_0 blocks [n_experts][k][ff/32], 4-byte aligned */
} q8_moe_layer;

/* Bytes of the workspace the calls below need for `rows` rows (0 for arguments
 * they refuse).  More rows than 64 need no more than 64 do.  The caller
 * zero-fills it once before its first use; every call leaves the counters at
 * its head at zero again, so one workspace, as large as the largest call's,
 * serves call after call of any layer.  Two calls in flight at once (two
 * streams, or two captured graphs that may run at the same time) must not share
 * one. */
int64_t q8_moe_workspace_bytes(const q8_moe_layer *layer, int64_t rows);

/* The router alone: ids and gates of `rows` tokens.
 *   x     : f32 [rows][k], 16-byte aligned.
 *   ids   : out, int32 [rows][top_k], 4-byte aligned, in descending order of z.
 *   gates : out, f32 [rows][top_k], 4-byte aligned.
 *   workspace : 16-byte aligned, at least q8_moe_workspace_bytes.
 * The layer's weight pointers are not used and may be NULL.
 * Errors: Q8_E_NULL, Q8_E_SHAPE, Q8_E_MODE, Q8_E_ALIGN, Q8_E_ALIAS, Q8_E_HIP. */
q8_status q8_moe_route(const q8_moe_layer *layer, const float *x, int64_t rows, int32_t *ids, float *gates,
                       void *workspace, int64_t workspace_bytes, void *stream);

/* The experts for choices the caller gives (a router of its own, or
 * q8_moe_route's): ids and gates [rows][top_k] as above, in any order.  An id
 * outside 0 .. n_experts-1 (a padded row; an expert another GPU holds) adds
 * nothing; a row without any choice gives y = residual (or 0).  The same expert
 * twice in a row counts with the sum of its gates.
 *   residual : f32 [rows][k] or NULL, 4-byte aligned.
 *   y        : out, f32 [rows][k], 4-byte aligned.  May be exactly `residual`;
 *              must not otherwise overlap any argument.
 * The layer's router is not used and may be NULL.
 * Errors: as q8_moe_route. */
q8_status q8_moe_experts(const q8_moe_layer *layer, const float *x, int64_t rows, const int32_t *ids,
                         const float *gates, const float *residual, float *y, void *workspace,
                         int64_t workspace_bytes, void *stream);

/* The whole layer: q8_moe_route, then q8_moe_experts on its choices.  ids and
 * gates are outputs as in q8_moe_route, and required.
 * Errors: as q8_moe_route. */
q8_status q8_moe(const q8_moe_layer *layer, const float *x, int64_t rows, const float *residual, float *y,
                 int32_t *ids, float *gates, void *workspace, int64_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * The next token
 *
 * Draws one token from each row of logits with given parameters and a given
 * random number, the counterpart of q8_matvec_argmax for sampled decoding.  A
 * row's candidates are its logits that are neither NaN nor -inf.  With m the
 * largest of them (T the row's temperature):
 *
 *   w_i = exp((l_i - m) * (1/T)) * 2^44, in f64, rounded to a whole number
 *
 * so that every sum below is exact.  In descending order of
 * the logits, the lowest index first among equals, with running sums C_j:
 *
 *   top-k : the first top_k tokens; top_k <= 0 (or NULL): all
 *   top-p : the shortest prefix with C_j >= top_p * C_top-k (at least one token);
 *           top_p >= 1, NaN or NULL: all
 *   min-p : the tokens with w_i >= min_p * 2^44 (at least one); min_p <= 0, NaN or
 *           NULL: all
 *
 * The shortest of the three prefixes is kept, W is its sum, and the token is the
 * first with C_j > u * W (the last kept one of non-zero weight if there is none).
 * Products and comparisons of sums are in f64.  prob = w / W.  T <= 0 or NaN: the
 * largest logit, the lowest index among equals, prob 1.  A row without
 * candidates: index -1, prob 0.
 *
 *   logits      : f32 [rows] rows of n values, `ld` values apart (ld >= n), 4-byte
 *                 aligned.
 *   temperature : f32 [rows], or NULL: 1.
 *   top_k       : int32 [rows] or NULL;  top_p, min_p : f32 [rows] or NULL.
 *   u           : f32 [rows], the random numbers, in [0, 1).
 *   idx         : out, int32 [rows];  prob : out, f32 [rows], or NULL.
 *   workspace   : 16-byte aligned, at least q8_sample_workspace_bytes; scratch,
 *                 which need not be cleared.  Calls in flight at once must not
 *                 share one.
 * All arrays 4-byte aligned; the outputs and the workspace must not overlap any
 * other argument.  Limits (else Q8_E_SHAPE): 1 <= n < 2^19, 0 <= rows <= 65536,
 * ld <= 2^40.
 * Errors: Q8_E_NULL, Q8_E_SHAPE, Q8_E_ALIGN, Q8_E_ALIAS, Q8_E_HIP.
 * ------------------------------------------------------------------------- */
q8_status q8_sample(const float *logits, int64_t ld, int64_t rows, int64_t n, const float *temperature,
                    const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *idx,
                    float *prob, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of the q8_sample workspace (0 for sizes it refuses).  They do not decrease
 * with rows or n: a workspace for the largest call serves the smaller ones. */
int64_t q8_sample_workspace_bytes(int64_t rows, int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* Q8PROJ_Q8_DECODE_H */
