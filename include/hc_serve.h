/*
 * hc_serve.h - C ABI of further operators of a serving step, beside those of hc_window.h and
 * in the same library: what a step needs whose tokens have positions, whose requests share a
 * long prefix, and whose next tokens are drawn.
 *
 *   hc_kv4_append_rotary      a layer's queries and keys normed by head and rotated by their
 *                             positions; the keys and values rounded into their slots
 *   hc_kv4_attention_shared   each new token against the prefix that its request shares with
 *                             others and against its request's own cache
 *   hc_sample_tokens          the next tokens from the logits: temperature, top-k, top-p,
 *                             min-p, from given uniform numbers
 *
 * The cache, its rounding and the types are those of hc_window.h; memory, ownership, ordering
 * and errors those of both headers: caller-owned device memory of the context's device
 * (hc_read_init, any max_tokens), asynchronous on `stream`, argument errors refused on the
 * host before anything is enqueued, calls on one context on one stream at a time (they share
 * its scratch). Large arrays are 16-byte aligned, arrays of 4- and 8-byte integers and floats
 * to their elements, logits to theirs. Outputs must not overlap inputs or each other. What the
 * device reads from index arrays is checked by the kernels, in every build: an entry that
 * points outside its array is reported by hc_read_status as HC_ERR_BOUNDS, and nothing outside
 * is touched.
 */
#ifndef HC_SERVE_H
#define HC_SERVE_H

#include "hc_window.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HC_ROTARY_MAX_AXES 4
#define HC_SAMPLE_MAX_VOCAB 262144

/* How queries and keys are normed and rotated. */
typedef struct hc_rotary {
    const float* cos_sin;      /* [length][2][dim / 2]: a position's cosines, then its sines */
    const int32_t* axis_of;    /* [dim / 2]: the axis of each frequency; NULL: axis 0 */
    const void* q_norm;        /* [head_dim] weights of the call's dtype; NULL: no norm */
    const void* k_norm;
    float eps;                 /* of the norm */
    int length;                /* positions of the table */
    int dim;                   /* leading dimensions that are rotated: a multiple of 16 up to
                                  head_dim, or 0 (cos_sin, axis_of, positions are not read) */
    int axes;                  /* 1..HC_ROTARY_MAX_AXES */
    int interleaved;           /* pairs (2i, 2i + 1); 0: pairs (i, i + dim / 2) */
} hc_rotary;

/* Norms and rotates the queries and keys of `tokens` tokens, writes the queries, and rounds
 * the keys and the values (which are neither normed nor rotated) into their slots as
 * hc_kv4_append does. For a head x of a token, in this order, every step a single fp32
 * operation rounded to nearest, so that what the cache holds is the same everywhere:
 *
 *   with a norm:  y_i = x_i x_i; neighbours added, y_2i + y_2i+1, until one is left;
 *                 r = 1 / sqrt(y (1 / head_dim) + eps)  (product, sum, root, quotient);
 *                 n_i = (x_i r) w_i                     without:  n_i = x_i
 *   a pair (a, b) of frequency i:  (a c - b s, b c + a s), each of two products and their
 *                 difference or sum; c = cos_sin[p][0][i], s = cos_sin[p][1][i], p the token's
 *                 position on the axis of i
 *
 * (A head whose squares pass fp32's range, |x| above 2^60, has r = 0 or NaN.)
 *
 *   q, k, v    as in hc_kv4_append, of `dtype`; q_heads query heads (0: none, q and q_out NULL)
 *   positions  [axes][tokens]. A token with a negative one is none: its row of q_out and its
 *              slot stay as they are. One at or past `length` counts as length - 1, and is
 *              reported; an axis that is none counts as axis 0, and is reported.
 *   slots      as in hc_kv4_append
 *   q_out      [tokens][q_heads][head_dim] of `dtype`, rounded to nearest even
 */
int hc_kv4_append_rotary(const hc_kv4_cache* cache, const hc_rotary* rotary, int tokens, int q_heads,
                         int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                         const void* k, int64_t k_token_stride, int64_t k_head_stride,
                         const void* v, int64_t v_token_stride, int64_t v_head_stride,
                         const int32_t* positions, const int64_t* slots, void* q_out,
                         void* stream);

/* hc_kv4_attention of requests in groups that share a prefix: group g has the requests
 * cu_groups[g] .. cu_groups[g + 1] - 1 (cu_groups[0] = 0, cu_groups[groups] = requests) and the
 * prefix_lens[g] tokens in the blocks prefix_table[g][0..prefix_width). A token sees its
 * group's whole prefix, and behind it what it sees of its request's own cache in
 * hc_kv4_attention (block_table and kv_lens hold the own tokens alone, without the prefix). A
 * prefix is read once for all tokens of its group, whatever their requests; a prefix of
 * length 0 is none.
 *
 *   max_shared   an upper bound of the new tokens of a group's requests together, as max_new is
 *                of one request's: a group with more reports HC_ERR_BOUNDS, and the tokens
 *                past it have no defined output. Nor have those of requests in no group.
 *   workspace    floats [tokens][q_heads][head_dim + 2]: sums over the prefixes. Written by the
 *                call; nothing is kept there for another.
 *
 * The host reads no lengths: kernels are chosen by max_new, max_shared and what the tables have
 * room for (width * block_size tokens). Results do not depend on it, the time does: a table no
 * wider than its longest row needs, and of own tokens one of at most 2048 where there are many
 * requests of few tokens, is the faster one. A prefix of whole blocks can also stand at the
 * beginning of each request's row in hc_kv4_attention, which needs no workspace: faster where the
 * prefix is short or the tokens are chunks of prompts, whose products are the same either way;
 * this call where tokens are few and the prefix is long, which that one reads once a request.
 *
 * Everything else is as in hc_kv4_attention, its roundings among them: the prefix's part and the
 * own one are each as exact as a call of it, and are joined in fp32 before the one rounding to
 * `dtype`. */
int hc_kv4_attention_shared(const hc_kv4_cache* cache, int requests, int groups, int tokens, int q_heads,
                            int max_new, int max_shared, int table_width, int prefix_width, float scale,
                            int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                            const int32_t* cu_lens, const int32_t* kv_lens, const int32_t* block_table,
                            const int32_t* cu_groups, const int32_t* prefix_lens,
                            const int32_t* prefix_table, const uint64_t* mask, float* workspace,
                            void* out, float* lse, void* stream);

/* Draws a token of each row of the logits (laid out as for hc_token_logprobs; 1 <= vocab <=
 * HC_SAMPLE_MAX_VOCAB). Row t, with M its largest logit:
 *
 *   w_i = exp((x_i - M) / temperature[t])
 *   top_k[t]   the k largest stay, of equal ones those of lower ids (k < 1 or >= vocab: all)
 *   top_p[t]   of these, from the largest on (equal ones by id), those stay before which less
 *              than top_p of their sum lies: the first always does (>= 1: all)
 *   min_p[t]   of these, those with w_i >= min_p stay (<= 0: all; above 1 it is 1)
 *   token      the first id at which the sum of what stays, in the order of the ids, is above
 *              uniform[t] times all of it (uniform is cut to [0, 1); the last one that stays has
 *              weight, at most)
 *   logprob    ln of its w_i over the sum of what stays
 *
 * A temperature below 2^-64 (0 and negative ones too) takes the largest logit, of equal ones the
 * lowest id, with logprob 0. temperature, top_k, top_p, min_p may be NULL: 1, all, 1, 0. A logit
 * of -inf has no weight. A row with a NaN or +inf, or of -inf alone, or with a NaN (or an
 * infinity as temperature) among its settings, has token -1 and logprob NaN.
 *
 * Weights are whole multiples of 2^-45, within 2^-27 of w_i (up to e^-24) or the multiple, and their sums
 * are exact, so that the token does not depend on the order of anything; it is the formula's
 * but where uniform lies within 2^-26 of a border between two tokens (two sums, each off by up
 * to 2^-27), or a filter's border as near to another weight. logprob within 2^-20 of 1 + its size.
 */
int hc_sample_tokens(int tokens, int vocab, int dtype, const void* logits, int64_t row_stride,
                     const float* uniform, const float* temperature, const int32_t* top_k,
                     const float* top_p, const float* min_p, int32_t* token_ids, float* logprob,
                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HC_SERVE_H */
