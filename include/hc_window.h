/*
 * hc_window.h - C ABI of the verify-window operators beside the hyper-connection read
 * (hc_read.h), in the same library.
 *
 * One step of a serving loop takes each request's new tokens (its window: one token of
 * a decode step, the 1-8 drafted tokens of a verify step, a chunk of a prompt) through
 * the layers. Around the read it needs, in this order:
 *
 *   hc_window_plan      cache blocks, slots and positions of the new tokens, built on
 *                       the GPU from the requests' lengths
 *   hc_kv4_append       the new tokens' keys and values, rounded to 4 bits, into their slots
 *   hc_kv4_attention    each new token against its request's cache
 *   hc_token_logprobs   the drafted tokens' log probabilities on the step's logits, with
 *                       the entropy and the most likely alternatives
 *
 * and hc_kv4_load reads slots of the cache back as numbers.
 *
 * The cache is paged: `blocks` blocks of `block_size` tokens; a slot is block *
 * block_size + offset (64 bits). Each token and kv head holds a key and a value as one
 * group of head_dim 4-bit codes with a step s and a minimum m, bf16 each:
 *
 *   value = m + s * code, code in 0..15
 *
 *   codes   uint8_t  [blocks][2][kv_heads][block_size][head_dim / 2]   keys at 0, values
 *                    at 1; element 2i in the low half of byte i, 2i + 1 in the high half
 *   scales  uint16_t [blocks][2][kv_heads][block_size][2]              bf16 bits of s, m
 *
 * Rounding a group x (every step a single fp32 operation, so that codes are the same
 * everywhere): m = the largest bf16 <= min x; s = the smallest bf16 >= fl(fl(max x - m) *
 * fl(1/15)), raised to 2^-126 where it lies between 0 and that; code = fl(fl(x - m) *
 * fl(1/s)) rounded to the nearest integer, ties to even, clamped to 0..15 (0 where s =
 * 0). Both directions of rounding keep every x within [m, m + 15 s] to fp32 accuracy.
 * A group with a NaN or an infinity, or whose width max x - m is infinite, is held as
 * s = m = NaN and reads back as NaN.
 *
 * Memory, ownership, ordering and errors are those of hc_read.h: caller-owned device
 * memory of the context's device (hc_read_init, any max_tokens), asynchronous on
 * `stream`, argument errors refused on the host before anything is enqueued. hc_kv4_*
 * and hc_token_logprobs share the context's scratch, whose size does not depend on any
 * argument (41 MB, allocated by hc_read_init): calls on one context must be issued on one
 * stream at a time. `codes`,
 * `scales`, q, k, v, their outputs, and the logits of hc_token_logprobs where noted, are
 * 16-byte aligned; arrays of 4- and 8-byte integers and floats are aligned to their
 * elements. Outputs must not overlap inputs or each other unless said.
 *
 * What the device reads from arrays (lengths, block ids, slots, offsets) is checked by
 * the kernels, in every build, and hc_read_status reports HC_ERR_BOUNDS for an entry that
 * points outside its array. A slot that does is skipped (hc_kv4_load: read as zeros);
 * hc_kv4_attention reads block 0 in place of a block that does not exist, so that the
 * request's output is wrong but no memory outside the cache is touched, and cuts lengths
 * that do not fit to what does.
 */
#ifndef HC_WINDOW_H
#define HC_WINDOW_H

#include "hc_read.h"

#ifdef __cplusplus
extern "C" {
#endif

enum hc_dtype {
    HC_DTYPE_BF16 = 0,
    HC_DTYPE_FP16 = 1,
    HC_DTYPE_FP32 = 2
};

#define HC_PLAN_MAX_REQUESTS 8192
#define HC_KV4_MAX_BLOCK 256
#define HC_KV4_MAX_GROUP 128
#define HC_KV4_MAX_MASKED 64
#define HC_LOGPROBS_MAX_TOP 32

/* One layer's cache. block_size: 16, 32, 64, 128 or 256; head_dim: 64 or 128; kv_heads: at
 * most 65535. */
typedef struct hc_kv4_cache {
    uint8_t* codes;
    uint16_t* scales;
    int blocks;
    int kv_heads;
    int block_size;
    int head_dim;
} hc_kv4_cache;

/* Blocks, slots and positions of a step's new tokens.
 *
 *   cached_lens[requests], new_lens[requests]   tokens held and tokens to add (< 0: 0)
 *   free_blocks[free_capacity], free_count[1]   a stack of free block ids; count is
 *                       clamped to 0..free_capacity; blocks are taken from its top
 *   block_table[requests][table_width]          in and out: a request's first
 *                       ceil(cached / block_size) entries are read, the entries of its
 *                       new blocks are written, the others stay
 *
 * Requests are served in order. A request is granted if its blocks fit the table's row
 * and, unless it needs none, the blocks wanted up to and including it are at most
 * free_count. Request b's j-th new block is free_blocks[free_count - 1 - (j-th of all
 * wanted before)]. One that is not granted keeps its cached tokens and takes nothing.
 *
 *   cu_lens[requests + 1]     first new token of each request, and their total
 *   kv_lens[requests]         cached + new where granted, else cached
 *   slots[capacity]           slot of each new token, -1 where its request was not
 *                             granted, where its block's id is negative (reported) and
 *                             past the total
 *   request_of, positions     [capacity] the token's request and its position in it,
 *                             -1 past the total
 *   free_left[1]              free_count less the blocks taken; must not be free_count
 *
 * Totals saturate at 2^31 - 1. 1 <= requests <= HC_PLAN_MAX_REQUESTS; block_size as in
 * a cache; requests * table_width < 2^31. */
int hc_window_plan(int requests, int table_width, int block_size, int capacity, int free_capacity,
                   const int32_t* cached_lens, const int32_t* new_lens,
                   const int32_t* free_blocks, const int32_t* free_count,
                   int32_t* block_table, int64_t* slots, int32_t* request_of,
                   int32_t* positions, int32_t* cu_lens, int32_t* kv_lens,
                   int32_t* free_left, void* stream);

/* Rounds the keys and values of `tokens` tokens to 4 bits and writes them to their
 * slots (slots[tokens]; negative: the token is skipped). Give a slot once in a call: of
 * several tokens given the same one, any may end in each 32-bit word of its codes and scales,
 * so that what it holds need not be one of them. k and v hold head_dim values of `dtype` at token * token_stride +
 * head * head_stride elements; strides are multiples of 16 bytes, but for that of an axis
 * of one, which is not used. */
int hc_kv4_append(const hc_kv4_cache* cache, int tokens, int dtype,
                  const void* k, int64_t k_token_stride, int64_t k_head_stride,
                  const void* v, int64_t v_token_stride, int64_t v_head_stride,
                  const int64_t* slots, void* stream);

/* Reads `tokens` slots back: k_out and v_out [tokens][kv_heads][head_dim] of `dtype`,
 * m + s * code rounded to nearest even. A negative slot reads as zeros. */
int hc_kv4_load(const hc_kv4_cache* cache, int tokens, const int64_t* slots, int dtype,
                void* k_out, void* v_out, void* stream);

/* Attention of each request's new tokens against its cache, which already holds them:
 *
 *   out = sum_j p_j v_j,  p = softmax over the visible keys j of scale * (q . k_j)
 *   lse = ln sum_j exp(scale * (q . k_j))
 *
 * Request b has the tokens cu_lens[b] .. cu_lens[b + 1] - 1 of q, the last ones of its
 * kv_lens[b] tokens in the cache. Token i of n sees positions 0 .. kv_len - n + i, or,
 * with a mask, every position below kv_len - n and position kv_len - n + j where bit j
 * of mask[token] is set (a draft tree; max_new <= HC_KV4_MAX_MASKED). A token that sees
 * nothing gets zeros and lse = -inf. Query head h reads kv head h / (q_heads / kv_heads).
 *
 *   q     head_dim values of `dtype` (bf16 or fp16) at token * q_token_stride + head *
 *         q_head_stride elements; strides as in hc_kv4_append
 *   out   [tokens][q_heads][head_dim] of `dtype`
 *   lse   [tokens][q_heads] fp32, or NULL
 *   max_new   an upper bound of the requests' new tokens, which chooses the kernel: a
 *             request with more reports HC_ERR_BOUNDS and the rest of it is not written
 *
 * A request that hc_window_plan did not grant has tokens in q and none in the cache: its rows
 * are computed as if its last cached tokens were they, and mean nothing.
 *
 * What is rounded: sums, maxima and softmax statistics are fp32, and keys and values enter
 * as the cache holds them, exactly. q is held as fp16 over a power of two of each row's own
 * (exact but for elements 2^-27 below the row's largest). Each weight p_j, or p_j times the
 * value's step, is rounded once to fp16 over a power of two of each row's own (so that no
 * row loses bits to what it does not see or hardly weighs): to 11 bits down to 2^-14 of the
 * largest that the row has seen, to 2^-25 of that below. For more than 16 rows (new tokens x
 * query heads of a kv head) the part m + 8 s that a key's dimensions have in common, and the
 * sum of q that it meets, are two fp16 terms each, 22 bits. So, while the sums of a logit's
 * terms stay below 2^8, out is within 2^-10 sum_j p_j (|s_j (c_j - 8)| + |m_j + 8 s_j|) +
 * 2^-22 n max_j p_j max_j s_j of the formula before it is rounded to `dtype`, n the keys that
 * weigh less than 2^-14 of the largest (2^17 equal keys of 2^-18 each are rounded the same
 * way and may be off by 2^-7 of what they add up to), and lse within 2^-19 of 1 + the largest
 * such sum. A row that sees a key or value held as NaN, or whose query is NaN, is NaN.
 *
 * Output is bitwise deterministic for given inputs. */
int hc_kv4_attention(const hc_kv4_cache* cache, int requests, int tokens, int q_heads,
                     int max_new, int table_width, float scale, int dtype,
                     const void* q, int64_t q_token_stride, int64_t q_head_stride,
                     const int32_t* cu_lens, const int32_t* kv_lens, const int32_t* block_table,
                     const uint64_t* mask, void* out, float* lse, void* stream);

/* Log probabilities of given tokens. Row t of the logits, `vocab` values of `dtype` at t *
 * row_stride elements, need only be aligned to its elements:
 *
 *   lse = ln sum exp(x);  logprob = x[token] - lse;  entropy = -sum p ln p
 *   rank = number of logits above x[token]
 *   top_ids, top_logprobs [tokens][top]   the `top` most likely tokens and their log
 *                     probabilities, equal ones in the order of their ids
 *
 * A logit of -inf has probability 0 and adds 0 to the entropy. A row of -inf alone has
 * lse = logprob = -inf, top_logprobs = -inf and entropy 0. A token id outside the
 * vocabulary has logprob = -inf and rank = vocab. A row with a NaN or +inf has NaN as
 * logprob, entropy and top_logprobs (lse NaN or +inf), and unspecified rank and ids.
 * All in fp32, with the hardware's powers of two (2^-22): lse within 2^-17 + 2^-22 of the
 * row's largest |x|, log probabilities, which are taken from differences of logits, within
 * 2^-17 + 2^-23 of the difference to the largest one for ordinary rows, the entropy within
 * 2^-17 + 2^-20 (28 + ln vocab).
 * 0 <= top <= min(vocab, HC_LOGPROBS_MAX_TOP); 1 <= vocab. */
int hc_token_logprobs(int tokens, int vocab, int top, int dtype, const void* logits,
                      int64_t row_stride, const int32_t* token_ids, float* logprob,
                      float* entropy, float* lse, int32_t* rank, int32_t* top_ids,
                      float* top_logprobs, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HC_WINDOW_H */
