/*
 * fa_kv4.h -- C ABI of the paged 4-bit key/value cache: planning a step's
 * pages and slots on the GPU, writing keys and values into the cache, reading
 * them back, and exact attention over the cache.
 *
 * The serving form of the operation in fa.h: queries are few (one new token,
 * some drafted ones, or a chunk of a prompt) and keys and values are those of
 * every earlier token of the request, held between calls.  The conventions of
 * fa.h hold (device pointers, caller-owned buffers, no allocation, work only
 * enqueued on `stream`, outputs that overlap nothing, statuses); sizes and
 * strides are in elements.
 *
 * Cache format.  The cache is uint8 [num_pages, Hkv, fa_kv4_page_bytes()]
 * (16-byte aligned).  A page holds page_size tokens (16, 32, 64 or 128) and a
 * group is `group` consecutive channels (32 or 64); the record of one page
 * of one head is
 *     K codes  [page_size][d / 2]      K params [page_size][d / group]
 *     V codes  [page_size][d / 2]      V params [page_size][d / group]
 * A param is a pair of bf16 (scale in the low half-word, minimum in the high
 * one), a code is 4 bits, and the value of a channel is minimum + scale * code.
 * Eight channels share a little-endian 32-bit word: channels 0, 2, 4, 6 are the
 * nibbles of its low half, 1, 3, 5, 7 those of its high half, low nibble first.
 * The cache need not be initialised: rows that were not written are never used.
 *
 * A slot is a token's place in the cache, page * page_size + offset; -1 stands
 * for none.  num_pages * page_size must be below 2^31 (byte offsets are 64-bit).
 *
 * Errors inside the data (a slot or a page id outside the cache, offsets in
 * cu_q that do not fit, an inconsistent free list) cannot be returned by a call
 * that only enqueues: the kernels touch no memory outside the buffers, skip the
 * row or the request concerned (a page id out of range gives that request an
 * undefined result), and fa_check_error() returns FA_ERR_INVALID_ARG.
 */
#ifndef FA_KV4_H_
#define FA_KV4_H_

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one page of one K/V head; 0 for a geometry that is not supported. */
size_t fa_kv4_page_bytes(int d, int page_size, int group);

/*
 * One step's bookkeeping, without a host round trip: from the lengths of B
 * requests (at most FA_KV4_MAX_BATCH) it takes pages from a free list,
 * completes the block tables, and lists where every new token goes.
 *   past_len    in    : int32 [B], tokens the request holds in the cache
 *   new_len     in    : int32 [B], tokens to add (>= 0), or -1: the request is
 *                       finished and its pages return to the free list
 *   block_table inout : int32 [B, max_pages]; row b's first
 *                       ceil(past_len / page_size) entries are its pages, the
 *                       pages taken now are written behind them
 *   free_list   inout : int32 [num_pages], a ring of page ids
 *   free_state  in    : int32 [2], the ring's first free entry and their number
 *   kv_len      out   : int32 [B], past_len + new_len (0 if finished)
 *   cu_q        out   : int32 [B + 1], prefix sums of the tokens added
 *   slots       out   : int32 [max_tokens], the slots of the new tokens, request
 *                       after request, -1 behind the last
 *   state_out   out   : int32 [4]: the ring's new first entry and number (the
 *                       next call's free_state), tokens added, requests served
 * Pages are taken from the ring's front in the order of the requests and
 * returned pages are put at its end (they are free from the next call on).
 * Requests are served in order until one does not fit -- the free pages, the
 * max_tokens places or its table row are used up, or its lengths are invalid
 * -- and from that one on none is: those keep kv_len = past_len and add
 * nothing, and state_out[3] is the number of requests before them.  Finished
 * requests return their pages in any case.  Same inputs, same outputs; the
 * call may be repeated with the inputs' values unchanged.
 */
#define FA_KV4_MAX_BATCH 8192
fa_status fa_kv4_plan(const int32_t* past_len, const int32_t* new_len, int B, int page_size,
                      int num_pages, int32_t* block_table, int max_pages, int32_t* free_list,
                      const int32_t* free_state, int max_tokens, int32_t* kv_len, int32_t* cu_q,
                      int32_t* slots, int32_t* state_out, fa_stream_t stream);

/*
 * Quantises T tokens' keys and values and writes them to their slots.
 *   K, V  in : bf16, element (t, h, c) at t * token_stride + h * head_stride + c
 *              (strides >= 0 and multiples of 8, base 16-byte aligned), so views
 *              of a packed projection need no copy
 *   slots in : int32 [T]; -1 skips the token; slots >= 0 must be distinct
 * Per (token, head, group): minimum = min x, scale = (max x - min x) / 15 rounded
 * to bf16, code = (x - minimum) / scale rounded to the nearest integer, ties to
 * even, at most 15 -- decided exactly.  Values of one size share scale 0 and
 * code 0.  A group that holds a NaN or an infinity reads back as NaN.
 */
fa_status fa_kv4_append(const void* K, const void* V, int T, int Hkv, int d, int k_token_stride,
                        int k_head_stride, int v_token_stride, int v_head_stride,
                        const int32_t* slots, void* cache, int num_pages, int page_size,
                        int group, fa_stream_t stream);

/*
 * Reads T tokens back: K, V out bf16 [T, Hkv, d] contiguous, minimum + scale *
 * code rounded to nearest even.  Rows whose slot is -1 are left as they were.
 */
fa_status fa_kv4_gather(const int32_t* slots, const void* cache, int num_pages, int page_size,
                        int group, int T, int Hkv, int d, void* K, void* V, fa_stream_t stream);

/*
 * Exact attention of new tokens over the cache:
 *     O = softmax(scale * Q K^T + mask) V,    L = rowwise logsumexp (natural log)
 * with K and V the values the cache holds.
 *   Q           in  : bf16, query t of the batch's list, head h, channel c at
 *                     t * q_token_stride + h * q_head_stride + c (strides as K's)
 *   block_table in  : int32 [B, max_pages]
 *   cu_q        in  : int32 [B + 1]; queries cu_q[b] .. cu_q[b + 1] - 1 belong to
 *                     request b, at most max_q of them (none is allowed)
 *   kv_len      in  : int32 [B]; keys of request b, clamped to
 *                     [0, max_pages * page_size].  The request's n queries are
 *                     its last n tokens: query i is at position kv_len - n + i
 *   O           out : bf16 [total_q, Hq, d];  L out: fp32 [total_q, Hq]
 *   causal          : key j is visible to a query at position p iff j <= p
 *   window          : -1 = none, w >= 0: only keys p - w <= j <= p
 *   workspace       : DEVICE, >= fa_kv4_attn_workspace_bytes() bytes, 256-byte
 *                     aligned; contents on entry are ignored; not to be shared
 *                     by calls that may overlap.  Calls for which
 *                     fa_kv4_attn_call_workspace_bytes() is 0 (short tables or
 *                     windows) may pass NULL and 0
 * Hq is a multiple of Hkv; query head h reads K/V head h / (Hq / Hkv).
 * d is 64, 128 or 256.  A query that sees no key gets O = 0, L = -inf.  Rows of
 * O and L behind cu_q[B] are left as they were.  Deterministic.  Keys have to be
 * below 2^116 in size; a key or value that is NaN reaches the queries that see
 * it and no others, and a query that is not finite its own row alone.  Requests
 * may share pages.  Make a first call with the same d, group, max_q, max_pages
 * and window before any stream capture (it may load device code).
 */
size_t fa_kv4_attn_workspace_bytes(int Hq, int Hkv, int d, int max_q);
size_t fa_kv4_attn_call_workspace_bytes(int B, int total_q, int max_q, int Hq, int Hkv, int d,
                                        int max_pages, int page_size, int window);
fa_status fa_kv4_attn(const void* Q, const void* cache, const int32_t* block_table,
                      const int32_t* cu_q, const int32_t* kv_len, void* O, float* L, int B,
                      int total_q, int max_q, int Hq, int Hkv, int d, int q_token_stride,
                      int q_head_stride, int num_pages, int max_pages, int page_size, int group,
                      float scale, int causal, int window, void* workspace,
                      size_t workspace_bytes, fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_KV4_H_ */
