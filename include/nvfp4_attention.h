/*
 * nvfp4_attention.h -- C ABI of the operators around the paged FP8 KV cache of nvfp4.h: block tables
 * and slot maps built on the device, attention of prompts (or of single tokens) over the cache, and
 * attention of trees of drafted tokens over it.  Part of libnvfp4.so (gfx950); the conventions of
 * nvfp4.h hold here too: device pointers, caller-owned buffers, no allocation, no host
 * synchronisation, every check before any HIP call, results deterministic.
 *
 * The cache is the one nvfp4_kv_fp8_store writes: [num_slots, cache_ld] E4M3 bytes for the keys and
 * as many for the values, a slot's row holding kv_heads * head_dim codes, each standing for
 * E4M3(code) * scale with one static scale per tensor.  Slots are grouped into blocks of block_size:
 * position p of request r lives in slot block_table[r][p / block_size] * block_size +
 * p % block_size.
 *
 * Source: ai.info summary of arXiv 2609.04098, "Main Findings" (FP8 KV cache with static per-tensor
 * scales under the attention layers of the hybrid model; the pages give no formula for the attention
 * itself, so the definitions below are this library's).
 */
#ifndef NVFP4_ATTENTION_H
#define NVFP4_ATTENTION_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of requests in one call. */
#define NVFP4_MAX_REQUESTS 8192

/* Largest number of 64-bit words of a drafted token's mask (64 drafted tokens a word). */
#define NVFP4_MAX_TREE_WORDS 64

/*
 * nvfp4_kv_block_tables -- bookkeeping of one serving step, from request lengths alone: which new
 * cache blocks each request gets, and where each new token's row goes.
 *
 * Request r has c = context_lens[r] tokens in the cache and brings n = query_lens[r] new ones
 * (negative lengths count as 0).  It holds have = ceil(c / block_size) blocks and needs
 * need = ceil((c + n) / block_size), both at most table_width.  Requests take new blocks in order:
 * with base_r the sum of need - have over the requests before r,
 *   block_table[r][have + k] = free_blocks[*free_start + base_r + k],   0 <= k < need - have,
 * or -1 where that index lies outside [0, num_free).  Other entries are left as they were.
 *   query_start[r]  = sum of n over the requests before r; query_start[requests] = their total
 *                     (sums above 2^31 - 1 give 2^31 - 1)
 *   seq_lens[r]     = c + n (at most 2^31 - 1)
 *   blocks_needed   = base_requests: above num_free - *free_start the blocks did not suffice
 *   token t = query_start[r] + i, at position p = c + i:
 *     positions[t]    = p
 *     slot_mapping[t] = block_table[r][p / block_size] * block_size + p % block_size, or -1 where
 *                       that entry is negative or outside the table
 *   t >= query_start[requests] (padding, up to max_tokens): slot_mapping -1, positions 0.  Tokens
 *   from max_tokens on are dropped.
 * slot_mapping is what nvfp4_kv_fp8_store takes; block_table, query_start and seq_lens are what the
 * attentions below take.  Calling it again with the same arguments gives the same results: the free
 * list itself is not changed (the caller advances *free_start by blocks_needed).
 *
 *   context_lens, query_lens  device, int32[requests].
 *   requests      0 .. NVFP4_MAX_REQUESTS.
 *   block_size    1 .. 2^24.
 *   free_blocks   device, int32[num_free] (may be NULL when num_free is 0); num_free < 2^31.
 *   free_start    device, one int32, or NULL for 0; not written.
 *   block_table   device, int32 [requests, table_width], row pitch table_ld (elements), read and
 *                 written; requests * table_ld < 2^40.
 *   slot_mapping  device, int64[max_tokens], 8-byte aligned; positions: int32[max_tokens];
 *   max_tokens    0 .. 2^31 - 257.
 *   query_start   int32[requests + 1]; seq_lens: int32[requests]; blocks_needed: one int32.
 * No output may overlap an input or another output.  Exact.
 * Errors: EINVAL (NULL), ESHAPE, EALIGN (int32 pointers 4 bytes).  requests == 0 still writes the
 * padding, query_start[0] = 0 and blocks_needed = 0.
 */
nvfp4_status nvfp4_kv_block_tables(const int32_t* context_lens, const int32_t* query_lens,
                                   int64_t requests, int64_t block_size,
                                   const int32_t* free_blocks, int64_t num_free,
                                   const int32_t* free_start, int32_t* block_table,
                                   int64_t table_width, int64_t table_ld, int64_t* slot_mapping,
                                   int32_t* positions, int64_t max_tokens, int32_t* query_start,
                                   int32_t* seq_lens, int32_t* blocks_needed, void* stream);

/*
 * nvfp4_kv_fp8_attention -- attention of each request's new tokens over the cache: whole prompts,
 * chunks of prompts and single tokens, mixed in one call.
 *
 * Request r owns the query rows t in [query_start[r], query_start[r + 1]) and the key positions
 * j in [0, seq_lens[r]); its n query rows are the last n positions, p_t = seq_lens[r] - n + i.  Head h
 * reads KV head h / (heads / kv_heads).  With K, V the decoded rows of position j,
 *   x_j = scale * (q . K_j)
 *   x_j = softcap * tanh(x_j / softcap)                  where softcap > 0
 *   x_j = x_j + slopes[h] * (j - p_t)                    where slopes is given
 *   out = sum_j exp(x_j) V_j / sum_j exp(x_j)            over the visible j
 * j is visible when doc_start[t] <= j (document mask: the position at which the token's document
 * begins; 0 where doc_start is NULL) and, besides, j <= p_t or j < prefix_lens[r] (prefix mask: the
 * positions below the prefix's end are seen ahead of the causal order too; 0 where prefix_lens is NULL).
 * By itself the prefix mask shows the prefix to every token of the request.  Together with documents it
 * is bounded by them: a token sees of the prefix what lies in or behind the beginning of its own document.
 * So the two belong together where the prefix ends within the request's first document; then only that
 * document's tokens see it, all of it, and no document sees another.  A prefix that ends further on shows
 * a document's tokens what follows their document up to there (the masks say where a token's document
 * begins, not where it ends).  A prefix that all documents share is not among these masks.
 * A position whose table column or slot lies outside the table or the cache is not visible.  A row that
 * sees nothing gives zeros.
 * Rows t < query_start[0] or >= query_start[requests], and rows of other requests' gaps, are left as
 * they were.  Values in positions a row does not see have no effect on it, NaN codes included.
 *
 * Arithmetic: q . K is formed by MFMA with exact FP32 products of the query type and the decoded
 * codes, FP32 sums, FP32 scores and softmax statistics; exp(x - reference) is rounded once to FP16
 * (by at most 2^-11 relative, or 2^-29 of the row's largest where that is more) for the product with the
 * decoded values, summed in FP32; the result is rounded once to the query type.  Scores (times log2(e)) of -1e37 and less count as -infinity.  The cap adds an error of at most
 * 2^-20 min(softcap, max(128, |x_j|)) to a score; caps below 1e-9 count as 1e-9, above 1e37 as 1e37.
 *
 *   q             device, [tokens, heads, head_dim] of dtype (BF16 or F16), token and head strides in
 *                 elements (multiples of 8; head_dim contiguous); 16-byte aligned.
 *   tokens        rows of q and out; query_start entries are clamped to [0, tokens].
 *   heads, kv_heads  1 <= kv_heads <= heads <= 1024, heads a multiple of kv_heads.
 *   head_dim      64, 128 or 256.
 *   key_cache, value_cache, num_slots, cache_ld  as nvfp4_kv_fp8_store wrote them (16-byte aligned,
 *                 cache_ld a multiple of 16, >= kv_heads * head_dim and < 2^31); 1 <= num_slots < 2^31.
 *   key_scale, value_scale  device, one float each (decode direction).
 *   block_table   device, int32 [requests, table_width], row pitch table_ld.  Columns from
 *                 (2^31 - 256) / block_size (rounded down) on are not looked at.
 *   query_start, seq_lens   device, int32[requests + 1] (not decreasing) and int32[requests].
 *   scale         finite; softcap >= 0 and finite (0: no cap).
 *   slopes        device, float[heads], or NULL.
 *   doc_start     device, int32[tokens], or NULL; prefix_lens: device, int32[requests], or NULL.
 *   max_query_len, max_seq_len  bounds of the requests' query and key counts, >= 1: they only choose
 *                 how the work is divided (the results of requests above them are right too).
 *   out           device, as q; q itself with q's strides, or without overlap with it.
 *   workspace     device, 16-byte aligned, at least the bytes that nvfp4_kv_fp8_attention_workspace
 *                 gives for the same arguments; its contents are used within the call only.  Calls
 *                 that may run at the same time need one each.  May be NULL where that gives 0.
 * Single tokens take part in the row tiles of 256 that a prompt in the same call asks for, and cost as
 * much as a tile full of rows: many of them over long contexts are faster in a call of their own.
 * Errors: EINVAL (NULL, dtype, scale or softcap not as above), ESHAPE (sizes, strides that let output
 * elements overlap, a workspace too small), EALIGN.  tokens == 0 or requests == 0 launches nothing.
 */
nvfp4_status nvfp4_kv_fp8_attention(
    const void* q, nvfp4_dtype dtype, int64_t tokens, int64_t heads, int64_t kv_heads,
    int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* key_cache,
    const uint8_t* value_cache, const float* key_scale, const float* value_scale,
    int64_t num_slots, int64_t cache_ld, const int32_t* block_table, int64_t requests,
    int64_t table_width, int64_t table_ld, int64_t block_size, const int32_t* query_start,
    const int32_t* seq_lens, float scale, float softcap, const float* slopes,
    const int32_t* doc_start, const int32_t* prefix_lens, int64_t max_query_len,
    int64_t max_seq_len, void* out, int64_t out_token_stride, int64_t out_head_stride,
    void* workspace, int64_t workspace_bytes, void* stream);

/*
 * nvfp4_kv_fp8_tree_attention -- attention of trees of drafted tokens: request r's n query rows are
 * drafted tokens whose keys and values are stored at positions c .. c + n - 1, c = seq_lens[r] - n.
 * Row i sees every position below c, and position c + d where bit d % 64 of word d / 64 of
 * tree_mask[t] is set (d < n; bits past the words are 0): its ancestors, and itself if its own bit is
 * set.  One drafted token with bit 0 set is an ordinary decode step.
 *
 *   tree_mask     device, int64 [tokens, tree_words], row pitch tree_ld (elements); 8-byte aligned.
 *   tree_words    1 .. NVFP4_MAX_TREE_WORDS.
 *   positions     device, int32[tokens], or NULL: the position each drafted token counts at in the
 *                 distance bias (context length + depth in the tree), of queries and of drafted keys
 *                 alike; NULL takes c + i.  Read only where slopes is given.
 *   other arguments, arithmetic and errors as nvfp4_kv_fp8_attention.
 */
nvfp4_status nvfp4_kv_fp8_tree_attention(
    const void* q, nvfp4_dtype dtype, int64_t tokens, int64_t heads, int64_t kv_heads,
    int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* key_cache,
    const uint8_t* value_cache, const float* key_scale, const float* value_scale,
    int64_t num_slots, int64_t cache_ld, const int32_t* block_table, int64_t requests,
    int64_t table_width, int64_t table_ld, int64_t block_size, const int32_t* query_start,
    const int32_t* seq_lens, float scale, float softcap, const float* slopes,
    const int64_t* tree_mask, int64_t tree_words, int64_t tree_ld, const int32_t* positions,
    int64_t max_query_len, int64_t max_seq_len, void* out, int64_t out_token_stride,
    int64_t out_head_stride, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace of either attention for these arguments; 0 where none is needed, and where the
 * arguments are invalid (the attention then reports the error). */
int64_t nvfp4_kv_fp8_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads,
                                         int64_t head_dim, int64_t requests,
                                         int64_t max_query_len, int64_t max_seq_len);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_ATTENTION_H */
