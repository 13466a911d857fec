/*
 * nvfp4_serving.h -- C ABI of the other operators of a serving step: norms and position rotation of
 * queries and keys, appending keys and values to the paged caches, attention over a cache held in 4 bits
 * (NVFP4), and verification of drafted tokens.  Part of libnvfp4.so (gfx950); the conventions of nvfp4.h
 * hold here too: device pointers, caller-owned buffers, no allocation, no host synchronisation, every
 * check before any HIP call, results deterministic.
 *
 * A step calls them in this order:
 *   nvfp4_kv_block_tables -> nvfp4_qk_norm_rope -> nvfp4_kv_fp8_append or nvfp4_kv_fp4_append ->
 *   nvfp4_kv_fp8_attention or nvfp4_kv_fp4_attention (their tree forms for drafted tokens) ->
 *   nvfp4_verify_drafted
 *
 * The 4-bit cache.  Keys are held in two arrays, values in two more:
 *   codes   [num_blocks, kv_heads, block_size, head_dim / 2]   E2M1 codes, element 2j low in byte j
 *   scales  [num_blocks, kv_heads, block_size, head_dim / 16]  E4M3 scale of each 16 elements
 * A head's row is encoded by the rules of nvfp4.h under a static global scale g (encode direction): element =
 * V(code) * E4M3(scale) / g.  One step differs: the block scale's factor is the product fl(g * fl(1/6)), not the
 * quotient fl(g / 6) of nvfp4_quantize.  The two are equal or neighbours, so a block takes another scale than there
 * only where its scaled maximum lies within 2^-22 of the middle between two scale codes, where either is as near.
 * Where g is six times a binary32 number the factors are the same number, and so are all codes and scales.  Slot s of a
 * slot map is row s % block_size of block
 * s / block_size, as in the FP8 cache, so nvfp4_kv_block_tables serves both.  A KV head's rows of a block
 * lie together: 9/16 byte an element, read in whole lines.
 *
 * Source: ai.info summary of arXiv 2609.04098, "Methodology in Plain English" (E2M1 values, one E4M3 scale
 * per 16 elements under an FP32 global scale) and "Key Contributions" (a KV cache with calibrated per-layer
 * scales).  The pages hold the cache in FP8 and give no formula for the norms, the rotation, the attention
 * or the verification: the definitions below are this library's.
 */
#ifndef NVFP4_SERVING_H
#define NVFP4_SERVING_H

#include "nvfp4_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head vector of nvfp4_qk_norm_rope, elements. */
#define NVFP4_MAX_HEAD_DIM 512

/*
 * nvfp4_qk_norm_rope -- norm and position rotation of the head vectors of queries and keys, in one pass.
 *
 * A head vector x[0 .. head_dim) of token t becomes
 *   n_i = x_i / sqrt(mean(x^2) + eps) * (weight_offset + weight_i)   where a weight is given, else x_i
 *   a' = a cos(w) - b sin(w),  b' = b cos(w) + a sin(w),   w = positions[t] * inv_freq[i]
 * for the pairs (a, b) = (n_i, n_{i + num_freq}), or (n_2i, n_{2i + 1}) where interleaved is 1,
 * i < num_freq; elements from 2 num_freq on are not rotated.  The result is rounded once to dtype (to
 * nearest even) from a value formed in binary64: angles, cosines and sums are right for every position, and
 * the result is the exact value's rounding unless that lies within about 2^-48 (|a| + |b|) of the middle
 * between two numbers.  Angles of more than 2^31 lose accuracy.  NaN and infinities spread over the head vector
 * that holds them.
 *
 *   q, k          device, [tokens, q_heads, head_dim] and [tokens, k_heads, head_dim] of dtype (F32, BF16 or
 *                 F16), token and head strides in elements (in bytes multiples of 16 and below 2^32, head_dim
 *                 contiguous); 16-byte aligned.  k may be absent: k_heads 0.
 *   head_dim      a multiple of 16, 16 .. NVFP4_MAX_HEAD_DIM; q_heads 1 .. 1024; k_heads 0 .. 1024.
 *   positions     device, int32[tokens]; inv_freq: device, float[num_freq].  Both NULL with num_freq 0: no
 *                 rotation.  num_freq: a multiple of 8, at most head_dim / 2.
 *   interleaved   0 or 1.
 *   q_weight, k_weight  device, head_dim elements of weight_dtype each (aligned to them), or NULL: no norm.
 *   eps           >= 0 and finite; weight_offset: finite (1 where weights are held less 1).
 *   q_out, k_out  device, as q and k with strides of their own; each may be its own input with the same
 *                 strides (in place), and overlaps nothing otherwise.
 * Errors: EINVAL (NULL, dtype, flag, eps or weight_offset not as above), ESHAPE, EALIGN.  tokens == 0 launches
 * nothing.
 */
nvfp4_status nvfp4_qk_norm_rope(const void* q, int64_t q_heads, int64_t q_token_stride,
                                int64_t q_head_stride, const void* k, int64_t k_heads,
                                int64_t k_token_stride, int64_t k_head_stride, nvfp4_dtype dtype,
                                int64_t tokens, int64_t head_dim, const int32_t* positions,
                                const float* inv_freq, int64_t num_freq, int interleaved,
                                const void* q_weight, const void* k_weight, nvfp4_dtype weight_dtype,
                                double eps, double weight_offset, void* q_out,
                                int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                                int64_t k_out_token_stride, int64_t k_out_head_stride, void* stream);

/*
 * nvfp4_kv_fp8_append -- norm and rotate the new tokens' keys, encode keys and values to FP8 and write them
 * into their slots: bit for bit what nvfp4_qk_norm_rope of the keys (rounded to dtype, as there) and then
 * nvfp4_kv_fp8_store give, without the rotated keys ever being written.
 *
 *   key, value    device, [tokens, kv_heads, head_dim] of dtype, strides as in nvfp4_qk_norm_rope.
 *   kv_heads      1 .. 1024; head_dim: 64, 128 or 256.
 *   positions .. weight_offset   as nvfp4_qk_norm_rope; k_weight is the keys' (values are stored as they are).
 *   key_scale, value_scale, slot_mapping, key_cache, value_cache, num_slots, cache_ld   as
 *                 nvfp4_kv_fp8_store: decode-direction scales, int64[tokens] slots (NULL: token t in slot t;
 *                 slots outside [0, num_slots) are skipped; two tokens with one slot race).
 * No cache overlaps an input or the other cache.  Errors as nvfp4_qk_norm_rope.
 */
nvfp4_status nvfp4_kv_fp8_append(const void* key, const void* value, nvfp4_dtype dtype, int64_t tokens,
                                 int64_t kv_heads, int64_t head_dim, int64_t key_token_stride,
                                 int64_t key_head_stride, int64_t value_token_stride,
                                 int64_t value_head_stride, const int32_t* positions,
                                 const float* inv_freq, int64_t num_freq, int interleaved,
                                 const void* k_weight, nvfp4_dtype weight_dtype, double eps,
                                 double weight_offset, const float* key_scale, const float* value_scale,
                                 const int64_t* slot_mapping, uint8_t* key_cache, uint8_t* value_cache,
                                 int64_t num_slots, int64_t cache_ld, void* stream);

/*
 * nvfp4_kv_fp4_append -- the same into the 4-bit cache: the keys as nvfp4_qk_norm_rope gives them and the values,
 * encoded as said above.  Codes and scales are bit-exact.
 *
 *   num_freq      a multiple of 16 where interleaved is 0 (a block of 16 then holds one half of its pairs).
 *   key_gscale, value_gscale  device, one float each (encode direction, positive and finite: not checked).
 *   key_codes, key_scales, value_codes, value_scales   device, as above, contiguous; 16-byte aligned.
 *   num_blocks, block_size    num_blocks >= 0, block_size 1 .. 2^24,
 *                             num_blocks * block_size * kv_heads < 2^31.
 *   slot_mapping  device, int64[tokens] or NULL; slots outside [0, num_blocks * block_size) are skipped.
 * Other arguments and errors as nvfp4_kv_fp8_append.
 */
nvfp4_status nvfp4_kv_fp4_append(const void* key, const void* value, nvfp4_dtype dtype, int64_t tokens,
                                 int64_t kv_heads, int64_t head_dim, int64_t key_token_stride,
                                 int64_t key_head_stride, int64_t value_token_stride,
                                 int64_t value_head_stride, const int32_t* positions,
                                 const float* inv_freq, int64_t num_freq, int interleaved,
                                 const void* k_weight, nvfp4_dtype weight_dtype, double eps,
                                 double weight_offset, const float* key_gscale,
                                 const float* value_gscale, const int64_t* slot_mapping,
                                 uint8_t* key_codes, uint8_t* key_scales, uint8_t* value_codes,
                                 uint8_t* value_scales, int64_t num_blocks, int64_t block_size,
                                 void* stream);

/*
 * nvfp4_kv_fp4_load -- gather slots of the 4-bit cache (keys or values) and decode them:
 * out = fl(V(code) * E4M3(scale) / g), one correctly rounded binary32 division, rounded once more to BF16
 * (nearest even) when out_dtype is BF16.  Bit 7 of a scale byte is not looked at; 0x7F, which the encoder
 * does not write, counts as 480 (so in the attentions).
 *
 *   codes, scales device, as above; head_dim 64, 128 or 256; kv_heads 1 .. 1024.
 *   gscale        device, one float.
 *   slot_mapping  device, int64[tokens], or NULL (slot t); a slot outside the cache gives zeros.
 *   out           device, [tokens, kv_heads, head_dim] of out_dtype (F32 or BF16), contiguous; 16-byte
 *                 aligned.  Overlaps no input.
 * Errors as nvfp4_kv_fp4_append.
 */
nvfp4_status nvfp4_kv_fp4_load(const uint8_t* codes, const uint8_t* scales, int64_t num_blocks,
                               int64_t kv_heads, int64_t block_size, int64_t head_dim,
                               const float* gscale, const int64_t* slot_mapping, int64_t tokens, void* out,
                               nvfp4_dtype out_dtype, void* stream);

/*
 * nvfp4_kv_fp4_attention -- nvfp4_kv_fp8_attention over the 4-bit cache: the same definition, masks and
 * arithmetic, with K and V the decoded rows V(code) * E4M3(scale) / g.  What the cache holds where nothing
 * was written (any bytes) has no effect on rows that do not see it.
 *
 *   key_codes, key_scales, value_codes, value_scales  device, as above, contiguous; 16-byte aligned.
 *   key_gscale, value_gscale  device, one float each (encode direction).
 *   num_blocks, block_size    as nvfp4_kv_fp4_append (num_blocks >= 1).
 *   other arguments and errors  as nvfp4_kv_fp8_attention; workspace as
 *                 nvfp4_kv_fp4_attention_workspace says.
 */
nvfp4_status nvfp4_kv_fp4_attention(
    const void* q, nvfp4_dtype dtype, int64_t tokens, int64_t heads, int64_t kv_heads,
    int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* key_codes,
    const uint8_t* key_scales, const uint8_t* value_codes, const uint8_t* value_scales,
    const float* key_gscale, const float* value_gscale, int64_t num_blocks, int64_t block_size,
    const int32_t* block_table, int64_t requests, int64_t table_width, int64_t table_ld,
    const int32_t* query_start, const int32_t* seq_lens, float scale, float softcap,
    const float* slopes, const int32_t* doc_start, const int32_t* prefix_lens, int64_t max_query_len,
    int64_t max_seq_len, void* out, int64_t out_token_stride, int64_t out_head_stride,
    void* workspace, int64_t workspace_bytes, void* stream);

/* nvfp4_kv_fp8_tree_attention over the 4-bit cache. */
nvfp4_status nvfp4_kv_fp4_tree_attention(
    const void* q, nvfp4_dtype dtype, int64_t tokens, int64_t heads, int64_t kv_heads,
    int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* key_codes,
    const uint8_t* key_scales, const uint8_t* value_codes, const uint8_t* value_scales,
    const float* key_gscale, const float* value_gscale, int64_t num_blocks, int64_t block_size,
    const int32_t* block_table, int64_t requests, int64_t table_width, int64_t table_ld,
    const int32_t* query_start, const int32_t* seq_lens, float scale, float softcap,
    const float* slopes, const int64_t* tree_mask, int64_t tree_words, int64_t tree_ld,
    const int32_t* positions, int64_t max_query_len, int64_t max_seq_len, void* out,
    int64_t out_token_stride, int64_t out_head_stride, void* workspace, int64_t workspace_bytes,
    void* stream);

/* Bytes of workspace of either attention over the 4-bit cache for these arguments; 0 where none is needed, and where
 * the arguments are invalid (the attention then reports the error). */
int64_t nvfp4_kv_fp4_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads,
                                         int64_t head_dim, int64_t requests, int64_t max_query_len,
                                         int64_t max_seq_len);

/*
 * nvfp4_verify_drafted -- verification of drafted tokens against the target's probabilities, from given
 * random numbers, so that what is emitted is distributed as the target's own samples are.
 *
 * Request r owns rows query_start[r] .. query_start[r + 1] - 1 of the step: its last accepted token, then its
 * drafted tokens, one after another (chains; drafted trees are not verified by this call).  With s =
 * query_start[r] and n + 1 its rows, row s + i holds the target's probabilities p_i of the token after input
 * token i, and, for i < n, the draft's q_i, from which token x_i = tokens[s + i + 1] was drawn.
 *   x_i is accepted while  accept_u[s + i] * q_i(x_i) < p_i(x_i)   (the products exact; a token outside
 *   [0, vocab) is not accepted); a = number of tokens accepted before the first that is not.
 *   The next token is sampled from the weights  w(v) = max(p_a(v) - q_a(v), 0)  if a < n, or p_n(v) if a = n:
 *   the lowest v with w(v) > 0 and  sum_{u <= v} w(u) > sample_u[r] * sum_u w(u).  Where all w are zero, p_a
 *   takes their place; sample_u of 1 or more (or NaN) takes the last v with w(v) > 0; a p_a without a positive
 *   value gives -1.
 * Without draft_probs the drafted tokens count as certain: q_i(x_i) = 1, q_i(v) = 0 otherwise.
 *   accepted[r] = a;  out_tokens[s + i] = x_i for i < a, the sampled token for i = a, -1 for a < i <= n.
 * A request without rows has accepted 0.  Entries of out_tokens of no request are left as they were.  Starts that fall
 * leave a request without rows, or rows with several requests: each is verified over all its rows, and the last of
 * them writes such a row.
 * Sums are formed in binary64 in a fixed order.  NaN probabilities count as 0 weights and are not accepted.
 *
 *   target_probs  device, float [rows, vocab], row pitch target_ld >= vocab (elements); 4-byte aligned.
 *   draft_probs   device, float [rows, vocab], row pitch draft_ld, or NULL; its row s + n is not read.
 *   rows, vocab   0 <= rows < 2^31 - 4096, 1 <= vocab < 2^31 - 4096; rows * ld <= 2^40.
 *   tokens        device, int32[rows]: the step's input tokens.
 *   query_start   device, int32[requests + 1]; entries are clamped to [0, rows].
 *   accept_u      device, float[rows] (entry s + n is not read); sample_u: device, float[requests]; both of [0, 1).
 *   accepted      device, int32[requests]; out_tokens: device, int32[rows].  Overlap no input and not each other.
 *   workspace     device, 16-byte aligned, at least the bytes that nvfp4_verify_drafted_workspace gives; used
 *                 within the call only.  Calls that may run at the same time need one each.
 * Errors: EINVAL (NULL), ESHAPE, EALIGN.  requests == 0 launches nothing.
 */
nvfp4_status nvfp4_verify_drafted(const float* target_probs, int64_t target_ld, const float* draft_probs,
                                  int64_t draft_ld, int64_t rows, int64_t vocab, const int32_t* tokens,
                                  const int32_t* query_start, int64_t requests, const float* accept_u,
                                  const float* sample_u, int32_t* accepted, int32_t* out_tokens,
                                  void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace of nvfp4_verify_drafted; 0 where the arguments are invalid or nothing is to be done. */
int64_t nvfp4_verify_drafted_workspace(int64_t requests, int64_t vocab);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_SERVING_H */
