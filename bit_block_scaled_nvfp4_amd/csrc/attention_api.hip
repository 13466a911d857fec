// Host layer of the cache's attention operators: argument validation (before any HIP call), division
// of the work, launch.  The contracts are in include/nvfp4_attention.h.
#include "attention_checks.h"

namespace {

nvfp4_status run(const Call& c, const Masks& m, void* stream) {
  const int64_t longest = query_bound(c.max_query_len, c.tokens);
  const nvfp4::AttnPlan p = nvfp4::plan_attention(c.tokens, c.heads, c.kv_heads, c.head_dim, c.requests, longest, c.max_seq_len);
  if (p.workspace > 0) {
    if (!c.workspace) return NVFP4_EINVAL;
    if (c.workspace_bytes < p.workspace) return NVFP4_ESHAPE;
  }
  return device_status(nvfp4::launch_attention(kernel_args(c, p, m), p, (int)c.head_dim, c.dtype == NVFP4_BF16,
                                               reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_kv_block_tables(const int32_t* context_lens, const int32_t* query_lens,
                                   int64_t requests, int64_t block_size,
                                   const int32_t* free_blocks, int64_t num_free,
                                   const int32_t* free_start, int32_t* block_table,
                                   int64_t table_width, int64_t table_ld, int64_t* slot_mapping,
                                   int32_t* positions, int64_t max_tokens, int32_t* query_start,
                                   int32_t* seq_lens, int32_t* blocks_needed, void* stream) {
  if (requests < 0 || requests > NVFP4_MAX_REQUESTS || block_size < 1 || block_size > kMaxBlockSize ||
      num_free < 0 || num_free > kMaxI32 || max_tokens < 0 || max_tokens > kMaxI32 - 256 ||
      !table_fits(requests, table_width, table_ld))
    return NVFP4_ESHAPE;
  if (!query_start || !blocks_needed || (num_free > 0 && !free_blocks)) return NVFP4_EINVAL;
  if (requests > 0 && (!context_lens || !query_lens || !seq_lens || (!block_table && table_width > 0)))
    return NVFP4_EINVAL;
  if (max_tokens > 0 && (!slot_mapping || !positions)) return NVFP4_EINVAL;
  if (!aligned(context_lens, 4) || !aligned(query_lens, 4) || !aligned(free_blocks, 4) ||
      !aligned(free_start, 4) || !aligned(block_table, 4) || !aligned(slot_mapping, 8) ||
      !aligned(positions, 4) || !aligned(query_start, 4) || !aligned(seq_lens, 4) ||
      !aligned(blocks_needed, 4))
    return NVFP4_EALIGN;
  nvfp4::TablesArgs a{};
  a.context_lens = context_lens;
  a.query_lens = query_lens;
  a.free_blocks = free_blocks;
  a.free_start = free_start;
  a.block_table = block_table;
  a.slot_mapping = slot_mapping;
  a.positions = positions;
  a.query_start = query_start;
  a.seq_lens = seq_lens;
  a.blocks_needed = blocks_needed;
  a.table_ld = table_ld;
  a.requests = (int32_t)requests;
  a.table_width = (int32_t)table_width;
  a.num_free = (int32_t)num_free;
  a.max_tokens = (int32_t)max_tokens;
  a.bs = nvfp4::make_fast_div((uint32_t)block_size);
  return device_status(nvfp4::launch_block_tables(a, reinterpret_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_fp8_attention(
    const void* q, nvfp4_dtype dtype, int64_t tokens, int64_t heads, int64_t kv_heads,
    int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* key_cache,
    const uint8_t* value_cache, const float* key_scale, const float* value_scale,
    int64_t num_slots, int64_t cache_ld, const int32_t* block_table, int64_t requests,
    int64_t table_width, int64_t table_ld, int64_t block_size, const int32_t* query_start,
    const int32_t* seq_lens, float scale, float softcap, const float* slopes,
    const int32_t* doc_start, const int32_t* prefix_lens, int64_t max_query_len,
    int64_t max_seq_len, void* out, int64_t out_token_stride, int64_t out_head_stride,
    void* workspace, int64_t workspace_bytes, void* stream) {
  const Call c{q, (int)dtype, tokens, heads, kv_heads, head_dim, q_token_stride, q_head_stride,
               key_cache, value_cache, key_scale, value_scale, num_slots, cache_ld, block_table,
               requests, table_width, table_ld, block_size, query_start, seq_lens, scale, softcap,
               slopes, max_query_len, max_seq_len, out, out_token_stride, out_head_stride,
               workspace, workspace_bytes, false, nullptr, nullptr};
  bool empty = false;
  const nvfp4_status st = check(c, &empty);
  if (st != NVFP4_OK) return st;
  if (!aligned(doc_start, 4) || !aligned(prefix_lens, 4)) return NVFP4_EALIGN;
  if (empty) return NVFP4_OK;
  return run(c, Masks{doc_start, prefix_lens, nullptr, 0, 0, nullptr}, stream);
}

nvfp4_status nvfp4_kv_fp8_tree_attention(
    const void* q, nvfp4_dtype dtype, int64_t tokens, int64_t heads, int64_t kv_heads,
    int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* key_cache,
    const uint8_t* value_cache, const float* key_scale, const float* value_scale,
    int64_t num_slots, int64_t cache_ld, const int32_t* block_table, int64_t requests,
    int64_t table_width, int64_t table_ld, int64_t block_size, const int32_t* query_start,
    const int32_t* seq_lens, float scale, float softcap, const float* slopes,
    const int64_t* tree_mask, int64_t tree_words, int64_t tree_ld, const int32_t* positions,
    int64_t max_query_len, int64_t max_seq_len, void* out, int64_t out_token_stride,
    int64_t out_head_stride, void* workspace, int64_t workspace_bytes, void* stream) {
  const Call c{q, (int)dtype, tokens, heads, kv_heads, head_dim, q_token_stride, q_head_stride,
               key_cache, value_cache, key_scale, value_scale, num_slots, cache_ld, block_table,
               requests, table_width, table_ld, block_size, query_start, seq_lens, scale, softcap,
               slopes, max_query_len, max_seq_len, out, out_token_stride, out_head_stride,
               workspace, workspace_bytes, false, nullptr, nullptr};
  bool empty = false;
  const nvfp4_status st = check(c, &empty);
  if (st != NVFP4_OK) return st;
  const Masks m{nullptr, nullptr, tree_mask, tree_words, tree_ld, positions};
  const nvfp4_status tree = check_tree(c, empty, m);
  if (tree != NVFP4_OK) return tree;
  if (empty) return NVFP4_OK;
  return run(c, m, stream);
}

int64_t nvfp4_kv_fp8_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads,
                                         int64_t head_dim, int64_t requests,
                                         int64_t max_query_len, int64_t max_seq_len) {
  if (!shape_ok(tokens, heads, kv_heads, head_dim, requests, max_query_len, max_seq_len)) return 0;
  if (tokens == 0 || requests == 0) return 0;
  return nvfp4::plan_attention(tokens, heads, kv_heads, head_dim, requests, query_bound(max_query_len, tokens), max_seq_len).workspace;
}

}  // extern "C"
