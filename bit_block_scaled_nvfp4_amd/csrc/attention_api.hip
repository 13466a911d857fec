// Host layer of the cache's attention operators: argument validation (before any HIP call), division
// of the work, launch.  The contracts are in include/nvfp4_attention.h.
#include <stdint.h>

#include "attention_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxI32 = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxSpan = int64_t(1) << 40;
constexpr int64_t kMaxPositions = kMaxI32 - 255;  // of a request that an attention looks at
constexpr int64_t kMaxBlockSize = int64_t(1) << 24;

nvfp4_status device_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_EDEVICE; }

// Row pitch and extent of a [rows, width] int32 table.
bool table_fits(int64_t rows, int64_t width, int64_t ld) {
  return width >= 0 && width <= kMaxI32 && ld >= width && ld >= 1 && ld <= kMaxSpan &&
         (rows == 0 || ld <= kMaxSpan / rows);
}

// Extent of [tokens, heads, head_dim] with these strides; false when a stride is negative or the
// extent too large.
bool span_fits(int64_t tokens, int64_t heads, int64_t head_dim, int64_t ts, int64_t hs) {
  if (ts < 0 || hs < 0 || ts > kMaxSpan || hs > kMaxSpan) return false;
  if (tokens > 1 && ts > kMaxSpan / (tokens - 1)) return false;
  if (heads > 1 && hs > kMaxSpan / (heads - 1)) return false;
  return (tokens - 1) * ts + (heads - 1) * hs + head_dim <= kMaxSpan;
}

// Whether no two elements of an output with these strides share an address.
bool distinct(int64_t tokens, int64_t heads, int64_t head_dim, int64_t ts, int64_t hs) {
  if (tokens == 1) return heads == 1 || hs >= head_dim;
  if (heads == 1) return ts >= head_dim;
  return (hs >= head_dim && ts >= (heads - 1) * hs + head_dim) ||
         (ts >= head_dim && hs >= (tokens - 1) * ts + head_dim);
}

bool shape_ok(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t requests,
              int64_t max_query_len, int64_t max_seq_len) {
  return tokens >= 0 && heads >= 1 && heads <= 1024 && kv_heads >= 1 && heads % kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) && tokens <= kMaxI32 / heads &&
         requests >= 0 && requests <= NVFP4_MAX_REQUESTS && max_query_len >= 1 &&
         max_query_len <= kMaxI32 && max_seq_len >= 1 && max_seq_len <= kMaxI32;
}

// A bound above what the tokens allow says nothing more.
int64_t query_bound(int64_t max_query_len, int64_t tokens) {
  return max_query_len < tokens ? max_query_len : tokens;
}

struct Call {
  const void* q;
  int dtype;
  int64_t tokens, heads, kv_heads, head_dim, q_ts, q_hs;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  int64_t num_slots, cache_ld;
  const int32_t* table;
  int64_t requests, table_width, table_ld, block_size;
  const int32_t *query_start, *seq_lens;
  float scale, softcap;
  const float* slopes;
  int64_t max_query_len, max_seq_len;
  void* out;
  int64_t out_ts, out_hs;
  void* workspace;
  int64_t workspace_bytes;
};

// Checks everything that both attentions take; `empty` says that there is nothing to compute.
nvfp4_status check(const Call& c, bool* empty) {
  if (c.dtype != NVFP4_BF16 && c.dtype != NVFP4_F16) return NVFP4_EINVAL;
  if (!shape_ok(c.tokens, c.heads, c.kv_heads, c.head_dim, c.requests, c.max_query_len, c.max_seq_len))
    return NVFP4_ESHAPE;
  *empty = c.tokens == 0 || c.requests == 0;
  if (!c.ks || !c.vs || !c.query_start) return NVFP4_EINVAL;
  if (!*empty && (!c.q || !c.out || !c.kc || !c.vc || !c.seq_lens || (!c.table && c.table_width > 0)))
    return NVFP4_EINVAL;
  // written so that a NaN fails
  if (!(c.scale - c.scale == 0.0f) || !(c.softcap - c.softcap == 0.0f) || !(c.softcap >= 0.0f))
    return NVFP4_EINVAL;
  if (!table_fits(c.requests, c.table_width, c.table_ld)) return NVFP4_ESHAPE;
  if (c.block_size < 1 || c.block_size > kMaxBlockSize) return NVFP4_ESHAPE;
  if (c.num_slots < 0 || c.num_slots > kMaxI32 || (!*empty && c.num_slots < 1)) return NVFP4_ESHAPE;
  if (c.cache_ld < c.kv_heads * c.head_dim || c.cache_ld > kMaxI32 ||
      (c.num_slots > 0 && c.cache_ld > kMaxSpan / c.num_slots))
    return NVFP4_ESHAPE;
  if (!*empty) {
    if (!span_fits(c.tokens, c.heads, c.head_dim, c.q_ts, c.q_hs) ||
        !span_fits(c.tokens, c.heads, c.head_dim, c.out_ts, c.out_hs) ||
        !distinct(c.tokens, c.heads, c.head_dim, c.out_ts, c.out_hs))
      return NVFP4_ESHAPE;
  }
  if (!aligned(c.q, 16) || !aligned(c.out, 16) || c.q_ts % 8 || c.q_hs % 8 || c.out_ts % 8 ||
      c.out_hs % 8 || !aligned(c.kc, 16) || !aligned(c.vc, 16) || c.cache_ld % 16 ||
      !aligned(c.ks, 4) || !aligned(c.vs, 4) || !aligned(c.table, 4) || !aligned(c.query_start, 4) ||
      !aligned(c.seq_lens, 4) || !aligned(c.slopes, 4) || !aligned(c.workspace, 16))
    return NVFP4_EALIGN;
  return NVFP4_OK;
}

nvfp4_status run(const Call& c, const int32_t* doc_start, const int32_t* prefix_lens,
                 const int64_t* tree, int64_t tree_words, int64_t tree_ld,
                 const int32_t* positions, void* stream) {
  const int64_t longest = query_bound(c.max_query_len, c.tokens);
  const nvfp4::AttnPlan p = nvfp4::plan_attention(c.tokens, c.heads, c.kv_heads, c.head_dim, c.requests, longest, c.max_seq_len);
  if (p.workspace > 0) {
    if (!c.workspace) return NVFP4_EINVAL;
    if (c.workspace_bytes < p.workspace) return NVFP4_ESHAPE;
  }
  nvfp4::AttnArgs a{};
  a.q = static_cast<const uint16_t*>(c.q);
  a.q_ts = c.q_ts;
  a.q_hs = c.q_hs;
  a.out = static_cast<uint16_t*>(c.out);
  a.out_ts = c.out_ts;
  a.out_hs = c.out_hs;
  a.kc = c.kc;
  a.vc = c.vc;
  a.cache_ld = c.cache_ld;
  a.ks = c.ks;
  a.vs = c.vs;
  a.table = c.table;
  a.table_ld = c.table_ld;
  a.query_start = c.query_start;
  a.seq_lens = c.seq_lens;
  a.slopes = c.slopes;
  a.doc_start = doc_start;
  a.prefix_lens = prefix_lens;
  a.tree = tree;
  a.tree_ld = tree_ld;
  a.tree_words = (int32_t)tree_words;
  a.positions = positions;
  a.num_slots = (int32_t)c.num_slots;
  // the end of a tile of keys has to stay below 2^31
  const int64_t columns = kMaxPositions / c.block_size;
  a.table_width = (int32_t)(c.table_width < columns ? c.table_width : columns);
  a.requests = (int32_t)c.requests;
  a.tokens = (int32_t)c.tokens;
  a.heads = (int32_t)c.heads;
  a.kv_heads = (int32_t)c.kv_heads;
  const int64_t group = c.heads / c.kv_heads;
  a.row_tiles = p.row_tiles;
  a.all_tiles = p.all_tiles;
  a.workers = p.workers;
  a.bs = nvfp4::make_fast_div((uint32_t)c.block_size);
  a.group = nvfp4::make_fast_div((uint32_t)group);
  a.scale = c.scale;
  // below 1e-9 the capped scores change no weight in FP32, and 1e37 bounds the scores that count: between them
  // the cap's factors are finite
  a.cap = c.softcap > 0.0f ? (c.softcap < 1e-9f ? 1e-9f : (c.softcap > 1e37f ? 1e37f : c.softcap)) : 0.0f;
  if (p.workers) {
    const int64_t rows = 2 * (int64_t)p.workers * p.rows;
    a.part = static_cast<float*>(c.workspace);
    a.part_ml = a.part + rows * c.head_dim;
    a.headers = reinterpret_cast<int32_t*>(a.part_ml + rows * 2);
  }
  return device_status(nvfp4::launch_attention(a, p, (int)c.head_dim, c.dtype == NVFP4_BF16,
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
               workspace, workspace_bytes};
  bool empty = false;
  const nvfp4_status st = check(c, &empty);
  if (st != NVFP4_OK) return st;
  if (!aligned(doc_start, 4) || !aligned(prefix_lens, 4)) return NVFP4_EALIGN;
  if (empty) return NVFP4_OK;
  return run(c, doc_start, prefix_lens, nullptr, 0, 0, nullptr, stream);
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
               workspace, workspace_bytes};
  bool empty = false;
  const nvfp4_status st = check(c, &empty);
  if (st != NVFP4_OK) return st;
  if (!empty && !tree_mask) return NVFP4_EINVAL;
  if (tree_words < 1 || tree_words > NVFP4_MAX_TREE_WORDS || tree_ld < tree_words ||
      tree_ld > kMaxSpan || (tokens > 0 && tree_ld > kMaxSpan / tokens))
    return NVFP4_ESHAPE;
  if (!aligned(tree_mask, 8) || !aligned(positions, 4)) return NVFP4_EALIGN;
  if (empty) return NVFP4_OK;
  return run(c, nullptr, nullptr, tree_mask, tree_words, tree_ld, positions, stream);
}

int64_t nvfp4_kv_fp8_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads,
                                         int64_t head_dim, int64_t requests,
                                         int64_t max_query_len, int64_t max_seq_len) {
  if (!shape_ok(tokens, heads, kv_heads, head_dim, requests, max_query_len, max_seq_len)) return 0;
  if (tokens == 0 || requests == 0) return 0;
  return nvfp4::plan_attention(tokens, heads, kv_heads, head_dim, requests, query_bound(max_query_len, tokens), max_seq_len).workspace;
}

}  // extern "C"
