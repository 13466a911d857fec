// What the host layers of the cache's attentions share: validation of a call's arguments and the kernels' arguments
// from them.
#pragma once

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
  // the 4-bit cache: block scales of keys and values (kc, vc: codes; num_slots: blocks * block_size; cache_ld unused)
  bool fp4;
  const uint8_t *kbs, *vbs;
};

// Whether the cache's extent fits: rows of cache_ld bytes, or (4-bit cache) rows of head_dim / 2 bytes that are
// numbered in 32 bits.
bool cache_fits(const Call& c) {
  if (c.fp4) return c.num_slots <= kMaxI32 / c.kv_heads;
  return c.cache_ld >= c.kv_heads * c.head_dim && c.cache_ld <= kMaxI32 &&
         (c.num_slots <= 0 || c.cache_ld <= kMaxSpan / c.num_slots);
}

// Checks everything that all attentions take; `empty` says that there is nothing to compute.
nvfp4_status check(const Call& c, bool* empty) {
  if (c.dtype != NVFP4_BF16 && c.dtype != NVFP4_F16) return NVFP4_EINVAL;
  if (!shape_ok(c.tokens, c.heads, c.kv_heads, c.head_dim, c.requests, c.max_query_len, c.max_seq_len))
    return NVFP4_ESHAPE;
  *empty = c.tokens == 0 || c.requests == 0;
  if (!c.ks || !c.vs || !c.query_start) return NVFP4_EINVAL;
  if (!*empty && (!c.q || !c.out || !c.kc || !c.vc || !c.seq_lens || (!c.table && c.table_width > 0)))
    return NVFP4_EINVAL;
  if (!*empty && c.fp4 && (!c.kbs || !c.vbs)) return NVFP4_EINVAL;
  // written so that a NaN fails
  if (!(c.scale - c.scale == 0.0f) || !(c.softcap - c.softcap == 0.0f) || !(c.softcap >= 0.0f))
    return NVFP4_EINVAL;
  if (!table_fits(c.requests, c.table_width, c.table_ld)) return NVFP4_ESHAPE;
  if (c.block_size < 1 || c.block_size > kMaxBlockSize) return NVFP4_ESHAPE;
  if (c.num_slots < 0 || c.num_slots > kMaxI32 || (!*empty && c.num_slots < 1)) return NVFP4_ESHAPE;
  if (!cache_fits(c)) return NVFP4_ESHAPE;
  if (!*empty) {
    if (!span_fits(c.tokens, c.heads, c.head_dim, c.q_ts, c.q_hs) ||
        !span_fits(c.tokens, c.heads, c.head_dim, c.out_ts, c.out_hs) ||
        !distinct(c.tokens, c.heads, c.head_dim, c.out_ts, c.out_hs))
      return NVFP4_ESHAPE;
  }
  if (!aligned(c.q, 16) || !aligned(c.out, 16) || c.q_ts % 8 || c.q_hs % 8 || c.out_ts % 8 ||
      c.out_hs % 8 || !aligned(c.kc, 16) || !aligned(c.vc, 16) || c.cache_ld % 16 ||
      !aligned(c.ks, 4) || !aligned(c.vs, 4) || !aligned(c.table, 4) || !aligned(c.query_start, 4) ||
      !aligned(c.seq_lens, 4) || !aligned(c.slopes, 4) || !aligned(c.workspace, 16) || !aligned(c.kbs, 16) ||
      !aligned(c.vbs, 16))
    return NVFP4_EALIGN;
  return NVFP4_OK;
}

// A tree's words, documents and prefixes: what one or the other attention takes besides.
struct Masks {
  const int32_t *doc_start, *prefix_lens;
  const int64_t* tree;
  int64_t tree_words, tree_ld;
  const int32_t* positions;
};

nvfp4_status check_tree(const Call& c, bool empty, const Masks& m) {
  if (!empty && !m.tree) return NVFP4_EINVAL;
  if (m.tree_words < 1 || m.tree_words > NVFP4_MAX_TREE_WORDS || m.tree_ld < m.tree_words ||
      m.tree_ld > kMaxSpan || (c.tokens > 0 && m.tree_ld > kMaxSpan / c.tokens))
    return NVFP4_ESHAPE;
  if (!aligned(m.tree, 8) || !aligned(m.positions, 4)) return NVFP4_EALIGN;
  return NVFP4_OK;
}

nvfp4::AttnArgs kernel_args(const Call& c, const nvfp4::AttnPlan& p, const Masks& m) {
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
  a.kbs = c.kbs;
  a.vbs = c.vbs;
  a.ks = c.ks;
  a.vs = c.vs;
  a.table = c.table;
  a.table_ld = c.table_ld;
  a.query_start = c.query_start;
  a.seq_lens = c.seq_lens;
  a.slopes = c.slopes;
  a.doc_start = m.doc_start;
  a.prefix_lens = m.prefix_lens;
  a.tree = m.tree;
  a.tree_ld = m.tree_ld;
  a.tree_words = (int32_t)m.tree_words;
  a.positions = m.positions;
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
  return a;
}

}  // namespace
