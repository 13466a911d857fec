// Internal declarations shared by the host layer and the kernels of the cache's attention operators
// (include/nvfp4_attention.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_attention.h"

namespace nvfp4 {

constexpr int kComputeUnits = 256;  // gfx950

// Quotient by a launch constant d >= 1 for 0 <= n < 2^31: with l = ceil(log2 d) and
// mul = ceil(2^(31 + l) / d), mul * d - 2^(31 + l) < d <= 2^l, so n * mul / 2^(31 + l) exceeds n / d by
// less than n / 2^31 / d < 1 / d and has the same floor.
struct FastDiv {
  uint32_t d, mul, shift;
};

inline FastDiv make_fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  const uint64_t two = uint64_t(1) << (31 + l);
  return FastDiv{d, (uint32_t)((two + d - 1) / d), 31 + l};
}

struct TablesArgs {
  const int32_t* context_lens;
  const int32_t* query_lens;
  const int32_t* free_blocks;
  const int32_t* free_start;
  int32_t* block_table;
  int64_t* slot_mapping;
  int32_t* positions;
  int32_t* query_start;
  int32_t* seq_lens;
  int32_t* blocks_needed;
  int64_t table_ld;
  int32_t requests, table_width, num_free, max_tokens;
  FastDiv bs;
};

// How an attention call is divided among workgroups.
enum class AttnKernel : int32_t {
  Stream16,  // a wavefront streams its own keys past 16 or 32 query rows
  Stream32,
  Tiled,  // key tiles staged in LDS for 256 query rows
};

struct AttnPlan {
  AttnKernel kernel;
  int32_t rows;     // query rows (token, head of the group) of a row tile
  int32_t join_rows;  // of them, as many as the longest request has
  int32_t workers;  // 0: one workgroup per (row tile, KV head, request); else the number of
                    // workgroups that share the whole key range, and a joining launch
  int32_t row_tiles;  // of the longest request as far as the caller told (grid bound)
  int32_t all_tiles;  // > 0 (tiled kernel without workers): the grid counts row tiles of all requests
  int64_t workspace;
};

struct AttnArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs;  // elements
  uint16_t* out;
  int64_t out_ts, out_hs;
  const uint8_t* kc;
  const uint8_t* vc;
  int64_t cache_ld;
  const float* ks;
  const float* vs;
  const int32_t* table;
  int64_t table_ld;
  const int32_t* query_start;
  const int32_t* seq_lens;
  const float* slopes;
  const int32_t* doc_start;
  const int32_t* prefix_lens;
  const int64_t* tree;  // not null: drafted trees
  int64_t tree_ld;
  const int32_t* positions;
  float* part;       // workspace: partial outputs, then their statistics, then headers
  float* part_ml;
  int32_t* headers;
  int32_t num_slots, table_width, requests, tokens;
  int32_t heads, kv_heads, tree_words;
  int32_t row_tiles, workers;  // as in the plan
  FastDiv bs, group;
  float scale, cap;
  int32_t all_tiles;  // as in the plan
};

// Workgroups that share a compute unit's registers: what a call is divided among.  More of them keep more
// loads in flight, as long as their operands fit: 4 KB a step and wavefront with 64 dims, 16 KB with 256.
constexpr int stream_groups(int head_dim, int rows) {
  if (head_dim == 64) return 3;
  if (head_dim == 128) return rows == 16 ? 3 : 2;
  return 1;
}

constexpr int kStreamUnit = 128;  // positions of a workgroup's step in the streaming kernel

AttnPlan plan_attention(int64_t tokens, int64_t heads, int64_t kv_heads,
                        int64_t head_dim, int64_t requests, int64_t max_query_len,
                        int64_t max_seq_len);

hipError_t launch_block_tables(const TablesArgs& a, hipStream_t stream);
// Launch the plan's kernel (and, with workers, the joining kernel).
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, int head_dim, bool bf16,
                            hipStream_t stream);
hipError_t launch_attention_tiled(const AttnArgs& a, int head_dim, bool bf16, hipStream_t stream);

}  // namespace nvfp4
