// The rule that divides an attention call's work: which kernel, how many workgroups, how large a workspace.  Host
// arithmetic on the call's sizes alone.
#include "attention_internal.h"

namespace nvfp4 {

namespace {

constexpr int64_t kMaxTiles = 4096;  // bound of a grid dimension
constexpr int64_t kShort = 8 * kStreamUnit;  // positions that a workgroup walks over alone

// `groups`: workgroups that share a compute unit in the streaming kernel; `most`: rows that it can take at once.
AttnPlan plan(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t requests,
              int64_t max_query_len, int64_t max_seq_len, int (*groups)(int, int), int64_t most) {
  AttnPlan p{};
  const int64_t group = heads / kv_heads, rows = max_query_len * group;
  // Short sequences: one launch of a workgroup per item and no join (one token over 500 and 1000 positions,
  // 256 dims: 14 and 16 us a call, shared among workers and joined 19 us; over 1500 21 and 19 us), by row
  // tiles of 32 where these all run at once (prompts of 37 and 500 tokens, 24 heads over 4 of 256 dims: 14 and
  // 28 us, tiles of 256 rows 20 and 46 us.  64 prompts of 60 tokens, which do not run at once: 29 against 16).
  const bool small = max_seq_len <= kShort && requests * kv_heads * ((rows + 31) / 32) <= kComputeUnits;
  if (rows <= 16) {
    p.kernel = AttnKernel::Stream16;
    p.rows = 16;
  } else if (rows <= 96 || small) {
    // Tiles of 32 rows re-read the keys from the caches and decode them again; tiles of 256 leave
    // wavefronts idle.  16 requests of up to 6001 positions, 32 against 256 rows: 48 rows of 128 dims 54
    // and 76 us, 96 rows of 128 and 256 dims 71 and 85, 79 and 102.  64 requests: 48 rows of 128 and 256
    // dims 217 and 234, 171 and 270; 96 rows of 256 dims 279 and 287, of 128 dims 321 and 250 (where the
    // device is full, the other side is ahead there already); 128 rows of 64 dims 289 and 184; 192 rows of
    // 128 and 256 dims (all 6001 long) 938 and 407, 854 and 412.
    p.kernel = AttnKernel::Stream32;
    p.rows = 32;
    // Over the 4-bit cache decoding is most of a tile's work, and tiles of 48 rows where they are fewer than those of 32
    // pay from some thousand positions on: below, a workgroup takes few steps and each is longer.  Trees of 12 tokens
    // with 4 heads each over 1500, 6001 and 24000 positions (32 against 48 rows): 16 requests of 128 dims 33 and 37, 54 and
    // 52, 149 and 121 us; 64 of them 57 and 72, 181 and 139, 662 and 427; 16 of 64 dims 29 and 32, 46 and 43, 108 and 94.
    // Of 24 tokens (three tiles or two), 128 dims: 42 and 45, 78 and 76, 224 and 201.
    if (most == 48 && max_seq_len >= 4096 && rows <= 96 && (rows + 47) / 48 < (rows + 31) / 32) {
      p.kernel = AttnKernel::Stream48;
      p.rows = 48;
    }
  } else {
    p.kernel = AttnKernel::Tiled;
    p.rows = 256;
  }
  p.join_rows = (int32_t)(rows < p.rows ? rows : p.rows);
  // Row tiles: every request may be as long as the longest, but together they have the call's tokens only
  // (sum of ceil(n / rows) <= sum of n / rows + requests).
  const int64_t each = (rows + p.rows - 1) / p.rows, any = tokens * group / p.rows + requests;
  const int64_t items = kv_heads * (requests * each < any ? requests * each : any);
  p.row_tiles = (int32_t)(each < kMaxTiles ? each : kMaxTiles);  // (the kernels' strides cover the others)
  if (p.kernel == AttnKernel::Tiled) {
    // Where the context is most of the work all row tiles cost alike, and sharing fills the device and
    // balances ragged lengths (4 trees of 64 over up to 60000: 505 us, a workgroup per item 3475; chunk of 512
    // over 6000, 32 heads of 128 dims: 121 and 206; 64 trees of 192 rows over up to 6001: 380 and 367).
    // A prompt's row tiles cost as much as they see; every one of them counts as the whole request here, so
    // that equal shares are not equal work.  Fresh prompts of fewer than 256 items are shared all the
    // same, and lose by it (prompts of 500 to 2000 tokens, 24 heads over 4 of 256 dims: 512 65 us against 48,
    // 1000 94 against 77, 2048 194 against 140; 32 over 8 of 128 dims: 512 75 and 27, 1500 111 and 56;
    // 8 heads of 64 dims: 2700 55 and 61, 4096 103 and 92).
    const bool deep = 4 * max_query_len <= max_seq_len;
    if (max_seq_len > 256 && items < (deep ? 4 : 1) * kComputeUnits) p.workers = kComputeUnits;
  } else if (max_seq_len > kShort && items < 4 * kComputeUnits) {
    p.workers = groups((int)head_dim, p.rows) * kComputeUnits;
  }
  // A grid of requests by the longest's row tiles is mostly empty where one prompt joins many single tokens,
  // and an empty workgroup takes the room of a full one: the grid counts all requests' row tiles then, and
  // a workgroup finds its own by summing the lengths (24 heads of 256 dims; 63 tokens over 2000 positions and
  // a prompt of 4096: 1.79 ms by requests, 0.39 so; 255 over 1000 and a prompt of 8192: 6.60 ms, 1.19).
  // Where at least half of the grid's places hold a tile, the place says it, with nothing to sum.
  if (p.kernel == AttnKernel::Tiled && p.workers == 0 && requests * each > 2 * any)
    p.all_tiles = (int32_t)(any < kMaxTiles ? any : kMaxTiles);
  if (p.workers)
    p.workspace = (int64_t)p.workers * (2 * (int64_t)p.rows * (head_dim + 2) + 8) * (int64_t)sizeof(float);
  return p;
}

}  // namespace

AttnPlan plan_attention(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                        int64_t requests, int64_t max_query_len, int64_t max_seq_len) {
  return plan(tokens, heads, kv_heads, head_dim, requests, max_query_len, max_seq_len, stream_groups, 32);
}

AttnPlan plan_attention_fp4(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t requests,
                            int64_t max_query_len, int64_t max_seq_len) {
  // The rules but for the 48 rows and the eight wavefronts are the FP8 cache's, with its figures.  What they give of fresh prompts was
  // timed over this cache too, shared out (where they share) against row tiles, us in a graph: 24 heads over 4 of 256 dims, 512
  // tokens 64 and 51, 1000 88 and 82, 2048 177 and 153; 32 over 8 of 128 dims, 300 36 and 20, 512 35 and 27, 1000 54 and 42, 2048 not shared 79
  // (shared 84); 8 heads of 64 dims, 2048 37 and 53, 2700 50 and 66.  As over the FP8 cache, shares lose but at 64 dims.
  AttnPlan p = plan(tokens, heads, kv_heads, head_dim, requests, max_query_len, max_seq_len, stream_groups_fp4,
                    head_dim <= 128 ? 48 : 32);
  // Eight wavefronts an item where each has a compute unit of its own and some steps to share: two a SIMD fill each
  // other's waits.  Four against eight (us on the device, one token, 16 heads over 4): 500 positions of 64 and 128 dims 8.8 and
  // 7.8, 9.9 and 9.0, 1000 positions 12.9 and 10.4, 14.9 and 12.6; 64 requests 15.3 and 12.1, 16.6 and 14.7; 6 tokens, 64
  // dims 11.2 and 10.2, 15.9 and 13.4.  Of 200 positions they gain nothing (7.4 and 7.3 of 128 dims, 64 requests 8.4 and 8.3).  Left out where
  // a SIMD's instructions are most of the time, so that they gain less there and lose at 200 positions: 256 dims 12.9 and 12.7, 19.5 and 18.1
  // (200 positions 8.9 and 9.5), 32 rows of 128 dims 12.2 and 12.1, 17.5 and 16.1 (200 positions 9.3 and 10.1).
  p.wide = p.workers == 0 && p.rows * head_dim <= 2048 && max_seq_len > 2 * kStreamUnit &&
           kv_heads * requests * p.row_tiles <= kComputeUnits;
  return p;
}

}  // namespace nvfp4
