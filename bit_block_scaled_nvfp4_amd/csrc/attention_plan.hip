// The rule that divides an attention call's work: which kernel, how many workgroups, how large a workspace.  Host
// arithmetic on the call's sizes alone.
#include "attention_internal.h"

namespace nvfp4 {

namespace {

constexpr int64_t kMaxTiles = 4096;  // bound of a grid dimension
constexpr int64_t kShort = 8 * kStreamUnit;  // positions that a workgroup walks over alone

}  // namespace

AttnPlan plan_attention(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                        int64_t requests, int64_t max_query_len, int64_t max_seq_len) {
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
    p.workers = stream_groups((int)head_dim, p.rows) * kComputeUnits;
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

}  // namespace nvfp4
