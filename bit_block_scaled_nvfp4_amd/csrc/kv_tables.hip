// Block tables and slot maps of one serving step, from request lengths (nvfp4_kv_block_tables).
//
// Two exclusive sums over the requests (new tokens, new blocks) decide everything; the rest is one
// independent lookup per new token and per new block.  The call is bound by latency: a few hundred KB
// at most, against a launch of several microseconds.  So there is one launch and no step that waits
// for another workgroup: every workgroup forms both sums of all requests itself (8 bytes read per
// request, from the L2 after the first), keeps them in LDS, and then serves its own stretch of tokens
// and of new blocks by binary search in them.  A token in a new block reads the block's number from the
// free list, not from the table entry that another workgroup may still be writing; entries below
// `have` are only read and entries from `have` on only written.
//
// Measured: 3.5 us on the device for 64 requests with one token each, 5.7 us for 500 requests with 29 thousand
// tokens; 10.4 and 10.8 us a call from Python, most of it the binding's (1 us: that no results overlap).
#include "attention_internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
// Tokens (and new blocks) of a workgroup in one turn.
constexpr int kChunk = 2 * kThreads;

__device__ __forceinline__ uint32_t div_of(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.mul) >> f.shift);
}

// Number of blocks that `len` tokens (0 .. 2^32) take, at most `width`.
__device__ __forceinline__ uint32_t blocks_of(uint64_t len, const FastDiv& f, uint32_t width) {
  if (len == 0) return 0;
  const uint64_t last = len - 1 < 0x7FFFFFFFull ? len - 1 : 0x7FFFFFFFull;
  const uint32_t b = div_of((uint32_t)last, f) + 1;
  return b < width ? b : width;
}

__device__ __forceinline__ uint32_t clamp31(uint64_t x) {
  return x < 0x7FFFFFFFull ? (uint32_t)x : 0x7FFFFFFFu;
}

// Saturating sums: operands are at most 2^31 - 1, so a 32-bit sum cannot wrap before the clamp.
__device__ __forceinline__ uint32_t add31(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < 0x7FFFFFFFu ? s : 0x7FFFFFFFu;
}

// Index r with sums[r] <= x < sums[r + 1], for sums[0] = 0 <= x < sums[n].
__device__ __forceinline__ int find(const uint32_t* sums, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) block_tables_kernel(TablesArgs a) {
  extern __shared__ uint32_t lds[];
  const int R = a.requests;
  uint32_t* tok = lds;            // R + 1 sums of new tokens
  uint32_t* blk = lds + R + 1;    // R + 1 sums of new blocks
  uint32_t* wsum = lds + 2 * (R + 1);  // 2 x kWaves
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t W = (uint32_t)a.table_width;
  const int32_t first_free = a.free_start ? *a.free_start : 0;

  // the sums, kThreads requests at a time; carry is uniform
  uint32_t carry_t = 0, carry_b = 0;
  for (int base = 0; base < R; base += kThreads) {
    const int r = base + tid;
    uint32_t n = 0, nb = 0;
    if (r < R) {
      const int32_t c0 = a.context_lens[r], n0 = a.query_lens[r];
      const uint32_t c = c0 > 0 ? (uint32_t)c0 : 0u;
      n = n0 > 0 ? (uint32_t)n0 : 0u;
      nb = blocks_of((uint64_t)c + n, a.bs, W) - blocks_of(c, a.bs, W);
      if (blockIdx.x == 0) a.seq_lens[r] = (int32_t)clamp31((uint64_t)c + n);
    }
    uint32_t st = n, sb = nb;  // inclusive sums over the wavefront
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t pt = __shfl_up(st, d), pb = __shfl_up(sb, d);
      if (lane >= d) {
        st = add31(st, pt);
        sb = add31(sb, pb);
      }
    }
    if (lane == 63) {
      wsum[wave] = st;
      wsum[kWaves + wave] = sb;
    }
    __syncthreads();
    uint32_t before_t = carry_t, before_b = carry_b, all_t = carry_t, all_b = carry_b;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) {
        before_t = all_t;
        before_b = all_b;
      }
      all_t = add31(all_t, wsum[w]);
      all_b = add31(all_b, wsum[kWaves + w]);
    }
    if (r < R) {
      tok[r + 1] = add31(before_t, st);
      blk[r + 1] = add31(before_b, sb);
    }
    carry_t = all_t;
    carry_b = all_b;
    __syncthreads();  // wsum is written again in the next turn
  }
  if (tid == 0) {
    tok[0] = 0;
    blk[0] = 0;
  }
  __syncthreads();
  const uint32_t tokens = carry_t, blocks = carry_b;
  if (blockIdx.x == 0) {
    for (int r = tid; r <= R; r += kThreads) a.query_start[r] = (int32_t)tok[r];
    if (tid == 0) *a.blocks_needed = (int32_t)blocks;
  }

  const uint32_t stride = gridDim.x * (uint32_t)kThreads;
  for (uint32_t t = blockIdx.x * (uint32_t)kThreads + tid; t < (uint32_t)a.max_tokens; t += stride) {
    int64_t slot = -1;
    uint32_t p = 0;
    if (t < tokens) {
      const int r = find(tok, R, t);
      const int32_t c0 = a.context_lens[r];
      const uint32_t c = c0 > 0 ? (uint32_t)c0 : 0u;
      p = clamp31((uint64_t)c + (t - tok[r]));
      const uint32_t col = div_of(p, a.bs);
      if (col < W) {
        const uint32_t have = blocks_of(c, a.bs, W);
        int32_t b = -1;
        if (col < have) {
          b = a.block_table[(int64_t)r * a.table_ld + col];
        } else {
          const int64_t k = (int64_t)first_free + blk[r] + (col - have);
          if (k >= 0 && k < a.num_free) b = a.free_blocks[k];
        }
        if (b >= 0) slot = (int64_t)b * a.bs.d + (p - col * a.bs.d);
      }
    }
    a.slot_mapping[t] = slot;
    a.positions[t] = (int32_t)p;
  }
  for (uint32_t x = blockIdx.x * (uint32_t)kThreads + tid; x < blocks; x += stride) {
    const int r = find(blk, R, x);
    const int32_t c0 = a.context_lens[r];
    const uint32_t col = blocks_of(c0 > 0 ? (uint32_t)c0 : 0u, a.bs, W) + (x - blk[r]);
    const int64_t k = (int64_t)first_free + x;
    a.block_table[(int64_t)r * a.table_ld + col] = (k >= 0 && k < a.num_free) ? a.free_blocks[k] : -1;
  }
}

}  // namespace

hipError_t launch_block_tables(const TablesArgs& a, hipStream_t stream) {
  // a workgroup for every kChunk tokens; the number of new blocks is known on the device only, and
  // the loops' strides cover what the grid does not
  int64_t grid = ((int64_t)a.max_tokens + kChunk - 1) / kChunk;
  if (grid < 1) grid = 1;
  if (grid > kComputeUnits) grid = kComputeUnits;
  const size_t lds = sizeof(uint32_t) * (2 * ((size_t)a.requests + 1) + 2 * kWaves);
  hipLaunchKernelGGL(block_tables_kernel, dim3((uint32_t)grid), dim3(kThreads), lds, stream, a);
  return hipGetLastError();
}

}  // namespace nvfp4
