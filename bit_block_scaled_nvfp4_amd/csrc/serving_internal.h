// Internal declarations shared by the host layer and the kernels of include/nvfp4_serving.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention_internal.h"
#include "nvfp4_serving.h"

namespace nvfp4 {

// Head vectors of one kind: queries, keys or values.
struct HeadGroup {
  const uint8_t* src;  // or null: no such vectors
  uint32_t ts, hs;     // bytes
  uint8_t* out;        // same type: rows with strides of their own
  uint32_t out_ts, out_hs;
  const uint8_t* weight;  // or null: no norm
  const float* scale;  // of a cache: decode direction (FP8), encode direction (4 bits)
  uint8_t* cache;      // codes
  uint8_t* cache_scales;
  FastDiv heads;
  int32_t turned;      // rotated
};

enum class HeadSink { Same, Fp8, Fp4 };

struct HeadArgs {
  HeadGroup group[2];
  const int32_t* positions;
  const float* inv_freq;
  const int64_t* slots;  // caches: null for slot t
  double eps, offset, per_dim;  // per_dim: 1 / head_dim
  int64_t num_slots, cache_ld;
  int32_t tokens, head_dim, num_freq, interleaved;
  int32_t weight_dtype;
  int32_t block_tokens;  // tokens of a workgroup
  FastDiv bs;
};

hipError_t launch_heads(HeadArgs a, nvfp4_dtype dt, HeadSink sink, hipStream_t stream);

struct Fp4LoadArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* g;
  const int64_t* slots;
  uint8_t* out;
  int64_t num_slots, tokens;
  int32_t head_bits;  // log2 of head_dim
  int32_t kv_heads;
  int32_t pieces;     // of 16 bytes of the result, a token
  FastDiv bs;
};

hipError_t launch_fp4_load(Fp4LoadArgs a, bool bf16_out, hipStream_t stream);

constexpr int kVerifyChunk = 4096;  // tokens of the vocabulary that a workgroup sums

struct VerifyArgs {
  const float* p;
  const float* q;  // or null: drafted tokens are certain
  int64_t p_ld, q_ld;
  const int32_t* tokens;
  const int32_t* query_start;
  const float* accept_u;
  const float* sample_u;
  int32_t* accepted;
  int32_t* out;
  double* sums;  // [requests, chunks, 2]: of the weights, of p
  int32_t rows, vocab, requests, chunks;
};

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream);

}  // namespace nvfp4
