// Host layer of the serving operators: argument validation (before any HIP call) and launch.  The contracts are in
// include/nvfp4_serving.h.
#include "attention_checks.h"
#include "serving_internal.h"

namespace {

bool valid_dtype(int d) { return d == NVFP4_F32 || d == NVFP4_BF16 || d == NVFP4_F16; }

constexpr int64_t kMaxStride = int64_t(1) << 32;  // bytes from one head vector to the next

int64_t bytes_of(int d) { return d == NVFP4_F32 ? 4 : 2; }

// Head vectors of one kind, as a call gives them.
struct Vectors {
  const void* x;
  int64_t heads, ts, hs;
};

// Norm and rotation, as a call gives them.
struct Turn {
  const int32_t* positions;
  const float* inv_freq;
  int64_t num_freq;
  int interleaved;
  int weight_dtype;
  double eps, offset;
};

// Whether the vectors may be read (or, `out`, written) with these strides.
nvfp4_status check_vectors(const Vectors& v, int dtype, int64_t tokens, int64_t head_dim, bool out) {
  const int64_t eb = bytes_of(dtype);
  if (!span_fits(tokens, v.heads, head_dim, v.ts, v.hs)) return NVFP4_ESHAPE;
  if ((tokens > 1 && v.ts * eb >= kMaxStride) || (v.heads > 1 && v.hs * eb >= kMaxStride)) return NVFP4_ESHAPE;
  if (out && !distinct(tokens, v.heads, head_dim, v.ts, v.hs)) return NVFP4_ESHAPE;
  if (!aligned(v.x, 16) || (tokens > 1 && v.ts * eb % 16) || (v.heads > 1 && v.hs * eb % 16)) return NVFP4_EALIGN;
  return NVFP4_OK;
}

nvfp4_status check_turn(const Turn& t, int64_t head_dim, bool any_weight) {
  if (t.interleaved != 0 && t.interleaved != 1) return NVFP4_EINVAL;
  if (t.num_freq < 0 || t.num_freq % 8 || t.num_freq > head_dim / 2) return NVFP4_ESHAPE;
  // written so that a NaN fails
  if (!(t.eps - t.eps == 0.0) || !(t.eps >= 0.0) || !(t.offset - t.offset == 0.0)) return NVFP4_EINVAL;
  if (any_weight && !valid_dtype(t.weight_dtype)) return NVFP4_EINVAL;
  return NVFP4_OK;
}

// Positions and frequencies of a call that is not empty; what an empty one has of them is not looked at.
nvfp4_status check_angles(const Turn& t) {
  if (t.num_freq > 0 && (!t.positions || !t.inv_freq)) return NVFP4_EINVAL;
  if (!aligned(t.positions, 4) || !aligned(t.inv_freq, 4)) return NVFP4_EALIGN;
  return NVFP4_OK;
}

nvfp4::HeadGroup group_of(const Vectors& v, int dtype, int64_t tokens, const void* weight, bool turned) {
  nvfp4::HeadGroup g{};
  const int64_t eb = bytes_of(dtype);
  g.src = static_cast<const uint8_t*>(v.x);
  g.ts = (uint32_t)(tokens > 1 ? v.ts * eb : 0);
  g.hs = (uint32_t)(v.heads > 1 ? v.hs * eb : 0);
  g.weight = static_cast<const uint8_t*>(weight);
  g.heads = nvfp4::make_fast_div((uint32_t)v.heads);
  g.turned = turned ? 1 : 0;
  return g;
}

nvfp4::HeadArgs args_of(const Turn& t, int64_t tokens, int64_t head_dim) {
  nvfp4::HeadArgs a{};
  a.positions = t.positions;
  a.inv_freq = t.inv_freq;
  a.num_freq = (int32_t)t.num_freq;
  a.interleaved = t.interleaved;
  a.weight_dtype = t.weight_dtype;
  a.eps = t.eps;
  a.offset = t.offset;
  a.tokens = (int32_t)tokens;
  a.head_dim = (int32_t)head_dim;
  a.bs = nvfp4::make_fast_div(1);
  return a;
}

bool cache_dim(int64_t head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }

// Blocks of a 4-bit cache whose rows are numbered in 32 bits.
bool blocks_fit(int64_t num_blocks, int64_t block_size, int64_t kv_heads) {
  return kv_heads >= 1 && kv_heads <= 1024 && num_blocks >= 0 && num_blocks <= kMaxI32 && block_size >= 1 && block_size <= kMaxBlockSize &&
         num_blocks <= kMaxI32 / (block_size * kv_heads);
}

// What both appends check of keys and values.
nvfp4_status check_append(const Vectors& k, const Vectors& v, int dtype, int64_t tokens, int64_t head_dim,
                          const Turn& t, const void* k_weight, const float* k_scale, const float* v_scale,
                          const int64_t* slots) {
  if (!valid_dtype(dtype) || !k_scale || !v_scale) return NVFP4_EINVAL;
  if (tokens < 0 || tokens > kMaxI32 || k.heads < 1 || k.heads > 1024 || !cache_dim(head_dim)) return NVFP4_ESHAPE;
  const nvfp4_status st = check_turn(t, head_dim, k_weight != nullptr);
  if (st != NVFP4_OK) return st;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(slots, 8)) return NVFP4_EALIGN;
  if (tokens == 0) return NVFP4_OK;
  if (!k.x || !v.x) return NVFP4_EINVAL;
  if (!aligned(k_weight, bytes_of(t.weight_dtype))) return NVFP4_EALIGN;
  const nvfp4_status sa = check_angles(t), sk = check_vectors(k, dtype, tokens, head_dim, false);
  if (sa != NVFP4_OK) return sa;
  return sk != NVFP4_OK ? sk : check_vectors(v, dtype, tokens, head_dim, false);
}

nvfp4_status run4(Call& c, int64_t num_blocks, const Masks& m, bool tree, void* stream) {
  c.fp4 = true;
  // rows have to be numbered in 32 bits; what does not fit has no slots, which the checks refuse
  c.num_slots = blocks_fit(num_blocks, c.block_size, c.kv_heads) ? num_blocks * c.block_size : -1;
  bool empty = false;
  nvfp4_status st = check(c, &empty);
  if (st != NVFP4_OK) return st;
  if (tree) {
    st = check_tree(c, empty, m);
    if (st != NVFP4_OK) return st;
  } else if (!aligned(m.doc_start, 4) || !aligned(m.prefix_lens, 4)) {
    return NVFP4_EALIGN;
  }
  if (empty) return NVFP4_OK;
  const int64_t longest = query_bound(c.max_query_len, c.tokens);
  const nvfp4::AttnPlan p = nvfp4::plan_attention_fp4(c.tokens, c.heads, c.kv_heads, c.head_dim, c.requests, longest, c.max_seq_len);
  if (p.workspace > 0) {
    if (!c.workspace) return NVFP4_EINVAL;
    if (c.workspace_bytes < p.workspace) return NVFP4_ESHAPE;
  }
  return device_status(nvfp4::launch_attention_fp4(kernel_args(c, p, m), p, (int)c.head_dim, c.dtype == NVFP4_BF16,
                                                   reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_qk_norm_rope(const void* q, int64_t q_heads, int64_t q_token_stride,
                                int64_t q_head_stride, const void* k, int64_t k_heads,
                                int64_t k_token_stride, int64_t k_head_stride, nvfp4_dtype dtype,
                                int64_t tokens, int64_t head_dim, const int32_t* positions,
                                const float* inv_freq, int64_t num_freq, int interleaved,
                                const void* q_weight, const void* k_weight, nvfp4_dtype weight_dtype,
                                double eps, double weight_offset, void* q_out,
                                int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                                int64_t k_out_token_stride, int64_t k_out_head_stride, void* stream) {
  const Turn t{positions, inv_freq, num_freq, interleaved, (int)weight_dtype, eps, weight_offset};
  if (!valid_dtype(dtype)) return NVFP4_EINVAL;
  if (tokens < 0 || tokens > kMaxI32 || q_heads < 1 || q_heads > 1024 || k_heads < 0 || k_heads > 1024 ||
      head_dim < 16 || head_dim > NVFP4_MAX_HEAD_DIM || head_dim % 16)
    return NVFP4_ESHAPE;
  nvfp4_status st = check_turn(t, head_dim, q_weight || k_weight);
  if (st != NVFP4_OK) return st;
  if (tokens == 0) return NVFP4_OK;
  if (!q || !q_out || (k_heads > 0 && (!k || !k_out))) return NVFP4_EINVAL;
  st = check_angles(t);
  if (st != NVFP4_OK) return st;
  if (!aligned(q_weight, bytes_of(weight_dtype)) || !aligned(k_weight, bytes_of(weight_dtype))) return NVFP4_EALIGN;
  const Vectors in[2] = {{q, q_heads, q_token_stride, q_head_stride}, {k, k_heads, k_token_stride, k_head_stride}};
  const Vectors out[2] = {{q_out, q_heads, q_out_token_stride, q_out_head_stride},
                          {k_out, k_heads, k_out_token_stride, k_out_head_stride}};
  nvfp4::HeadArgs a = args_of(t, tokens, head_dim);
  for (int i = 0; i < (k_heads > 0 ? 2 : 1); ++i) {
    st = check_vectors(in[i], dtype, tokens, head_dim, false);
    if (st != NVFP4_OK) return st;
    st = check_vectors(out[i], dtype, tokens, head_dim, true);
    if (st != NVFP4_OK) return st;
    a.group[i] = group_of(in[i], dtype, tokens, i ? k_weight : q_weight, num_freq > 0);
    const nvfp4::HeadGroup o = group_of(out[i], dtype, tokens, nullptr, false);
    a.group[i].out = static_cast<uint8_t*>(const_cast<void*>(out[i].x));
    a.group[i].out_ts = o.ts;
    a.group[i].out_hs = o.hs;
  }
  return device_status(nvfp4::launch_heads(a, dtype, nvfp4::HeadSink::Same, reinterpret_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_fp8_append(const void* key, const void* value, nvfp4_dtype dtype, int64_t tokens,
                                 int64_t kv_heads, int64_t head_dim, int64_t key_token_stride,
                                 int64_t key_head_stride, int64_t value_token_stride,
                                 int64_t value_head_stride, const int32_t* positions,
                                 const float* inv_freq, int64_t num_freq, int interleaved,
                                 const void* k_weight, nvfp4_dtype weight_dtype, double eps,
                                 double weight_offset, const float* key_scale, const float* value_scale,
                                 const int64_t* slot_mapping, uint8_t* key_cache, uint8_t* value_cache,
                                 int64_t num_slots, int64_t cache_ld, void* stream) {
  const Turn t{positions, inv_freq, num_freq, interleaved, (int)weight_dtype, eps, weight_offset};
  const Vectors k{key, kv_heads, key_token_stride, key_head_stride}, v{value, kv_heads, value_token_stride, value_head_stride};
  const nvfp4_status st = check_append(k, v, dtype, tokens, head_dim, t, k_weight, key_scale, value_scale, slot_mapping);
  if (st != NVFP4_OK) return st;
  if (num_slots < 0 || num_slots > kMaxSpan || cache_ld < kv_heads * head_dim || cache_ld > kMaxSpan ||
      (num_slots > 0 && cache_ld > kMaxSpan / num_slots))
    return NVFP4_ESHAPE;
  if (!aligned(key_cache, 16) || !aligned(value_cache, 16) || cache_ld % 16) return NVFP4_EALIGN;
  if (tokens == 0 || num_slots == 0) return NVFP4_OK;
  if (!key_cache || !value_cache) return NVFP4_EINVAL;
  nvfp4::HeadArgs a = args_of(t, tokens, head_dim);
  a.group[0] = group_of(k, dtype, tokens, k_weight, num_freq > 0);
  a.group[1] = group_of(v, dtype, tokens, nullptr, false);
  a.group[0].scale = key_scale;
  a.group[1].scale = value_scale;
  a.group[0].cache = key_cache;
  a.group[1].cache = value_cache;
  a.slots = slot_mapping;
  a.num_slots = num_slots;
  a.cache_ld = cache_ld;
  return device_status(nvfp4::launch_heads(a, dtype, nvfp4::HeadSink::Fp8, reinterpret_cast<hipStream_t>(stream)));
}

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
                                 void* stream) {
  const Turn t{positions, inv_freq, num_freq, interleaved, (int)weight_dtype, eps, weight_offset};
  const Vectors k{key, kv_heads, key_token_stride, key_head_stride}, v{value, kv_heads, value_token_stride, value_head_stride};
  const nvfp4_status st = check_append(k, v, dtype, tokens, head_dim, t, k_weight, key_gscale, value_gscale, slot_mapping);
  if (st != NVFP4_OK) return st;
  if (!blocks_fit(num_blocks, block_size, kv_heads) || (interleaved == 0 && num_freq % 16)) return NVFP4_ESHAPE;
  if (!aligned(key_codes, 16) || !aligned(key_scales, 16) || !aligned(value_codes, 16) || !aligned(value_scales, 16))
    return NVFP4_EALIGN;
  if (tokens == 0 || num_blocks == 0) return NVFP4_OK;
  if (!key_codes || !key_scales || !value_codes || !value_scales) return NVFP4_EINVAL;
  nvfp4::HeadArgs a = args_of(t, tokens, head_dim);
  a.group[0] = group_of(k, dtype, tokens, k_weight, num_freq > 0);
  a.group[1] = group_of(v, dtype, tokens, nullptr, false);
  a.group[0].scale = key_gscale;
  a.group[1].scale = value_gscale;
  a.group[0].cache = key_codes;
  a.group[1].cache = value_codes;
  a.group[0].cache_scales = key_scales;
  a.group[1].cache_scales = value_scales;
  a.slots = slot_mapping;
  a.num_slots = num_blocks * block_size;
  a.bs = nvfp4::make_fast_div((uint32_t)block_size);
  return device_status(nvfp4::launch_heads(a, dtype, nvfp4::HeadSink::Fp4, reinterpret_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_fp4_load(const uint8_t* codes, const uint8_t* scales, int64_t num_blocks,
                               int64_t kv_heads, int64_t block_size, int64_t head_dim,
                               const float* gscale, const int64_t* slot_mapping, int64_t tokens, void* out,
                               nvfp4_dtype out_dtype, void* stream) {
  if (!gscale || (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16)) return NVFP4_EINVAL;
  if (kv_heads < 1 || kv_heads > 1024 || !cache_dim(head_dim) || !blocks_fit(num_blocks, block_size, kv_heads) ||
      tokens < 0 || tokens > kMaxI32 || tokens > kMaxSpan / (kv_heads * head_dim))
    return NVFP4_ESHAPE;
  if (tokens > 0 && (!out || (num_blocks > 0 && (!codes || !scales)))) return NVFP4_EINVAL;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16) || !aligned(gscale, 4) || !aligned(slot_mapping, 8))
    return NVFP4_EALIGN;
  if (tokens == 0) return NVFP4_OK;
  nvfp4::Fp4LoadArgs a{};
  a.codes = codes;
  a.scales = scales;
  a.g = gscale;
  a.slots = slot_mapping;
  a.out = static_cast<uint8_t*>(out);
  a.num_slots = num_blocks * block_size;
  a.tokens = tokens;
  a.head_bits = head_dim == 64 ? 6 : (head_dim == 128 ? 7 : 8);
  a.kv_heads = (int32_t)kv_heads;
  a.bs = nvfp4::make_fast_div((uint32_t)block_size);
  return device_status(nvfp4::launch_fp4_load(a, out_dtype == NVFP4_BF16, reinterpret_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_fp4_attention(
    const void* q, nvfp4_dtype dtype, int64_t tokens, int64_t heads, int64_t kv_heads,
    int64_t head_dim, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* key_codes,
    const uint8_t* key_scales, const uint8_t* value_codes, const uint8_t* value_scales,
    const float* key_gscale, const float* value_gscale, int64_t num_blocks, int64_t block_size,
    const int32_t* block_table, int64_t requests, int64_t table_width, int64_t table_ld,
    const int32_t* query_start, const int32_t* seq_lens, float scale, float softcap,
    const float* slopes, const int32_t* doc_start, const int32_t* prefix_lens, int64_t max_query_len,
    int64_t max_seq_len, void* out, int64_t out_token_stride, int64_t out_head_stride,
    void* workspace, int64_t workspace_bytes, void* stream) {
  Call c{q, (int)dtype, tokens, heads, kv_heads, head_dim, q_token_stride, q_head_stride,
         key_codes, value_codes, key_gscale, value_gscale, 0, 0, block_table,
         requests, table_width, table_ld, block_size, query_start, seq_lens, scale, softcap,
         slopes, max_query_len, max_seq_len, out, out_token_stride, out_head_stride,
         workspace, workspace_bytes, true, key_scales, value_scales};
  return run4(c, num_blocks, Masks{doc_start, prefix_lens, nullptr, 0, 0, nullptr}, false, stream);
}

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
    void* stream) {
  Call c{q, (int)dtype, tokens, heads, kv_heads, head_dim, q_token_stride, q_head_stride,
         key_codes, value_codes, key_gscale, value_gscale, 0, 0, block_table,
         requests, table_width, table_ld, block_size, query_start, seq_lens, scale, softcap,
         slopes, max_query_len, max_seq_len, out, out_token_stride, out_head_stride,
         workspace, workspace_bytes, true, key_scales, value_scales};
  return run4(c, num_blocks, Masks{nullptr, nullptr, tree_mask, tree_words, tree_ld, positions}, true, stream);
}

int64_t nvfp4_kv_fp4_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads,
                                         int64_t head_dim, int64_t requests, int64_t max_query_len,
                                         int64_t max_seq_len) {
  if (!shape_ok(tokens, heads, kv_heads, head_dim, requests, max_query_len, max_seq_len)) return 0;
  if (tokens == 0 || requests == 0) return 0;
  return nvfp4::plan_attention_fp4(tokens, heads, kv_heads, head_dim, requests, query_bound(max_query_len, tokens), max_seq_len).workspace;
}

nvfp4_status nvfp4_verify_drafted(const float* target_probs, int64_t target_ld, const float* draft_probs,
                                  int64_t draft_ld, int64_t rows, int64_t vocab, const int32_t* tokens,
                                  const int32_t* query_start, int64_t requests, const float* accept_u,
                                  const float* sample_u, int32_t* accepted, int32_t* out_tokens,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  // (the kernels' steps over rows and tokens stay below 2^31 too)
  if (rows < 0 || rows > kMaxI32 - nvfp4::kVerifyChunk || vocab < 1 || vocab > kMaxI32 - nvfp4::kVerifyChunk || requests < 0 ||
      requests > NVFP4_MAX_REQUESTS || target_ld < vocab || (draft_probs && draft_ld < vocab))
    return NVFP4_ESHAPE;
  if (rows > 0 && (target_ld > kMaxSpan / rows || (draft_probs && draft_ld > kMaxSpan / rows))) return NVFP4_ESHAPE;
  if (requests == 0) return NVFP4_OK;
  if (!query_start || !sample_u || !accepted) return NVFP4_EINVAL;
  if (rows > 0 && (!target_probs || !tokens || !accept_u || !out_tokens)) return NVFP4_EINVAL;
  const int64_t need = nvfp4_verify_drafted_workspace(requests, vocab);
  if (!workspace) return NVFP4_EINVAL;
  if (workspace_bytes < need) return NVFP4_ESHAPE;
  if (!aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(tokens, 4) || !aligned(query_start, 4) ||
      !aligned(accept_u, 4) || !aligned(sample_u, 4) || !aligned(accepted, 4) || !aligned(out_tokens, 4) ||
      !aligned(workspace, 16))
    return NVFP4_EALIGN;
  nvfp4::VerifyArgs a{};
  a.p = target_probs;
  a.q = draft_probs;
  a.p_ld = target_ld;
  a.q_ld = draft_probs ? draft_ld : 0;
  a.tokens = tokens;
  a.query_start = query_start;
  a.accept_u = accept_u;
  a.sample_u = sample_u;
  a.accepted = accepted;
  a.out = out_tokens;
  a.sums = static_cast<double*>(workspace);
  a.rows = (int32_t)rows;
  a.vocab = (int32_t)vocab;
  a.requests = (int32_t)requests;
  a.chunks = (int32_t)((vocab + nvfp4::kVerifyChunk - 1) / nvfp4::kVerifyChunk);
  return device_status(nvfp4::launch_verify(a, reinterpret_cast<hipStream_t>(stream)));
}

int64_t nvfp4_verify_drafted_workspace(int64_t requests, int64_t vocab) {
  if (requests < 1 || requests > NVFP4_MAX_REQUESTS || vocab < 1 || vocab > kMaxI32 - nvfp4::kVerifyChunk) return 0;
  return requests * ((vocab + nvfp4::kVerifyChunk - 1) / nvfp4::kVerifyChunk) * 16;
}

}  // extern "C"
