// Device code shared by the attention kernels over the paged caches (gfx950): which part of the
// work a workgroup takes, which positions a query row sees, how scores are capped and biased, and how
// partial results of one row tile are kept and joined.
//
// Terms.  Query rows of one request and one KV head are numbered row = i * group + g (token i, head
// g of the group of query heads that share the KV head), so that all rows of a tile read the same
// keys.  An item is one (request, row tile, KV head); its keys are counted in units (a fixed number
// of positions, aligned at position 0).
//
// All exponentials are base 2: scores are multiplied by log2(e) once.  The softmax keeps a reference
// value m per row instead of the running maximum: m is raised to kBelow under the largest score so far
// (scaling down what is accumulated) only when a lane's sum of exp2(x - m) over one tile passes kRaise.
// Below that every single term is below kRaise too, inside FP16, no maximum is formed and nothing is
// rescaled; on most tiles that is the case.
//
// exp2(x - m) goes into the output's product in FP16, into the sum of the weights in FP32.  FP16 ends at
// 2^-25 (half its smallest number): with m at the largest score itself, weights of less than 2^-25 were in
// the sum and not in the output, however many there were.  kBelow moves that to 2^-29 of the largest, less
// than half a step of the result for 2^18 keys in FP16 and 2^20 in BF16.  A lane's terms of a tile are 64 at
// most, so just after a raise their sum is 2^10 at most; up to kRaise, a factor of 2 within FP16, scores
// may grow by 11 (log2) before the next one.  More than 4 costs time: chunk of 2048 over 30011 with a bias
// 960 us at 4 and at 0, 1005 us at 5 and 8 (-4 is a constant that an instruction holds); ragged capped prompts
// 444 us at 4 and at 0, 448 at 5, 455 at 8 (raises).
#pragma once

#include "attention_internal.h"

namespace nvfp4 {
namespace attn {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kBelow = 4.0f;
constexpr float kRaise = 32768.0f;
// Reference of a row that has seen nothing: so far below every score that the first one seen raises it
// (exp2 overflows to infinity), and finite, so that exp2(-inf - m) is 0 and not NaN.
constexpr float kNoScore = -1e37f;
constexpr uint32_t kMinusInf = 0xFF800000u, kPlusInf = 0x7F800000u;

__device__ __forceinline__ uint32_t div_of(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.mul) >> f.shift);
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The kernel's arguments (its only parameter).  They are read anew wherever this is called: held in
// scalar registers from the kernel's entry to its end, the sixty of them do not fit, and what the
// compiler spills of them costs the loops vector registers.
__device__ __forceinline__ const AttnArgs& args() {
  typedef const __attribute__((address_space(4))) AttnArgs* Ptr;
  Ptr p = (Ptr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnArgs*)p;
}

// A condition that rarely holds: registers are kept for the other side.
__device__ __forceinline__ bool rarely(bool x) { return __builtin_expect(x, 0); }

__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ uint64_t uniform64(uint64_t x) {
  return (uint64_t)(uint32_t)uniform((int32_t)(x >> 32)) << 32 | (uint32_t)uniform((int32_t)x);
}

// ---- which positions a row sees -------------------------------------------------------------

// One query row as a lane holds it.  Visible: lo <= j < hi, or (drafted trees) hi <= j and the
// row's bit of j - ctx set.
struct Row {
  int32_t lo, hi;
  int32_t pos;    // position for the distance bias
  int32_t token;  // row of q, or -1 where the tile has no such row
  int32_t head;
  float slope;    // times log2(e); 0 without a bias
};

struct Request {
  int32_t start, count;  // query rows
  int32_t len, ctx;      // positions of the request; len - count
  int32_t keys;          // of them, as many as the block table has columns for
};

__device__ __forceinline__ Request request_of(const AttnArgs& a, int32_t r) {
  Request q;
  int32_t s = a.query_start[r], e = a.query_start[r + 1];
  s = s < 0 ? 0 : (s > a.tokens ? a.tokens : s);
  e = e < s ? s : (e > a.tokens ? a.tokens : e);
  q.start = s;
  q.count = e - s;
  const int32_t l = a.seq_lens[r];
  q.len = l > 0 ? l : 0;
  q.ctx = q.len - q.count;
  const int64_t room = (int64_t)a.table_width * a.bs.d;
  q.keys = q.len < room ? q.len : (int32_t)room;
  return q;
}

// Row of q that holds query row `row` of the request, or -1 past its rows; tokens * heads < 2^31.
__device__ __forceinline__ int32_t token_of(const AttnArgs& a, const Request& q, uint32_t row) {
  return row < (uint32_t)q.count * a.group.d ? q.start + (int32_t)div_of(row, a.group) : -1;
}

__device__ __forceinline__ int32_t head_of(const AttnArgs& a, const Request& q, int32_t kv_head, uint32_t row) {
  return kv_head * (int32_t)a.group.d + (int32_t)(row - div_of(row, a.group) * a.group.d);
}

__device__ __forceinline__ Row row_of(const AttnArgs& a, int32_t r, const Request& q, int32_t kv_head,
                                      uint32_t row) {
  Row w;
  w.lo = 0;
  w.hi = 0;
  w.pos = 0;
  w.token = token_of(a, q, row);
  w.head = 0;
  w.slope = 0.0f;
  if (w.token < 0) return w;
  w.head = head_of(a, q, kv_head, row);
  w.pos = q.ctx + (w.token - q.start);
  if (a.slopes) w.slope = a.slopes[w.head] * kLog2e;
  if (a.tree) {
    w.hi = q.ctx > 0 ? (q.ctx < q.keys ? q.ctx : q.keys) : 0;
    if (a.slopes && a.positions) w.pos = a.positions[w.token];
  } else {
    int32_t end = w.pos + 1;
    if (a.prefix_lens) {
      const int32_t p = a.prefix_lens[r];
      end = end > p ? end : p;
    }
    w.hi = end < 0 ? 0 : (end > q.keys ? q.keys : end);
    if (a.doc_start) {
      const int32_t s = a.doc_start[w.token];
      w.lo = s > 0 ? s : 0;
    }
  }
  return w;
}

// Bits b of a 64-bit word with lo <= b < hi.
__device__ __forceinline__ uint64_t bits_below(int32_t x) {
  return x <= 0 ? 0ull : (x >= 64 ? ~0ull : (1ull << x) - 1);
}

// Which of positions j0 .. j0 + 63 a row sees, bit by bit (positions at or beyond the request's length
// may be set too: they have no slot).  `token`: of a row of a drafted tree, else -1.
__device__ __forceinline__ uint64_t sees64(int32_t lo, int32_t hi, int32_t token, int32_t ctx, int32_t j0) {
  uint64_t bits = bits_below(hi - j0) & ~bits_below(lo - j0);
  if (token >= 0 && j0 + 64 > ctx) {
    // the row's mask bits from drafted token d on, d = j0 - ctx > -64
    const AttnArgs& a = args();
    const int64_t* words = a.tree + (int64_t)token * a.tree_ld;
    const int32_t d = j0 - ctx;
    if (d < 0) {
      bits |= (uint64_t)words[0] << -d;
    } else if ((d >> 6) < a.tree_words) {
      bits |= (uint64_t)words[d >> 6] >> (d & 63);
      if ((d & 63) && (d >> 6) + 1 < a.tree_words) bits |= (uint64_t)words[(d >> 6) + 1] << (64 - (d & 63));
    }
  }
  return bits;
}

// x where bit b of `seen` is set, else the value with bits `none`, an infinity.  (In integer arithmetic: a
// tile's selections by condition would hold as many lane masks in scalar registers.)
__device__ __forceinline__ float kept(float x, uint32_t seen, int b, uint32_t none) {
  const uint32_t m = (uint32_t)((int32_t)(seen << (31 - b)) >> 31);
  return __uint_as_float((__float_as_uint(x) & m) | (~m & none));
}

// Position at which key j counts in the distance bias; positions: of the drafted tokens, or NULL.
__device__ __forceinline__ int32_t key_position(const int32_t* positions, const Request& q, int32_t j) {
  if (!positions || j < q.ctx || j >= q.len) return j;
  return positions[q.start + (j - q.ctx)];
}

// The cap in units of log2(e): cap tanh(y) log2(e) = L - 2 L r with L = cap log2(e) and
// r = 1 / (exp(2 y) + 1).  This is r, for to_r = 2 log2(e) / cap times what turns x into a score; the
// product with -2 L joins the scaling that every score goes through.  r is off by a few 2^-24, the
// capped score by as much times 2 L: an error that goes with the cap, not with the score, so it is used
// up to kSmallCap only (there it is 3e-5, a fifteenth of the rounding of the exponentials to FP16).
__device__ __forceinline__ float cap_term(float x, float to_r) {
  return __builtin_amdgcn_rcpf(exp2_of(x * to_r) + 1.0f);
}

constexpr float kSmallCap = 128.0f;

// Where the cap is larger: y = x / cap (x a score) and the capped score in units of log2(e).  For
// |y| >= 1/2 the error above is one of the score itself.  Below, tanh(y) / y is Lambert's continued
// fraction 1 / (1 + y^2 / (3 + y^2 / (5 + y^2 / 7))) = (105 + 10 y^2) / (105 + 45 y^2 + y^4), off by less
// than 2^-24 of itself there.
__device__ __forceinline__ float capped_near(float x, float c, float to_y) {
  const float y = x * to_y, z = y * y;
  return (x * c) * (__builtin_fmaf(z, 10.0f, 105.0f) * __builtin_amdgcn_rcpf(__builtin_fmaf(z, z + 45.0f, 105.0f)));
}

__device__ __forceinline__ float capped_wide(float x, float c, float to_y, float to_r, float base) {
  const float far = __builtin_fmaf(cap_term(x, to_r), -2.0f * base, base);
  return __builtin_fabsf(x * to_y) < 0.5f ? capped_near(x, c, to_y) : far;
}

// N scores of a lane.  Scores rarely reach half of a wide cap: the other form is formed where one of the
// wavefront's does (8192-token prompt, 32 heads of 128 dims, cap 200: 911 us, both forms of every score
// 1086 us, the form for small caps 728 us).
template <int N, typename V>
__device__ __forceinline__ void cap_wide(V& x, float c, float cap) {
  float to_y = c / (cap * kLog2e), top = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(x[i]));
  if (rarely(__any(!(top * __builtin_fabsf(to_y) < 0.5f)))) {
    asm volatile("" : "+v"(to_y));  // the two sides share nothing: it would be kept through the branch
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = capped_wide(x[i], c, to_y, 2.0f * kLog2e * to_y, cap * kLog2e);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = capped_near(x[i], c, to_y);
      if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// What becomes of a score before the softmax.  A kernel for each: what one of them needs costs the others
// registers (the wide cap beside the other, behind a branch: up to 27 more spilled in the tiled kernel).
enum class Scores {
  Plain,
  Modified,  // capped by kSmallCap at most, or biased, or both
  WideCap    // capped by more, and biased where slopes is given
};

inline Scores scores_of(const AttnArgs& a) {
  if (a.cap > kSmallCap) return Scores::WideCap;
  return a.cap > 0.0f || a.slopes ? Scores::Modified : Scores::Plain;
}

// ---- cache rows -----------------------------------------------------------------------------

// The block table's entry for position j (a position without one gets some other entry: slot_of masks
// it).  Loaded a step before slot_of looks at it, so that nothing waits for the load.
__device__ __forceinline__ int32_t entry_of(const AttnArgs& a, const int32_t* table_row, uint32_t j) {
  if (a.table_width <= 0) return -1;
  const uint32_t col = div_of(j, a.bs), last = (uint32_t)a.table_width - 1;
  return table_row[col < last ? col : last];
}

// How the cache holds keys and values.
enum class Cache {
  Fp8,  // E4M3 codes, a slot's row [kv_heads * head_dim] after another
  Fp4   // NVFP4: E2M1 codes, two a byte, and an E4M3 scale for each 16; blocks [kv_heads, block_size, head_dim]
};

// Slot of position j, or -1 where it is not in the cache or not below `end`.  In the 4-bit cache: the number of the
// KV head's row (blocks * kv_heads * block_size < 2^31).
template <Cache C = Cache::Fp8>
__device__ __forceinline__ int32_t slot_of(const AttnArgs& a, int32_t entry, int32_t end, uint32_t j, int32_t kv_head = 0) {
  const uint32_t col = div_of(j, a.bs);
  const int64_t s = (int64_t)entry * a.bs.d + (j - col * a.bs.d);
  const bool there = j < (uint32_t)end && col < (uint32_t)a.table_width && entry >= 0 && s < a.num_slots;
  if constexpr (C == Cache::Fp4)
    return there ? (int32_t)(((uint32_t)entry * (uint32_t)a.kv_heads + (uint32_t)kv_head) * a.bs.d + (j - col * a.bs.d)) : -1;
  return there ? (int32_t)s : -1;
}

// What a key's products and a value's sums are multiplied by: a decode-direction scale, or the inverse of an
// encode-direction one.
template <Cache C>
__device__ __forceinline__ float scale_of(const float* s) {
  if constexpr (C == Cache::Fp4) return 1.0f / *s;
  return *s;
}

// Address of a slot's row: cache_ld < 2^31.
__device__ __forceinline__ const uint8_t* row_at(const uint8_t* base, int32_t slot, const AttnArgs& a) {
  return base + (uint64_t)(uint32_t)slot * (uint32_t)a.cache_ld;
}

// ---- 4-bit codes ----------------------------------------------------------------------------
//
// A code times its block's scale has at most 2 + 4 significant bits and lies in [2^-10, 2880]: exact in FP16 and
// in BF16.  Scale bytes are taken as magnitudes: bit 7 is not looked at, and 0x7F, which the encoder does not
// write, counts as 480, the next number of the grid.  So whatever the cache holds where nothing was written is
// finite, and masked by a weight of 0.

// Scale bytes 0 and 1 (or 2 and 3) of w as FP16 times 2^-8: the byte's fields stand 7 bits up in FP16's, whose exponent
// counts from 15 and not from 7.
template <int PAIR>
__device__ __forceinline__ f16x2 scale_pair(uint32_t w) {
  const uint32_t two = __builtin_amdgcn_perm(0u, w, PAIR ? 0x0C030C02u : 0x0C010C00u);
  return __builtin_bit_cast(f16x2, (two & 0x007F007Fu) << 7);
}

// Codes 2 B and 2 B + 1 of w, times 2^8 (what scale_pair lacks).
template <int B>
__device__ __forceinline__ f16x2 two_codes(uint32_t w) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, B));
}

template <int B>
__device__ __forceinline__ uint32_t two_f16(uint32_t w, f16x2 scales) {
  return __builtin_bit_cast(uint32_t, two_codes<B>(w) * scales);
}

// The same in BF16, which has no packed product: in FP32, whose upper half it is.  `scale`: byte << 20 as FP32, the
// scale times 2^-120.
template <int B>
__device__ __forceinline__ uint32_t two_bf16(uint32_t w, float scale) {
  const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 0x1p120f, B);
  return __builtin_amdgcn_perm(__float_as_uint(v.y * scale), __float_as_uint(v.x * scale), 0x07060302u);
}

// Eight codes of a key in the query's type; `byte`: which of the bytes of `scales` is their block's.
template <bool BF16>
__device__ __forceinline__ u32x4 decode_key8(uint32_t w, uint32_t scales, int byte) {
  if constexpr (BF16) {
    const float s = __uint_as_float((scales >> (8 * byte) & 0x7Fu) << 20);
    return u32x4{two_bf16<0>(w, s), two_bf16<1>(w, s), two_bf16<2>(w, s), two_bf16<3>(w, s)};
  }
  const f16x2 two = byte & 2 ? scale_pair<1>(scales) : scale_pair<0>(scales);
  const f16x2 s = byte & 1 ? f16x2{two[1], two[1]} : f16x2{two[0], two[0]};
  return u32x4{two_f16<0>(w, s), two_f16<1>(w, s), two_f16<2>(w, s), two_f16<3>(w, s)};
}

// Codes of the same 8 dims of two keys, put together by dim: byte b of `even` holds dim 2 b of both keys, of `odd`
// dim 2 b + 1.
__device__ __forceinline__ void pair_keys(uint32_t k0, uint32_t k1, uint32_t& even, uint32_t& odd) {
  constexpr uint32_t low = 0x0F0F0F0Fu;
  even = (k0 & low) | ((k1 << 4) & ~low);
  odd = ((k0 >> 4) & low) | (k1 & ~low);
}

// Scale bytes of two keys (in the low byte of each) as scale_pair gives them.
__device__ __forceinline__ f16x2 scales_of_keys(uint32_t s0, uint32_t s1) {
  return __builtin_bit_cast(f16x2, ((s0 | s1 << 16) & 0x007F007Fu) << 7);
}

// Non-zero where one of the four codes is NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// The four codes with NaN replaced by 0.
__device__ __forceinline__ uint32_t without_nans(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xFFu); }

// 4 x 4 byte transpose: out[t] holds byte t of in[0 .. 3].
__device__ __forceinline__ void transpose4(const uint32_t in[4], uint32_t out[4]) {
  const uint32_t p0 = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u);
  const uint32_t p1 = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);
  const uint32_t q0 = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u);
  const uint32_t q1 = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(q0, p0, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(q0, p0, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(q1, p1, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(q1, p1, 0x07060302u);
}

// Four codes as four 16-bit values (exact: every E4M3 value is an FP16 and a BF16 value).
__device__ __forceinline__ u32x2 decode_f16(uint32_t w) {
  u32x2 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, false));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, true));
  return o;
}

__device__ __forceinline__ u32x2 decode_bf16(uint32_t w) {
  u32x2 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, false));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, true));
  return o;
}

// Keys are decoded to the query's type, values to FP16.
template <bool BF16>
__device__ __forceinline__ u32x2 decode_key(uint32_t w) {
  if constexpr (BF16) return decode_bf16(w);
  return decode_f16(w);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  f16x2 p;
  p[0] = (_Float16)a;
  p[1] = (_Float16)b;
  return __builtin_bit_cast(uint32_t, p);
}

// One output element in the query's type, rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
  if constexpr (BF16) {
    bf16x2 p;
    p[0] = (__bf16)a;
    p[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, p);
  }
  return pack_f16(a, b);
}

// ---- division of the work -------------------------------------------------------------------

// A stretch of one item's key units.
struct Segment {
  int32_t r, tile, kv_head;
  int32_t u0, u1;    // units
  bool first, last;  // it holds the item's first / last unit
  int32_t last_worker;  // worker that holds the item's last unit
};

// What every workgroup leaves for the joining kernel.
struct Header {
  int32_t r, tile, kv_head;
  int32_t last_worker;  // of the item that begins in this worker and ends in a later one, else -1
  int32_t worker;
  int32_t unused[3];
};

// Work of request r in units, all its items: every item counts the units of the whole request.  (An
// item of a prompt whose rows see less skips the rest; such calls are divided by row tiles unless
// the new tokens are few beside their context.)
__device__ __forceinline__ void weight_of(const AttnArgs& a, int32_t r, int32_t rows, int32_t unit,
                                          uint32_t& units, uint64_t& total) {
  const Request q = request_of(a, r);
  const uint64_t tiles = ((uint64_t)q.count * a.group.d + rows - 1) / (uint32_t)rows;
  units = ((uint32_t)q.keys + (uint32_t)unit - 1) / (uint32_t)unit;
  if (units == 0) units = 1;  // the rows still get their zeros
  total = (uint64_t)units * tiles * (uint32_t)a.kv_heads;
}

__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int d) {
  const uint32_t lo = __shfl_up((uint32_t)x, d), hi = __shfl_up((uint32_t)(x >> 32), d);
  return (uint64_t)hi << 32 | lo;
}

// Quotient of 64-bit numbers that mostly fit 32 bits.
__device__ __forceinline__ uint64_t quotient(uint64_t n, uint64_t d) {
  return ((n | d) >> 32) == 0 ? (uint32_t)n / (uint32_t)d : n / d;
}

// Workgroup b runs on XCD b % 8, so worker numbers run through one XCD after another: workers next to
// each other, which read the same rows for neighbouring KV heads, share an L2 (with 64 dims two heads
// share every cache line).
__device__ __forceinline__ uint32_t worker_of(uint32_t b, uint32_t P) {
  const uint32_t per = (P + 7) / 8, k = b / 8;
  return k < per ? (b % 8) * per + k : 0xFFFFFFFFu;
}

// The workers' shares: worker w takes units [W w / P, W (w + 1) / P) of the W units of all items, one
// after another.  Every workgroup finds its own start by summing the requests' weights (one pass over
// the lengths, or two where there are more requests than threads), with no launch before it and
// nothing kept.  The state lies in LDS and the first thread advances it: it is used once a segment.
template <int NT>
struct Share {
  uint64_t W, x, end;  // all units; the next unit and the end of this worker's share
  uint64_t base;       // units before request r
  uint64_t total;      // of request r
  uint64_t sums[NT / 64];
  uint32_t units;      // of an item of request r
  uint32_t P;
  int32_t r;
  int32_t worker;  // this workgroup's number
  int32_t more;
  Segment segment;

  // Sum over the wavefronts before this one, and over all; `t` becomes the wavefront's inclusive sum.
  __device__ __forceinline__ void scan(uint64_t& t, uint64_t& before, uint64_t& all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t p = shfl_up64(t, d);
      if (lane >= d) t += p;
    }
    if (lane == 63) sums[wave] = t;
    __syncthreads();
    before = all = 0;
    for (int k = 0; k < NT / 64; ++k) {
      if (k < wave) before += sums[k];
      all += sums[k];
    }
    __syncthreads();
  }

  __device__ __forceinline__ void begin(int32_t rows, int32_t unit) {
    const AttnArgs& a = args();
    const int tid = threadIdx.x;
    const int R = a.requests;
    uint64_t sum = 0, first = 0, mine = 0, own = 0;
    for (int b = 0; b < R; b += NT) {
      const int i = b + tid;
      uint64_t t = 0, before, all;
      uint32_t u;
      if (i < R) weight_of(a, i, rows, unit, u, t);
      own = t;
      scan(t, before, all);
      first = sum + before + t - own;  // of the last pass: used only where it is the first too
      mine = own;
      sum += all;
    }
    // a worker takes two units at least: smaller shares cost more to join than to compute
    const uint64_t most = (sum + 1) / 2, limit = (uint64_t)a.workers;
    const uint32_t p = (uint32_t)(most < limit ? (most > 0 ? most : 1) : limit);
    const uint32_t w = worker_of(blockIdx.x, p);
    const uint64_t x0 = w < p ? quotient(sum * w, p) : 0, x1 = w < p ? quotient(sum * (w + 1), p) : 0;
    if (tid == 0) {
      W = sum;
      P = p;
      worker = (int32_t)w;
      x = x0;
      end = x1;
      r = 0;
      base = 0;
    }
    __syncthreads();
    if (x0 < x1) {
      // the request that holds unit x0
      if (R <= NT) {
        if (tid < R && first <= x0 && x0 < first + mine) {
          base = first;
          r = tid;
        }
      } else {
        uint64_t s = 0;
        for (int b = 0; b < R && s <= x0; b += NT) {
          const int i = b + tid;
          uint64_t t = 0, before, all;
          uint32_t u;
          if (i < R) weight_of(a, i, rows, unit, u, t);
          const uint64_t o = t;
          scan(t, before, all);
          const uint64_t f = s + before + t - o;
          if (i < R && f <= x0 && x0 < f + o) {
            base = f;
            r = i;
          }
          s += all;
        }
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t u;
        uint64_t t;
        weight_of(a, r, rows, unit, u, t);
        units = u;
        total = t;
      }
    }
  }

  __device__ __forceinline__ bool take(Segment& s) const {
    if (!uniform(more)) return false;
    s.r = uniform(segment.r);
    s.tile = uniform(segment.tile);
    s.kv_head = uniform(segment.kv_head);
    s.u0 = uniform(segment.u0);
    s.u1 = uniform(segment.u1);
    s.first = uniform(segment.first);
    s.last = uniform(segment.last);
    s.last_worker = uniform(segment.last_worker);
    return true;
  }

  // Without sharing: row tile number `worker` of all requests' (of one KV head; a request's last tile first:
  // it sees the most keys), and the grid's height further at the next call.  False past the last.
  // Uniform over the workgroup, which has to pass a barrier before the first call and between two.
  __device__ __forceinline__ bool next_tile(int32_t rows, int32_t unit, Segment& s) {
    const AttnArgs& a = args();
    const int tid = threadIdx.x;
    const int R = a.requests;
    const uint64_t y = (uint32_t)uniform(worker);
    if (tid == 0) more = false;
    uint64_t sum = 0;
    for (int b = 0; b < R && sum <= y; b += NT) {
      const int i = b + tid;
      uint64_t t = i < R ? ((uint64_t)request_of(a, i).count * a.group.d + rows - 1) / (uint32_t)rows : 0, before, all;
      const uint64_t own = t;
      scan(t, before, all);
      const uint64_t first = sum + before + t - own;
      if (first <= y && y < first + own) {
        const uint32_t keys = (uint32_t)request_of(a, i).keys;
        segment = Segment{i, (int32_t)(first + own - 1 - y), (int32_t)blockIdx.x, 0, (int32_t)((keys + (uint32_t)unit - 1) / (uint32_t)unit), true, true, 0};
        more = true;
      }
      sum += all;
    }
    if (tid == 0) worker = (int32_t)y + a.all_tiles;  // (behind a barrier of the sums; read again a call later)
    __syncthreads();
    return take(s);
  }

  // The next segment, or false when the share is done.  Uniform over the workgroup, which has to pass
  // a barrier between two calls.
  __device__ __forceinline__ bool next(int32_t rows, int32_t unit, Segment& s) {
    if (threadIdx.x == 0) {
      more = x < end;
      if (x < end) {
        const AttnArgs& a = args();
        while (x >= base + total) {  // ends before r leaves the requests: x < W, the sum of all totals
          base += total;
          ++r;
          uint32_t u;
          uint64_t t;
          weight_of(a, r, rows, unit, u, t);
          units = u;
          total = t;
        }
        const uint64_t y = x - base;
        const uint64_t item = quotient(y, units);
        const uint32_t off = (uint32_t)(y - item * units);
        uint64_t n = units - off;
        if (n > end - x) n = end - x;
        segment.r = r;
        // row tiles of one KV head lie next to each other: neighbouring workers read the same keys
        const uint32_t tiles = (uint32_t)quotient(total, (uint64_t)units * (uint32_t)a.kv_heads);
        segment.kv_head = (int32_t)quotient(item, tiles);
        segment.tile = (int32_t)(item - (uint64_t)segment.kv_head * tiles);
        segment.u0 = (int32_t)off;
        segment.u1 = (int32_t)(off + n);
        segment.first = off == 0;
        segment.last = off + n == units;
        const uint64_t tail = base + (item + 1) * units;  // one past the item's last unit
        // worker of unit tail - 1: the largest w with W w / P <= tail - 1, that is W w < tail P
        segment.last_worker = (int32_t)quotient(tail * P - 1, W);
        x += n;
      }
    }
    __syncthreads();
    return take(s);
  }
};

// Partial results: worker w keeps two slots, 2 w for a segment that continues an item of an earlier
// worker and 2 w + 1 for one whose item goes on in a later one.
__device__ __forceinline__ int64_t part_slot(uint32_t w, bool first) { return 2 * (int64_t)w + (first ? 1 : 0); }

}  // namespace attn
}  // namespace nvfp4
