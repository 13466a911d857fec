// Attention of few query rows over the paged FP8 cache: decode steps, drafted trees, short chunks.
// Also the kernel that joins partial results.
//
// What bounds it: every key and value code is read once per (request, KV head) and used by 16 or
// 32 rows, so the call is bound by HBM reads.  The kernel therefore keeps as many loads in flight as
// its registers hold and touches LDS only to join its wavefronts at the end of an item.  A wavefront
// takes 32 positions at a time, from the cache straight into MFMA operand registers:
//
//   scores   S^T[key][row] = K Q^T, v_mfma_f32_16x16x32 with the keys as rows of A.  Lane l holds
//            key l % 16; the dims of a 32-deep step are permuted (the same way in Q) so that the four
//            lanes of a key load 64 contiguous bytes at a time.
//   softmax  a column of S^T is a query row, so a lane's statistics are scalars; lanes l, l ^ 16,
//            l ^ 32, l ^ 48 share the row.
//   output   O^T[dim][row] += V^T P^T.  P^T leaves the first product in the operand layout of the
//            second (its 8 keys of a lane are {4 g .. 4 g + 3} and {16 + 4 g ..}, g = l / 16), so V^T
//            is loaded in that key order: 8 rows of the cache, head_dim / 16 contiguous bytes each,
//            16 lanes covering a row; 4 x 4 byte transposes put a dim's keys side by side.
//
// Keys are requested two steps ahead and values one, their slots looked up a step before that, so the
// chain block table -> address -> row is never waited for.  What the loop needs has to fit the registers
// of the workgroups that share a compute unit: one spilled value read back in the loop waits for every
// load in flight.
//
// Measured (HBM reads at 6.4 TB/s in a plain read kernel, copies at 4.9 TB/s): 64 requests x up to 8000
// positions, one token each, 4 KV heads x 256 dims, 569 MB: 112 us a call, 5.1 TB/s; 8 KV heads x 128
// dims, 569 MB: 122 us; 8 x 64 dims, 285 MB: 91 us, 3.1 TB/s.  One request of 100000 positions, 205 MB:
// 50 us.
#include "kv_attention_common.h"

namespace nvfp4 {
namespace {

using namespace attn;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kStep = 32;              // positions of a wavefront's step
constexpr int kUnit = kWaves * kStep;  // positions of a workgroup's step
static_assert(kUnit == kStreamUnit, "the division of the work counts in these");

// Codes of 32 positions as a lane holds them.
template <int D>
struct Keys {
  u32x4 k[2][D / 64];  // keys l % 16 and 16 + l % 16
};

template <int D>
struct Values {
  uint32_t v[8][D / 64];  // keys 4 g + i and 16 + 4 g + i
};

template <bool ONCE, typename T>
__device__ __forceinline__ T read(const T* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(p);
  return *p;
}

// A position that is not in the cache reads slot 0 (there is one) and is masked afterwards.  ONCE: the
// request's rows fit one tile, every line is read by one workgroup once, and the loads do not ask to be
// kept in the caches -- except those of keys of 64 and 128 dims, whose lines are read in two or more
// goes (64 x up to 8000 positions, 128 dims: 122 us so, keys not kept 127, all kept 138; 64 dims: 94, 105,
// 90; 256 dims: 118 us so, keys kept 113, all kept 125; one request of 100000 positions, 256 dims: 50, 44,
// 44).  Several row tiles of a request read the same lines at about the same time, and asking for them to
// be kept pays (16 x up to 6001 positions, 2 and 3 tiles of 128 dims: 60 and 80 us, not kept 68 and 88 us).
template <int D, bool ONCE>
__device__ __forceinline__ void load_keys(const AttnArgs& a, int32_t slot, const uint8_t* kbase, int lane, Keys<D>& c) {
  const int32_t s = slot < 0 ? 0 : slot;
  const uint8_t* base = kbase + (lane >> 4) * 16;
  const int from = (lane & 15) * 4;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const uint8_t* p = row_at(base, __builtin_amdgcn_ds_bpermute(from + 64 * t, s), a);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const u32x4* q = reinterpret_cast<const u32x4*>(p + 64 * j);
      c.k[t][j] = read<ONCE && D == 256>(q);
    }
  }
}

template <int D, bool ONCE>
__device__ __forceinline__ void load_values(const AttnArgs& a, int32_t slot, const uint8_t* vbase, int lane, Values<D>& c) {
  const int32_t s = slot < 0 ? 0 : slot;
  const uint8_t* base = vbase + (lane & 15) * (D / 16);
  const int from = (lane >> 4) * 16;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint8_t* p = row_at(base, __builtin_amdgcn_ds_bpermute(from + (16 * (e >> 2) + (e & 3)) * 4, s), a);
    if constexpr (D == 256) {
      const u32x4 w = read<ONCE>(reinterpret_cast<const u32x4*>(p));
      c.v[e][0] = w.x; c.v[e][1] = w.y; c.v[e][2] = w.z; c.v[e][3] = w.w;
    } else if constexpr (D == 128) {
      const u32x2 w = read<ONCE>(reinterpret_cast<const u32x2*>(p));
      c.v[e][0] = w.x; c.v[e][1] = w.y;
    } else {
      c.v[e][0] = read<ONCE>(reinterpret_cast<const uint32_t*>(p));
    }
  }
}

__device__ __forceinline__ float max_over_groups(float x) {
  x = __builtin_fmaxf(x, __shfl_xor(x, 16));
  return __builtin_fmaxf(x, __shfl_xor(x, 32));
}

__device__ __forceinline__ float sum_over_groups(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

template <bool BF16>
__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 y, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
}

// State of a wavefront over one segment: NQ column tiles of 16 query rows.
template <int D, int NQ>
struct State {
  u32x4 q[NQ][D / 32];
  f32x4 acc[NQ][D / 16];  // acc[.][t][i]: dim (4 g + i) * (D / 16) + t
  float m[NQ], l[NQ];     // l: this lane's keys only
  int32_t lo[NQ], hi[NQ];  // of the lane's rows, as in Row; their numbers are formed again where needed
  int32_t pos[NQ];
  float slope[NQ];
  int32_t lo_all, hi_all;  // positions every row of the tile sees: [lo_all, hi_all)
};

template <int D, bool BF16, int NQ, Scores SCORES>
__device__ __forceinline__ void step(const Segment& sg, const Request& rq, const Keys<D>& kc, Values<D>& vc, int32_t slot,
                                     int32_t j0, float c, float cap, int lane, State<D, NQ>& s) {
  const int g = lane >> 4;
  f32x4 x[2][NQ];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int n = 0; n < NQ; ++n) x[t][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < D / 64; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const u32x2 lo = decode_key<BF16>(kc.k[t][j][2 * h]);
        const u32x2 hi = decode_key<BF16>(kc.k[t][j][2 * h + 1]);
        const u32x4 k = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int n = 0; n < NQ; ++n) x[t][n] = mfma16<BF16>(k, s.q[n][2 * j + h], x[t][n]);
        // decode a few operands at a time: all of them at once take twice the registers of their codes
        if (t == 1) __builtin_amdgcn_sched_barrier(0);
      }

  __builtin_amdgcn_sched_barrier(0);  // the phases' instructions stay apart, to keep their registers few
  // wave-uniform: every position of the step is in the cache and seen by every row of the tile
  const uint64_t in_cache = __ballot(slot >= 0);
  const bool whole = in_cache == ~0ull && j0 >= s.lo_all && j0 + kStep <= s.hi_all;
  // scores are x cm + base, in units of log2
  float cm = c, base = 0.0f;
  if constexpr (SCORES != Scores::Plain) {
    if (cap > 0.0f) {
      if constexpr (SCORES == Scores::WideCap) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int n = 0; n < NQ; ++n) cap_wide<4>(x[t][n], c, cap);
        cm = 1.0f;
      } else {
        const float to_r = cm / cap * 2.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[t][n][i] = cap_term(x[t][n][i], to_r);
        base = cap * kLog2e;
        cm = -2.0f * base;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[t][n][i] = __builtin_fmaf(x[t][n][i], cm, base);
  if constexpr (SCORES != Scores::Plain) {
    const AttnArgs& a = args();
    if (a.slopes) {
      const int32_t* positions = a.tree ? a.positions : nullptr;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t kp = key_position(positions, rq, j0 + 16 * t + 4 * g + i);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            x[t][n][i] = __builtin_fmaf(s.slope[n], (float)(kp - s.pos[n]), x[t][n][i]);
        }
    }
  }
  // bit 16 t + i of seen[n] >> 4 g: whether row n sees position 16 t + 4 g + i of the step
  uint32_t seen[NQ];
  if (rarely(!whole)) {
    const AttnArgs& a = args();
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int32_t token = a.tree ? token_of(a, rq, (uint32_t)((sg.tile * NQ + n) * 16 + (lane & 15))) : -1;
      seen[n] = ((uint32_t)sees64(s.lo[n], s.hi[n], token, rq.ctx, j0) & (uint32_t)in_cache) >> (4 * g);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][n][i] = kept(x[t][n][i], seen[n], 16 * t + i, kMinusInf);
    }
  }

  u32x4 p[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float e[8], sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = exp2_of(x[i >> 2][n][i & 3] - s.m[n]);
    sum = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    if (rarely(__any(sum > kRaise))) {
      float top = x[0][n][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, x[i >> 2][n][i & 3]);
      const float m = __builtin_fmaxf(s.m[n], max_over_groups(top) - kBelow);
      const float f = exp2_of(s.m[n] - m);
      s.m[n] = m;
      s.l[n] *= f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) s.acc[n][t] *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = exp2_of(x[i >> 2][n][i & 3] - m);
      sum = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    }
    s.l[n] += sum;
    p[n] = u32x4{pack_f16(e[0], e[1]), pack_f16(e[2], e[3]), pack_f16(e[4], e[5]), pack_f16(e[6], e[7])};
  }

  // Values of positions outside the cache count as zeros.  A NaN code in a position that only some rows
  // see must reach those rows alone, which a product with 0 would not give: it counts as 0 here too
  // and the rows that see it are set to NaN afterwards.
  __builtin_amdgcn_sched_barrier(0);
  bool nans = false;
  if (rarely(!whole)) {
    const uint32_t mine = (uint32_t)in_cache >> (4 * g);  // bit 16 t + i: position 16 t + 4 g + i
    uint32_t bad = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t there = (uint32_t)((int32_t)(mine << (31 - (16 * (e >> 2) + (e & 3)))) >> 31);
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
        vc.v[e][d] &= there;
        const uint32_t b = nan_codes(vc.v[e][d]);
        bad |= b;
        vc.v[e][d] &= ~((b >> 7) * 0xFFu);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    nans = __any(bad != 0);
  }
#pragma unroll
  for (int d = 0; d < D / 64; ++d) {
    uint32_t a0[4], a1[4], t0[4], t1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a0[i] = vc.v[i][d];
      a1[i] = vc.v[4 + i][d];
    }
    transpose4(a0, t0);
    transpose4(a1, t1);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const u32x2 lo = decode_f16(t0[b]), hi = decode_f16(t1[b]);
      const u32x4 w = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
      for (int n = 0; n < NQ; ++n) s.acc[n][4 * d + b] = mfma16<false>(w, p[n], s.acc[n][4 * d + b]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (rarely(nans)) {
    const AttnArgs& a = args();
    const uint8_t* vbase = a.vc + (int64_t)sg.kv_head * D;
#pragma unroll 1
    for (int o = 0; o < kStep; ++o) {
      const int32_t at = __shfl(slot, o);
      if (at < 0) continue;
      // this lane's dims are the D / 4 from g * D / 4 on
      const uint8_t* p8 = row_at(vbase, at, a) + g * (D / 4);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int32_t token = a.tree ? token_of(a, rq, (uint32_t)((sg.tile * NQ + n) * 16 + (lane & 15))) : -1;
        const bool see = (sees64(s.lo[n], s.hi[n], token, rq.ctx, j0) >> o) & 1;
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {
          const uint32_t bad = see ? nan_codes(*reinterpret_cast<const uint32_t*>(p8 + 4 * w)) : 0u;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            constexpr int T = D / 16;
            f32x4& o4 = s.acc[n][(4 * w + b) % T];
            o4[(4 * w + b) / T] = __uint_as_float(__float_as_uint(o4[(4 * w + b) / T]) | ((bad >> (8 * b + 7)) & 1) * 0x7FFFFFFFu);
          }
        }
      }
    }
  }
}

template <int D, bool BF16, int NQ, Scores SCORES>
__device__ __forceinline__ void segment(const Segment& sg, bool split, int32_t worker, float* lds) {
  const AttnArgs& a = args();
  constexpr int kRows = 16 * NQ;
  constexpr int kPitch = D + 4;  // floats; 16 bytes a row apart, so a store's 8 lanes differ in banks
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, d16 = lane & 15;
  const Request rq = request_of(a, sg.r);
  State<D, NQ> s;
  const float c = a.scale * *a.ks * kLog2e, cap = SCORES != Scores::Plain ? a.cap : 0.0f;

  int32_t lo_min = 0x7FFFFFFF, hi_max = 0, lo_max = 0, hi_min = 0x7FFFFFFF;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const Row w = row_of(a, sg.r, rq, sg.kv_head, (uint32_t)(sg.tile * kRows + 16 * n + d16));
    s.lo[n] = w.lo;
    s.hi[n] = w.hi;
    s.pos[n] = w.pos;
    s.slope[n] = w.slope;
    s.m[n] = kNoScore;
    s.l[n] = 0.0f;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) s.acc[n][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t* qp = a.q + (int64_t)w.token * a.q_ts + (int64_t)w.head * a.q_hs + g * 16;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      s.q[n][j] = w.token >= 0 ? *reinterpret_cast<const u32x4*>(qp + 64 * (j >> 1) + 8 * (j & 1)) : u32x4{0, 0, 0, 0};
    if (w.token >= 0) {
      // a tree's rows see at most the request's keys, and below ctx all of them
      lo_min = min(lo_min, w.lo);
      hi_max = max(hi_max, a.tree ? rq.keys : w.hi);
      lo_max = max(lo_max, w.lo);
      hi_min = min(hi_min, w.hi);
    }
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    lo_min = min(lo_min, __shfl_xor(lo_min, d));
    hi_max = max(hi_max, __shfl_xor(hi_max, d));
    lo_max = max(lo_max, __shfl_xor(lo_max, d));
    hi_min = min(hi_min, __shfl_xor(hi_min, d));
  }
  s.lo_all = __builtin_amdgcn_readfirstlane(lo_max);
  s.hi_all = __builtin_amdgcn_readfirstlane(hi_min);
  lo_min = __builtin_amdgcn_readfirstlane(lo_min);
  hi_max = __builtin_amdgcn_readfirstlane(hi_max);
  int32_t u0 = sg.u0, u1 = sg.u1;
  if (lo_min >= hi_max) {
    u1 = u0;
  } else {
    u0 = max(u0, lo_min / kUnit);
    u1 = min(u1, (hi_max + kUnit - 1) / kUnit);
  }

  const int32_t* table_row = a.table + (int64_t)sg.r * a.table_ld;
  const uint8_t* kbase = a.kc + (int64_t)sg.kv_head * D;
  const uint8_t* vbase = a.vc + (int64_t)sg.kv_head * D;
  const uint32_t off = wave * kStep + (lane & 31);
  // slots of step u from the table entries e loaded before; entries of a unit before the
  // first are loaded too (of some position) and not used
  const auto slots = [&](int32_t e, int32_t u) { return slot_of(a, e, hi_max, (uint32_t)u * kUnit + off); };
  const auto entries = [&](int32_t u) { return entry_of(a, table_row, (uint32_t)u * kUnit + off); };
  // from the last unit to the first: what is nearest, and with a distance bias weighs most, comes first
  // and sets the reference
  if (u0 < u1) {
    int32_t u = u1 - 1;
    int32_t s0 = slots(entries(u), u), s1;
    int32_t e1 = entries(u - 1);
    __builtin_amdgcn_sched_barrier(0);
    Keys<D> k0, k1;
    Values<D> v;
    load_keys<D, NQ == 1>(a, s0, kbase, lane, k0);
    for (;; u -= 2) {
      // lane offsets are formed anew in each turn: kept through the loop, they push operands out to
      // scratch memory, and reading those back waits for the codes in flight
      int ln = lane;
      asm volatile("" : "+v"(ln));
      // (table entries are requested ahead of the codes: loads land in order, and looking at an entry
      // that was requested after them would wait for the codes)
      s1 = slots(e1, u - 1);
      const int32_t e2 = entries(u - 2);
      __builtin_amdgcn_sched_barrier(0);
      load_values<D, NQ == 1>(a, s0, vbase, ln, v);
      if (u > u0) load_keys<D, NQ == 1>(a, s1, kbase, ln, k1);
      step<D, BF16, NQ, SCORES>(sg, rq, k0, v, s0, u * kUnit + wave * kStep, c, cap, ln, s);
      if (u - 1 < u0) break;
      s0 = slots(e2, u - 2);
      e1 = entries(u - 3);
      __builtin_amdgcn_sched_barrier(0);
      load_values<D, NQ == 1>(a, s1, vbase, ln, v);
      if (u - 1 > u0) load_keys<D, NQ == 1>(a, s0, kbase, ln, k0);
      step<D, BF16, NQ, SCORES>(sg, rq, k1, v, s1, (u - 1) * kUnit + wave * kStep, c, cap, ln, s);
      if (u - 2 < u0) break;
    }
  }

  // join the wavefronts
  const AttnArgs& ea = args();
  float* ml = lds + kWaves * 16 * kPitch;  // [wave][kRows][2]
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float l = sum_over_groups(s.l[n]);
    if (g == 0) {
      ml[(wave * kRows + 16 * n + d16) * 2] = s.m[n];
      ml[(wave * kRows + 16 * n + d16) * 2 + 1] = l;
    }
  }
  const float vs = *ea.vs;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    __syncthreads();
    float m = kNoScore;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) m = __builtin_fmaxf(m, ml[(k * kRows + 16 * n + d16) * 2]);
    const float f = exp2_of(s.m[n] - m);
    float* mine = lds + (wave * 16 + d16) * kPitch + g * (D / 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < D / 16; t += 4) {
        f32x4 o = {s.acc[n][t][i], s.acc[n][t + 1][i], s.acc[n][t + 2][i], s.acc[n][t + 3][i]};
        *reinterpret_cast<f32x4*>(mine + i * (D / 16) + t) = o * f;
      }
    __syncthreads();
    // 16 threads a row, D / 16 contiguous dims each
    const int row = tid >> 4, part = tid & 15;
    float mr = kNoScore, lr = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) mr = __builtin_fmaxf(mr, ml[(k * kRows + 16 * n + row) * 2]);
#pragma unroll
    for (int k = 0; k < kWaves; ++k)
      lr += ml[(k * kRows + 16 * n + row) * 2 + 1] * exp2_of(ml[(k * kRows + 16 * n + row) * 2] - mr);
    float o[D / 16];
#pragma unroll
    for (int t = 0; t < D / 16; t += 4) {
      f32x4 sum = *reinterpret_cast<f32x4*>(lds + row * kPitch + part * (D / 16) + t);
#pragma unroll
      for (int k = 1; k < kWaves; ++k)
        sum += *reinterpret_cast<f32x4*>(lds + (k * 16 + row) * kPitch + part * (D / 16) + t);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t + i] = sum[i];
    }
    const uint32_t rr = (uint32_t)(sg.tile * kRows + 16 * n + row);
    if (rr < (uint32_t)rq.count * ea.group.d) {
      if (split && !(sg.first && sg.last)) {
        const int64_t at = part_slot((uint32_t)worker, sg.first) * kRows + 16 * n + row;
        float* op = ea.part + at * D + part * (D / 16);
#pragma unroll
        for (int t = 0; t < D / 16; t += 4) *reinterpret_cast<f32x4*>(op + t) = f32x4{o[t], o[t + 1], o[t + 2], o[t + 3]};
        if (part == 0) *reinterpret_cast<f32x2*>(ea.part_ml + 2 * at) = f32x2{mr, lr};
      } else {
        const int32_t i = (int32_t)div_of(rr, ea.group);
        const int32_t head = sg.kv_head * (int32_t)ea.group.d + (int32_t)(rr - (uint32_t)i * ea.group.d);
        const float inv = lr == 0.0f ? 0.0f : vs / lr;
        uint16_t* op = ea.out + (int64_t)(rq.start + i) * ea.out_ts + (int64_t)head * ea.out_hs + part * (D / 16);
#pragma unroll
        for (int t = 0; t < D / 16; t += 4)
          *reinterpret_cast<u32x2*>(op + t) = u32x2{pack_out<BF16>(o[t] * inv, o[t + 1] * inv), pack_out<BF16>(o[t + 2] * inv, o[t + 3] * inv)};
      }
    }
  }
  __syncthreads();  // the next segment writes ml and the tiles again
}

template <int D, bool BF16, int NQ, Scores SCORES>
__global__ void __launch_bounds__(kThreads, stream_groups(D, 16 * NQ)) attention_stream_kernel(AttnArgs) {
  constexpr int kRows = 16 * NQ;
  __shared__ __align__(16) float lds[kWaves * 16 * (D + 4) + kWaves * kRows * 2];
  __shared__ Share<kThreads> share;
  Segment s;
  if (args().workers == 0) {
    const AttnArgs& a = args();
    s.kv_head = blockIdx.x;
    s.r = blockIdx.y;
    s.first = s.last = true;
    s.last_worker = 0;
    const Request q = request_of(a, s.r);
    s.u0 = 0;
    s.u1 = (int32_t)(((uint32_t)q.keys + kUnit - 1) / kUnit);
    const int32_t tiles = (int32_t)(((uint32_t)q.count * a.group.d + kRows - 1) / kRows);
    for (s.tile = blockIdx.z; s.tile < tiles; s.tile += gridDim.z) segment<D, BF16, NQ, SCORES>(s, false, 0, lds);
    return;
  }
  share.begin(kRows, kUnit);
  Header* header = reinterpret_cast<Header*>(args().headers) + blockIdx.x;
  if (threadIdx.x == 0) header->last_worker = -1;
  while (share.next(kRows, kUnit, s)) {
    if (s.first && !s.last && threadIdx.x == 0) *header = Header{s.r, s.tile, s.kv_head, s.last_worker, share.worker, {0, 0, 0}};
    segment<D, BF16, NQ, SCORES>(s, true, uniform(share.worker), lds);
  }
}

// Pieces [k0, k1) of one row of an item that several workers computed, under the reference m: their sums
// of exponentials (l, the same in every lane) and of outputs (this lane's D / 64 dims).  Pieces are summed
// in the workers' order, whatever order they were computed in.
template <int D>
__device__ __forceinline__ void join_pieces(const AttnArgs& a, const Header& h, int32_t rows, int32_t local, int32_t k0,
                                            int32_t k1, float m, int lane, float& l, float (&o)[D / 64]) {
  constexpr int E = D / 64, kAtOnce = 16;
  const uint32_t w0 = (uint32_t)h.worker;
  l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int32_t b = k0; b < k1; b += kAtOnce) {
    // kAtOnce pieces are requested together; past the last, the last again, with weight 0
    float v[kAtOnce][E];
    const int32_t mine = min(b + (lane & (kAtOnce - 1)), k1 - 1);
    const f32x2 ml = *reinterpret_cast<const f32x2*>(a.part_ml + 2 * (part_slot(w0 + mine, mine == 0) * rows + local));
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int32_t at = min(b + k, k1 - 1);
      const float* p = a.part + (part_slot(w0 + at, at == 0) * rows + local) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = p[e];
    }
    const float f = exp2_of(ml.x - m);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const bool there = b + k < k1;
      const float fk = __shfl(f, k), lk = __shfl(ml.y, k);
      l = there ? __builtin_fmaf(lk, fk, l) : l;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = there ? __builtin_fmaf(v[k][e], fk, o[e]) : o[e];
    }
  }
}

// Joins the pieces of the items that were shared out: blocks (b, y) take rows of the item that begins in
// workgroup b's share and ends in that of worker last_worker.  With few pieces a wavefront takes a whole
// row and a block four; with more (one long request over all workers) a block takes one row and its
// wavefronts a quarter of the pieces each.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) attention_join_kernel(AttnArgs a, int32_t rows) {
  constexpr int E = D / 64;
  __shared__ float sums[kWaves][D + 1];
  const Header h = reinterpret_cast<const Header*>(a.headers)[blockIdx.x];
  if (h.last_worker < 0) return;
  const Request rq = request_of(a, h.r);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t n = h.last_worker - h.worker + 1;
  const bool alone = n <= 16;  // a wavefront joins a row by itself
  const int32_t per = alone ? kWaves : 1;
  for (int32_t first = (int32_t)blockIdx.y * per; first < rows; first += (int32_t)gridDim.y * per) {
    const int32_t local = alone ? first + wave : first;
    const uint32_t row = (uint32_t)(h.tile * rows + local);
    const int32_t token = token_of(a, rq, row);
    if (!alone && token < 0) return;  // the same in all wavefronts; so are later rows
    if (token < 0) continue;
    float m = kNoScore;
    for (int32_t k = lane; k < n; k += 64)
      m = __builtin_fmaxf(m, a.part_ml[2 * (part_slot((uint32_t)(h.worker + k), k == 0) * rows + local)]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d));
    float o[E], l;
    const int32_t share = (n + kWaves - 1) / kWaves;
    join_pieces<D>(a, h, rows, local, alone ? 0 : min(wave * share, n), alone ? n : min((wave + 1) * share, n), m, lane, l, o);
    if (!alone) {
#pragma unroll
      for (int e = 0; e < E; ++e) sums[wave][lane * E + e] = o[e];
      if (lane == 0) sums[wave][D] = l;
      __syncthreads();
      l = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        l += sums[w][D];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += sums[w][lane * E + e];
      }
      __syncthreads();
      if (wave != 0) continue;
    }
    const float inv = l == 0.0f ? 0.0f : *a.vs / l;
    uint16_t* op = a.out + (int64_t)token * a.out_ts + (int64_t)head_of(a, rq, h.kv_head, row) * a.out_hs + lane * E;
    if constexpr (E == 1) {
      *op = (uint16_t)pack_out<BF16>(o[0] * inv, 0.0f);
    } else if constexpr (E == 2) {
      *reinterpret_cast<uint32_t*>(op) = pack_out<BF16>(o[0] * inv, o[1] * inv);
    } else {
      *reinterpret_cast<u32x2*>(op) = u32x2{pack_out<BF16>(o[0] * inv, o[1] * inv), pack_out<BF16>(o[2] * inv, o[3] * inv)};
    }
  }
}

template <int D, bool BF16, int NQ, Scores SCORES>
void launch_stream(const AttnArgs& a, hipStream_t stream) {
  const dim3 grid = a.workers ? dim3((uint32_t)a.workers) : dim3((uint32_t)a.kv_heads, (uint32_t)a.requests, (uint32_t)a.row_tiles);
  hipLaunchKernelGGL((attention_stream_kernel<D, BF16, NQ, SCORES>), grid, dim3(kThreads), 0, stream, a);
}

template <int D, bool BF16, int NQ>
void launch_stream(const AttnArgs& a, hipStream_t stream) {
  switch (scores_of(a)) {
    case Scores::Plain: launch_stream<D, BF16, NQ, Scores::Plain>(a, stream); break;
    case Scores::Modified: launch_stream<D, BF16, NQ, Scores::Modified>(a, stream); break;
    case Scores::WideCap: launch_stream<D, BF16, NQ, Scores::WideCap>(a, stream); break;
  }
}

template <int D, bool BF16>
hipError_t launch_all(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  switch (p.kernel) {
    case AttnKernel::Stream16: launch_stream<D, BF16, 1>(a, stream); break;
    case AttnKernel::Stream32: launch_stream<D, BF16, 2>(a, stream); break;
    case AttnKernel::Tiled: {
      const hipError_t t = launch_attention_tiled(a, D, BF16, stream);
      if (t != hipSuccess) return t;
      break;
    }
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.workers == 0) return e;
  // enough blocks for the rows that a tile has as far as the caller told, one row or four a block; the
  // kernel's stride covers the others
  const uint32_t y = (uint32_t)(p.join_rows <= 16 ? p.join_rows : (p.join_rows + kWaves - 1) / kWaves);
  hipLaunchKernelGGL((attention_join_kernel<D, BF16>), dim3((uint32_t)a.workers, y), dim3(kThreads), 0, stream, a, p.rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, int head_dim, bool bf16,
                            hipStream_t stream) {
  switch (head_dim) {
    case 64: return bf16 ? launch_all<64, true>(a, p, stream) : launch_all<64, false>(a, p, stream);
    case 128: return bf16 ? launch_all<128, true>(a, p, stream) : launch_all<128, false>(a, p, stream);
    default: return bf16 ? launch_all<256, true>(a, p, stream) : launch_all<256, false>(a, p, stream);
  }
}

}  // namespace nvfp4
