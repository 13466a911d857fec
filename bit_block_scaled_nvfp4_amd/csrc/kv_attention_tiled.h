// Attention of many query rows over the paged caches: prompts, long chunks, wide drafted trees.  Kernels are
// templates over the cache's format; kv_attention_tiled.hip has those of the FP8 cache,
// kv_attention_tiled_fp4.hip those of the 4-bit cache.
//
// What bounds it: the matrix cores, 4 FLOP per query row, visible position and dim, and next to them
// the vector unit, with about 11 instructions a score (256 dims; staging and addresses included).  A workgroup of 8
// wavefronts takes 256 query rows, 32 a wavefront, and walks over the keys in tiles of 8192 / head_dim
// positions (16 KB of keys and 16 KB of values in 16 bits), so a tile costs every wavefront 16 MFMAs of
// 32 x 32 x 16 for the scores and 16 for the output whatever the head size, and the 32 operand reads
// from LDS that go with them: at 128 bytes a clock the reads of 8 wavefronts take as long as their
// MFMAs, no longer.  Codes are decoded once a workgroup, on the way into LDS, not once a wavefront.
//
//   scores   S^T[key][row] = K Q^T; the query operand stays in registers.  A lane holds one row's
//            scores (row = lane % 32; lanes l and l ^ 32 share it), so statistics are lane scalars.
//   output   O^T[dim][row] += V^T P^T, P^T straight from the scores' registers: the 8 keys of a lane
//            in a 16-key step are {4 h .. 4 h + 3} and {8 + 4 h ..}, h = lane / 32, and V^T lies in LDS
//            with its keys in that order.
//
// Two LDS buffers: while a tile is multiplied out of one, the next goes from registers into the other,
// the two after it are on their way from the cache into registers (one was not enough to cover a read
// of HBM) and the slots of the one after those are looked up; one barrier a tile.
//
// Measured (a dense bf16 library product of 8192^3 reaches 1.24 PFLOP/s on such a card): 16384-token prompt,
// 24 heads of 256 dims over 4 KV heads, 3.30 ms, 1.00 PFLOP/s; 32 heads of 128 dims 1.00, of 64 dims 0.78,
// of 128 dims with capped scores 0.77 PFLOP/s.  The matrix cores are busy 45 % of the time at 256 dims, LDS has
// no bank conflicts.  Tiles with half their rows empty take as long as full ones: with one wavefront a
// SIMD its own chain (operand reads, scores, softmax, output) shows in full.  The loop's time depends on its
// address modulo 32 (chunk of 2048 over 30011 with a bias: 964 to 1030 us over the eight places).
//
// Over the 4-bit cache staging costs more: a load for the codes and one for the scale of each piece, a product with the scale,
// and for keys in BF16, which has no packed product, a step by way of FP32.  Chunk of 2048 over 30011, 24 heads of 256 dims over
// 4 KV heads: 1.72 ms and 33 us for the join under the profiler, 0.89 PFLOP/s together, the matrix cores busy 38 % of the time; a
// call among others, not profiled, 1.70 ms, 0.92 PFLOP/s.
#pragma once

#include "kv_attention_common.h"

namespace nvfp4 {
namespace {

using namespace attn;

constexpr int kThreads = 512;
constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves;
constexpr int kTileBytes = 16384;
constexpr int kLookUp = 4;  // wavefronts 4 .. 7 look up slots in turn

template <int D>
constexpr int kKeys = 8192 / D;  // positions of a tile: 32, 64, 128

// LDS layouts.  Tiles are rows of 256 bytes, 16 columns of 16; the column number is scrambled (an exclusive
// or that depends on the key or dim) so that 16 neighbouring lanes, or 8 of each half of a wavefront,
// reading one granule (lane half: two neighbouring ones) of as many neighbouring keys or dims, touch 16
// different columns, and so do the stores.  With 8 columns scrambled an operand read took 12 clocks
// instead of 8.

// Byte offset of granule `gr` (8 dims) of key `key` in a K tile [key][D].
template <int D>
__device__ __forceinline__ int k_offset(int key, int gr) {
  const int k0 = key & 1, k1 = (key >> 1) & 1, k2 = (key >> 2) & 1, k3 = (key >> 3) & 1;
  if constexpr (D == 64)  // two keys a row
    return ((key >> 1) << 8) + ((((k0 << 3) | gr) ^ ((k1 << 2) | (k2 << 1) | k3)) << 4);
  return key * (2 * D) + ((gr ^ ((k0 << 3) | (k1 << 2) | (k2 << 1) | k3)) << 4);
}

// Byte offset of granule `gr` (8 keys) of dim `dim` in a V^T tile [dim][keys]; 1, 2 or 4 dims a row.  Stores
// write half granules: 8 dims that lie 4 apart, 4 quads of keys.
template <int D>
__device__ __forceinline__ int v_offset(int dim, int gr) {
  const int d0 = dim & 1, d1 = (dim >> 1) & 1, d2 = (dim >> 2) & 1, d3 = (dim >> 3) & 1, d4 = (dim >> 4) & 1;
  if constexpr (D == 256)
    return ((dim >> 2) << 8) + ((((d1 << 3) | (d0 << 2) | gr) ^ ((d4 << 3) | (d3 << 2) | (d2 << 1) | d3)) << 4);
  if constexpr (D == 128)
    return ((dim >> 1) << 8) + ((((d0 << 3) | gr) ^ ((d4 << 3) | (d2 << 2) | ((d1 ^ d3) << 1) | d3)) << 4);
  return (dim << 8) + ((gr ^ (((d0 ^ d4) << 3) | ((d1 ^ d3) << 2) | (d2 << 1) | d3)) << 4);
}

// What a lane reads of those tiles, granule 2 e + h of key or dim 32 n + r, from its offset for e = n = 0:
// the scramble depends on r alone, so e's low bits are exchanged into the column and the rest is a
// constant offset.
template <int D>
__device__ __forceinline__ u32x4 read_k(const char* tile, int at, int n, int e) {
  return *reinterpret_cast<const u32x4*>(tile + (at ^ ((e & 7) << 5)) + n * (64 * D) + (e >> 3) * 256);
}

template <int D>
__device__ __forceinline__ u32x4 read_v(const char* tile, int at, int n, int e) {
  return *reinterpret_cast<const u32x4*>(tile + (at ^ (e << 5)) + n * (64 * kKeys<D>));
}

template <bool BF16>
__device__ __forceinline__ f32x16 mfma32(u32x4 x, u32x4 y, f32x16 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
}

// Whether one of n elements of q (a multiple of 8) is infinite or NaN: all bits of its exponent are set, and the
// lowest of them added carries into the sign's place.
template <bool BF16>
__device__ __forceinline__ bool no_numbers(const uint16_t* q, int n) {
  constexpr uint32_t exponent = BF16 ? 0x7F807F80u : 0x7C007C00u, lowest = BF16 ? 0x00800080u : 0x04000400u;
  uint32_t bad = 0;
#pragma unroll 1
  for (int i = 0; i < n; i += 8) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(q + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) bad |= ((v[k] & exponent) + lowest) & 0x80008000u;
  }
  return bad != 0;
}

__device__ __forceinline__ float other_half_max(float x) { return __builtin_fmaxf(x, __shfl_xor(x, 32)); }

// Barrier that orders LDS only: loads from the cache stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Which of a tile's positions are in the cache, bit per position.
template <int D>
struct There {
  uint64_t lo;
  __device__ __forceinline__ bool all() const { return lo == ~0ull; }
  __device__ __forceinline__ uint64_t half(int) const { return lo; }
};
template <>
struct There<64> {
  uint64_t lo, hi;  // hi: positions 64 .. 127
  __device__ __forceinline__ bool all() const { return (lo & hi) == ~0ull; }
  __device__ __forceinline__ uint64_t half(int n) const { return n ? hi : lo; }
};

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// This thread's codes of a tile on their way from the cache to LDS.
struct Fetched {
  u32x2 k[2];     // 8 dims of one key, twice
  uint32_t v[4];  // 4 dims of 4 consecutive keys
};

// The same over the 4-bit cache.
struct Fetched4 {
  uint32_t k[2];  // a block of 16 dims of one key
  uint32_t ks;    // its scale
  uint32_t v[2];  // 8 dims of 2 consecutive keys
  uint32_t vs[2];  // the scales of the block that holds these dims
};

template <Cache C>
struct FetchedOf {
  using Type = Fetched;
};
template <>
struct FetchedOf<Cache::Fp4> {
  using Type = Fetched4;
};

template <int D>
__device__ __forceinline__ int k_key(int tid) { return tid / (D / 16); }
template <int D>
__device__ __forceinline__ int k_chunk(int tid) { return tid % (D / 16); }
template <int D>
__device__ __forceinline__ int v_quad(int lane, int wave) { return (lane & 3) + 4 * (wave % (kKeys<D> / 16)); }
template <int D>
__device__ __forceinline__ int v_dim(int lane, int wave) { return 4 * ((lane >> 2) + 16 * (wave / (kKeys<D> / 16))); }

// The 4-bit cache's: a pair of keys and 8 dims; 8 lanes read 32 bytes of a row.  (4 keys and 4 dims, as above, are eight
// loads where these are four: chunk of 2048 over 30011, 32 heads over 8 of 128 dims 1290 us, so 1202; of 64 dims 824 and 799; 24
// over 4 of 256 dims 1878 and 1830.)  A store waits two clocks for banks; 16 pairs and 4 eights of 256 dims a wavefront have
// no such wait, read 16 bytes of a row, and take as long (1793 and 1800 us).
template <int D>
__device__ __forceinline__ int v_pair(int lane, int wave) { return (lane & 7) + 8 * (wave % (kKeys<D> / 16)); }
template <int D>
__device__ __forceinline__ int v_dim8(int lane, int wave) { return 8 * ((lane >> 3) + 8 * (wave / (kKeys<D> / 16))); }

// Slots of a tile (`sl`, in LDS) and which of them are in the cache; the codes are requested.
template <int D>
__device__ __forceinline__ void fetch(const AttnArgs& a, const int32_t* sl, const uint64_t* in_cache, const uint8_t* kbase,
                                      const uint8_t* vbase, int tid, Fetched& f, There<D>& there) {
  const int lane = tid & 63, wave = tid >> 6;
  // a position that is not in the cache reads slot 0 (there is one): its scores are masked, its values
  // replaced by zeros
  const int32_t sk = max(sl[k_key<D>(tid)], 0);
  const i32x4 sv = *reinterpret_cast<const i32x4*>(sl + 4 * v_quad<D>(lane, wave));
  there.lo = uniform64(in_cache[0]);
  if constexpr (D == 64) there.hi = uniform64(in_cache[1]);
  const uint8_t* kp = row_at(kbase, sk, a) + 8 * k_chunk<D>(tid);
  f.k[0] = *reinterpret_cast<const u32x2*>(kp);
  f.k[1] = *reinterpret_cast<const u32x2*>(kp + D / 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = *reinterpret_cast<const uint32_t*>(row_at(vbase, max(sv[i], 0), a) + v_dim<D>(lane, wave));
}

// Rows of a tile instead of slots: the KV head is in their number.
template <int D>
__device__ __forceinline__ void fetch(const AttnArgs& a, const int32_t* sl, const uint64_t* in_cache, const uint8_t* kbase,
                                      const uint8_t* vbase, int tid, Fetched4& f, There<D>& there) {
  const int lane = tid & 63, wave = tid >> 6;
  const uint64_t sk = (uint32_t)max(sl[k_key<D>(tid)], 0);
  const int64_t sv = *reinterpret_cast<const int64_t*>(sl + 2 * v_pair<D>(lane, wave));
  there.lo = uniform64(in_cache[0]);
  if constexpr (D == 64) there.hi = uniform64(in_cache[1]);
  const u32x2 k = *reinterpret_cast<const u32x2*>(kbase + sk * (D / 2) + 8 * k_chunk<D>(tid));
  f.k[0] = k.x;
  f.k[1] = k.y;
  f.ks = a.kbs[sk * (D / 16) + k_chunk<D>(tid)];
  const uint32_t dim = v_dim8<D>(lane, wave);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t row = (uint32_t)max((int32_t)(sv >> (32 * i)), 0);
    f.v[i] = *reinterpret_cast<const uint32_t*>(vbase + row * (D / 2) + dim / 2);
    f.vs[i] = a.vbs[row * (D / 16) + dim / 16];
  }
}

// Decode into LDS.  `whole`: every row of the workgroup sees every position of the tile; else values
// of positions that are not in the cache, and NaN codes, are staged as zeros.  Returns whether this
// wavefront's values held such a code.
template <int D, bool BF16>
__device__ __forceinline__ bool stage(const Fetched& f, const There<D>& there, bool whole, char* kt, char* vt, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  const int kk = k_key<D>(tid), c = k_chunk<D>(tid);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const u32x2 lo = decode_key<BF16>(f.k[e].x), hi = decode_key<BF16>(f.k[e].y);
    *reinterpret_cast<u32x4*>(kt + k_offset<D>(kk, c + e * (D / 16))) = u32x4{lo.x, lo.y, hi.x, hi.y};
  }
  const int quad = v_quad<D>(lane, wave), dim = v_dim<D>(lane, wave);
  uint32_t in[4] = {f.v[0], f.v[1], f.v[2], f.v[3]}, t[4];
  bool any = false;
  if (rarely(!whole)) {
    const uint64_t from = there.half(wave >= 4);
    const uint32_t four = (uint32_t)(from >> ((4 * quad) & 63));
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      in[i] = (four >> i) & 1 ? in[i] : 0u;
      bad |= nan_codes(in[i]);
      in[i] = without_nans(in[i]);
    }
    any = __any(bad != 0);
  }
  transpose4(in, t);
  // keys 16 s + 8 e + 4 h + i are half e of granule 2 s + h
  const int gr = (quad >> 2) * 2 + (quad & 1), half = (quad >> 1) & 1;
#pragma unroll
  for (int b = 0; b < 4; ++b) *reinterpret_cast<u32x2*>(vt + v_offset<D>(dim + b, gr) + 8 * half) = decode_f16(t[b]);
  return any;
}

// From the 4-bit cache: whatever its codes are, they are finite, and a weight of 0 masks them.
template <int D, bool BF16>
__device__ __forceinline__ bool stage(const Fetched4& f, const There<D>&, bool, char* kt, char* vt, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  const int kk = k_key<D>(tid), c = k_chunk<D>(tid);
  // Granules 2 c and 2 c + 1 of the key: which of them first is chosen so that 16 neighbouring lanes of a store, which
  // differ in c or in the key's low bits, touch 16 different columns, and each 8 of them columns that differ modulo 8 (without
  // the second, half of the stores' bank conflicts: 1843 us for 1793, at 64 dims 783 for 760, each pair in one run)
  const int odd = (D == 256 ? c >> 2 ^ c >> 3 : D == 128 ? c >> 2 ^ kk : kk ^ kk >> 1) & 1;
  const uint32_t k0 = f.k[0], k1 = f.k[1];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    *reinterpret_cast<u32x4*>(kt + k_offset<D>(kk, 2 * c + (e ^ odd))) = decode_key8<BF16>(e ^ odd ? k1 : k0, f.ks, 0);
  const int pair = v_pair<D>(lane, wave), dim = v_dim8<D>(lane, wave);
  uint32_t even, odds;
  pair_keys(f.v[0], f.v[1], even, odds);
  const f16x2 by = scales_of_keys(f.vs[0], f.vs[1]);
  // (granules as in the other stage)
  const int quad = pair >> 1, gr = (quad >> 2) * 2 + (quad & 1), at = 8 * ((quad >> 1) & 1) + 4 * (pair & 1);
  const auto put = [&](int d, uint32_t two) { *reinterpret_cast<uint32_t*>(vt + v_offset<D>(dim + d, gr) + at) = two; };
  put(0, two_f16<0>(even, by));
  put(1, two_f16<0>(odds, by));
  put(2, two_f16<1>(even, by));
  put(3, two_f16<1>(odds, by));
  put(4, two_f16<2>(even, by));
  put(5, two_f16<2>(odds, by));
  put(6, two_f16<3>(even, by));
  put(7, two_f16<3>(odds, by));
  return false;
}

// Score of element i of x[n], less m: x cm + (slope * offset + (bias - m)).
template <Scores SCORES>
__device__ __forceinline__ float score(float x, float cm, float slope, float shift, int n, int i) {
  if constexpr (SCORES != Scores::Plain) shift = __builtin_fmaf(slope, (float)(32 * n + 8 * (i >> 2) + (i & 3)), shift);
  return __builtin_fmaf(x, cm, shift);
}

// exp2 of the scores less m in FP16, in the output product's operand layout; returns their sum in FP32.
template <int N, Scores SCORES>
__device__ __forceinline__ float exponentials(const f32x16 (&x)[N], float cm, float slope, float shift, u32x4 (&p)[2 * N]) {
  float sum = 0.0f;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = exp2_of(score<SCORES>(x[n][8 * u + i], cm, slope, shift, n, 8 * u + i));
      sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      p[2 * n + u] = u32x4{pack_f16(e[0], e[1]), pack_f16(e[2], e[3]), pack_f16(e[4], e[5]), pack_f16(e[6], e[7])};
    }
  return sum;
}

// Query operands of a wavefront that stay in registers; with 256 dims they, the output and the scores
// do not fit 256 registers together, and the other half is read from LDS (8 more operand reads a tile,
// beside 32).
template <int D>
constexpr int kQueryRegs = D == 256 ? 8 : D / 16;

template <int D>
struct WaveState {
  u32x4 q[kQueryRegs<D>];
  f32x16 acc[D / 32];  // acc[.][4 j + i]: dim 32 . + 8 j + 4 h + i
  float m, l;
  int32_t lo, hi;  // of the lane's row, as in Row; the rest of it is formed again where it is needed
  int32_t pos;
  float slope;
  int32_t lo_min, hi_max, lo_all, hi_all;  // over the wavefront's rows
};

template <int D, bool BF16, Scores SCORES>
__device__ __forceinline__ void multiply(float cap, const Request& rq, const char* qt, const char* kt, const char* vt, const There<D>& there,
                                         bool nans, bool moved, float* away, const Segment& now, uint32_t my_row, int32_t j0, float c, float inv_cap, int lane, WaveState<D>& s) {
  constexpr int N = kKeys<D> / 32;
  const int r = lane & 31, h = lane >> 5;
  const int kat = k_offset<D>(r, h), vat = v_offset<D>(r, h);
  f32x16 x[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[n][i] = 0.0f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e)
      x[n] = mfma32<BF16>(read_k<D>(kt, kat, n, e), e < kQueryRegs<D> ? s.q[e < kQueryRegs<D> ? e : 0] : *reinterpret_cast<const u32x4*>(qt + (e - kQueryRegs<D>) * 1024), x[n]);
  }
  // the phases' instructions stay apart: mixed, they need more registers than there are
  __builtin_amdgcn_sched_barrier(0);
  const bool whole = there.all() && j0 >= s.lo_all && j0 + kKeys<D> <= s.hi_all;
  // scores are x cm + bias, in units of log2; `bias` starts from the position's distance and each
  // element adds its offset in the tile
  float cm = c, bias = 0.0f;
  uint32_t none = kMinusInf;  // times cm: -inf
  if constexpr (SCORES != Scores::Plain) {
    float base = 0.0f;
    if (cap > 0.0f) {
      if constexpr (SCORES == Scores::WideCap) {
#pragma unroll
        for (int n = 0; n < N; ++n) cap_wide<16>(x[n], c, cap);
        cm = 1.0f;
      } else {
        const float to_r = c * inv_cap * 2.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[n][i] = cap_term(x[n][i], to_r);
          __builtin_amdgcn_sched_barrier(0);
        }
        base = cap * kLog2e;
        cm = -2.0f * base;
        none = kPlusInf;
      }
    }
    bias = __builtin_fmaf(s.slope, (float)(j0 + 4 * h - s.pos), base);
    if (rarely(moved && j0 + kKeys<D> > rq.ctx)) {
      // drafted keys count at positions of their own: their difference from the place in the cache, by
      // way of LDS (this wavefront's part)
      const int32_t* positions = args().positions;
#pragma unroll
      for (int k = 0; k < kKeys<D>; k += 64) {
        const int32_t j = j0 + k + lane;
        if (k + lane < kKeys<D>) away[k + lane] = (float)(key_position(positions, rq, j) - j);
      }
      const float per = s.slope / cm;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 w = *reinterpret_cast<const f32x4*>(away + 32 * n + 8 * g + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[n][4 * g + i] = __builtin_fmaf(per, w[i], x[n][4 * g + i]);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  }
  if (rarely(!whole)) {
    const AttnArgs& ra = args();
    const int32_t token = ra.tree ? token_of(ra, rq, my_row) : -1;
#pragma unroll
    for (int n2 = 0; n2 < N; n2 += 2) {
      const uint64_t bits = sees64(s.lo, s.hi, token, rq.ctx, j0 + 32 * n2) & there.half(n2);
      // bit 8 j + i: whether the row sees position 32 n + 8 j + 4 h + i
      const uint32_t seen0 = (uint32_t)bits >> (4 * h), seen1 = (uint32_t)(bits >> 32) >> (4 * h);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[n2][i] = kept(x[n2][i], seen0, 8 * (i >> 2) + (i & 3), none);
        if constexpr (N > 1) x[n2 + 1][i] = kept(x[n2 + 1][i], seen1, 8 * (i >> 2) + (i & 3), none);
      }
    }
  }
  u32x4 p[2 * N];
  float sum = exponentials<N, SCORES>(x, cm, s.slope, bias - s.m, p);
  if (rarely(__any(sum > kRaise))) {
    const float lower = bias - kBelow;
    float top = score<SCORES>(x[0][0], cm, s.slope, lower, 0, 0);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, score<SCORES>(x[n][i], cm, s.slope, lower, n, i));
    const float m = __builtin_fmaxf(s.m, other_half_max(top));
    const float f = exp2_of(s.m - m);
    s.m = m;
    s.l *= f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) s.acc[d] *= f;
    sum = exponentials<N, SCORES>(x, cm, s.slope, bias - m, p);
  }
  s.l += sum;
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 2 * N; ++e)
      s.acc[d] = mfma32<false>(read_v<D>(vt, vat, d, e), p[e], s.acc[d]);
  if (rarely(nans)) {
    // NaN codes among the tile's values were staged as zeros, so that they cannot reach rows that do not
    // see them; the rows that do are set here, from the cache
    const AttnArgs& ra = args();
    const int32_t token = ra.tree ? token_of(ra, rq, my_row) : -1;
    const int32_t request = uniform(now.r), kv_head = uniform(now.kv_head);
    const int32_t* table_row = ra.table + (int64_t)request * ra.table_ld;
#pragma unroll 1
    for (int o = 0; o < kKeys<D>; ++o) {
      const int32_t at = slot_of(ra, entry_of(ra, table_row, j0 + o), s.hi_max, j0 + o);
      if (at < 0) continue;
      const bool see = sees64(s.lo, s.hi, token, rq.ctx, j0 + o) & 1;
      const uint8_t* p8 = row_at(ra.vc + (int64_t)kv_head * D, at, ra) + 4 * h;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t bad = see ? nan_codes(*reinterpret_cast<const uint32_t*>(p8 + 32 * d + 8 * j)) : 0u;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            s.acc[d][4 * j + b] = __uint_as_float(__float_as_uint(s.acc[d][4 * j + b]) | ((bad >> (8 * b + 7)) & 1) * 0x7FFFFFFFu);
        }
    }
  }
}

template <int D>
struct Shared {
  char tiles[2][2][kTileBytes];  // [buffer][K, V^T]
  char query[D == 256 ? kWaves * 8192 : 16];  // [wavefront][operand][lane]
  int32_t limits[kWaves][4];
  int32_t nans[2][kWaves];
  float away[kWaves][kKeys<D>];  // drafted keys' positions less their places
  int32_t slots[8][128];    // of the tiles t with t % 8 = index
  uint64_t in_cache[8][2];
  Share<kThreads> share;
};

template <Cache C, int D, bool BF16, Scores SCORES, bool SPLIT>
__device__ __forceinline__ void segment(const Segment& sg, Shared<D>& lds) {
  const AttnArgs& a = args();
  constexpr int BN = kKeys<D>;
  int tid = threadIdx.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const Request rq = request_of(a, sg.r);
  WaveState<D> s;
  float c = a.scale * scale_of<C>(a.ks) * kLog2e;
  // a negative factor goes into the query, so that the largest raw product is the largest score
  const uint32_t flip = c < 0.0f ? 0x80008000u : 0u;
  c = __builtin_fabsf(c);
  // (and a factor of 0 too: -inf, a masked score, times 0 would be NaN; elements that are no numbers, times 0, are
  // looked at behind the loop)
  const uint32_t keep = c == 0.0f ? 0u : 0xFFFFFFFFu;
  if (c == 0.0f) c = 1.0f;
  const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
  const bool moved = SCORES != Scores::Plain && a.tree && a.slopes && a.positions;
  const uint32_t my_row = (uint32_t)(sg.tile * kRows + 32 * wave + r);
  const Row row = row_of(a, sg.r, rq, sg.kv_head, my_row);
  s.lo = row.lo;
  s.hi = row.hi;
  s.pos = row.pos;
  s.slope = row.slope;
  s.m = kNoScore;
  s.l = 0.0f;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) s.acc[d][i] = 0.0f;
  const uint16_t* qp = a.q + (int64_t)row.token * a.q_ts + (int64_t)row.head * a.q_hs + 8 * h;
  char* qt = lds.query + (D == 256 ? wave * 8192 + lane * 16 : 0);
#pragma unroll
  for (int e = 0; e < D / 16; ++e) {
    u32x4 v = {0, 0, 0, 0};
    if (row.token >= 0) v = (*reinterpret_cast<const u32x4*>(qp + 16 * e) ^ flip) & keep;
    if (e < kQueryRegs<D>) s.q[e < kQueryRegs<D> ? e : 0] = v;
    else *reinterpret_cast<u32x4*>(qt + (e - kQueryRegs<D>) * 1024) = v;  // read back by this lane only
  }
  int32_t lo_min = 0x7FFFFFFF, hi_max = 0, lo_all = 0, hi_all = 0x7FFFFFFF;
  if (row.token >= 0) {
    lo_min = lo_all = row.lo;
    hi_max = a.tree ? rq.keys : row.hi;
    hi_all = row.hi;
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    lo_min = min(lo_min, __shfl_xor(lo_min, d));
    hi_max = max(hi_max, __shfl_xor(hi_max, d));
    lo_all = max(lo_all, __shfl_xor(lo_all, d));
    hi_all = min(hi_all, __shfl_xor(hi_all, d));
  }
  s.lo_min = __builtin_amdgcn_readfirstlane(lo_min);
  s.hi_max = __builtin_amdgcn_readfirstlane(hi_max);
  s.lo_all = __builtin_amdgcn_readfirstlane(lo_all);
  s.hi_all = __builtin_amdgcn_readfirstlane(hi_all);
  if (lane == 0) {
    lds.limits[wave][0] = s.lo_min;
    lds.limits[wave][1] = s.hi_max;
    lds.limits[wave][2] = s.lo_all;
    lds.limits[wave][3] = s.hi_all;
  }
  __syncthreads();
  lo_min = hi_all = 0x7FFFFFFF;
  hi_max = lo_all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    lo_min = min(lo_min, lds.limits[w][0]);
    hi_max = max(hi_max, lds.limits[w][1]);
    lo_all = max(lo_all, lds.limits[w][2]);
    hi_all = min(hi_all, lds.limits[w][3]);
  }
  lo_all = __builtin_amdgcn_readfirstlane(lo_all);
  hi_all = __builtin_amdgcn_readfirstlane(hi_all);
  lo_min = __builtin_amdgcn_readfirstlane(lo_min);
  hi_max = __builtin_amdgcn_readfirstlane(hi_max);
  int32_t t0 = sg.u0, t1 = sg.u1;
  if (lo_min >= hi_max) {
    t1 = t0;
  } else {
    t0 = max(t0, lo_min / BN);
    t1 = min(t1, (hi_max + BN - 1) / BN);
  }

  const int32_t* table_row = a.table + (int64_t)sg.r * a.table_ld;
  const int64_t head_at = C == Cache::Fp4 ? 0 : (int64_t)sg.kv_head * D;
  const uint8_t* kbase = a.kc + head_at;
  const uint8_t* vbase = a.vc + head_at;
  // One wavefront looks up a tile's slots for all: the table entries are loaded in one turn, turned into
  // slots in the next and used by everybody in the one after, two turns before the tile is multiplied.
  const uint32_t o0 = lane & (BN - 1), o1 = 64 + lane;
  int32_t e0 = 0, e1 = 0;
  const auto load_entries = [&](int32_t t) {
    e0 = entry_of(a, table_row, (uint32_t)t * BN + o0);
    if constexpr (D == 64) e1 = entry_of(a, table_row, (uint32_t)t * BN + o1);
  };
  const auto put_slots = [&](int32_t t) {
    const int32_t x = slot_of<C>(a, e0, hi_max, (uint32_t)t * BN + o0, sg.kv_head);
    const uint64_t b = __ballot(x >= 0);
    if (lane < BN) lds.slots[t & 7][o0] = x;
    uint64_t c1 = ~0ull;
    if constexpr (D == 64) {
      const int32_t y = slot_of<C>(a, e1, hi_max, (uint32_t)t * BN + o1, sg.kv_head);
      c1 = __ballot(y >= 0);
      lds.slots[t & 7][o1] = y;
    }
    if (lane == 0) {
      lds.in_cache[t & 7][0] = b;
      lds.in_cache[t & 7][1] = c1;
    }
  };
  // from the last tile to the first: what is nearest, and with a distance bias weighs most, comes first
  // and sets the reference
  if (t0 < t1) {
    typename FetchedOf<C>::Type f;
    There<D> cur, nxt;
    // whether every row of the workgroup sees all of tile t
    const auto whole = [&](int32_t t, const There<D>& th) { return th.all() && t * BN >= lo_all && (t + 1) * BN <= hi_all; };
    // the first four tiles by one wavefront each, and the first entries of the loop's own look-ups
    const int32_t te = t1 - 1;
    load_entries(te - (wave < 4 ? wave : 4));
    if (wave < 4) put_slots(te - wave);
    lds_barrier();
    typename FetchedOf<C>::Type f0;
    There<D> nx2;
    fetch<D>(a, lds.slots[te & 7], lds.in_cache[te & 7], kbase, vbase, tid, f0, cur);
    fetch<D>(a, lds.slots[(te - 1) & 7], lds.in_cache[(te - 1) & 7], kbase, vbase, tid, f, nxt);
    const bool bad = stage<D, BF16>(f0, cur, whole(te, cur), lds.tiles[0][0], lds.tiles[0][1], tid);
    if (lane == 0) lds.nans[0][wave] = bad;
    fetch<D>(a, lds.slots[(te - 2) & 7], lds.in_cache[(te - 2) & 7], kbase, vbase, tid, f0, nx2);
    lds_barrier();
    // Turn of tile t out of buffer b: `x` holds the codes of tile t - 1, and then takes those of t - 3.
    const auto turn = [&](int32_t t, int b, typename FetchedOf<C>::Type& x) {
      // LDS and cache offsets are formed anew in each turn (a few instructions): kept in registers
      // through the loop, they push operands out to scratch memory
      if constexpr (D != 128) asm volatile("" : "+v"(tid));
      There<D> after = nx2;
      if (t > t0) {
        const bool bad2 = stage<D, BF16>(x, nxt, whole(t - 1, nxt), lds.tiles[b ^ 1][0], lds.tiles[b ^ 1][1], tid);
        if (lane == 0) lds.nans[b ^ 1][wave] = bad2;
        if (wave == kLookUp + (t & 3)) put_slots(t - 4);
        // (ahead of the codes: loads land in order, and an entry requested after them would be waited for
        // with them)
        if (wave == kLookUp + ((t - 1) & 3)) load_entries(t - 5);
        __builtin_amdgcn_sched_barrier(0);
        // tiles before the first have negative positions, which have no slot: they read slot 0 and are
        // not used
        fetch<D>(a, lds.slots[(t - 3) & 7], lds.in_cache[(t - 3) & 7], kbase, vbase, tid, x, after);
      }
      const int32_t j0 = t * BN;
      if (j0 < s.hi_max && j0 + BN > s.lo_min) {
        int32_t nans = 0;
        if (C == Cache::Fp8 && rarely(!whole(t, cur))) {
#pragma unroll
          for (int w = 0; w < kWaves; ++w) nans |= lds.nans[b][w];
        }
        multiply<D, BF16, SCORES>(a.cap, rq, qt, lds.tiles[b][0], lds.tiles[b][1], cur, C == Cache::Fp8 && uniform(nans) != 0, moved, lds.away[wave], lds.share.segment, my_row, j0, c, inv_cap, lane, s);
      }
      cur = nxt;
      nxt = nx2;
      nx2 = after;
      lds_barrier();
    };
    for (int32_t t = te;; t -= 2) {
      turn(t, 0, f);
      if (t - 1 < t0) break;
      turn(t - 1, 1, f0);
      if (t - 2 < t0) break;
    }
  }

  float l = s.l + __shfl_xor(s.l, 32);
  const AttnArgs& ea = args();
  const int32_t token = token_of(ea, rq, my_row);
  if (rarely(ea.scale * scale_of<C>(ea.ks) * kLog2e == 0.0f)) {
    // (here, and not where the query is read: what stands before the loop moves it, and its time depends on
    // its address modulo 32 by up to 7 %)
    bool none = false;
    if (token >= 0) {
      const int32_t head = head_of(ea, rq, uniform(lds.share.segment.kv_head), my_row);
      none = no_numbers<BF16>(ea.q + (int64_t)token * ea.q_ts + (int64_t)head * ea.q_hs, D);
    }
    if (none && l > 0.0f) l = __builtin_nanf("");  // a row that sees nothing stays 0
  }
  if (token >= 0) {
    const Segment& now = lds.share.segment;
    const bool first = uniform(now.first), last = uniform(now.last);
    if (SPLIT && !(first && last)) {
      const int64_t at = part_slot((uint32_t)uniform(lds.share.worker), first) * kRows + 32 * wave + r;
      float* op = ea.part + at * D + 4 * h;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4*>(op + 32 * d + 8 * j) = f32x4{s.acc[d][4 * j], s.acc[d][4 * j + 1], s.acc[d][4 * j + 2], s.acc[d][4 * j + 3]};
      if (h == 0) *reinterpret_cast<f32x2*>(ea.part_ml + 2 * at) = f32x2{s.m, l};
    } else {
      const float inv = l == 0.0f ? 0.0f : scale_of<C>(ea.vs) / l;
      const int32_t head = head_of(ea, rq, uniform(lds.share.segment.kv_head), my_row);
      uint16_t* op = ea.out + (int64_t)token * ea.out_ts + (int64_t)head * ea.out_hs + 4 * h;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<u32x2*>(op + 32 * d + 8 * j) =
              u32x2{pack_out<BF16>(s.acc[d][4 * j] * inv, s.acc[d][4 * j + 1] * inv), pack_out<BF16>(s.acc[d][4 * j + 2] * inv, s.acc[d][4 * j + 3] * inv)};
    }
  }
  __syncthreads();  // the next segment writes the limits and the tiles again
}

// How a workgroup finds its work: the row tile that its place in the grid says; a row tile among all
// requests' (next_tile); a share of all items' keys.  Three kernels, since what one of them needs beside
// segment() costs the others registers.
enum class Work { Place, Search, Share };

template <Cache C, int D, bool BF16, Scores SCORES, Work WORK>
__global__ void __launch_bounds__(kThreads) attention_tiled_kernel(AttnArgs) {
  __shared__ __align__(16) Shared<D> lds;
  Segment s;
  if constexpr (WORK == Work::Place) {
    const AttnArgs& a = args();
    s.kv_head = blockIdx.x;
    s.r = blockIdx.y;
    s.first = s.last = true;
    s.last_worker = 0;
    const Request q = request_of(a, s.r);
    s.u0 = 0;
    s.u1 = (int32_t)(((uint32_t)q.keys + kKeys<D> - 1) / kKeys<D>);
    const int32_t tiles = (int32_t)(((uint32_t)q.count * a.group.d + kRows - 1) / kRows);
    // the last row tiles see the most keys: they start first
    for (int32_t k = blockIdx.z; k < tiles; k += gridDim.z) {
      s.tile = tiles - 1 - k;
      if (threadIdx.x == 0) lds.share.segment = s;  // read again behind segment()'s first barrier
      segment<C, D, BF16, SCORES, false>(s, lds);
    }
  } else if constexpr (WORK == Work::Search) {
    if (threadIdx.x == 0) lds.share.worker = blockIdx.y;
    __syncthreads();
    while (lds.share.next_tile(kRows, kKeys<D>, s)) segment<C, D, BF16, SCORES, false>(s, lds);
  } else {
    lds.share.begin(kRows, kKeys<D>);
    Header* header = reinterpret_cast<Header*>(args().headers) + blockIdx.x;
    if (threadIdx.x == 0) header->last_worker = -1;
    while (lds.share.next(kRows, kKeys<D>, s)) {
      if (s.first && !s.last && threadIdx.x == 0) *header = Header{s.r, s.tile, s.kv_head, s.last_worker, lds.share.worker, {0, 0, 0}};
      segment<C, D, BF16, SCORES, true>(s, lds);
    }
  }
}

template <Cache C, int D, bool BF16, Scores SCORES>
void launch(const AttnArgs& a, hipStream_t stream) {
  const dim3 threads(kThreads), workers((uint32_t)a.workers), search((uint32_t)a.kv_heads, (uint32_t)a.all_tiles);
  const dim3 place((uint32_t)a.kv_heads, (uint32_t)a.requests, (uint32_t)a.row_tiles);
  if (a.workers)
    hipLaunchKernelGGL((attention_tiled_kernel<C, D, BF16, SCORES, Work::Share>), workers, threads, 0, stream, a);
  else if (a.all_tiles)
    hipLaunchKernelGGL((attention_tiled_kernel<C, D, BF16, SCORES, Work::Search>), search, threads, 0, stream, a);
  else
    hipLaunchKernelGGL((attention_tiled_kernel<C, D, BF16, SCORES, Work::Place>), place, threads, 0, stream, a);
}

template <Cache C, int D, bool BF16>
void launch(const AttnArgs& a, hipStream_t stream) {
  switch (scores_of(a)) {
    case Scores::Plain: launch<C, D, BF16, Scores::Plain>(a, stream); break;
    case Scores::Modified: launch<C, D, BF16, Scores::Modified>(a, stream); break;
    case Scores::WideCap: launch<C, D, BF16, Scores::WideCap>(a, stream); break;
  }
}

template <Cache C, int D>
void launch(const AttnArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) launch<C, D, true>(a, stream); else launch<C, D, false>(a, stream);
}

template <Cache C>
hipError_t launch_tiled(const AttnArgs& a, int head_dim, bool bf16, hipStream_t stream) {
  switch (head_dim) {
    case 64: launch<C, 64>(a, bf16, stream); break;
    case 128: launch<C, 128>(a, bf16, stream); break;
    default: launch<C, 256>(a, bf16, stream); break;
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace nvfp4
