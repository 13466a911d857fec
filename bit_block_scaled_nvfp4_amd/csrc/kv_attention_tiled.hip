// Attention of many query rows over the paged FP8 cache: prompts, long chunks, wide drafted trees.
//
// What bounds it: the matrix cores, 4 FLOP per query row, visible position and dim, and next to them
// the vector unit, which spends about 8 instructions a score on the softmax.  A workgroup of 8
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
// Two LDS buffers: while tile t is multiplied out of one, tile t + 1 goes from registers into the
// other, tile t + 2 is on its way from the cache into those registers and the slots of tile t + 3 are
// looked up; one barrier a tile.
#include "kv_attention_common.h"

namespace nvfp4 {
namespace {

using namespace attn;

constexpr int kThreads = 512;
constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves;
constexpr int kTileBytes = 16384;

template <int D>
constexpr int kKeys = 8192 / D;  // positions of a tile: 32, 64, 128

// Byte offset of 16-byte granule `gr` of key `key` in a K tile [key][D].  The granule index is
// scrambled by the key so that 8 lanes reading one granule of 8 keys touch 8 different bank groups.
template <int D>
__device__ __forceinline__ int k_offset(int key, int gr) {
  return key * (2 * D) + ((gr ^ (key & 7)) << 4);
}

// Byte offset of granule `gr` (8 keys) of dim `dim` in a V^T tile [dim][keys].  Reads take one granule
// of 8 consecutive dims, writes half granules of 4 dims that lie 4 apart: the scramble separates both.
template <int D>
__device__ __forceinline__ int v_offset(int dim, int gr) {
  if constexpr (D == 256) {
    // rows of 64 bytes, two to a bank cycle
    const int k = dim >> 1;
    return (k << 7) + (((((dim & 1) << 2) | gr) ^ (k & 7)) << 4);
  } else {
    const int f = (dim & 1) | ((dim >> 1) & 2) | (((dim << 1) ^ (dim >> 1)) & 4);
    return dim * (2 * kKeys<D>) + ((gr ^ f) << 4);
  }
}

// What a lane reads of those tiles, granule 2 e + h of key or dim 32 n + r: the scramble depends on r
// alone, so four addresses and constant offsets serve all e and n.
template <int D>
__device__ __forceinline__ u32x4 read_k(const char* const (&kp)[4], int n, int e) {
  return *reinterpret_cast<const u32x4*>(kp[e & 3] + n * (64 * D) + (e >> 2) * 128);
}

template <int D>
__device__ __forceinline__ u32x4 read_v(const char* const (&vp)[4], int n, int e) {
  return *reinterpret_cast<const u32x4*>(vp[e & 3] + n * (64 * kKeys<D>) + (e >> 2) * 128);
}

template <bool BF16>
__device__ __forceinline__ f32x16 mfma32(u32x4 x, u32x4 y, f32x16 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
}

__device__ __forceinline__ float other_half_max(float x) { return __builtin_fmaxf(x, __shfl_xor(x, 32)); }

// Barrier that orders LDS only: loads from the cache stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Slots of a tile's positions: lane l holds position l (and 64 + l).
template <int D>
struct Slots {
  int32_t s[D == 64 ? 2 : 1];
};

template <int D>
__device__ __forceinline__ Slots<D> look_up(const AttnArgs& a, const int32_t* table_row, int32_t end, int32_t j0, int lane) {
  Slots<D> r;
  r.s[0] = slot_at(a, table_row, end, j0 + (lane & (kKeys<D> - 1)));
  if constexpr (D == 64) r.s[1] = slot_at(a, table_row, end, j0 + 64 + lane);
  return r;
}

// Which of a tile's positions are in the cache, bit per position.
struct There {
  uint64_t lo, hi;  // hi: positions 64 .. 127, all ones in a shorter tile
  __device__ __forceinline__ bool all() const { return (lo & hi) == ~0ull; }
};

// This thread's codes of a tile on their way from the cache to LDS.
struct Fetched {
  u32x4 k;        // 16 dims of one key
  uint32_t v[4];  // 4 dims of 4 consecutive keys
};

template <int D>
__device__ __forceinline__ int k_key(int tid) { return tid / (D / 16); }
template <int D>
__device__ __forceinline__ int k_chunk(int tid) { return tid % (D / 16); }
template <int D>
__device__ __forceinline__ int v_quad(int lane, int wave) { return (lane & 3) + 4 * (wave % (kKeys<D> / 16)); }
template <int D>
__device__ __forceinline__ int v_dim(int lane, int wave) { return 4 * ((lane >> 2) + 16 * (wave / (kKeys<D> / 16))); }

template <int D>
__device__ __forceinline__ void fetch(const AttnArgs& a, const Slots<D>& sl, const uint8_t* kbase, const uint8_t* vbase,
                                      int tid, Fetched& f, There& there) {
  const int lane = tid & 63, wave = tid >> 6;
  there.lo = __ballot(sl.s[0] >= 0);
  there.hi = ~0ull;
  if constexpr (D == 64) there.hi = __ballot(sl.s[1] >= 0);
  const int kk = k_key<D>(tid), q4 = 4 * v_quad<D>(lane, wave);
  // the halves of a 128-position tile are uniform over a wavefront
  int32_t from_k = sl.s[0], from_v = sl.s[0];
  if constexpr (D == 64) {
    from_k = wave >= 4 ? sl.s[1] : sl.s[0];
    from_v = (wave & 7) >= 4 ? sl.s[1] : sl.s[0];
  }
  const int32_t sk = __shfl(from_k, kk & 63);
  // a position that is not in the cache reads slot 0 (there is one): its scores are masked, its values
  // replaced by zeros
  f.k = *reinterpret_cast<const u32x4*>(kbase + (int64_t)(sk < 0 ? 0 : sk) * a.cache_ld + 16 * k_chunk<D>(tid));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t sv = __shfl(from_v, (q4 + i) & 63);
    f.v[i] = *reinterpret_cast<const uint32_t*>(vbase + (int64_t)(sv < 0 ? 0 : sv) * a.cache_ld + v_dim<D>(lane, wave));
  }
}

// Decode into LDS, values that are NaN as zeros; returns whether this wavefront's values hold one.
template <int D, bool BF16>
__device__ __forceinline__ bool stage(const Fetched& f, const There& there, char* kt, char* vt, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  const int kk = k_key<D>(tid), c = k_chunk<D>(tid);
  const u32x2 k0 = decode_key<BF16>(f.k.x), k1 = decode_key<BF16>(f.k.y), k2 = decode_key<BF16>(f.k.z), k3 = decode_key<BF16>(f.k.w);
  *reinterpret_cast<u32x4*>(kt + k_offset<D>(kk, 2 * c)) = u32x4{k0.x, k0.y, k1.x, k1.y};
  *reinterpret_cast<u32x4*>(kt + k_offset<D>(kk, 2 * c + 1)) = u32x4{k2.x, k2.y, k3.x, k3.y};
  const int quad = v_quad<D>(lane, wave), dim = v_dim<D>(lane, wave);
  uint64_t from = there.lo;
  if constexpr (D == 64) from = (wave & 7) >= 4 ? there.hi : there.lo;
  const uint32_t four = (uint32_t)(from >> ((4 * quad) & 63));
  uint32_t in[4], t[4], bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    in[i] = (four >> i) & 1 ? f.v[i] : 0u;
    bad |= nan_codes(in[i]);
  }
  const bool any = __any(bad != 0);
  if (any) {
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = without_nans(in[i]);
  }
  transpose4(in, t);
  // keys 16 s + 8 e + 4 h + i are half e of granule 2 s + h
  const int gr = (quad >> 2) * 2 + (quad & 1), half = (quad >> 1) & 1;
#pragma unroll
  for (int b = 0; b < 4; ++b) *reinterpret_cast<u32x2*>(vt + v_offset<D>(dim + b, gr) + 8 * half) = decode_f16(t[b]);
  return any;
}

template <int D>
struct WaveState {
  u32x4 q[D / 16];
  f32x16 acc[D / 32];  // acc[.][4 j + i]: dim 32 . + 8 j + 4 h + i
  float m, l;
  Row row;
  int32_t lo_min, hi_max, lo_all, hi_all;  // over the wavefront's rows
};

template <int D, bool BF16>
__device__ __forceinline__ void multiply(const AttnArgs& a, const Request& rq, const char* kt, const char* vt, const There& there,
                                         bool nans, const int32_t* table_row, const uint8_t* vbase, int32_t j0, float c, float inv_cap, int lane, WaveState<D>& s) {
  constexpr int N = kKeys<D> / 32;
  const int r = lane & 31, h = lane >> 5;
  const char *kp[4], *vp[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kp[e] = kt + k_offset<D>(r, 2 * e + h);
    vp[e] = vt + v_offset<D>(r, (2 * e + h) & (kKeys<D> / 8 - 1));
  }
  f32x16 x[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[n][i] = 0.0f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e)
      x[n] = mfma32<BF16>(read_k<D>(kp, n, e), s.q[e], x[n]);
  }
  const bool whole = there.all() && j0 >= s.lo_all && j0 + kKeys<D> <= s.hi_all;
  float cm = c;
  if (a.cap > 0.0f || a.slopes || c == 0.0f) {
    cm = 1.0f;
    if (a.cap > 0.0f) {
      const float mul = c * (1.0f / kLog2e);
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[n][i] = capped(x[n][i] * mul, a.cap, inv_cap) * kLog2e;
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] *= c;
    }
    if (a.slopes) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int32_t kp = key_position(a, rq, j0 + 32 * n + 8 * (i >> 2) + 4 * h + (i & 3));
          x[n][i] = __builtin_fmaf(s.row.slope, (float)(kp - s.row.pos), x[n][i]);
        }
    }
  }
  if (!whole) {
#pragma unroll
    for (int n2 = 0; n2 < N; n2 += 2) {
      const uint64_t bits = sees64(a, s.row, rq, j0 + 32 * n2) & (n2 ? there.hi : there.lo);
      // bit 8 j + i: whether the row sees position 32 n + 8 j + 4 h + i
      const uint32_t seen0 = (uint32_t)bits >> (4 * h), seen1 = (uint32_t)(bits >> 32) >> (4 * h);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[n2][i] = kept(x[n2][i], seen0, 8 * (i >> 2) + (i & 3));
        if constexpr (N > 1) x[n2 + 1][i] = kept(x[n2 + 1][i], seen1, 8 * (i >> 2) + (i & 3));
      }
    }
  }
  float top = x[0][0];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, x[n][i]);
  if (__any(top * cm > s.m + kSlack)) {
    const float m = __builtin_fmaxf(s.m, other_half_max(top * cm));
    const float f = exp2_of(s.m - m);
    s.m = m;
    s.l *= f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) s.acc[d] *= f;
  }
  u32x4 p[2 * N];
  float sum = 0.0f;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = exp2_of(__builtin_fmaf(x[n][8 * u + i], cm, -s.m));
      sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      p[2 * n + u] = u32x4{pack_f16(e[0], e[1]), pack_f16(e[2], e[3]), pack_f16(e[4], e[5]), pack_f16(e[6], e[7])};
    }
  s.l += sum;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 2 * N; ++e)
      s.acc[d] = mfma32<false>(read_v<D>(vp, d, e), p[e], s.acc[d]);
  if (nans) {
    // NaN codes among the tile's values were staged as zeros, so that they cannot reach rows that do not
    // see them; the rows that do are set here, from the cache
#pragma unroll 1
    for (int o = 0; o < kKeys<D>; ++o) {
      const int32_t at = slot_at(a, table_row, s.hi_max, j0 + o);
      if (at < 0) continue;
      const bool see = sees64(a, s.row, rq, j0 + o) & 1;
      const uint8_t* p8 = vbase + (int64_t)at * a.cache_ld + 4 * h;
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

struct Shared {
  char tiles[2][2][kTileBytes];  // [buffer][K, V^T]
  int32_t limits[kWaves][4];
  int32_t nans[2][kWaves];
  uint64_t scratch[kWaves + 2];
};

template <int D, bool BF16, bool SPLIT>
__device__ __forceinline__ void segment(const AttnArgs& a, const Segment& sg, Shared& lds) {
  constexpr int BN = kKeys<D>;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const Request rq = request_of(a, sg.r);
  WaveState<D> s;
  float c = a.scale * *a.ks * kLog2e;
  // a negative factor goes into the query, so that the largest raw product is the largest score
  const uint32_t flip = c < 0.0f ? 0x80008000u : 0u;
  c = __builtin_fabsf(c);
  const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
  const uint32_t my_row = (uint32_t)(sg.tile * kRows + 32 * wave + r);
  s.row = row_of(a, sg.r, rq, sg.kv_head, my_row);
  s.m = kNoScore;
  s.l = 0.0f;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) s.acc[d][i] = 0.0f;
  const uint16_t* qp = a.q + (int64_t)s.row.token * a.q_ts + (int64_t)s.row.head * a.q_hs + 8 * h;
#pragma unroll
  for (int e = 0; e < D / 16; ++e) {
    s.q[e] = u32x4{0, 0, 0, 0};
    if (s.row.token >= 0) s.q[e] = *reinterpret_cast<const u32x4*>(qp + 16 * e) ^ flip;
  }
  int32_t lo_min = 0x7FFFFFFF, hi_max = 0, lo_all = 0, hi_all = 0x7FFFFFFF;
  if (s.row.token >= 0) {
    lo_min = lo_all = s.row.lo;
    hi_max = a.tree ? rq.len : s.row.hi;
    hi_all = s.row.hi;
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    lo_min = min(lo_min, __shfl_xor(lo_min, d));
    hi_max = max(hi_max, __shfl_xor(hi_max, d));
    lo_all = max(lo_all, __shfl_xor(lo_all, d));
    hi_all = min(hi_all, __shfl_xor(hi_all, d));
  }
  s.lo_min = __builtin_amdgcn_readfirstlane(lo_min);
  s.hi_max = min(__builtin_amdgcn_readfirstlane(hi_max), rq.len);
  s.lo_all = __builtin_amdgcn_readfirstlane(lo_all);
  s.hi_all = __builtin_amdgcn_readfirstlane(hi_all);
  if (lane == 0) {
    lds.limits[wave][0] = s.lo_min;
    lds.limits[wave][1] = s.hi_max;
  }
  __syncthreads();
  lo_min = 0x7FFFFFFF;
  hi_max = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    lo_min = min(lo_min, lds.limits[w][0]);
    hi_max = max(hi_max, lds.limits[w][1]);
  }
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
  const uint8_t* kbase = a.kc + (int64_t)sg.kv_head * D;
  const uint8_t* vbase = a.vc + (int64_t)sg.kv_head * D;
  if (t0 < t1) {
    Fetched f;
    There cur, nxt;
    Slots<D> sl = look_up<D>(a, table_row, hi_max, t0 * BN, lane);
    fetch<D>(a, sl, kbase, vbase, tid, f, cur);
    sl = look_up<D>(a, table_row, hi_max, (t0 + 1) * BN, lane);
    const bool bad = stage<D, BF16>(f, cur, lds.tiles[0][0], lds.tiles[0][1], tid);
    if (lane == 0) lds.nans[0][wave] = bad;
    fetch<D>(a, sl, kbase, vbase, tid, f, nxt);
    sl = look_up<D>(a, table_row, hi_max, (t0 + 2) * BN, lane);
    lds_barrier();
    for (int32_t t = t0; t < t1; ++t) {
      const int b = (t - t0) & 1;
      There after = nxt;
      if (t + 1 < t1) {
        const bool bad2 = stage<D, BF16>(f, nxt, lds.tiles[b ^ 1][0], lds.tiles[b ^ 1][1], tid);
        if (lane == 0) lds.nans[b ^ 1][wave] = bad2;
        // positions past the last tile have no slot; they read slot 0 and are not used
        fetch<D>(a, sl, kbase, vbase, tid, f, after);
        sl = look_up<D>(a, table_row, hi_max, (t + 3) * BN, lane);
      }
      const int32_t j0 = t * BN;
      if (j0 < s.hi_max && j0 + BN > s.lo_min) {
        int32_t nans = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) nans |= lds.nans[b][w];
        multiply<D, BF16>(a, rq, lds.tiles[b][0], lds.tiles[b][1], cur, __builtin_amdgcn_readfirstlane(nans) != 0, table_row, vbase, j0, c, inv_cap, lane, s);
      }
      cur = nxt;
      nxt = after;
      lds_barrier();
    }
  }

  const float l = s.l + __shfl_xor(s.l, 32);
  if (s.row.token >= 0) {
    if (SPLIT && !(sg.first && sg.last)) {
      const int64_t at = part_slot(blockIdx.x, sg.first) * kRows + 32 * wave + r;
      float* op = a.part + at * D + 4 * h;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4*>(op + 32 * d + 8 * j) = f32x4{s.acc[d][4 * j], s.acc[d][4 * j + 1], s.acc[d][4 * j + 2], s.acc[d][4 * j + 3]};
      if (h == 0) *reinterpret_cast<f32x2*>(a.part_ml + 2 * at) = f32x2{s.m, l};
    } else {
      const float inv = l == 0.0f ? 0.0f : *a.vs / l;
      uint16_t* op = a.out + (int64_t)s.row.token * a.out_ts + (int64_t)s.row.head * a.out_hs + 4 * h;
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

// SPLIT: the workgroups share the items' keys; else each takes whole items.
template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kThreads) attention_tiled_kernel(AttnArgs a) {
  __shared__ __align__(16) Shared lds;
  if constexpr (!SPLIT) {
    Segment s;
    s.kv_head = blockIdx.x;
    s.r = blockIdx.y;
    s.first = s.last = true;
    s.last_worker = 0;
    const Request q = request_of(a, s.r);
    s.u0 = 0;
    s.u1 = (q.len + kKeys<D> - 1) / kKeys<D>;
    const int32_t tiles = (int32_t)(((uint32_t)q.count * a.group.d + kRows - 1) / kRows);
    // the last row tiles see the most keys: they start first
    for (int32_t k = blockIdx.z; k < tiles; k += gridDim.z) {
      s.tile = tiles - 1 - k;
      segment<D, BF16, false>(a, s, lds);
    }
  } else {
    Share<kThreads> share;
    share.begin(a, kRows, kKeys<D>, lds.scratch);
    Segment s;
    Header hd{0, 0, 0, -1};
    while (share.next(a, s)) {
      if (s.first && !s.last) hd = Header{s.r, s.tile, s.kv_head, s.last_worker};
      segment<D, BF16, true>(a, s, lds);
    }
    if (threadIdx.x == 0) *reinterpret_cast<Header*>(a.headers + 4 * blockIdx.x) = hd;
  }
}

template <int D, bool BF16>
void launch(const AttnArgs& a, hipStream_t stream) {
  if (a.workers) {
    hipLaunchKernelGGL((attention_tiled_kernel<D, BF16, true>), dim3((uint32_t)a.workers), dim3(kThreads), 0, stream, a);
  } else {
    const dim3 grid((uint32_t)a.kv_heads, (uint32_t)a.requests, (uint32_t)a.row_tiles);
    hipLaunchKernelGGL((attention_tiled_kernel<D, BF16, false>), grid, dim3(kThreads), 0, stream, a);
  }
}

template <int D>
void launch(const AttnArgs& a, bool bf16, hipStream_t stream) {
  if (bf16)
    launch<D, true>(a, stream);
  else
    launch<D, false>(a, stream);
}

}  // namespace

hipError_t launch_attention_tiled(const AttnArgs& a, int head_dim, bool bf16, hipStream_t stream) {
  switch (head_dim) {
    case 64: launch<64>(a, bf16, stream); break;
    case 128: launch<128>(a, bf16, stream); break;
    default: launch<256>(a, bf16, stream); break;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
