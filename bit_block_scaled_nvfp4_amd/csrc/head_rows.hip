// Norm and position rotation of head vectors, and where they go: rows of the same type, the FP8 cache or the
// 4-bit cache (gfx950).
//
// A head vector is served by L lanes of one wavefront (L the power of two >= head_dim / 16), two chunks of 8 elements a
// lane: the lane that holds elements i .. i + 7 of the first half of the pairs holds the same of the second half, so a
// rotation needs no other lane, and the norm one sum over L lanes.  The other chunks, those of neighbouring pairs and
// those of values are halved in the same way, so that lanes next to each other always read and write chunks next to each
// other, and a block of 16 elements lies in a lane and its neighbour.
//
// Everything between the input and the one rounding is binary64.  What it buys is that the rounding to the input's
// type is that of the exact value, so that what follows it, a code of 4 or 8 bits, does not depend on how a sum was
// ordered or a cosine approximated.  Cosines and sines are formed once a workgroup for its tokens, in LDS, and shared
// by all heads.  The next row is requested before the present one is worked on.
//
// What bounds it: HBM reads and writes, and beside them the binary64 instructions.  Measured (copies at 4.9 TB/s): 8192
// tokens of 24 and 4 heads of 256 dims with norms, a quarter rotated, 235 MB: 45 us, 5.2 TB/s; 3001 of 32 and 8 heads of
// 128 dims in FP16, all rotated, 61 MB: 14.6 us.  16384 tokens of 4 heads of 256 dims into the 4-bit cache, 86 MB: 26 us, 17 of
// them issue of vector instructions; 2047 of 8 heads of 128 dims into the FP8 cache, 13 MB: 7.3 us.  One
// token: 4.2 us.
#include "codec.h"
#include "serving_internal.h"

namespace nvfp4 {
namespace {

using namespace codec;

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 20;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef double f64x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t div_of(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.mul) >> f.shift);
}

// cos and sin of position * frequency, to about 2^-51 below 2^31: the product (31 and 24 bits) in two numbers, less the
// nearest multiple of pi / 2, which is taken off in two pieces of 53 bits, then Taylor's series up to the first term
// below 2^-55 on [-pi / 4, pi / 4].
__device__ __forceinline__ f64x2 cos_sin(double position, double frequency) {
  constexpr double kHigh = 0x1.921fb54442d18p0, kLow = 0x1.1a62633145c07p-54;  // pi / 2
  const double x = position * frequency, rest = __builtin_fma(position, frequency, -x);
  const double k = __builtin_rint(x * 0.63661977236758134308);  // 2 / pi
  const double r = __builtin_fma(-k, kHigh, x) + __builtin_fma(-k, kLow, rest);
  const double z = r * r;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;  // 1 / 15!, 1 / 16!
  s = __builtin_fma(s, z, 1.0 / 6227020800.0);
  c = __builtin_fma(c, z, -1.0 / 87178291200.0);
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  s = __builtin_fma(s * z, r, r);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  // the quadrant, k mod 4
  const int q = (int)(k - 4.0 * __builtin_floor(k * 0.25));
  const double cq = q & 1 ? s : c, sq = q & 1 ? c : s;
  return f64x2{(q + 1) & 2 ? -cq : cq, q & 2 ? -sq : sq};
}

// x cut to binary32 with the last bit set where anything is lost: rounding that to fewer bits gives what rounding x
// itself would (rounding twice to nearest does not).
__device__ __forceinline__ float cut(double x) {
  const float f = (float)x;
  const double back = (double)f;
  uint32_t u = __float_as_uint(f);
  u -= __builtin_fabs(back) > __builtin_fabs(x) ? 1u : 0u;
  u |= back != x ? 1u : 0u;
  return __uint_as_float(u);
}

// Whether rounding f, itself rounded from binary64, to DT may differ from rounding once: f lies in the middle between
// two of DT's numbers.  (FP16's subnormal numbers lie further apart: there every f with 12 zeros at its end.)
template <nvfp4_dtype DT>
__device__ __forceinline__ bool in_the_middle(float f) {
  const uint32_t u = __float_as_uint(f);
  if constexpr (DT == NVFP4_BF16) return (uint16_t)u == 0x8000u;
  if constexpr (DT == NVFP4_F16) return (u & 0x0FFFu) == 0 && ((u & 0x1000u) || __builtin_fabsf(f) < 0x1p-14f);
  return false;
}

// Two numbers of a 16-bit type, the first one low.
template <nvfp4_dtype DT>
__device__ __forceinline__ uint32_t two(float f, float g) {
  if constexpr (DT == NVFP4_BF16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f, (__bf16)g});
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)f, (_Float16)g});
}

// Two chunks of 8 elements as they lie in memory.
template <nvfp4_dtype DT>
struct Raw {
  u32x4 w[DT == NVFP4_F32 ? 4 : 2];
};

// x rounded once to DT: by way of binary32 where that is the same (all but one element in 2^16, or 2^13 of FP16).
template <nvfp4_dtype DT>
__device__ __forceinline__ void round16(const double (&x)[16], Raw<DT>& r) {
  float v[16];
  bool middle = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = (float)x[i];
    middle |= in_the_middle<DT>(v[i]);
  }
  if (DT != NVFP4_F32 && __builtin_expect(__any(middle), 0)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = cut(x[i]);
  }
  if constexpr (DT == NVFP4_F32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) r.w[i >> 2][i & 3] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i >> 2][i & 3] = two<DT>(v[2 * i], v[2 * i + 1]);
  }
}

// x of the lane that a DPP control names.
template <int CONTROL>
__device__ __forceinline__ float from_lane(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), CONTROL, 0xF, 0xF, true));
}

template <int CONTROL>
__device__ __forceinline__ double from_lane(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CONTROL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CONTROL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

constexpr int kNeighbour = 0xB1, kOtherPair = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

// Sum over groups of 2^bits lanes (32 at most), the same in all of a group.  What is summed so far is the same in the
// lanes that a mirror exchanges.
__device__ __forceinline__ double sum_over(double x, int bits) {
  if (bits > 0) x += from_lane<kNeighbour>(x);
  if (bits > 1) x += from_lane<kOtherPair>(x);
  if (bits > 2) x += from_lane<kMirror8>(x);
  if (bits > 3) x += from_lane<kMirror16>(x);
  if (bits > 4) x += __shfl_xor(x, 16);
  return x;
}

// 1 / sqrt(x), to about 2^-52: the instruction's value and two steps of Newton's method.
__device__ __forceinline__ double inverse_root(double x) {
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(y * 0.5, __builtin_fma(-x * y, y, 1.0), y);
  return y;
}

template <nvfp4_dtype DT>
__device__ __forceinline__ void load_raw(const uint8_t* p, int c0, int c1, Raw<DT>& r) {
  if constexpr (DT == NVFP4_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r.w[i] = *(reinterpret_cast<const u32x4*>(p + c0 * 32) + i);
      r.w[2 + i] = *(reinterpret_cast<const u32x4*>(p + c1 * 32) + i);
    }
  } else {
    r.w[0] = *(reinterpret_cast<const u32x4*>(p + c0 * 16));
    r.w[1] = *(reinterpret_cast<const u32x4*>(p + c1 * 16));
  }
}

template <nvfp4_dtype DT>
__device__ __forceinline__ void widen(const Raw<DT>& r, float (&v)[16]) {
  if constexpr (DT == NVFP4_F32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i >> 2][i & 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t word = r.w[i >> 2][i & 3];  // (a bit cast of a vector's element takes its first)
      if constexpr (DT == NVFP4_BF16) {
        v[2 * i] = __uint_as_float(word << 16);
        v[2 * i + 1] = __uint_as_float(word & 0xFFFF0000u);
      } else {
        const f16x2 h = __builtin_bit_cast(f16x2, word);
        v[2 * i] = (float)h[0];
        v[2 * i + 1] = (float)h[1];
      }
    }
  }
}

template <nvfp4_dtype DT>
__device__ __forceinline__ void store_raw(uint8_t* p, int c0, int c1, const Raw<DT>& r) {
  if constexpr (DT == NVFP4_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      __builtin_nontemporal_store(r.w[i], reinterpret_cast<u32x4*>(p + c0 * 32) + i);
      __builtin_nontemporal_store(r.w[2 + i], reinterpret_cast<u32x4*>(p + c1 * 32) + i);
    }
  } else {
    __builtin_nontemporal_store(r.w[0], reinterpret_cast<u32x4*>(p + c0 * 16));
    __builtin_nontemporal_store(r.w[1], reinterpret_cast<u32x4*>(p + c1 * 16));
  }
}

// An element of a weight as it lies in memory, and its value.
__device__ __forceinline__ uint32_t weight_bits(const uint8_t* w, int32_t dt, int i) {
  return dt == NVFP4_F32 ? reinterpret_cast<const uint32_t*>(w)[i] : reinterpret_cast<const uint16_t*>(w)[i];
}

__device__ __forceinline__ double weight_of(uint32_t bits, int32_t dt) {
  if (dt == NVFP4_F32) return __uint_as_float(bits);
  if (dt == NVFP4_BF16) return __uint_as_float(bits << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

__device__ __forceinline__ float absmax8(const float* v) {
  float m = __builtin_fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// grid: z and x over groups of block_tokens tokens, y over stretches of their head vectors.
template <nvfp4_dtype DT, HeadSink SINK, bool PAIRS>
__global__ void __launch_bounds__(kThreads) heads_kernel(HeadArgs a, int lane_bits) {
  extern __shared__ __align__(16) char lds[];
  const int lanes = a.head_dim / 16;  // that hold elements of a head vector
  const int turning = a.num_freq / 8;  // of them, those with pairs whose halves are apart
  const int tid = threadIdx.x, j = tid & ((1 << lane_bits) - 1);
  const bool there = j < lanes;
  // chunk of 8 elements that lane i holds: the halves of the pairs, and the halves of the rest
  const auto chunk = [&](int i, int half, bool turned) {
    if (PAIRS || !turned) return i + half * lanes;
    return i < turning ? i + half * turning : turning + i + half * (lanes - turning);
  };
  const int64_t b0 = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * a.block_tokens;
  if (b0 >= a.tokens) return;
  const int32_t t0 = (int32_t)b0;
  const uint32_t count = min(a.block_tokens, a.tokens - t0);
  const uint32_t step = (kThreads * gridDim.y) >> lane_bits, wave_rows = 64u >> lane_bits;
  // the second kind's rows go on with the wavefront behind the one that the first kind's end with
  const uint32_t first = (blockIdx.y * kThreads + tid) >> lane_bits, used = (count * a.group[0].heads.d + wave_rows - 1) & ~(wave_rows - 1);
  const uint32_t shifted = first + step - used % step, second = shifted < step ? shifted : shifted - step;
  const auto request = [&](const HeadGroup& g, uint32_t row, Raw<DT>& r, int64_t& slot) {
    if (row >= count * g.heads.d) return;
    const uint32_t token = div_of(row, g.heads), head = row - token * g.heads.d;
    if (SINK != HeadSink::Same) slot = a.slots ? a.slots[t0 + token] : (int64_t)(t0 + token);  // looked at a turn later
    const uint8_t* src = g.src + t0 * (int64_t)g.ts;
    if (there) load_raw<DT>(src + (uint64_t)token * g.ts + (uint64_t)head * g.hs, chunk(j, 0, g.turned), chunk(j, 1, g.turned), r);
  };
  Raw<DT> raw[2] = {}, ahead{};
  int64_t slot[2] = {-1, -1}, slot_ahead = -1;
  request(a.group[0], first, raw[0], slot[0]);
  request(a.group[1], second, raw[1], slot[1]);

  // [token][8][turning], or neighbouring pairs: [token][4][2 turning], the second number counting chunks
  f64x2* turns = reinterpret_cast<f64x2*>(lds);
  double* weights = reinterpret_cast<double*>(turns + a.block_tokens * a.num_freq);  // [group][16][lanes]
  constexpr int kOfChunk = PAIRS ? 4 : 8;  // pairs that a chunk begins
  const int chunks = a.num_freq / kOfChunk, all = (int)count * a.num_freq;
  // what the first turns of both loops take is requested ahead of the cosines: none of these loads waits for another
  const auto element = [&](int g, int i) { return 8 * chunk(i >> 4, (i >> 3) & 1, a.group[g].turned) + (i & 7); };
  uint32_t bits[2] = {0, 0};
#pragma unroll
  for (int g = 0; g < 2; ++g)
    if (a.group[g].weight && tid < a.head_dim) bits[g] = weight_bits(a.group[g].weight, a.weight_dtype, element(g, tid));
  int i = tid, t = i < all ? i / a.num_freq : 0, f = i - t * a.num_freq;
  int32_t position = i < all ? a.positions[t0 + t] : 0;
  float frequency = i < all ? a.inv_freq[f] : 0.0f;
  while (i < all) {
    turns[(t * kOfChunk + f % kOfChunk) * chunks + f / kOfChunk] = cos_sin(position, frequency);
    i += kThreads;
    if (i >= all) break;
    t = i / a.num_freq;
    f = i - t * a.num_freq;
    position = a.positions[t0 + t];
    frequency = a.inv_freq[f];
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (!a.group[g].weight) continue;
    for (int i = tid; i < a.head_dim; i += kThreads) {
      if (i != tid) bits[g] = weight_bits(a.group[g].weight, a.weight_dtype, element(g, i));
      weights[(g * 16 + (i & 15)) * lanes + (i >> 4)] = a.offset + weight_of(bits[g], a.weight_dtype);
    }
  }
  __syncthreads();
  // one kind of vectors after the other (not one loop over both: what a kind's loop needs of the arguments stays in
  // scalar registers)
  const auto rows_of = [&](const HeadGroup& g, int kind, uint32_t row, Raw<DT> raw, int64_t slot) {
    // (loaded here: a load in the loop would be waited for together with the next row)
    const float scale = SINK == HeadSink::Same ? 0.0f : *g.scale;
    const float inv = SINK == HeadSink::Fp8 ? 1.0f / scale : 0.0f;  // correctly rounded, as in the store without rotation
    for (; row < count * g.heads.d; row += step) {
      request(g, row + step, ahead, slot_ahead);
      const uint32_t token = div_of(row, g.heads), head = row - token * g.heads.d;
      const int c0 = chunk(j, 0, g.turned), c1 = chunk(j, 1, g.turned);
      const bool turned = g.turned && there && (PAIRS ? c0 < chunks : j < turning);  // (PAIRS: the second chunk is asked below)
      if (g.weight || turned) {
        float v[16];
        widen<DT>(raw, v);
        double x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = v[i];
        if (g.weight) {
          double sum = 0.0, more = 0.0;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            sum = __builtin_fma(x[i], x[i], sum);
            more = __builtin_fma(x[i + 1], x[i + 1], more);
          }
          sum += more;
          sum = sum_over(sum, lane_bits);
          const double by = inverse_root(__builtin_fma(sum, a.per_dim, a.eps));
          const double* w = weights + (kind * 16) * lanes + (there ? j : 0);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= by * w[i * lanes];
        }
        if (turned) {
          if constexpr (PAIRS) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = h ? c1 : c0;
              if (c >= chunks) continue;
              const f64x2* at = turns + token * 4 * chunks + c;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const f64x2 cs = at[k * chunks];
                const double xa = x[8 * h + 2 * k], xb = x[8 * h + 2 * k + 1];
                x[8 * h + 2 * k] = __builtin_fma(-xb, cs.y, xa * cs.x);
                x[8 * h + 2 * k + 1] = __builtin_fma(xa, cs.y, xb * cs.x);
              }
            }
          } else {
            const f64x2* at = turns + token * 8 * turning + j;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const f64x2 cs = at[k * turning];
              const double xa = x[k], xb = x[8 + k];
              x[k] = __builtin_fma(-xb, cs.y, xa * cs.x);
              x[8 + k] = __builtin_fma(xa, cs.y, xb * cs.x);
            }
          }
        }
        round16<DT>(x, raw);
      }
      if constexpr (SINK == HeadSink::Same) {
        if (there) {
          uint8_t* out = g.out + t0 * (int64_t)g.out_ts;
          store_raw<DT>(out + (uint64_t)token * g.out_ts + (uint64_t)head * g.out_hs, c0, c1, raw);
        }
      } else if constexpr (SINK == HeadSink::Fp8) {
        float v[16];
        widen<DT>(raw, v);
        if (there && slot >= 0 && slot < a.num_slots) {
          uint8_t* o = g.cache + slot * a.cache_ld + head * (uint32_t)a.head_dim;
          *reinterpret_cast<u32x2*>(o + c0 * 8) = u32x2{e4m3_pack4(v, inv), e4m3_pack4(v + 4, inv)};
          *reinterpret_cast<u32x2*>(o + c1 * 8) = u32x2{e4m3_pack4(v + 8, inv), e4m3_pack4(v + 12, inv)};
        }
      } else {
        // a block of 16 is the same chunk of this lane and its neighbour (lanes and, where it counts, turning are even):
        // the even one forms the first block's scale, the odd one the second's
        float v[16];
        widen<DT>(raw, v);
        float m0 = absmax8(v), m1 = absmax8(v + 8);
        m0 = fmaxf(m0, from_lane<kNeighbour>(m0));
        m1 = fmaxf(m1, from_lane<kNeighbour>(m1));
        // nearest even, subnormal codes kept: what e4m3_encode gives
        const float scaled = __builtin_fminf((j & 1 ? m1 : m0) * (scale * (1.0f / 6.0f)), 448.0f);
        const uint32_t sc = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(scaled, scaled, 0, false) & 0xFFu;
        const float sd = __builtin_amdgcn_cvt_f32_fp8((int)sc, 0);
        const float r = sd > 0.0f ? scale / sd : 0.0f, other = from_lane<kNeighbour>(r);
        const float r0 = j & 1 ? other : r, r1 = j & 1 ? r : other;
        uint32_t w0 = e2m1_pack8(v, r0), w1 = e2m1_pack8(v + 8, r1);
        if (__builtin_expect(__any(!(r < __builtin_inff())), 0)) {
          if (!(r0 < __builtin_inff())) w0 = e2m1_pack8_wide(v, r0);
          if (!(r1 < __builtin_inff())) w1 = e2m1_pack8_wide(v + 8, r1);
        }
        if (slot >= 0 && slot < a.num_slots) {
          const uint32_t block = div_of((uint32_t)slot, a.bs);
          const int64_t at = (int64_t)(block * g.heads.d + head) * a.bs.d + ((uint32_t)slot - block * a.bs.d);
          uint8_t* o = g.cache + at * (a.head_dim / 2);
          *reinterpret_cast<uint32_t*>(o + 4 * c0) = w0;
          *reinterpret_cast<uint32_t*>(o + 4 * c1) = w1;
          g.cache_scales[at * lanes + ((j & 1 ? c1 : c0) >> 1)] = (uint8_t)sc;
        }
      }
      raw = ahead;
      slot = slot_ahead;
    }
  };
  rows_of(a.group[0], 0, first, raw[0], slot[0]);
  if (a.group[1].src) rows_of(a.group[1], 1, second, raw[1], slot[1]);
}

template <nvfp4_dtype DT, HeadSink SINK>
void launch(const HeadArgs& a, int lane_bits, dim3 grid, size_t lds, hipStream_t stream) {
  if (a.interleaved)
    hipLaunchKernelGGL((heads_kernel<DT, SINK, true>), grid, dim3(kThreads), lds, stream, a, lane_bits);
  else
    hipLaunchKernelGGL((heads_kernel<DT, SINK, false>), grid, dim3(kThreads), lds, stream, a, lane_bits);
}

template <nvfp4_dtype DT>
void launch(const HeadArgs& a, HeadSink sink, int lane_bits, dim3 grid, size_t lds, hipStream_t stream) {
  switch (sink) {
    case HeadSink::Same: launch<DT, HeadSink::Same>(a, lane_bits, grid, lds, stream); break;
    case HeadSink::Fp8: launch<DT, HeadSink::Fp8>(a, lane_bits, grid, lds, stream); break;
    case HeadSink::Fp4: launch<DT, HeadSink::Fp4>(a, lane_bits, grid, lds, stream); break;
  }
}

// x / g, correctly rounded, from y = 1 / g (correctly rounded): a quotient within two units, and Markstein's step, which
// is exact from a quotient within one, twice.  For x = V * E4M3(scale) >= 2^-10 and g of [2^-100, 2^100]: nothing on the
// way leaves the normal numbers.
__device__ __forceinline__ float divided(float x, float g, float y) {
  float q = x * y;
  q = __builtin_fmaf(__builtin_fmaf(-q, g, x), y, q);
  q = __builtin_fmaf(__builtin_fmaf(-q, g, x), y, q);
  return __builtin_copysignf(q, x);  // a zero keeps its sign
}

// Bound by its writes: 16384 tokens of 4 heads of 256 dims to binary32, 77 MB, 15.2 us, 5.1 TB/s.
// A lane decodes 16 bytes of the result: 8 elements (BF16) or 4 of one head's row.  grid: x over groups of
// kThreads >> lane_bits tokens, y over stretches of 1 << lane_bits pieces of a token.
template <bool BF16_OUT>
__global__ void __launch_bounds__(kThreads) fp4_load_kernel(Fp4LoadArgs a, int lane_bits) {
  constexpr int E = BF16_OUT ? 8 : 4;
  const int32_t c = (int32_t)(blockIdx.y << lane_bits) + (int32_t)(threadIdx.x & ((1u << lane_bits) - 1));
  if (c >= a.pieces) return;
  const int shift = a.head_bits - (BF16_OUT ? 3 : 2);  // log2 of a head's pieces
  const uint32_t head = (uint32_t)c >> shift, at = (uint32_t)c & ((1u << shift) - 1);
  const float g = *a.g, y = 1.0f / g;
  const bool plain = g >= 0x1p-100f && g <= 0x1p100f;
  const int64_t step = (int64_t)gridDim.x * (kThreads >> lane_bits);
  for (int64_t t = (int64_t)blockIdx.x * (kThreads >> lane_bits) + (threadIdx.x >> lane_bits); t < a.tokens; t += step) {
    const int64_t s = a.slots ? a.slots[t] : t;
    float v[E];
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = 0.0f;
    if (s >= 0 && s < a.num_slots) {
      const uint32_t block = div_of((uint32_t)s, a.bs);
      const int64_t row = (int64_t)(block * (uint32_t)a.kv_heads + head) * a.bs.d + ((uint32_t)s - block * a.bs.d);
      const uint8_t* p = a.codes + (row << (a.head_bits - 1)) + at * (E / 2);
      const uint32_t w = BF16_OUT ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
      const float sd = e4m3_value(a.scales[(row << (a.head_bits - 4)) + at * E / 16] & 0x7Fu);
      const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
      v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
      if constexpr (BF16_OUT) {
        const auto lo2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), hi2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        v[4] = lo2[0]; v[5] = lo2[1]; v[6] = hi2[0]; v[7] = hi2[1];
      }
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] *= sd;  // exact
      if (plain) {
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = divided(v[k], g, y);
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] /= g;
      }
    }
    u32x4 o;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (BF16_OUT) o[k] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * k], (__bf16)v[2 * k + 1]});
      else o[k] = __float_as_uint(v[k]);
    }
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(a.out) + t * a.pieces + c);
  }
}

}  // namespace

hipError_t launch_heads(HeadArgs a, nvfp4_dtype dt, HeadSink sink, hipStream_t stream) {
  int lane_bits = 0;
  while (16 << lane_bits < a.head_dim) ++lane_bits;
  // lanes that a token takes, of each kind
  const int64_t tasks[2] = {(int64_t)a.group[0].heads.d << lane_bits, a.group[1].src ? (int64_t)a.group[1].heads.d << lane_bits : 0};
  // Tokens of a workgroup: what gives its lanes four turns, but no more than leave every compute unit two workgroups,
  // nor than 32 KB of cosines.  Fewer do not pay for a workgroup's start, more leave its end uneven.  Measured with calls back to
  // back in a graph, on inputs in turn (us): 8192 tokens of 28 heads of 256 dims, four turns at 2 tokens: 45 at 1, 41 at 2, 44 at 4,
  // 47 at 8; 16384 tokens of 4 heads of 256 dims into the 4-bit cache, four turns at 8: 32 at 2, 27 at 4, 24 at 8, 25 at 14, into the
  // FP8 cache 35, 31, 27, 31; of 8 heads of 128 dims into the FP8 cache, neighbouring pairs, four turns at 8: 16384 tokens 34, 30, 28,
  // 33, 8192 tokens 19, 17.5, 16.6, 19; 2047 tokens, where 4 are two workgroups a compute unit, 8.8 at 1, 7.2 at 2, 7.7 at 4, 7.9 at 8:
  // four workgroups a unit would be 6 % ahead there.
  int64_t block = 4 * kThreads / (tasks[0] + tasks[1]);
  const int64_t spread = (a.tokens + 2 * kComputeUnits - 1) / (2 * kComputeUnits);
  if (block > spread) block = spread;
  if (a.num_freq && block > 2048 / a.num_freq) block = 2048 / a.num_freq;
  if (block < 1) block = 1;
  a.block_tokens = (int32_t)block;
  a.per_dim = 1.0 / a.head_dim;
  const int64_t x = (a.tokens + block - 1) / block;
  // few tokens: their heads are shared out
  int64_t y = ((block * tasks[0] + 63) / 64 * 64 + block * tasks[1] + kThreads - 1) / kThreads;
  const int64_t room = (2 * kComputeUnits + x - 1) / x;
  if (y > room) y = room;
  const bool weights = a.group[0].weight || a.group[1].weight;
  const size_t lds = (size_t)block * a.num_freq * 16 + (weights ? (size_t)a.head_dim * 16 : 0);
  // (a dimension of a grid has fewer than 2^32 threads)
  const dim3 grid((uint32_t)(x < kMaxBlocks ? x : kMaxBlocks), (uint32_t)y, (uint32_t)((x + kMaxBlocks - 1) / kMaxBlocks));
  switch (dt) {
    case NVFP4_F32: launch<NVFP4_F32>(a, sink, lane_bits, grid, lds, stream); break;
    case NVFP4_BF16: launch<NVFP4_BF16>(a, sink, lane_bits, grid, lds, stream); break;
    default: launch<NVFP4_F16>(a, sink, lane_bits, grid, lds, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_fp4_load(Fp4LoadArgs a, bool bf16_out, hipStream_t stream) {
  a.pieces = a.kv_heads << (a.head_bits - (bf16_out ? 3 : 2));
  int lane_bits = 0;
  while (lane_bits < 8 && (1 << lane_bits) < a.pieces) ++lane_bits;
  const int64_t group = kThreads >> lane_bits, x = (a.tokens + group - 1) / group;
  const dim3 grid((uint32_t)(x < kMaxBlocks ? x : kMaxBlocks), (uint32_t)((a.pieces + (1 << lane_bits) - 1) >> lane_bits));
  if (bf16_out)
    hipLaunchKernelGGL(fp4_load_kernel<true>, grid, dim3(kThreads), 0, stream, a, lane_bits);
  else
    hipLaunchKernelGGL(fp4_load_kernel<false>, grid, dim3(kThreads), 0, stream, a, lane_bits);
  return hipGetLastError();
}

}  // namespace nvfp4
