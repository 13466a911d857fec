// Norm and position rotation of head vectors, and where they go: rows of the same type, the FP8 cache or the
// 4-bit cache (gfx950).
//
// A head vector is served by L lanes of one wavefront (L the power of two >= head_dim / 16), 16 elements a lane: the
// lane that holds elements i .. i + 7 of the first half of the pairs holds the same of the second half, so a rotation
// needs no other lane, and the norm one sum over L lanes.  Elements beyond the rotated ones, neighbouring pairs and
// values go 16 in a row.
//
// Everything between the input and the one rounding is binary64, which a matrix-free kernel has room for beside its
// memory traffic: a lane has about a dozen operations an element.  What it buys is that the rounding to the input's
// type is that of the exact value, so that what follows it, a code of 4 or 8 bits, does not depend on how a sum was
// ordered or a cosine approximated.  Cosines and sines are formed once a workgroup for its tokens, in LDS, and shared
// by all heads.
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

// The type's number nearest to x, as binary32.
template <nvfp4_dtype DT>
__device__ __forceinline__ float rounded(double x) {
  if constexpr (DT == NVFP4_F32) return (float)x;
  if constexpr (DT == NVFP4_BF16) return (float)(__bf16)cut(x);
  return (float)(_Float16)cut(x);
}

template <nvfp4_dtype DT>
__device__ __forceinline__ void load8(const uint8_t* p, float* v) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
  if constexpr (DT == NVFP4_F32) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(p + 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(w[i]);
      v[4 + i] = __uint_as_float(x[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == NVFP4_BF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const uint32_t word = w[i];  // (a bit cast of a vector's element takes its first)
        const f16x2 h = __builtin_bit_cast(f16x2, word);
        v[2 * i] = (float)h[0];
        v[2 * i + 1] = (float)h[1];
      }
    }
  }
}

// Numbers of the type, held as binary32: exact.
template <nvfp4_dtype DT>
__device__ __forceinline__ void store8(uint8_t* p, const float* v) {
  u32x4 w, x;
  if constexpr (DT == NVFP4_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = __float_as_uint(v[i]);
      x[i] = __float_as_uint(v[4 + i]);
    }
    *reinterpret_cast<u32x4*>(p + 16) = x;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == NVFP4_BF16)
        w[i] = __float_as_uint(v[2 * i]) >> 16 | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
      else
        w[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
    }
  }
  *reinterpret_cast<u32x4*>(p) = w;
}

__device__ __forceinline__ double weight_at(const uint8_t* w, int32_t dt, int i) {
  if (dt == NVFP4_F32) return reinterpret_cast<const float*>(w)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(w)[i];
  if (dt == NVFP4_BF16) return __uint_as_float((uint32_t)b << 16);
  return (float)__builtin_bit_cast(_Float16, b);
}

__device__ __forceinline__ float absmax8(const float* v) {
  float m = __builtin_fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// Slot of token t, or -1 where it is not stored.
__device__ __forceinline__ int64_t slot_of(const HeadArgs& a, int32_t t) {
  const int64_t s = a.slots ? a.slots[t] : (int64_t)t;
  return s >= 0 && s < a.num_slots ? s : -1;
}

// grid: x over groups of block_tokens tokens, y over stretches of their head vectors.
template <nvfp4_dtype DT, HeadSink SINK, bool PAIRS>
__global__ void __launch_bounds__(kThreads) heads_kernel(HeadArgs a, int lane_bits) {
  extern __shared__ __align__(16) char lds[];
  const int lanes = a.head_dim / 16;   // that hold elements of a head vector
  const int turning = a.num_freq / 8;  // of them, those with pairs
  f64x2* turns = reinterpret_cast<f64x2*>(lds);                                // [token][8][turning]
  double* weights = reinterpret_cast<double*>(turns + a.block_tokens * a.num_freq);  // [group][16][lanes]
  const int tid = threadIdx.x;
  // chunks of 8 elements that lane j holds
  const auto chunk = [&](int j, int half, bool turned) {
    if (!PAIRS && turned && j < turning) return j + half * turning;
    return 2 * j + half;
  };
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (!a.group[g].weight) continue;
    for (int i = tid; i < a.head_dim; i += kThreads) {
      const int j = i >> 4, k = i & 15;
      weights[(g * 16 + k) * lanes + j] = a.offset + weight_at(a.group[g].weight, a.weight_dtype, 8 * chunk(j, k >> 3, a.group[g].turned) + (k & 7));
    }
  }
  constexpr int kEb = DT == NVFP4_F32 ? 4 : 2;
  const int j = tid & ((1 << lane_bits) - 1);
  for (int64_t b0 = (int64_t)blockIdx.x * a.block_tokens; b0 < a.tokens; b0 += (int64_t)gridDim.x * a.block_tokens) {
    const int32_t t0 = (int32_t)b0, count = min(a.block_tokens, a.tokens - t0);
    for (int i = tid; i < count * a.num_freq; i += kThreads) {
      const int t = i / a.num_freq, f = i - t * a.num_freq;
      turns[(t * 8 + (f & 7)) * turning + (f >> 3)] = cos_sin(a.positions[t0 + t], a.inv_freq[f]);
    }
    __syncthreads();
    const uint32_t rows = (uint32_t)count * a.all_heads.d, step = (kThreads * gridDim.y) >> lane_bits;
    for (uint32_t row = (blockIdx.y * kThreads + tid) >> lane_bits; row < rows; row += step) {
      const uint32_t tl = div_of(row, a.all_heads);
      int32_t head = (int32_t)(row - tl * a.all_heads.d);
      const int32_t t = t0 + (int32_t)tl;
      const bool second = head >= a.group[0].heads;
      const HeadGroup& g = second ? a.group[1] : a.group[0];
      if (second) head -= a.group[0].heads;
      const bool there = j < lanes, turned = g.turned && j < turning;
      const int c0 = chunk(j, 0, g.turned), c1 = chunk(j, 1, g.turned);
      const int64_t slot = SINK == HeadSink::Same ? 0 : slot_of(a, t);
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
      if (there) {
        const uint8_t* p = g.src + (int64_t)t * g.ts + (int64_t)head * g.hs;
        load8<DT>(p + c0 * 8 * kEb, v);
        load8<DT>(p + c1 * 8 * kEb, v + 8);
      }
      if (g.weight || turned) {
        double x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = v[i];
        if (g.weight) {
          double sum = 0.0;
#pragma unroll
          for (int i = 0; i < 16; ++i) sum = __builtin_fma(x[i], x[i], sum);
          for (int d = 1; d < 1 << lane_bits; d <<= 1) sum += __shfl_xor(sum, d);
          const double by = 1.0 / __builtin_sqrt(sum / a.head_dim + a.eps);
          if (there) {
            const double* w = weights + (second ? 16 : 0) * lanes + j;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= by * w[i * lanes];
          }
        }
        if (turned) {
          const f64x2* at = turns + tl * 8 * turning + j;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const f64x2 cs = at[k * turning];
            const int ia = PAIRS ? 2 * k : k, ib = PAIRS ? 2 * k + 1 : 8 + k;
            const double xa = x[ia], xb = x[ib];
            x[ia] = __builtin_fma(-xb, cs.y, xa * cs.x);
            x[ib] = __builtin_fma(xa, cs.y, xb * cs.x);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = rounded<DT>(x[i]);
      }
      if constexpr (SINK == HeadSink::Same) {
        if (there) {
          uint8_t* o = g.out + (int64_t)t * g.out_ts + (int64_t)head * g.out_hs;
          store8<DT>(o + c0 * 8 * kEb, v);
          store8<DT>(o + c1 * 8 * kEb, v + 8);
        }
      } else if constexpr (SINK == HeadSink::Fp8) {
        const float inv = 1.0f / *g.scale;  // correctly rounded, as in the store without rotation
        if (there && slot >= 0) {
          uint8_t* o = g.cache + slot * a.cache_ld + head * a.head_dim;
          *reinterpret_cast<u32x2*>(o + c0 * 8) = u32x2{e4m3_pack4(v, inv), e4m3_pack4(v + 4, inv)};
          *reinterpret_cast<u32x2*>(o + c1 * 8) = u32x2{e4m3_pack4(v + 8, inv), e4m3_pack4(v + 12, inv)};
        }
      } else {
        // A block of 16 is two neighbouring chunks: this lane's own, or (the first half of the pairs in one block, the
        // second in another) the same ones of this lane and its neighbour.
        const bool across = !PAIRS && turned;
        float m0 = absmax8(v), m1 = absmax8(v + 8);
        const float n0 = __shfl_xor(m0, 1), n1 = __shfl_xor(m1, 1);
        if (across) {
          m0 = fmaxf(m0, n0);
          m1 = fmaxf(m1, n1);
        } else {
          m0 = m1 = fmaxf(m0, m1);
        }
        const float gs = *g.scale, gs6 = gs * (1.0f / 6.0f);
        const uint32_t s0 = e4m3_encode(m0 * gs6), s1 = e4m3_encode(m1 * gs6);
        const float d0 = e4m3_value(s0), d1 = e4m3_value(s1);
        const float r0 = d0 > 0.0f ? gs / d0 : 0.0f, r1 = d1 > 0.0f ? gs / d1 : 0.0f;
        const uint32_t w0 = r0 < __builtin_inff() ? e2m1_pack8(v, r0) : e2m1_pack8_wide(v, r0);
        const uint32_t w1 = r1 < __builtin_inff() ? e2m1_pack8(v + 8, r1) : e2m1_pack8_wide(v + 8, r1);
        if (there && slot >= 0) {
          const uint32_t block = div_of((uint32_t)slot, a.bs);
          const int64_t at = (int64_t)(block * (uint32_t)g.heads + (uint32_t)head) * a.bs.d + ((uint32_t)slot - block * a.bs.d);
          uint8_t* o = g.cache + at * (a.head_dim / 2);
          uint8_t* os = g.cache_scales + at * lanes;
          *reinterpret_cast<uint32_t*>(o + 4 * c0) = w0;
          *reinterpret_cast<uint32_t*>(o + 4 * c1) = w1;
          const bool odd = across && (j & 1);
          os[(odd ? c1 : c0) >> 1] = (uint8_t)(odd ? s1 : s0);
        }
      }
    }
    __syncthreads();  // the cosines are written again
  }
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

// A lane decodes 8 elements of one row.
template <bool BF16_OUT>
__global__ void __launch_bounds__(kThreads) fp4_load_kernel(Fp4LoadArgs a) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.pieces; i += (int64_t)gridDim.x * kThreads) {
    const int per_head = a.head_dim / 8;
    const int64_t token_head = i / per_head;
    const int c = (int)(i - token_head * per_head);
    const int64_t t = token_head / a.kv_heads;
    const uint32_t head = (uint32_t)(token_head - t * a.kv_heads);
    const int64_t s = a.slots ? a.slots[t] : t;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    if (s >= 0 && s < a.num_slots) {
      const uint32_t block = div_of((uint32_t)s, a.bs);
      const int64_t row = (int64_t)(block * (uint32_t)a.kv_heads + head) * a.bs.d + ((uint32_t)s - block * a.bs.d);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(a.codes + row * (a.head_dim / 2) + 4 * c);
      const float sd = e4m3_value(a.scales[row * (a.head_dim / 16) + c / 2] & 0x7Fu), g = *a.g;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float m = e2m1_value(w >> (4 * k) & 7u) * sd / g;
        v[k] = __uint_as_float(__float_as_uint(m) | (w >> (4 * k + 3) & 1u) << 31);
      }
    }
    if constexpr (BF16_OUT) {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * k], (__bf16)v[2 * k + 1]});
      *reinterpret_cast<u32x4*>(a.out + i * 16) = o;
    } else {
      store8<NVFP4_F32>(a.out + i * 32, v);
    }
  }
}

}  // namespace

hipError_t launch_heads(HeadArgs a, nvfp4_dtype dt, HeadSink sink, hipStream_t stream) {
  int lane_bits = 0;
  while (16 << lane_bits < a.head_dim) ++lane_bits;
  const int heads = a.group[0].heads + a.group[1].heads;
  const int64_t tasks = (int64_t)heads << lane_bits;  // lanes that a token takes
  // a workgroup takes as many tokens as give each thread four head vectors, but no more than leave two workgroups for
  // each compute unit, nor than 32 KB of cosines
  int64_t block = (4 * kThreads + tasks - 1) / tasks;
  const int64_t spread = (a.tokens + 2 * kComputeUnits - 1) / (2 * kComputeUnits);
  if (block > spread) block = spread;
  if (a.num_freq && block > 2048 / a.num_freq) block = 2048 / a.num_freq;
  if (block < 1) block = 1;
  a.block_tokens = (int32_t)block;
  a.all_heads = make_fast_div((uint32_t)heads);
  const int64_t x = (a.tokens + block - 1) / block;
  // few tokens: their heads are shared out
  int64_t y = (block * tasks + kThreads - 1) / kThreads;
  const int64_t room = (2 * kComputeUnits + x - 1) / x;
  if (y > room) y = room;
  const bool weights = a.group[0].weight || a.group[1].weight;
  const size_t lds = (size_t)block * a.num_freq * 16 + (weights ? (size_t)a.head_dim * 16 : 0);
  // (a grid has fewer than 2^32 threads; the kernel's stride covers the others)
  const dim3 grid((uint32_t)(x < kMaxBlocks ? x : kMaxBlocks), (uint32_t)y);
  switch (dt) {
    case NVFP4_F32: launch<NVFP4_F32>(a, sink, lane_bits, grid, lds, stream); break;
    case NVFP4_BF16: launch<NVFP4_BF16>(a, sink, lane_bits, grid, lds, stream); break;
    default: launch<NVFP4_F16>(a, sink, lane_bits, grid, lds, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_fp4_load(const Fp4LoadArgs& a, bool bf16_out, int64_t tokens, hipStream_t stream) {
  Fp4LoadArgs b = a;
  b.pieces = tokens * a.kv_heads * (a.head_dim / 8);
  const int64_t x = (b.pieces + kThreads - 1) / kThreads;
  const dim3 grid((uint32_t)(x < kMaxBlocks ? x : kMaxBlocks));
  if (bf16_out)
    hipLaunchKernelGGL(fp4_load_kernel<true>, grid, dim3(kThreads), 0, stream, b);
  else
    hipLaunchKernelGGL(fp4_load_kernel<false>, grid, dim3(kThreads), 0, stream, b);
  return hipGetLastError();
}

}  // namespace nvfp4
