// Verification of drafted tokens (gfx950): how many of a request's drafts the target accepts, and the token sampled
// behind them.
//
// What bounds it: HBM reads of two rows of the vocabulary a request (target and draft at the first token that was not
// accepted; where all were, the target's last row alone).  A row is cut into chunks of 4096 that workgroups of a first
// launch sum, each after finding the row by itself (64 drafts a look, one lane each: three dependent loads); a second
// launch, a workgroup a request, finds the chunk that the random number falls into, sums that chunk again element by
// element and writes the tokens.  Sums are binary64 in a fixed order: weights are differences of binary32 numbers, so
// two orders differ by about 2^-50 of the sum.
#include "serving_internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kEach = kVerifyChunk / kThreads;  // elements of a thread

struct Rows {
  int32_t start, last;  // first and last row of the request; last < start: none
};

__device__ __forceinline__ Rows rows_of(const VerifyArgs& a, int32_t r) {
  const int32_t s = min(max(a.query_start[r], 0), a.rows), e = min(max(a.query_start[r + 1], 0), a.rows);
  return Rows{s, max(e, s) - 1};
}

// First row of the request that goes no further: its drafted token is not accepted, or it is the last.  By every
// wavefront for itself.
__device__ __forceinline__ int32_t row_reached(const VerifyArgs& a, const Rows& q) {
  const int lane = threadIdx.x & 63;
  for (int32_t b = q.start; b < q.last; b += 64) {
    const int32_t t = b + lane;
    bool yes = false;
    if (t < q.last) {
      const int32_t x = a.tokens[t + 1];
      if (x >= 0 && x < a.vocab) {
        const double likely = a.q ? (double)a.q[(int64_t)t * a.q_ld + x] : 1.0;
        yes = (double)a.accept_u[t] * likely < (double)a.p[(int64_t)t * a.p_ld + x];
      }
    }
    const uint64_t not_yet = ~__ballot(yes);
    if (not_yet) return min(b + (int32_t)__builtin_ctzll(not_yet), q.last);
  }
  return q.last;
}

// Where a token's weight comes from.
struct Weights {
  const float* p;
  const float* q;   // or null
  int32_t without;  // a token that counts as 0 (a certain draft that was not accepted), or -1
};

__device__ __forceinline__ Weights weights_of(const VerifyArgs& a, const Rows& q, int32_t row) {
  const bool drafted = row < q.last;
  return Weights{a.p + (int64_t)row * a.p_ld, drafted && a.q ? a.q + (int64_t)row * a.q_ld : nullptr, drafted && !a.q ? a.tokens[row + 1] : -1};
}

__device__ __forceinline__ double positive(float x) { return x > 0.0f ? (double)x : 0.0; }

__device__ __forceinline__ double weight_at(const Weights& w, int32_t v, float p, float q) {
  if (w.q) return p > q ? (double)p - (double)q : 0.0;
  return v == w.without ? 0.0 : positive(p);
}

// Sum over the workgroup, the same in all threads; in the threads' order.
__device__ __forceinline__ double sum_all(double x, double* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += lds[w];
  __syncthreads();
  return s;
}

// Inclusive sum over the threads up to this one, and over all.
__device__ __forceinline__ double scan_all(double x, double* lds, double& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double up = __shfl_up(x, d);
    if (lane >= d) x += up;
  }
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  double before = 0.0;
  all = 0.0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w == wave) before = all;
    all += lds[w];
  }
  __syncthreads();
  return before + x;
}

// Lowest (LEAST) or highest of the workgroup's numbers.
template <bool LEAST>
__device__ __forceinline__ int32_t extreme(int32_t x, int32_t* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = LEAST ? min(x, __shfl_xor(x, d)) : max(x, __shfl_xor(x, d));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  int32_t s = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s = LEAST ? min(s, lds[w]) : max(s, lds[w]);
  __syncthreads();
  return s;
}

// grid: x over chunks of the vocabulary, y over requests.
__global__ void __launch_bounds__(kThreads) verify_sum_kernel(VerifyArgs a) {
  __shared__ double lds[kWaves];
  const int32_t r = blockIdx.y;
  const Rows q = rows_of(a, r);
  if (q.last < q.start) {
    if (blockIdx.x == 0 && threadIdx.x == 0) a.accepted[r] = 0;
    return;
  }
  const int32_t row = row_reached(a, q);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.accepted[r] = row - q.start;
  const Weights w = weights_of(a, q, row);
  const int32_t v0 = blockIdx.x * kVerifyChunk + threadIdx.x;
  float p[kEach], d[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int32_t v = v0 + i * kThreads;
    p[i] = v < a.vocab ? w.p[v] : 0.0f;
    d[i] = w.q && v < a.vocab ? w.q[v] : 0.0f;
  }
  double left = 0.0, whole = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    left += weight_at(w, v0 + i * kThreads, p[i], d[i]);
    whole += positive(p[i]);
  }
  left = sum_all(left, lds);
  whole = sum_all(whole, lds);
  if (threadIdx.x == 0) {
    double* to = a.sums + ((int64_t)r * a.chunks + blockIdx.x) * 2;
    to[0] = left;
    to[1] = whole;
  }
}

__global__ void __launch_bounds__(kThreads) verify_pick_kernel(VerifyArgs a) {
  __shared__ double lds[kWaves];
  __shared__ int32_t ints[kWaves];
  __shared__ double carry;
  constexpr int32_t kNone = 0x7FFFFFFF;
  const int32_t r = blockIdx.x;
  const Rows q = rows_of(a, r);
  if (q.last < q.start) return;
  const int tid = threadIdx.x;
  const int32_t row = q.start + a.accepted[r];
  Weights w = weights_of(a, q, row);
  const double* sums = a.sums + (int64_t)r * a.chunks * 2;
  // the row's sum, of the weights or, where they are all zero, of the target's probabilities
  double left = 0.0, whole = 0.0;
  for (int32_t b = 0; b < a.chunks; b += kThreads) {
    const int32_t c = b + tid;
    double l, p;
    scan_all(c < a.chunks ? sums[2 * c] : 0.0, lds, l);
    scan_all(c < a.chunks ? sums[2 * c + 1] : 0.0, lds, p);
    left += l;
    whole += p;
  }
  const bool plain = !(left > 0.0);
  if (plain) w = Weights{w.p, nullptr, -1};
  const double aim = (double)a.sample_u[r] * (plain ? whole : left);
  // the first chunk whose sum passes the aim, or the last that has any weight
  int32_t chosen = kNone, last = -1;
  double before = 0.0, base = 0.0;
  for (int32_t b = 0; b < a.chunks && chosen == kNone; b += kThreads) {
    const int32_t c = b + tid;
    const double x = c < a.chunks ? sums[2 * c + (plain ? 1 : 0)] : 0.0;
    double all;
    const double upto = before + scan_all(x, lds, all);
    last = max(last, extreme<false>(x > 0.0 ? c : -1, ints));
    chosen = extreme<true>(x > 0.0 && upto > aim ? c : kNone, ints);
    if (c == chosen) carry = upto - x;
    before += all;
  }
  __syncthreads();
  if (chosen != kNone) base = carry;
  const bool at_end = chosen == kNone;
  if (at_end) chosen = last;
  int32_t token = -1;
  if (chosen >= 0) {
    const int32_t v0 = chosen * kVerifyChunk + tid * kEach;
    double x[kEach], sum = 0.0, all;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int32_t v = v0 + i;
      x[i] = v < a.vocab ? weight_at(w, v, w.p[v], w.q ? w.q[v] : 0.0f) : 0.0;
      sum += x[i];
    }
    double upto = base + (scan_all(sum, lds, all) - sum);
    int32_t first = kNone, end = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      upto += x[i];
      if (x[i] > 0.0) {
        end = v0 + i;
        if (first == kNone && upto > aim) first = v0 + i;
      }
    }
    // (where rounding leaves the chunk's sum at the aim: its last token with a weight)
    first = extreme<true>(at_end ? kNone : first, ints);
    end = extreme<false>(end, ints);
    token = first == kNone ? end : first;
  }
  for (int32_t t = q.start + tid; t <= q.last; t += kThreads) a.out[t] = t < row ? a.tokens[t + 1] : t == row ? token : -1;
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(verify_sum_kernel, dim3((uint32_t)a.chunks, (uint32_t)a.requests), dim3(kThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_pick_kernel, dim3((uint32_t)a.requests), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace nvfp4
