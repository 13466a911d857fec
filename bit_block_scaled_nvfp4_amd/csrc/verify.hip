// Verification of drafted tokens (gfx950): how many of a request's drafts the target accepts, and the token sampled
// behind them.
//
// What bounds it: HBM reads of two rows of the vocabulary a request (target and draft at the first token that was not
// accepted; where all were, the target's last row alone).  A row is cut into chunks of 4096 that workgroups of a first
// launch sum, each after finding the row by itself (64 drafts a look, one lane each: three dependent loads); a second
// launch, a workgroup a request, finds the chunk that the random number falls into, sums that chunk again element by
// element and writes the tokens.  Sums are binary64 in a fixed order: weights are differences of binary32 numbers, so
// two orders differ by about 2^-50 of the sum.
//
// Measured (copies at 4.9 TB/s): 64 requests of up to 8 drafts over 131077 tokens, 64 MB: 13.6 us for the sums and 5.8 for the
// tokens (10 with barriers and single loads); one request over 32000: 4.8 and 5.1, the start of a launch and the chain of
// loads.
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

// Whether a request behind r owns row t too.  That takes starts that fall: the row is then the last such request's, and no
// other writes it (two writers in no order would leave either's token).
__device__ bool taken_later(const VerifyArgs& a, int32_t r, int32_t t) {
  for (int32_t i = r + 2; i < a.requests; ++i) {
    const Rows q = rows_of(a, i);
    if (q.start <= t && t <= q.last) return true;
  }
  return false;
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

// Inclusive sum over a wavefront's lanes up to this one.
__device__ __forceinline__ double scan_wave(double x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double up = __shfl_up(x, d);
    if (lane >= d) x += up;
  }
  return x;
}

// kEach numbers of a row from v on: whole where `all`, else those below the vocabulary's end.
struct __attribute__((packed, aligned(4))) Four {
  float x[4];
};

__device__ __forceinline__ void load_row(const float* row, int32_t v, int32_t vocab, float (&x)[kEach]) {
  if (v + kEach <= vocab) {
#pragma unroll
    for (int i = 0; i < kEach; i += 4) {
      const Four f = *reinterpret_cast<const Four*>(row + v + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i + k] = f.x[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = v + i < vocab ? row[v + i] : 0.0f;
  }
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

// A workgroup a request.  Every wavefront finds the chunk by itself (64 chunks a look), with no barrier.
__global__ void __launch_bounds__(kThreads) verify_pick_kernel(VerifyArgs a) {
  __shared__ double totals[kWaves];
  __shared__ int32_t firsts[kWaves], ends[kWaves];
  __shared__ bool met[kWaves];
  constexpr int32_t kNone = 0x7FFFFFFF;
  const int32_t r = blockIdx.x;
  const Rows q = rows_of(a, r);
  if (q.last < q.start) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t row = q.start + a.accepted[r];
  const double u = a.sample_u[r];
  // the rows of a request behind the next one, which starts behind this one's rows (looked at before the end only)
  int32_t next = r + 2 + tid;
  int32_t from = 0, to = 0;
  if (r + 2 < a.requests) {
    from = a.query_start[min(next, a.requests)];
    to = a.query_start[min(next + 1, a.requests)];
  }
  const double* sums = a.sums + (int64_t)r * a.chunks * 2;
  // the row's sum, of the weights or, where they are all zero, of the target's probabilities
  double left = 0.0, whole = 0.0;
  for (int32_t b = 0; b < a.chunks; b += 64) {
    const int32_t c = b + lane;
    double l = c < a.chunks ? sums[2 * c] : 0.0, p = c < a.chunks ? sums[2 * c + 1] : 0.0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      l += __shfl_xor(l, d);
      p += __shfl_xor(p, d);
    }
    left += l;
    whole += p;
  }
  const bool plain = !(left > 0.0);
  Weights w = weights_of(a, q, row);
  if (plain) w = Weights{w.p, nullptr, -1};
  // (of 1 and more, and NaN: the last token with a weight.  The total, and running sums, added in another order, may lie
  // either side of one another)
  const double aim = u < 1.0 ? u * (plain ? whole : left) : __builtin_inf();
  // the first chunk whose sum passes the aim, or the last that has any weight
  int32_t chosen = -1, last = -1;
  double before = 0.0, base = 0.0;
  for (int32_t b = 0; b < a.chunks && chosen < 0; b += 64) {
    const int32_t c = b + lane;
    const double x = c < a.chunks ? sums[2 * c + (plain ? 1 : 0)] : 0.0;
    const double sum = scan_wave(x), upto = before + sum;
    const uint64_t some = __ballot(x > 0.0), passed = __ballot(x > 0.0 && upto > aim);
    if (some) last = b + 63 - __builtin_clzll(some);
    if (passed) {
      const int at = __builtin_ctzll(passed);
      chosen = b + at;
      base = __shfl(upto - x, at);
    }
    before = __shfl(upto, 63);
  }
  const bool at_end = chosen < 0;
  if (at_end) chosen = last;
  // whether one of them has some of this request's rows
  const auto meets = [&](int32_t x, int32_t y) { return x < y && x <= q.last && y > q.start; };
  bool meet = meets(from, to);
  while ((next += kThreads) < a.requests) meet |= meets(a.query_start[next], a.query_start[next + 1]);
  int32_t token = -1;
  bool shared = false;
  if (chosen >= 0) {
    const int32_t v0 = chosen * kVerifyChunk + tid * kEach;
    float p[kEach], d[kEach];
    load_row(w.p, v0, a.vocab, p);
    if (w.q) load_row(w.q, v0, a.vocab, d);
    double x[kEach], sum = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      x[i] = weight_at(w, v0 + i, p[i], w.q ? d[i] : 0.0f);
      sum += x[i];
    }
    const double mine = scan_wave(sum);
    if (lane == 63) totals[wave] = mine;
    __syncthreads();
    double upto = base;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) upto += k < wave ? totals[k] : 0.0;
    upto += mine - sum;
    int32_t first = kNone, end = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      upto += x[i];
      if (x[i] > 0.0) {
        end = v0 + i;
        if (first == kNone && upto > aim) first = v0 + i;
      }
    }
    // the lowest of the lanes' first, the highest of their ends: lanes hold rising parts of the chunk
    const uint64_t found = __ballot(first != kNone), some = __ballot(end >= 0);
    const int32_t f = found ? __shfl(first, __builtin_ctzll(found)) : kNone, e = some ? __shfl(end, 63 - __builtin_clzll(some)) : -1;
    const bool wave_meets = __any(meet);
    if (lane == 0) {
      firsts[wave] = f;
      ends[wave] = e;
      met[wave] = wave_meets;
    }
    __syncthreads();
    int32_t at = kNone, tail = -1;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      at = min(at, firsts[k]);
      tail = max(tail, ends[k]);
      shared |= met[k];
    }
    // (where rounding leaves the chunk's sum at the aim: its last token with a weight)
    token = at_end || at == kNone ? tail : at;
  } else {
    shared = __syncthreads_or(meet);
  }
  for (int32_t t = q.start + tid; t <= q.last; t += kThreads) {
    if (__builtin_expect(shared, 0) && taken_later(a, r, t)) continue;
    a.out[t] = t < row ? a.tokens[t + 1] : t == row ? token : -1;
  }
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
