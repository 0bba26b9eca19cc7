// Device-side helpers of the linear attention's sweeps: powers of a head's decay and the segment
// that a block works on.
#pragma once

#include <cuda_fp16.h>

#include "linattn.cuh"
#include "ptx.cuh"

namespace mmf {

// Two fp32 operations at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
// max(|a|, |b|, |c|)
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float v;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(a), "f"(b), "f"(c));
  return v;
}

// log2 of a head's decay.  Decays lie in [0, 1]: a logarithm above 0 (or not a number) counts
// as 0, that of a decay of 0 is -inf.
__device__ __forceinline__ double lin_lg2_of(float log_decay) {
  return static_cast<double>(fminf(log_decay, 0.0f)) * 1.4426950408889634;
}
__device__ __forceinline__ double lin_lg2(const LinCall& c, int h) {
  return lin_lg2_of(__ldg(c.log_decay + h));
}
// gamma^n: the exponent is multiplied in double and rounded once to float, which puts at most
// n |log2 gamma| 2^-24 on the power, relative to it; exp2f's own error, up to 2 ulp, comes on top and is
// the larger one while n |log2 gamma| is small.  For weights that are used once; a state's decay is
// LinDecay or LinTurns.  gamma^0 is 1 for every decay.
__device__ __forceinline__ float lin_power(double lg2, int64_t n) {
  return n == 0 ? 1.0f : exp2f(static_cast<float>(lg2 * static_cast<double>(n)));
}

// Factors in fp16, kept finite.  Only a token whose values are all zero can have one beyond its range (the
// scales come from the others), and its products have to stay zero.
__device__ __forceinline__ __half2 lin_half2_finite(float lo, float hi) {
  uint32_t v;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  return *reinterpret_cast<const __half2*>(&v);
}

// The decay gamma^n of a state that is carried on many times, as whole + part, whole 1 or 0.  Rounded to
// one float it would be off the same way every time (a log decay of -1e-4: 9e-5 of a state after 4096
// tokens).  part is off by 2^-24 of 1 - gamma^n (of gamma^n below a half, where a state lasts for a few
// steps).  next = x + (part x + u) then rounds the state once, at a place that u moves about; with
// part x alone rounded into x, decays next to 1 would come to nothing.
struct LinDecay {
  float whole, part;
  LinDecay() = default;
  __device__ __forceinline__ LinDecay(double lg2, int64_t n) {
    const double g = n == 0 ? 1.0 : exp2(lg2 * static_cast<double>(n));
    whole = g >= 0.5 ? 1.0f : 0.0f;
    part = static_cast<float>(g - static_cast<double>(whole));
  }
  // gamma^n x + u
  __device__ __forceinline__ float next(float x, float u) const {
    return fmaf(whole, x, fmaf(part, x, u));
  }
};

// The decay gamma^n of chunks of n tokens, for states that take a chunk's product in the same operation,
// gamma^n x + u rounded once, where u moves the rounding about.  Rounded to one float the decay would be
// off the same way every time (4.7e-6 of a state after 16384 tokens at a log decay of -1e-4), so the two
// floats around it take turns, in proportion.  `last`: of the `left` tokens of a shorter last chunk.
struct alignas(16) LinTurns {
  float lo, hi;
  uint32_t share;   // of the turns that are hi's, in 2^-32
  float last;
  LinTurns() = default;
  __device__ __forceinline__ LinTurns(double lg2, int n, int left) {
    const double g = exp2(lg2 * n);
    lo = __double2float_rd(g);
    hi = __double2float_ru(g);
    share = hi > lo ? __double2uint_rn((g - lo) / (static_cast<double>(hi) - lo) * 0x1p32) : 0u;
    last = left == 0 ? 1.0f : static_cast<float>(exp2(lg2 * left));
  }
  __device__ __forceinline__ float of(int chunk) const {
    // hi when a sum of shares, from a half on, passes a whole one
    return (static_cast<uint32_t>(chunk) + 1u) * share + 0x80000000u < share ? hi : lo;
  }
};

// An infinity in a start state as a NaN, which the maxima that scales come from pass over: neither
// leaves its column finite, but an infinity would take the range from the other columns.
__device__ __forceinline__ float lin_nan_if_inf(float x) {
  return isinf(x) ? __int_as_float(0x7fffffff) : x;
}

struct LinSeg {
  bool valid;      // false: the item is past the last segment
  bool first, last;
  int seq;
  int64_t begin;   // the first token taken (forwards the lowest, backwards the highest)
  int64_t n;       // tokens
  int step;        // +1 or -1
  __device__ __forceinline__ int64_t token(int64_t p) const { return begin + step * p; }
};

// Bounds of a sequence.  Bounds read from the device are clamped to [0, T] and to one another, so
// that no value of them reaches outside the tensors; a clamped one is reported.
__device__ __forceinline__ void lin_bounds(const LinCall& c, int b, int64_t* lo, int64_t* hi,
                                           bool* bad) {
  if (c.cu == nullptr) {
    const int64_t len = c.T / c.B;
    *lo = b * len;
    *hi = *lo + len;
    return;
  }
  const int64_t x = __ldg(c.cu + b), y = __ldg(c.cu + b + 1);
  *lo = min(max(x, static_cast<int64_t>(0)), c.T);
  *hi = min(max(y, *lo), c.T);
  if (x != *lo || y != *hi) *bad = true;
}

// Zeros for the rows of head h of a sweep's output that belong to no sequence, shared out over the
// blocks of gridDim.x.
template <typename T>
__device__ __forceinline__ void lin_clear(const LinCall& c, const LinSweep& w, int h) {
  if (!c.clear || c.cu == nullptr) return;
  const int64_t x = __ldg(c.cu), y = __ldg(c.cu + c.B);
  const int64_t lo = min(max(x, static_cast<int64_t>(0)), c.T), hi = min(max(y, lo), c.T);
  const int64_t vecs = w.dv * static_cast<int>(sizeof(T)) / 16, n = (lo + c.T - hi) * vecs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / vecs, t = row < lo ? row : row - lo + hi;
    uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(w.o) + t * w.o_t + h * w.o_h);
    o[i - row * vecs] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// A sequence without tokens has one (empty) segment, which passes its state on.
__device__ __forceinline__ int64_t lin_count(const LinCall& c, int64_t len) {
  return len <= c.seg_len ? 1 : (len + c.seg_len - 1) / c.seg_len;
}

// Number of segments of sequence b, the item of its first and its length.  Every warp of the block works it
// out for itself; all lanes of a warp call it together.
__device__ __forceinline__ int64_t lin_segments(const LinCall& c, int b, int64_t* first,
                                                int64_t* len) {
  int64_t lo, hi;
  bool bad = false;
  if (c.cu == nullptr) {
    lin_bounds(c, b, &lo, &hi, &bad);
    const int64_t n = lin_count(c, hi - lo);
    *first = b * n;
    *len = hi - lo;
    return n;
  }
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int i = lane; i < b; i += 32) {
    lin_bounds(c, i, &lo, &hi, &bad);
    before += lin_count(c, hi - lo);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  lin_bounds(c, b, &lo, &hi, &bad);
  *first = before;
  *len = hi - lo;
  const int64_t n = lin_count(c, hi - lo);
  // bounds that overlap can ask for more items than the call has: those are left out
  return max(min(n, c.n_items - before), static_cast<int64_t>(0));
}

// The segment of item x (the same for every thread of the block; all lanes of a warp together).
__device__ __forceinline__ LinSeg lin_find(const LinCall& c, int64_t x, bool backwards) {
  LinSeg g = {};
  int64_t lo = 0, hi = 0, k = 0;
  bool bad = false;
  if (!c.split) {   // one item for each sequence
    g.seq = static_cast<int>(x);
    lin_bounds(c, g.seq, &lo, &hi, &bad);
    if (bad) atomicOr(c.status, kStatusBadPlan);
  } else if (c.cu == nullptr) {
    const int64_t per = lin_count(c, c.T / c.B);
    g.seq = static_cast<int>(x / per);
    k = x - g.seq * per;
    lin_bounds(c, g.seq, &lo, &hi, &bad);
  } else {
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    int found = -1;
    for (int b0 = 0; b0 < c.B && found < 0; b0 += 32) {
      int64_t n = 0;
      if (b0 + lane < c.B) {
        lin_bounds(c, b0 + lane, &lo, &hi, &bad);
        n = lin_count(c, hi - lo);
      }
      int64_t sum = n;   // inclusive prefix sum over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + sum > x);
      if (past) {
        const int l = __ffs(past) - 1;
        found = b0 + l;
        k = x - base - __shfl_sync(0xffffffffu, sum - n, l);
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (bad) atomicOr(c.status, kStatusBadPlan);
    if (found < 0) return g;
    g.seq = found;
    lin_bounds(c, found, &lo, &hi, &bad);
  }
  const int64_t len = hi - lo, n = lin_count(c, len);
  g.valid = true;
  g.first = k == 0;
  g.last = k == n - 1;
  const int64_t p0 = k * c.seg_len;
  g.n = min(c.seg_len, len - p0);
  g.step = backwards ? -1 : 1;
  g.begin = backwards ? hi - 1 - p0 : lo + p0;
  return g;
}

}  // namespace mmf
