// Linear attention with a decay for each head: S_t = gamma S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.
//
// A token mixer of the family of the MLGRU (an element-wise recurrence, "MatMul-freie LLMs:
// Zentrale Konzepte erklärt", section "Kernkomponenten: MLGRU und GLU"), with a matrix for a
// state.  This file holds the token-by-token sweep for every type and head size, the pass that
// joins the segments of a split sequence, and the single-token step.
//
// Splitting.  A sweep is serial in the tokens, so when (sequence, head) pairs are too few to fill
// the GPU every sequence is cut into segments of L tokens: one pass finds each segment's own
// contribution to the state from k and v alone (kState), a second joins them,
//   start_{s+1} = gamma^(tokens of s) start_s + own_s,
// which also gives the state after the last, and the third runs all segments at once from their
// start states.  A sequence of one segment is left to the third alone.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "linattn.cuh"
#include "linattn_dev.cuh"
#include "ptx.cuh"

namespace mmf {
namespace {

// ------------------------------------------------------------------ token-by-token sweep
// Block: one segment, one head, 32 columns of the state.  Thread (r, c) holds rows 4 r + 64 j ..
// + 3 and columns 4 c .. + 3: 4 KR values in registers, in fp32 throughout (the products too).
// k, q and v (each v twice, as both halves of a pair) come from shared memory as 16-byte broadcasts, a
// tile of kTok tokens at a time.
//
// Decay.  For a slow one (gamma^kTok at least 2^-8, which keeps the scaled sums in range) the state is
// held over gamma^i at a tile's token i: v is scaled by gamma^-i once, outputs by gamma^i, so that a token
// costs a state element an update and a product with q, and the state takes gamma^kTok once for
// each tile, with the next tile's first token (LinDecay).  Fast decays, whose states last for a few tokens,
// are taken at every token.  A product of the state with one token's decay at every token, even with the
// two floats around it in turn, is rounded the same way as long as the state moves little: 5e-5 of a
// state after 8192 tokens at a log decay of -1e-7, so 1e-5 at most at any (test_gpu_linattn_drift.py).
//
// Bound by latency: the fp32 operations, two rows at a time (f32x2), are a fourth to a third of the time,
// the rest is each token's chain of loads from shared memory, operations and shuffles with 12 warps on an
// SM to hide it.  Measured: 1500 tokens, 8 heads of 96 x 128 in fp32, a call 80 us (89 with the registers
// for a fourth block on an SM).  o is summed over the 16 row groups: four in a warp by shuffles, four
// warps through shared memory once every kTok tokens.
constexpr int kSweepThreads = 128;
constexpr int kTok = 16;
constexpr int kCols = 32;

template <typename T>
__device__ __forceinline__ float4 ld4(const T* p);
template <>
__device__ __forceinline__ float4 ld4<float>(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 ld4<__half>(const __half* p) {
  const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
  const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&a.x));
  const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&a.y));
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__half* p, float v) { *p = __float2half_rn(v); }

template <typename T, int KR, bool kState>
__global__ void __launch_bounds__(kSweepThreads, KR == 16 ? 2 : 3) lin_sweep_kernel(const __grid_constant__ LinCall c) {
  constexpr int kRows = 16 * KR;           // padded dk
  constexpr int kVecRow = kRows / 4;       // 4-value vectors of a k or q row
  constexpr int kLoads = kTok * kVecRow / kSweepThreads;   // of k (and of q) per thread
  static_assert(kTok * (kCols / 4) == kSweepThreads, "one v vector per thread");
  __shared__ __align__(16) float s_k[kTok][kRows];
  __shared__ __align__(16) float s_q[kState ? 1 : kTok][kState ? 4 : kRows];
  __shared__ __align__(16) float s_v[kTok][2 * kCols];
  __shared__ float s_o[kState ? 1 : 4][kState ? 1 : kTok][kCols];
  __shared__ float s_up[kTok + 1], s_down[kTok + 1];   // gamma^-n, gamma^n; 1 for fast decays
  __shared__ LinDecay s_decay[2];

  const int slices = (max(c.sw[0].dv, c.sw[0].dk) + kCols - 1) / kCols;
  const LinSweep& w = c.sw[blockIdx.z / slices];
  const int col0 = static_cast<int>(blockIdx.z % slices) * kCols;
  if (col0 >= w.dv) return;
  const int h = blockIdx.y;
  if (!kState && col0 == 0) lin_clear<T>(c, w, h);
  const LinSeg g = lin_find(c, blockIdx.x, w.backwards != 0);
  const bool whole = g.first && g.last;   // an unsplit sequence: nothing to start from
  if (!g.valid || (kState && whole)) return;

  const int tid = threadIdx.x, cg = tid & 7, rg = tid >> 3, warp = tid >> 5;
  const double lg2 = lin_lg2(c, h);
  const int lag = w.backwards ? 1 : 0;   // backwards the decay acts after a token, not before it
  const bool slow = lg2 * kTok >= -8.0;
  // the decay still due after the last token: of the last tile's tokens, of one backwards, or none
  const int64_t left = g.n == 0 ? 0 : slow ? (g.n - 1) % kTok + 1 : lag;
  if (tid <= kTok) s_up[tid] = slow ? static_cast<float>(exp2(-lg2 * tid)) : 1.0f;
  if (tid >= 32 && tid <= 32 + kTok) s_down[tid - 32] = slow ? static_cast<float>(exp2(lg2 * (tid - 32))) : 1.0f;
  if (tid == 64) s_decay[0] = LinDecay(lg2, slow ? kTok : 1);
  if (tid == 96) s_decay[1] = LinDecay(lg2, left);
  const size_t state0 = (static_cast<size_t>(g.seq) * c.H + h) * w.dk * w.dv;
  float* seg = w.seg ? w.seg + (static_cast<size_t>(blockIdx.x) * c.H + h) * w.dk * w.dv : nullptr;

  // the state before the first token: the split's start state [dk x dv], or s0
  uint64_t S[KR / 2][4];   // pairs of rows
  auto row_of = [&](int i) { return 4 * rg + (i & 3) + 64 * (i >> 2); };
#pragma unroll
  for (int i = 0; i < KR; i += 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[2] = {0.0f, 0.0f};
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int row = row_of(i + z), col = col0 + 4 * cg + j;
        if (!kState && row < w.dk && col < w.dv) {
          if (c.split && !whole)
            x[z] = seg[static_cast<size_t>(row) * w.dv + col];
          else if (w.s0)
            x[z] = w.s0[state0 + static_cast<size_t>(row) * w.s_key + static_cast<size_t>(col) * w.s_val];
        }
      }
      S[i / 2][j] = pair(x[0], x[1]);
    }

  const T* kp = static_cast<const T*>(w.k) + h * w.k_h;
  const T* vp = static_cast<const T*>(w.v) + h * w.v_h;
  const T* qp = static_cast<const T*>(w.q) + h * w.q_h;
  T* op = static_cast<T*>(w.o) + h * w.o_h;
  const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 rk[kLoads], rq[kState ? 1 : kLoads], rv;

  auto fetch = [&](int64_t p0) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int x = tid + i * kSweepThreads, tok = x / kVecRow, d = (x % kVecRow) * 4;
      const bool in = p0 + tok < g.n && d < w.dk;
      const int64_t t = g.token(p0 + tok);
      rk[i] = in ? ld4<T>(kp + t * w.k_t + d) : zero4;
      if constexpr (!kState) rq[i] = in ? ld4<T>(qp + t * w.q_t + d) : zero4;
    }
    const int tok = tid / (kCols / 4), d = col0 + (tid % (kCols / 4)) * 4;
    rv = (p0 + tok < g.n && d < w.dv) ? ld4<T>(vp + g.token(p0 + tok) * w.v_t + d) : zero4;
  };

  fetch(0);
  __syncthreads();
  // the decay that the state has still to take, with the next token of the full form
  const LinDecay decay = s_decay[0];
  LinDecay due = decay;
  if (slow || lag) due.whole = 1.0f, due.part = 0.0f;
  const float va = w.a * s_up[tid / (kCols / 4) + 1 - lag];
  for (int64_t p0 = 0; p0 < g.n; p0 += kTok) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int x = tid + i * kSweepThreads, tok = x / kVecRow, d = (x % kVecRow) * 4;
      *reinterpret_cast<float4*>(&s_k[tok][d]) = rk[i];
      if constexpr (!kState) *reinterpret_cast<float4*>(&s_q[tok][d]) = rq[i];
    }
    float4* v2 = reinterpret_cast<float4*>(&s_v[tid / (kCols / 4)][(tid % (kCols / 4)) * 8]);
    v2[0] = make_float4(rv.x * va, rv.x * va, rv.y * va, rv.y * va);
    v2[1] = make_float4(rv.z * va, rv.z * va, rv.w * va, rv.w * va);
    __syncthreads();
    if (p0 + kTok < g.n) fetch(p0 + kTok);
    const int nt = static_cast<int>(min(static_cast<int64_t>(kTok), g.n - p0));
    auto token = [&](int tok, auto full) {
      const ulonglong2 vlo = *reinterpret_cast<const ulonglong2*>(&s_v[tok][8 * cg]);
      const ulonglong2 vhi = *reinterpret_cast<const ulonglong2*>(&s_v[tok][8 * cg + 4]);
      const uint64_t v2[4] = {vlo.x, vlo.y, vhi.x, vhi.y};
      const uint64_t whole2 = pair(due.whole, due.whole), part2 = pair(due.part, due.part);
      [[maybe_unused]] uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};   // of the even and of the odd rows
#pragma unroll
      for (int i4 = 0; i4 < KR / 4; ++i4) {
        const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(&s_k[tok][4 * rg + 64 * i4]);
        ulonglong2 q4 = make_ulonglong2(0ull, 0ull);
        if constexpr (!kState) q4 = *reinterpret_cast<const ulonglong2*>(&s_q[tok][4 * rg + 64 * i4]);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          uint64_t* Sr = S[2 * i4 + z];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (full.value)
              Sr[j] = fma2(whole2, Sr[j], fma2(part2, Sr[j], mul2(z ? k4.y : k4.x, v2[j])));
            else
              Sr[j] = fma2(z ? k4.y : k4.x, v2[j], Sr[j]);
            if constexpr (!kState) sum[j] = fma2(z ? q4.y : q4.x, Sr[j], sum[j]);
          }
        }
      }
      if constexpr (full.value) due = decay;
      if constexpr (!kState) {
        // sum over the warp's four row groups (lane bits 3 and 4); each lane ends with a column
        float acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpair(sum[j]);
          acc[j] = x.x + x.y;
        }
        const bool hi16 = tid & 16, hi8 = tid & 8;
        float a0 = hi16 ? acc[2] : acc[0], a1 = hi16 ? acc[3] : acc[1];
        const float b0 = hi16 ? acc[0] : acc[2], b1 = hi16 ? acc[1] : acc[3];
        a0 += __shfl_xor_sync(0xffffffffu, b0, 16);
        a1 += __shfl_xor_sync(0xffffffffu, b1, 16);
        const float m = hi8 ? a1 : a0, y = hi8 ? a0 : a1;
        s_o[warp][tok][4 * cg + (hi16 ? 2 : 0) + (hi8 ? 1 : 0)] =
            m + __shfl_xor_sync(0xffffffffu, y, 8);
      }
    };
    token(0, std::true_type{});
    if (slow) {
      for (int tok = 1; tok < nt; ++tok) token(tok, std::false_type{});
    } else {
      for (int tok = 1; tok < nt; ++tok) token(tok, std::true_type{});
    }
    __syncthreads();
    if constexpr (!kState) {
      // read before the next tile's second barrier, which comes before s_o is written again
#pragma unroll
      for (int i = 0; i < kTok * kCols / kSweepThreads; ++i) {
        const int x = tid + i * kSweepThreads, tok = x / kCols, cc = x % kCols;
        if (tok < nt && col0 + cc < w.dv) {
          const float y = (s_o[0][tok][cc] + s_o[1][tok][cc]) + (s_o[2][tok][cc] + s_o[3][tok][cc]);
          st1(op + g.token(p0 + tok) * w.o_t + col0 + cc, y * (w.b * s_down[tok + 1 - lag]));
        }
      }
    }
  }

  if (!kState && !(whole && w.sT)) return;
  const LinDecay end = s_decay[1];
#pragma unroll
  for (int i = 0; i < KR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = row_of(i), col = col0 + 4 * cg + j;
      if (row >= w.dk || col >= w.dv) continue;
      const float2 p = unpair(S[i / 2][j]);
      const float x = left > 0 ? end.next((i & 1) ? p.y : p.x, 0.0f) : (i & 1) ? p.y : p.x;
      if (kState)
        seg[static_cast<size_t>(row) * w.dv + col] = x;
      else
        w.sT[state0 + static_cast<size_t>(row) * w.s_key + static_cast<size_t>(col) * w.s_val] = x;
    }
}

// -------------------------------------------------------------------- joining the segments
// Every thread takes four elements of a state through the segments of its sequence.  On entry
// slot s holds segment s's own contribution, on exit the state before it; sT gets the state after
// the last.  The first slot becomes a copy of s0, which may be sT itself.
__global__ void __launch_bounds__(256) lin_join_kernel(const __grid_constant__ LinCall c) {
  const int blocks = (c.sw[0].dk * c.sw[0].dv / 4 + 255) / 256;
  const LinSweep& w = c.sw[blockIdx.z];
  const int b = static_cast<int>(blockIdx.x) / blocks, h = blockIdx.y;
  const int e = (static_cast<int>(blockIdx.x) % blocks * 256 + static_cast<int>(threadIdx.x)) * 4;
  int64_t first, len;
  const int64_t n = lin_segments(c, b, &first, &len);   // whole warps
  if (n < 2) return;   // all threads
  __shared__ LinDecay s_decay[2];
  if (threadIdx.x < 2)
    s_decay[threadIdx.x] = LinDecay(lin_lg2(c, h), threadIdx.x == 0 ? c.seg_len
                                    : max(len - (n - 1) * c.seg_len, static_cast<int64_t>(0)));
  __syncthreads();
  if (e >= w.dk * w.dv) return;
  const LinDecay gl = s_decay[0], glast = s_decay[1];
  const int i = e / w.dv, j = e % w.dv;
  const size_t state = static_cast<size_t>(w.dk) * w.dv;
  const size_t at = (static_cast<size_t>(b) * c.H + h) * state + static_cast<size_t>(i) * w.s_key +
                    static_cast<size_t>(j) * w.s_val;
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (w.s0) {
    const float* p = w.s0 + at;
    S = make_float4(p[0], p[w.s_val], p[2 * w.s_val], p[3 * w.s_val]);
  }
  float* slot = w.seg + (static_cast<size_t>(first) * c.H + h) * state + e;
  const size_t step = static_cast<size_t>(c.H) * state;
  constexpr int kAhead = 4;   // slots in flight
  float4 own[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (u < n) own[u] = *reinterpret_cast<const float4*>(slot + u * step);
  for (int64_t x0 = 0; x0 < n; x0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t x = x0 + u;
      if (x < n) {
        const float4 o = own[u];
        if (x + kAhead < n) own[u] = *reinterpret_cast<const float4*>(slot + kAhead * step);
        *reinterpret_cast<float4*>(slot) = S;
        slot += step;
        const LinDecay& f = x + 1 < n ? gl : glast;
        S.x = f.next(S.x, o.x);
        S.y = f.next(S.y, o.y);
        S.z = f.next(S.z, o.z);
        S.w = f.next(S.w, o.w);
      }
    }
  }
  if (w.sT) {
    float* p = w.sT + at;
    p[0] = S.x;
    p[w.s_val] = S.y;
    p[2 * w.s_val] = S.z;
    p[3 * w.s_val] = S.w;
  }
}

// ------------------------------------------------------------------------ single token
// Block: one sequence, one head, up to 128 columns of the state; eight warps share its rows, a
// warp's lane holds four columns.  The state is read and written once, 16 bytes a lane and
// contiguous along a row, with kUnroll rows in flight; everything else is small.  Bound by that
// stream: 256 sequences of 16 heads of 128 x 128 take 86 us, 6280 GB/s, 96 % of a copy's rate.
constexpr int kStepThreads = 256;
constexpr int kStepWarps = kStepThreads / 32;

template <typename T>
__device__ __forceinline__ float ld1(const T* p);
template <>
__device__ __forceinline__ float ld1<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float ld1<__half>(const __half* p) { return __half2float(__ldg(p)); }

template <typename T>
__global__ void __launch_bounds__(kStepThreads) lin_step_kernel(const __grid_constant__ LinStep c) {
  constexpr int kUnroll = 8;
  __shared__ float s_k[256], s_q[256];
  __shared__ __align__(16) float s_o[kStepWarps][128];
  const int64_t b = blockIdx.x;
  const int h = blockIdx.y, col0 = static_cast<int>(blockIdx.z) * 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int64_t slot = b;
  bool skip = false;
  if (c.slots) {
    slot = c.slots[b];
    // a slot named by an earlier sequence has its one update there
    bool twice = false;
    for (int64_t i = tid; i < b; i += kStepThreads) twice |= c.slots[i] == slot;
    const bool out = slot < 0 || slot >= c.n_slots;
    twice = __syncthreads_or(twice && !out);
    skip = out || twice;
    if ((twice || slot >= c.n_slots) && tid == 0) atomicOr(c.status, kStatusBadPlan);
  }
  T* op = static_cast<T*>(c.o) + b * c.o_b + h * c.o_h;
  if (skip) {
    if (tid < 128 && col0 + tid < c.dv) st1(op + col0 + tid, 0.0f);
    return;
  }
  const T* kp = static_cast<const T*>(c.k) + b * c.k_b + h * c.k_h;
  const T* qp = static_cast<const T*>(c.q) + b * c.q_b + h * c.q_h;
  const T* vp = static_cast<const T*>(c.v) + b * c.v_b + h * c.v_h;
  if (tid < c.dk) {
    s_k[tid] = ld1<T>(kp + tid);
    s_q[tid] = ld1<T>(qp + tid);
  }
  __shared__ LinDecay s_decay;
  if (tid == kStepThreads - 1) s_decay = LinDecay(lin_lg2_of(c.log_decay[h]), 1);
  const int col = col0 + 4 * lane;
  const bool in = col < c.dv;
  const float4 v4 = in ? ld4<T>(vp + col) : make_float4(0.f, 0.f, 0.f, 0.f);
  float* st = c.state + (static_cast<size_t>(slot) * c.H + h) * c.dk * c.dv + col;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  const LinDecay gamma = s_decay;
  for (int r0 = warp; in && r0 < c.dk; r0 += kStepWarps * kUnroll) {
    float4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kStepWarps;
      if (r < c.dk) x[u] = __ldcs(reinterpret_cast<const float4*>(st + static_cast<size_t>(r) * c.dv));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kStepWarps;
      if (r < c.dk) {
        const float k = s_k[r], q = s_q[r];
        x[u].x = gamma.next(x[u].x, k * v4.x);
        x[u].y = gamma.next(x[u].y, k * v4.y);
        x[u].z = gamma.next(x[u].z, k * v4.z);
        x[u].w = gamma.next(x[u].w, k * v4.w);
        acc.x = fmaf(q, x[u].x, acc.x);
        acc.y = fmaf(q, x[u].y, acc.y);
        acc.z = fmaf(q, x[u].z, acc.z);
        acc.w = fmaf(q, x[u].w, acc.w);
        __stcs(reinterpret_cast<float4*>(st + static_cast<size_t>(r) * c.dv), x[u]);
      }
    }
  }
  *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = acc;
  __syncthreads();
  if (tid < 128 && col0 + tid < c.dv) {
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < kStepWarps; ++i) y += s_o[i][tid];
    st1(op + col0 + tid, y * c.scale);
  }
}

template <typename T, int KR>
cudaError_t sweeps(const LinCall& c, cudaStream_t s) {
  const int slices = (std::max(c.sw[0].dk, c.sw[0].dv) + kCols - 1) / kCols;
  const dim3 grid(static_cast<unsigned>(c.n_items), static_cast<unsigned>(c.H),
                  static_cast<unsigned>(slices * c.n_sweeps));
  if (c.split) {
    lin_sweep_kernel<T, KR, true><<<grid, kSweepThreads, 0, s>>>(c);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if ((e = launch_lin_join(c, s)) != cudaSuccess) return e;
  }
  lin_sweep_kernel<T, KR, false><<<grid, kSweepThreads, 0, s>>>(c);
  return cudaGetLastError();
}

template <typename T>
cudaError_t sweeps_of(const LinCall& c, cudaStream_t s) {
  const int d = std::max(c.sw[0].dk, c.n_sweeps > 1 ? c.sw[0].dv : 0);
  if (d <= 64) return sweeps<T, 4>(c, s);
  if (d <= 128) return sweeps<T, 8>(c, s);
  return sweeps<T, 16>(c, s);
}

}  // namespace

cudaError_t launch_lin_join(const LinCall& c, cudaStream_t s) {
  const int blocks = (c.sw[0].dk * c.sw[0].dv / 4 + 255) / 256;
  const dim3 grid(static_cast<unsigned>(blocks * c.B), static_cast<unsigned>(c.H),
                  static_cast<unsigned>(c.n_sweeps));
  lin_join_kernel<<<grid, 256, 0, s>>>(c);
  return cudaGetLastError();
}

size_t lin_seg_bytes(int64_t n_items, int H, int dk, int dv) {
  return (static_cast<size_t>(n_items) * H * dk * dv * 4 + 255) / 256 * 256;
}

LinForm lin_form(int H, int dk, int dv, int dt, int n_sweeps, const int64_t (*strides)[2]) {
  if (dt != kInF16) return kLinTokens;
  if (dk == 128 && dv == 128) {
    // tensor maps: none for a row that every token shares, columns counted in 31 bits, rows in 40
    bool maps = true;
    for (int i = 0; i < (n_sweeps > 1 ? 4 : 3); ++i)
      maps &= strides[i][0] > 0 && strides[i][0] < (1ll << 38) &&
              (H == 1 || strides[i][1] <= (0x7fffffff - 128) / (H - 1));
    if (maps) return kLinTc;
  }
  // a sweep's dk is 64 or 128, its dv a multiple of 64; the backward's have both orders
  auto keys = [](int d) { return d == 64 || d == 128; };
  return keys(dk) && (n_sweeps > 1 ? keys(dv) : dv % 64 == 0) ? kLinMma : kLinTokens;
}

void lin_plan(int64_t T, int64_t B, bool ragged, int H, int dk, int dv, LinForm form, int n_sweeps,
              int64_t* seg_len, int64_t* n_items, int* split) {
  // A model of the time, of the kernel that the call takes.  A block handles `step` tokens at a
  // time and `each` of them run on an SM (blocks beyond 148 each wait for the next wave); a step
  // takes t0 + t1 n us with n blocks on an SM, a block's start and end `start` us, a pass over k and v
  // alone about half of a whole one, and the two launches that a split adds `more` us.  The constants were
  // fitted to whole calls (16 heads of 128 or 64, in fp32 8 of 128), so they hold a part of the starts and
  // of the last, shorter segments.  A step alone, measured from the slope over long sequences: 128 tokens with
  // tcgen05 4.4; 64 in the register form 2.9 alone on an SM, 5.0 with three; 16 token by token 4.9
  // with three.  With these for constants the model would choose other segments in one call of ten, and
  // by itself gain 1 % at most on the average.  The split is worth (us, split /
  // whole): one prompt of 1024 28 / 36, of 4096 45 / 125, heads of 64, 4 of 512 21 / 30, fp32, one of
  // 512 40 / 104; it is not: backward of 1024 40 / 36, heads of 64, 8 of 512 35 / 31.
  const bool tc = form == kLinTc, mma = form == kLinMma;
  int64_t step, each, width;
  double t0, t1, start, more;
  if (tc) {
    step = 128, each = 1, width = 1;
    t0 = 4.1, t1 = 0.0, start = 3.5, more = 16.0;
  } else if (mma) {
    const int tile = dv % 128 == 0 ? 128 : 64;
    const double size = dk * tile / 4096.0;
    step = 64, each = dk == 128 ? 2 : 3, width = dv / tile;
    t0 = 2.0 * size, t1 = 1.7 * size, start = 3.0, more = 8.0;
  } else {
    const int most = std::max(dk, dv);
    const double size = most <= 64 ? 0.75 : most <= 128 ? 1.0 : 2.0;
    step = 16, each = most > 128 ? 2 : 3, width = (most + 31) / 32;
    t0 = 1.8 * size, t1 = 1.45 * size, start = 3.0, more = 10.0;
  }
  // Of a ragged batch the host knows the sum of the lengths alone: it takes the longest for three
  // times the mean, and half a segment more for each sequence.
  const int64_t mean = (T + B - 1) / B;
  const int64_t longest = ragged ? std::min(T, 3 * mean) : mean;
  const double units = static_cast<double>(H) * n_sweeps * width;
  auto time = [&](double steps, double segments) {
    const double blocks = units * segments;
    const double waves = std::ceil(blocks / (148.0 * each));
    const double on = std::min<double>(each, std::max(1.0, blocks / 148.0));
    return waves * (start + steps * (t0 + t1 * on));
  };
  const int64_t n = (longest + step - 1) / step, all = (T + step - 1) / step;
  double best = time(static_cast<double>(n), static_cast<double>(B));
  int64_t most_steps = 0;   // of a segment; none: no split
  auto consider = [&](int64_t l) {
    l = std::max<int64_t>(l, tc || mma ? 2 : 4);
    if (l >= n) return;
    const double segments = ragged ? static_cast<double>(all) / l + 0.5 * B
                                   : static_cast<double>(B * ((n + l - 1) / l));
    const double t = 1.5 * time(static_cast<double>(l), segments) + more;
    if (t < best) {
      best = t;
      most_steps = l;
    }
  };
  // segments that fill whole waves, and short ones
  for (int waves = 1; waves <= 4; ++waves) {
    const double room = 148.0 * each * waves / units;   // segments
    const int64_t segments = static_cast<int64_t>(ragged ? room - 0.5 * B : room / B);
    if (segments > 0) consider(((ragged ? all : n) + segments - 1) / segments);
  }
  for (int64_t l = 2; l <= 16; ++l) consider(l);
  *split = most_steps > 0;
  const int64_t L = most_steps * step;
  *seg_len = *split ? L : std::max<int64_t>(ragged ? T : mean, 1);
  *n_items = !*split ? B : ragged ? T / L + B : B * ((mean + L - 1) / L);
}

cudaError_t launch_linattn(const LinCall& c, cudaStream_t s) {
  if (c.form == kLinTc) return launch_lin_tc(c, s);
  if (c.form == kLinMma) return launch_lin_mma(c, s);
  return c.dt == kInF16 ? sweeps_of<__half>(c, s) : sweeps_of<float>(c, s);
}

cudaError_t launch_linattn_step(const LinStep& c, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(c.B), static_cast<unsigned>(c.H),
                  static_cast<unsigned>((c.dv + 127) / 128));
  if (c.dt == kInF16)
    lin_step_kernel<__half><<<grid, kStepThreads, 0, s>>>(c);
  else
    lin_step_kernel<float><<<grid, kStepThreads, 0, s>>>(c);
  return cudaGetLastError();
}

}  // namespace mmf
