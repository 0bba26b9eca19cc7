// Linear attention with a decay for each head on the tensor cores: chunks of 64 tokens, fp16.
//
// With S the state before a chunk of n tokens (rows i, j below), a, b the sweep's factors and lag 0
// forwards, 1 backwards (the decay then acts after a token):
//   P_ij  = a gamma^(i-j) q_i . k_j                    for j <= i, else 0
//   o_i   = b (gamma^(i+1-lag) S^T q_i + sum_j P_ij v_j)
//   S    <- gamma^n S + sum_j (a gamma^(n-1-j+lag) v_j) k_j^T
//
// Layout.  A block is four warps on one (segment, head, tile of DV columns).  A warp owns DV/4
// columns of the state and keeps them in registers, as fp32, in the accumulator layout of S^T
// (rows: columns of v; columns: those of k) for the whole segment.  That layout is at once the B
// operand of Q S after packing to fp16, so the state never goes through shared memory; Q, K, V
// and the scores P do, Q, K, V by 16-byte asynchronous copies a chunk ahead (rows past the end
// arrive as zeros), all swizzled for ldmatrix.
//
// Numbers.  Q, K and V are exact in fp16.  Three operands are rounded to fp16, each scaled by a
// power of two that brings its largest value to 2^14 .. 2^15: P (a power for each row, from its largest
// score), the state in Q S (one for each warp's columns and chunk), and the decayed V of the state's
// update (likewise).  So fp16's range does not matter, and its subnormals do for what is more than 2^28
// below the largest under the same power (in two parts, as the update's: more than 2^18).  P and the
// state cost a rounding of 2^-11 each, of different parts of an output that is rounded to 2^-11 itself.
// The decayed V is carried as two fp16 parts, 22 bits: the state is an fp32 output, and a third rounding
// would cost more than it saves (one part alone, measured: error against 64 bits 0.00035 instead of
// 0.00029, the output's own rounding being 0.00021).  All sums are fp32; the state takes a chunk's
// product in one fp32 rounding, so the tensor cores' own accumulation spans 64 tokens.
//
// What bounds it.  Heads of 64: 64 tokens are 32 KB, 0.7 us of an SM's share of the HBM; the products
// 0.5 us of mma.sync (555 TFLOP/s measured on this part).  Neither is reached: at 12 warps an SM the
// issue and latency of about 1800 instructions a warp and chunk are what counts (0.4 of a scheduler's
// slots).  Measured: 13 ragged prompts of 9001 tokens, 16 heads of 64, 41 us, their states 23, a call
// 71 us (with the registers for a fourth block on an SM, spilling, a tenth more; for two: as three,
// backward a fifth slower).  Four warps with a quarter of the columns each, because a warp with 32
// columns uses every operand it loads from Q, K and P twice: with 16 the loads would take as long as
// the products.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "linattn.cuh"
#include "linattn_dev.cuh"
#include "ptx.cuh"

namespace mmf {
namespace {

constexpr int kC = 64;            // tokens of a chunk
constexpr int kThreads = 128;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// The power of two that brings a magnitude (as the bits of a float) to 2^14 .. 2^15, as an exponent.
// Zeros take none; the limits keep products of two of them and an fp32 sum finite.
__device__ __forceinline__ int up_to_half(uint32_t bits, int most) {
  const int e = 14 + 127 - static_cast<int>(bits >> 23);
  return bits == 0u ? 0 : max(-60, min(e, most));
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Address of 16-byte vector `vec` of row `row` of a tile with kVecs vectors a row: the eight rows
// of a matrix that ldmatrix takes fall on the eight bank groups.
template <int kVecs>
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int row, int vec) {
  return base + static_cast<uint32_t>(row * kVecs + (vec ^ (row & 7))) * 16u;
}

template <int DK, int DV>
struct Tiles {
  static constexpr int kQ = kC * DK * 2;
  static constexpr int kV = kC * DV * 2;
  static constexpr int kP = kC * kC * 2;
  static constexpr int kStageOut = 2 * kQ + kV;     // Q, K, V
  static constexpr int kStageState = kQ + kV;       // K, V
  static constexpr int kStagesOut = 2;
  static constexpr int kStagesState = 3;
  static constexpr int kSmemOut = kStagesOut * kStageOut + kP;
  static constexpr int kSmemState = kStagesState * kStageState;
};

template <int DK, int DV, bool kState>
__global__ void __launch_bounds__(kThreads, DK == 128 ? 2 : 3)
lin_mma_kernel(const __grid_constant__ LinCall c, int sweep0, int tiles) {
  using L = Tiles<DK, DV>;
  constexpr int kStages = kState ? L::kStagesState : L::kStagesOut;
  constexpr int kStage = kState ? L::kStageState : L::kStageOut;
  constexpr int RV = DV / 4;          // state columns of v per warp
  constexpr int MT = RV / 16;         // as row tiles of S^T
  constexpr int NV = RV / 8;          // as column tiles of o
  constexpr int NK = DK / 8;          // column tiles of S^T
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float s_pow[kC + 1];     // gamma^0 .. gamma^64
  __shared__ int s_exp[kC];           // exponent of each row of P
  __shared__ LinTurns s_decay;

  const LinSweep& w = c.sw[sweep0 + blockIdx.z / tiles];
  const int h = blockIdx.y;
  if (!kState && blockIdx.z % tiles == 0) lin_clear<__half>(c, w, h);
  const LinSeg g = lin_find(c, blockIdx.x, w.backwards != 0);
  const bool whole = g.first && g.last;        // an unsplit sequence: nothing to start from
  if (!g.valid || (kState && whole)) return;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t4 = lane & 3;
  const int v0 = static_cast<int>(blockIdx.z % tiles) * DV + warp * RV;   // first column of v
  const int lag = w.backwards ? 1 : 0;
  const double lg2 = lin_lg2(c, h);
  if (tid <= kC) s_pow[tid] = lin_power(lg2, tid);

  const size_t state0 = (static_cast<size_t>(g.seq) * c.H + h) * w.dk * w.dv;
  float* seg = w.seg ? w.seg + (static_cast<size_t>(blockIdx.x) * c.H + h) * w.dk * w.dv : nullptr;
  float S[MT][NK][4];
  {
    const float* from = nullptr;
    size_t sk = 0, sv = 0;
    if (!kState && c.split && !whole) {
      from = seg;
      sk = static_cast<size_t>(w.dv);
      sv = 1;
    } else if (!kState && w.s0) {
      from = w.s0 + state0;
      sk = static_cast<size_t>(w.s_key);
      sv = static_cast<size_t>(w.s_val);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = v0 + 16 * m + gq + 8 * (e >> 1), col = 8 * n + 2 * t4 + (e & 1);
          const float x = from ? from[col * sk + row * sv] : 0.0f;
          S[m][n][e] = g.n > 0 ? lin_nan_if_inf(x) : x;
        }
  }
  float top = 0.0f;                   // largest magnitude of the state (but for NaN)
  if constexpr (!kState) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 4; e += 2) top = max3_abs(top, S[m][n][e], S[m][n][e + 1]);
  }

  const __half* kp = static_cast<const __half*>(w.k) + h * w.k_h;
  const __half* vp = static_cast<const __half*>(w.v) + h * w.v_h + (v0 - warp * RV);
  const __half* qp = static_cast<const __half*>(w.q) + h * w.q_h;
  __half* op = static_cast<__half*>(w.o) + h * w.o_h + v0;
  const uint32_t base = smem_u32(smem);
  auto tile_k = [&](int s) { return base + static_cast<uint32_t>(s * kStage); };
  auto tile_v = [&](int s) { return base + static_cast<uint32_t>(s * kStage + L::kQ); };
  auto tile_q = [&](int s) { return base + static_cast<uint32_t>(s * kStage + L::kQ + L::kV); };
  const uint32_t tile_p = base + static_cast<uint32_t>(kStages * kStage);

  const int64_t chunks = (g.n + kC - 1) / kC;
  // A thread's vectors of a tile: one column of vectors, rows a multiple of eight apart (so that the
  // swizzle is the same for all); pointers move on by a chunk at a time.
  constexpr int kRowsK = kThreads / (DK / 8), kRowsV = kThreads / (DV / 8);
  const int rk = tid / (DK / 8), rv = tid / (DV / 8);
  const uint32_t at_k = tile_at<DK / 8>(0u, rk, tid % (DK / 8));
  const uint32_t at_v = tile_at<DV / 8>(0u, rv, tid % (DV / 8));
  const __half* next_k = kp + g.token(rk) * w.k_t + tid % (DK / 8) * 8;
  const __half* next_q = qp + g.token(rk) * w.q_t + tid % (DK / 8) * 8;
  const __half* next_v = vp + g.token(rv) * w.v_t + tid % (DV / 8) * 8;
  const int64_t step_k = g.step * kRowsK * w.k_t, step_q = g.step * kRowsK * w.q_t;
  const int64_t step_v = g.step * kRowsV * w.v_t;
  auto load = [&](int64_t chunk) {
    if (chunk < chunks) {
      const int s = static_cast<int>(chunk % kStages);
      const int left = static_cast<int>(min(static_cast<int64_t>(kC), g.n - chunk * kC));
#pragma unroll
      for (int i = 0; i < kC / kRowsK; ++i) {
        const bool in = rk + i * kRowsK < left;
        const uint32_t at = at_k + static_cast<uint32_t>(i * kRowsK * DK * 2);
        cp_async16(tile_k(s) + at, in ? next_k + i * step_k : kp, in);
        if constexpr (!kState) cp_async16(tile_q(s) + at, in ? next_q + i * step_q : qp, in);
      }
#pragma unroll
      for (int i = 0; i < kC / kRowsV; ++i) {
        const bool in = rv + i * kRowsV < left;
        cp_async16(tile_v(s) + at_v + static_cast<uint32_t>(i * kRowsV * DV * 2),
                   in ? next_v + i * step_v : vp, in);
      }
      next_k += (kC / kRowsK) * step_k;
      next_q += (kC / kRowsK) * step_q;
      next_v += (kC / kRowsV) * step_v;
    }
    cp_async_commit();   // (possibly empty) one group for each chunk
  };
  // matrices of an ldmatrix.x4, by lane: row in the low three bits, which matrix above
  const int lr = lane & 7, lm = lane >> 3;

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i);
  if (tid == 0) s_decay = LinTurns(lg2, kC, static_cast<int>(g.n % kC));
  for (int64_t chunk = 0; chunk < chunks; ++chunk) {
    const int s = static_cast<int>(chunk % kStages);
    const int n = static_cast<int>(min(static_cast<int64_t>(kC), g.n - chunk * kC));
    cp_async_wait<kStages - 2>();
    __syncthreads();                  // the chunk is in, and the one before it is done with
    load(chunk + kStages - 1);
    const float decay = n < kC ? s_decay.last : s_decay.of(static_cast<int>(chunk));
    bool strange = false;             // the warp's part of V has a value that is not finite

    if constexpr (!kState) {
      // ---- scores: warp = 16 rows, the column tiles up to its diagonal
      {
        float P[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) P[j][e] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
          uint32_t a[4];
          ldsm4(a, tile_at<DK / 8>(tile_q(s), 16 * warp + lr + 8 * (lm & 1), 2 * kk + (lm >> 1)));
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            if (j <= 2 * warp) {
              uint32_t b[4];
              ldsm4(b, tile_at<DK / 8>(tile_k(s), 8 * j + lr + 8 * (lm >> 1), 2 * kk + (lm & 1)));
              mma16816(P[j], a, b[0], b[1]);
              mma16816(P[j + 1], a, b[2], b[3]);
            }
          }
        }
        float m[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 16 * warp + gq + 8 * (e >> 1), d = i - (8 * j + 2 * t4 + (e & 1));
            // not a product with 0: the score of a later token may be anything
            P[j][e] = d >= 0 ? P[j][e] * (w.a * s_pow[d]) : 0.0f;
            if (e & 1) m[e >> 1] = max3_abs(m[e >> 1], P[j][e - 1], P[j][e]);
          }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 1));
          m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 2));
          const int row = 16 * warp + gq + 8 * r;
          const int e = up_to_half(__float_as_uint(m[r]), 40);
          const float f = pow2(e);
          if (t4 == 0) s_exp[row] = e;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j <= 2 * warp + 1)
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(tile_at<8>(tile_p, row, j) + 4u * t4),
                           "r"(pack2(P[j][2 * r] * f, P[j][2 * r + 1] * f))
                           : "memory");
        }
      }

      // ---- Q S for the warp's columns, the state packed as it is needed
      float O[4][NV][4];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[m][v][e] = 0.0f;
      const int es = up_to_half(__reduce_max_sync(0xffffffffu, __float_as_uint(top)), 60);
      const float fs = pow2(es);
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        uint32_t b[NV][2];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float* x = S[v >> 1][2 * kk + z] + 2 * (v & 1);
            b[v][z] = pack2(x[0] * fs, x[1] * fs);
          }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint32_t a[4];
          ldsm4(a, tile_at<DK / 8>(tile_q(s), 16 * m + lr + 8 * (lm & 1), 2 * kk + (lm >> 1)));
#pragma unroll
          for (int v = 0; v < NV; ++v) mma16816(O[m][v], a, b[v][0], b[v][1]);
        }
      }
      __syncthreads();                // P and its exponents are in

      // ---- bring the rows to P's scale, then add P V
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = 16 * m + gq + 8 * r;
          const float f = s_pow[i + 1 - lag] * pow2(max(-126, min(127, s_exp[i] - es)));
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            O[m][v][2 * r] *= f;
            O[m][v][2 * r + 1] *= f;
          }
        }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t b[NV / 2][4];
        __half2 sum = __float2half2_rn(0.0f);   // 0 times what is not finite is NaN
#pragma unroll
        for (int v = 0; v < NV / 2; ++v) {
          ldsm4t(b[v], tile_at<DV / 8>(tile_v(s), 16 * kk + lr + 8 * (lm & 1),
                                       warp * (RV / 8) + 2 * v + (lm >> 1)));
#pragma unroll
          for (int z = 0; z < 4; ++z)
            sum = __hfma2(*reinterpret_cast<const __half2*>(&b[v][z]), __float2half2_rn(0.0f), sum);
        }
        const bool odd = __any_sync(0xffffffffu, !__hbeq2(sum, __float2half2_rn(0.0f)));
        strange |= odd;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m < kk) continue;
          uint32_t a[4];
          ldsm4(a, tile_at<8>(tile_p, 16 * m + lr + 8 * (lm & 1), 2 * kk + (lm >> 1)));
          if (m == kk && odd) {
            // 0 times an infinity or a NaN of a later token is not 0: on the diagonal such tokens
            // are added one at a time, to the rows from their own on
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {
#pragma unroll
              for (int v = 0; v < NV; ++v) {
                uint32_t x[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const int k0 = 2 * t4 + 8 * z;   // the two tokens of this register
                  const uint32_t keep = (k0 == j ? 0xffffu : 0u) | (k0 + 1 == j ? 0xffff0000u : 0u);
                  x[z] = b[v >> 1][2 * (v & 1) + z] & keep;
                }
                float y[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816(y, a, x[0], x[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (gq + 8 * (e >> 1) >= j) O[m][v][e] += y[e];
              }
            }
          } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
              mma16816(O[m][v], a, b[v >> 1][2 * (v & 1)], b[v >> 1][2 * (v & 1) + 1]);
          }
        }
      }
      __half* o_row = op + g.token(chunk * kC + gq) * w.o_t + 2 * t4;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = 16 * m + gq + 8 * r;
          if (i < n) {
            const float f = w.b * pow2(-s_exp[i]);
            __half* row = o_row + (2 * m + r) * (8 * g.step * w.o_t);
#pragma unroll
            for (int v = 0; v < NV; ++v)
              *reinterpret_cast<uint32_t*>(row + 8 * v) =
                  pack2(O[m][v][2 * r] * f, O[m][v][2 * r + 1] * f);
          }
        }
      if (chunk + 1 == chunks && !(whole && w.sT != nullptr)) break;   // no more readers
    }

    // ---- the state's update
    uint32_t hi[4][MT][4], lo[4][MT][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        // rows of S^T (columns of v) in the low bit of the matrix, tokens in the high one
        ldsm4t(hi[kk][m], tile_at<DV / 8>(tile_v(s), 16 * kk + lr + 8 * (lm >> 1),
                                          warp * (RV / 8) + 2 * m + (lm & 1)));
    // Their decay, in fp16 pairs of tokens: with a factor w 2^e = wh + wl, hi = v wh rounded and lo
    // the rest (v wh - hi, exact, plus v wl), an error of about 2^-22.  e brings the warp's largest
    // product to 2^14 .. 2^15, or the largest factor of a token that is not zero if that is less.
    auto weight = [&](int j) { return w.a * s_pow[max(n - 1 - j + lag, 0)]; };   // v is 0 past n
    float vtop = 0.0f, wide = 0.0f;
    auto scan = [&](auto clean) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          __half2 m2 = __float2half2_rn(0.0f);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t u = hi[kk][m][2 * z + y];
              if constexpr (clean.value)
                u &= ((u & 0x7c00u) == 0x7c00u ? 0u : 0xffffu) |
                     ((u & 0x7c000000u) == 0x7c000000u ? 0u : 0xffff0000u);
              m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __half2*>(&u)));
            }
          const float2 x = __half22float2(m2);
          const int j = 16 * kk + 2 * t4 + 8 * z;
          const float w0 = fabsf(weight(j)), w1 = fabsf(weight(j + 1));
          vtop = fmaxf(vtop, fmaxf(x.x * w0, x.y * w1));
          wide = fmaxf(wide, fmaxf(x.x != 0.0f ? w0 : 0.0f, x.y != 0.0f ? w1 : 0.0f));
        }
    };
    if constexpr (kState) {
      __half2 check = __float2half2_rn(0.0f);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int z = 0; z < 4; ++z)
            check = __hfma2(*reinterpret_cast<const __half2*>(&hi[kk][m][z]), __float2half2_rn(0.0f), check);
      strange = __any_sync(0xffffffffu, !__hbeq2(check, __float2half2_rn(0.0f)));
    }
    // the scale comes from what is finite: the rest stays as it is under any
    if (strange)
      scan(std::true_type{});
    else
      scan(std::false_type{});
    const int ev = min(up_to_half(__reduce_max_sync(0xffffffffu, magnitude(vtop)), 60),
                       up_to_half(__reduce_max_sync(0xffffffffu, magnitude(wide)), 60));
    const float fv = pow2(ev);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int j = 16 * kk + 2 * t4 + 8 * z;
        const float w0 = weight(j) * fv, w1 = weight(j + 1) * fv;
        const __half2 wh = lin_half2_finite(w0, w1);
        const float2 r = __half22float2(wh);
        const __half2 wl = lin_half2_finite(w0 - r.x, w1 - r.y);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const __half2 v2 = *reinterpret_cast<const __half2*>(&hi[kk][m][2 * z + y]);
            const __half2 h2 = __hmul2(v2, wh);
            hi[kk][m][2 * z + y] = *reinterpret_cast<const uint32_t*>(&h2);
            const __half2 l2 = __hfma2(v2, wl, __hfma2(v2, wh, __hneg2(h2)));
            lo[kk][m][2 * z + y] = *reinterpret_cast<const uint32_t*>(&l2);
          }
      }
    const float back = pow2(-ev);
    top = 0.0f;
    constexpr int NG = 4;             // column tiles of S^T at a time
#pragma unroll
    for (int n0 = 0; n0 < NK; n0 += NG) {
      float D[MT][NG][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < NG; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) D[m][x][e] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int x = 0; x < NG; x += 2) {
          uint32_t b[4];
          ldsm4t(b, tile_at<DK / 8>(tile_k(s), 16 * kk + lr + 8 * (lm & 1), n0 + x + (lm >> 1)));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma16816(D[m][x], hi[kk][m], b[0], b[1]);
            mma16816(D[m][x + 1], hi[kk][m], b[2], b[3]);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma16816(D[m][x], lo[kk][m], b[0], b[1]);
            mma16816(D[m][x + 1], lo[kk][m], b[2], b[3]);
          }
        }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < NG; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& y = S[m][n0 + x][e];
            y = fmaf(decay, y, D[m][x][e] * back);
            if constexpr (!kState) {
              if (e & 1) top = max3_abs(top, S[m][n0 + x][e - 1], y);
            }
          }
    }
  }
  cp_async_wait<0>();

  float* to = nullptr;
  size_t sk, sv;
  if (kState) {
    to = seg;
    sk = static_cast<size_t>(w.dv);
    sv = 1;
  } else {
    if (!whole || !w.sT) return;
    to = w.sT + state0;
    sk = static_cast<size_t>(w.s_key);
    sv = static_cast<size_t>(w.s_val);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = v0 + 16 * m + gq + 8 * (e >> 1), col = 8 * n + 2 * t4 + (e & 1);
        to[col * sk + row * sv] = S[m][n][e];
      }
}

template <int DK, int DV>
cudaError_t launch(const LinCall& c, int sweep0, int n, bool state, cudaStream_t s) {
  using L = Tiles<DK, DV>;
  static std::once_flag once[kMaxDevices];
  static cudaError_t attr[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    attr[dev] = cudaFuncSetAttribute(lin_mma_kernel<DK, DV, false>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemOut);
    if (attr[dev] == cudaSuccess)
      attr[dev] = cudaFuncSetAttribute(lin_mma_kernel<DK, DV, true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemState);
  });
  if (attr[dev] != cudaSuccess) return attr[dev];
  const int tiles = c.sw[sweep0].dv / DV;
  const dim3 grid(static_cast<unsigned>(c.n_items), static_cast<unsigned>(c.H),
                  static_cast<unsigned>(tiles * n));
  if (state)
    lin_mma_kernel<DK, DV, true><<<grid, kThreads, L::kSmemState, s>>>(c, sweep0, tiles);
  else
    lin_mma_kernel<DK, DV, false><<<grid, kThreads, L::kSmemOut, s>>>(c, sweep0, tiles);
  return cudaGetLastError();
}

cudaError_t launch_sizes(const LinCall& c, int sweep0, int n, bool state, cudaStream_t s) {
  const int dk = c.sw[sweep0].dk, dv = c.sw[sweep0].dv;
  if (dk == 64) return dv % 128 == 0 ? launch<64, 128>(c, sweep0, n, state, s)
                                     : launch<64, 64>(c, sweep0, n, state, s);
  return dv % 128 == 0 ? launch<128, 128>(c, sweep0, n, state, s)
                       : launch<128, 64>(c, sweep0, n, state, s);
}

// Sweeps of the same sizes go in one launch.
cudaError_t launch_all(const LinCall& c, bool state, cudaStream_t s) {
  for (int i = 0; i < c.n_sweeps;) {
    int n = 1;
    while (i + n < c.n_sweeps && c.sw[i + n].dk == c.sw[i].dk && c.sw[i + n].dv == c.sw[i].dv) ++n;
    cudaError_t e = launch_sizes(c, i, n, state, s);
    if (e != cudaSuccess) return e;
    i += n;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_lin_mma(const LinCall& c, cudaStream_t s) {
  if (c.split) {
    cudaError_t e = launch_all(c, true, s);
    if (e == cudaSuccess) e = launch_lin_join(c, s);
    if (e != cudaSuccess) return e;
  }
  return launch_all(c, false, s);
}

}  // namespace mmf
