// Linear attention with a decay for each head on the 5th-generation tensor cores (tcgen05,
// kind::f16): fp16 heads of 128 x 128, chunks of 128 tokens, one block on an SM.
//
// The arithmetic of a chunk (q_i, k_j, v_j: its tokens in the sweep's order, n of them; S the state
// before it; lag 0 forwards, 1 backwards):
//   P_ij  = a gamma^(i-j) q_i . k_j                     for j <= i, else 0
//   o_i   = b (gamma^(i+1-lag) S^T q_i + sum_j P_ij v_j)
//   S    <- gamma^n S + sum_j (a gamma^(n-1-j+lag) k_j) v_j^T
// as four products of 128 x 128 x 128:
//   Q K^T (both as loaded) -> P,  Q S -> o_i's first part,  P V (P from TMEM) -> its second part,
//   V^T K' with K' the decayed K (contracted over the tokens: both operands "MN-major").
// All operands sit in shared memory as the 128-byte-swizzled tiles that TMA writes, so the same
// image of K serves Q K^T (K-major) and V^T K' (MN-major), and V likewise.
//
// Warps: 0 TMA, 1 TMEM and MMA issue; then groups of four, a thread for each row of their tile:
// 4-7 the state's (row = column of v; its 128 values stay in the thread's registers), 8-11 K -> K',
// 12-15 and 16-19 the tokens' (scores and outputs), taking turns at the chunks, so that one's
// outputs overlap the other's scores.  Registers go from the first group to the state's.
// K' has two fp16 parts (22 bits), so that the state, an fp32 output, keeps its precision; the first
// overwrites K once Q K^T is done.  Shared memory, 32 KB each: two stages of K and V, the second
// part of K', Q (loaded again as soon as Q S is done), the fp16 state.  TMEM: P, Q S, P V, V^T K', 128
// columns each; the fp16 P overwrites P.  Loops over blocks of columns are not unrolled: the groups' code
// together has to stay in the instruction cache.
//
// Numbers: as in the register form of this sweep (linattn_mma.cu): Q, K, V exact; P, the state and
// K' scaled by powers of two (a row's, the whole state's, the chunk's) before they are rounded, and what
// is more than 2^28 (K': 2^18) below the largest under its power loses bits to fp16's subnormals.  P's
// power comes from a bound, some 2^10 above the scores, so 2^18 there too.  The state takes a chunk's
// product in one fp32 rounding.
//
// A v that is not finite would reach earlier tokens through P V as 0 times infinity.  Such values
// are replaced by zero on arrival and their place is noted: from that token on the column's
// outputs and state are NaN.
//
// kState: the state alone (pass one of a split sequence).  There the tokens' two groups turn K into
// K', a panel of 64 columns each, and the group for it looks after V.
//
// What bounds it.  Bytes that the sweep cannot do without: 128 KB a chunk (3 us of an SM's share of
// the HBM).  Five products of 512 cycles on the tensor pipe, which read both operands from shared
// memory at all of its bandwidth, and about 1800 cycles more of that for the conversions: no unit is
// full, the hand-overs between them and the fetch of the roles' code fill the rest.  Measured: 4.4 us
// a chunk, 5.0 where every row comes from HBM; 32768 tokens of 16 heads in 150 us, their states alone
// (kState, 64 KB a chunk) in 68; whole call 240 us (a register form on mma.sync: 553, two of its waves;
// token by token: 2991).
//
// Every wait is bounded; on a timeout the block records kStatusTimeout, every role stops, the
// copies and MMAs in flight are drained and TMEM is freed.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "linattn.cuh"
#include "linattn_dev.cuh"
#include "ptx.cuh"

namespace mmf {
namespace {

constexpr int kD = 128;                      // head size, k and v
constexpr int kC = 128;                      // tokens of a chunk
constexpr int kPanel = kC * 128;             // 128 rows x 64 fp16
constexpr int kTile = 2 * kPanel;            // 32 KB
constexpr int kThreads = 640;
// Registers of the groups' threads; together 5 * 96, what the block is launched with.
constexpr int kRegsIssue = 40, kRegsState = 184, kRegsDecay = 64, kRegsRows = 96;
static_assert(kRegsIssue + kRegsState + kRegsDecay + 2 * kRegsRows <= 5 * 96, "registers");
constexpr int kKeyBits = 6;                  // keys of a chunk that count as alike
constexpr int kGroup = 128;                  // threads of the state warps, and of the row warps
constexpr uint64_t kDrainNs = 2000000000ull;

template <bool kState>
struct Lay {
  static constexpr int kStages = 2;
  // kState: a stage is K, V and the second part of K'
  static constexpr int kStage = (kState ? 3 : 2) * kTile;
  static constexpr int kLo = kState ? 2 * kTile : kStages * kStage;   // kState: within the stage
  static constexpr int kQ = kLo + kTile;
  static constexpr int kS = kQ + kTile;
  static constexpr int kSmem = 1024 + (kState ? kStages * kStage : kS + kTile);
  static constexpr int kCols = kState ? 128 : 512;
};

// kind::f16, fp32 accumulator, fp16 operands, M = N = 128; bits 15 and 16: A and B MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((kD / 8) << 17) |
         ((kC / 16) << 24);
}

// Descriptor of an MN-major operand: 64 values of M or N are the 128 bytes of a swizzled row, the
// contraction runs over the rows.  Leading offset: to the next 64 values (the second panel);
// stride offset: to the next eight rows.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(kPanel >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Products of 128 x 128 x 128: eight MMAs of depth 16, issued by one elected lane of a converged
// warp.  Offsets are in 16-byte units of shared memory (TMEM: columns).
// Both K-major: 16 values are 32 bytes of a row, 64 a panel.
__device__ __forceinline__ void product_kk(uint32_t d, uint32_t a, uint32_t b) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b;\n\t.reg .b64 a;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 1024;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 1026;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 1028;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 1030;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d),
      "l"(smem_desc_kmajor_sw128(a)), "l"(smem_desc_kmajor_sw128(b)), "r"(idesc_f16(false, false)), "r"(0)
      : "memory");
}
// Both MN-major: contraction over the tiles' 128 rows, 16 of them 2048 bytes.
__device__ __forceinline__ void product_mn(uint32_t d, uint32_t a, uint32_t b, int add) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b;\n\t.reg .b64 a;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a, %1, 128;\n\tadd.s64 b, %2, 128;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 256;\n\tadd.s64 b, %2, 256;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 384;\n\tadd.s64 b, %2, 384;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 512;\n\tadd.s64 b, %2, 512;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 640;\n\tadd.s64 b, %2, 640;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 768;\n\tadd.s64 b, %2, 768;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 896;\n\tadd.s64 b, %2, 896;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d),
      "l"(desc_mn(a)), "l"(desc_mn(b)), "r"(idesc_f16(true, true)), "r"(add)
      : "memory");
}
// A in TMEM (16 fp16 are eight columns), B MN-major.
__device__ __forceinline__ void product_tm(uint32_t d, uint32_t a, uint32_t b) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 32;\n\tadd.s64 b, %2, 512;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 40;\n\tadd.s64 b, %2, 640;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 48;\n\tadd.s64 b, %2, 768;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 56;\n\tadd.s64 b, %2, 896;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(desc_mn(b)), "r"(idesc_f16(false, true)), "r"(0)
      : "memory");
}

__device__ __forceinline__ void st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Exponent of the power of two that brings a magnitude to 2^14 .. 2^15; zeros take none.
__device__ __forceinline__ int up_to_half(float top) {
  return top == 0.0f ? 0 : max(-100, min(14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 100));
}
__device__ __forceinline__ float warp_max(float magnitude) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(magnitude)));
}
template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
  return m;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Row r of a two-panel tile, and its 16-byte vector x (0..15): in a swizzled row of 128 bytes vector
// x is at x ^ (r mod 8), so that its address is the row's with three bits flipped.
__device__ __forceinline__ uint32_t row_at(uint32_t tile, int r) {
  return tile + static_cast<uint32_t>(r * 128 + ((r & 7) << 4));
}
__device__ __forceinline__ uint32_t vec_of(uint32_t row, int x) {
  return (row ^ static_cast<uint32_t>((x & 7) << 4)) + static_cast<uint32_t>((x >> 3) * kPanel);
}

template <int N>
__device__ __forceinline__ float min_of(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fminf(m, x[i]);
  return m;
}

// Tensor maps of each sweep's k, v and q.
struct LinMaps {
  CUtensorMap m[3 * kMaxSweeps];
};

// A wait of at most kTries tries, each of which may suspend the warp for up to kTryNs, so that
// waiting warps leave the issue slots and the shared-memory pipe to the working ones.
constexpr int kTries = 1 << 17;
constexpr uint32_t kTryNs = 20000;
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kTryNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort,
                                             unsigned* status) {
  int left = kTries;
  while (!try_wait(bar, parity)) {
    if (--left == 0) {
      *abort = 1;
      atomicOr(status, kStatusTimeout);
    }
    if (*abort) return false;
  }
  return true;
}

// A wait names a phase by its parity, so whoever waits must come before the phase after the next
// has completed, and not before the phase before has.  Barriers with two places (the even and the
// odd chunks') are handed over by groups that can run a chunk ahead of the waiting one, or are
// waited for every other chunk; stages are reused only after every hand-over of their chunk, which
// keeps either from getting two chunks ahead.
struct Bars {
  uint64_t full[2], empty[2];
  uint64_t scores[2], p[2], out[2], drained[2], k[2], v[2], state[2];
  uint64_t q_full[2];
  uint64_t q_read, qk, upd, drain;
};

template <bool kState>
struct Shared {
  Bars bars;
  float pow[kC + 4];        // gamma^0 .. gamma^128
  LinTurns decay;
  // diag[32 - row + column], from 3 on forwards: gamma^(i-j) of a diagonal block, 0 if j > i.  In it stand also a
  // column's powers of the blocks before, gamma^(31-j) forwards, gamma^j backwards, 16-byte aligned
  alignas(16) float diag[68];
  float red_k[2][kState ? 8 : 4], red_w[2][kState ? 8 : 4], red_s[4];   // of each warp (a panel's four)
  float top_k[2][4], low_k[2][4];   // largest magnitudes of rows of K: the largest and the least of each warp
  uint8_t key[2][kC];               // and each as the exponent of a power of two that it does not pass
  int exp_s[2];             // exponent of the fp16 state, by chunk
  int exp_k[4];             // of K'
  int bad_at[kD];           // first position of the segment whose v is not finite, by column
  int any_bad;
  uint32_t tmem;
  int abort;
};
static_assert(Lay<false>::kSmem + sizeof(Shared<false>) <= 227 * 1024, "shared memory per block");
static_assert(Lay<true>::kSmem + sizeof(Shared<true>) <= 227 * 1024, "shared memory per block");

template <bool kState>
__global__ void __launch_bounds__(kThreads, 1)
lin_tc_kernel(const __grid_constant__ LinCall c, const __grid_constant__ LinMaps maps) {
  using L = Lay<kState>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<kState> sh;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto tile_k = [&](int s) { return base + static_cast<uint32_t>(s * L::kStage); };
  auto tile_v = [&](int s) { return base + static_cast<uint32_t>(s * L::kStage + kTile); };
  auto tile_lo = [&](int s) { return base + static_cast<uint32_t>((kState ? s * L::kStage : 0) + L::kLo); };
  const uint32_t tile_q = base + static_cast<uint32_t>(L::kQ);
  const uint32_t tile_s = base + static_cast<uint32_t>(L::kS);

  const int sweep = blockIdx.z, h = blockIdx.y;
  const LinSweep& w = c.sw[sweep];
  if (!kState) lin_clear<__half>(c, w, h);
  const LinSeg g = lin_find(c, blockIdx.x, w.backwards != 0);
  const bool whole = g.first && g.last;
  if (!g.valid || (kState && whole)) return;

  // (broadcast, so that the roles' branches are known to be the same for a whole warp)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool back = w.backwards != 0;
  const int lag = back ? 1 : 0;
  const int chunks = static_cast<int>((g.n + kC - 1) / kC);
  const CUtensorMap* mk = &maps.m[3 * sweep];
  const CUtensorMap* mv = &maps.m[3 * sweep + 1];
  const CUtensorMap* mq = &maps.m[3 * sweep + 2];

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.bars.full[s]), 1);
      mbar_init(smem_u32(&sh.bars.empty[s]), 1);
      mbar_init(smem_u32(&sh.bars.scores[s]), 1);
      mbar_init(smem_u32(&sh.bars.p[s]), 4);
      mbar_init(smem_u32(&sh.bars.out[s]), 1);
      mbar_init(smem_u32(&sh.bars.drained[s]), 4);
      mbar_init(smem_u32(&sh.bars.k[s]), kState ? 8 : 4);
      mbar_init(smem_u32(&sh.bars.v[s]), 4);
      mbar_init(smem_u32(&sh.bars.state[s]), 4);
      mbar_init(smem_u32(&sh.bars.q_full[s]), 1);
    }
    mbar_init(smem_u32(&sh.bars.q_read), 4);
    mbar_init(smem_u32(&sh.bars.qk), 1);
    mbar_init(smem_u32(&sh.bars.upd), 1);
    mbar_init(smem_u32(&sh.bars.drain), 1);
    sh.abort = 0;
    sh.any_bad = 0;
    fence_mbar_init();
    tma_prefetch_desc(mk);
    tma_prefetch_desc(mv);
    if (!kState) tma_prefetch_desc(mq);
  }
  if (tid <= kC) sh.pow[tid] = lin_power(lin_lg2(c, h), tid);
  if (!kState && tid < 64) {
    const int d = back ? tid - 32 : 32 - tid;
    sh.diag[(back ? 0 : 3) + tid] = d >= 0 ? lin_power(lin_lg2(c, h), d) : 0.0f;
  }
  if (tid == kThreads - 1) sh.decay = LinTurns(lin_lg2(c, h), kC, static_cast<int>(g.n % kC));
  if (tid < kD) sh.bad_at[tid] = 0x7fffffff;
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), L::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t t_p = tmem, t_qs = tmem + 128, t_pv = tmem + 256, t_upd = tmem + (kState ? 0 : 384);
  volatile int* abort_flag = &sh.abort;
  // waits of a whole warp, with one outcome
  auto wait = [&](uint64_t& bar, int parity) {
    return __all_sync(0xffffffffu, wait_bounded(smem_u32(&bar), static_cast<uint32_t>(parity),
                                                abort_flag, c.status));
  };
  auto arrive = [&](uint64_t& bar) {   // once for the warp, after all its lanes
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar));
  };
  // first token row of a chunk's tile: rows ascend with the tokens in both directions
  auto row0 = [&](int chunk) {
    return g.begin + (back ? -(static_cast<int64_t>(chunk) * kC + kC - 1) : static_cast<int64_t>(chunk) * kC);
  };
  auto tokens = [&](int chunk) {
    return static_cast<int>(min(static_cast<int64_t>(kC), g.n - static_cast<int64_t>(chunk) * kC));
  };

  // Thread r of a group of four warps: row r of V made safe for the products: zeros where the row is
  // no token of the segment and where a value is not finite.
  auto clean_v = [&](int chunk, int r) {
    const int pos = back ? kC - 1 - r : r;
    const uint32_t row = row_at(tile_v(chunk & 1), r);
    if (pos >= tokens(chunk)) {
#pragma unroll 1
      for (int x = 0; x < 16; ++x) sts128(vec_of(row, x), make_uint4(0u, 0u, 0u, 0u));
    } else {
      // 0 times what is not finite is NaN
      __half2 odd[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) odd[e] = __float2half2_rn(0.0f);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const uint4 v = lds128(vec_of(row, x));
        const __half2* hv = reinterpret_cast<const __half2*>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) odd[e] = __hfma2(hv[e], __float2half2_rn(0.0f), odd[e]);
      }
      const float2 sum = __half22float2(__hadd2(__hadd2(odd[0], odd[1]), __hadd2(odd[2], odd[3])));
      if (!(sum.x + sum.y == 0.0f)) {
#pragma unroll 1
        for (int col = 0; col < kD; ++col) {
          const uint32_t a = vec_of(row, col >> 3) + 2u * (col & 7);
          uint16_t x;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a) : "memory");
          if ((x & 0x7c00u) == 0x7c00u) {
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(0)) : "memory");
            atomicMin(&sh.bad_at[col], chunk * kC + pos);
            sh.any_bad = 1;
          }
        }
      }
    }
    fence_proxy_async_smem();
  };
  // Largest magnitude in row r of a tile of K or Q, infinity or NaN if one of it is not finite.
  constexpr int kVecs = kState ? 8 : 16;   // vectors of a row that a thread takes (kState: a panel)
  auto row_top = [&](uint32_t row) {
    __half2 m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = __float2half2_rn(0.0f);
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {
      const uint4 v = lds128(vec_of(row, x));
      const __half2* hv = reinterpret_cast<const __half2*>(&v);
#pragma unroll
      for (int e = 0; e < 4; ++e) m[e] = __hmax2_nan(m[e], __habs2(hv[e]));
    }
    const float2 y = __half22float2(__hmax2_nan(__hmax2_nan(m[0], m[1]), __hmax2_nan(m[2], m[3])));
    return y.x >= y.y || y.x != y.x ? y.x : y.y;
  };
  // Row r of K' from row r of K: a gamma^(tokens after it) k_j in two fp16 parts, scaled by the
  // chunk's power of two.  With the factor w 2^e = wh + wl in fp16, hi = k wh rounded, and the rest
  // (k wh - hi, exact, plus k wl) is lo: three half2 operations, an error of about 2^-22.  e brings
  // the largest product to 2^14 .. 2^15, or the largest factor of a row that is not zero there if
  // that is less.
  // find_exp: e and row r's factor w 2^e; false if one of the warps gave up (`ok`).  Named barrier `id` is
  // that of the threads that share the tile: a group, or two with a panel each.
  auto find_exp = [&](int chunk, int r, int panel, int id, bool ok, float* f) {
    const int set = chunk & 1;   // written again only after all of them handed the chunk over
    const int n = tokens(chunk), pos = back ? kC - 1 - r : r;
    const bool in = pos < n;
    const float wt = in ? w.a * sh.pow[n - 1 - pos + lag] : 0.0f;
    float top = 0.0f;
    if (ok && in) top = row_top(row_at(tile_k(chunk & 1) + panel * kPanel, r));
    if (!(top <= 65504.0f)) {
      // the scales come from what is finite: the rest stays as it is under any of them
      sh.any_bad = 1;
      top = 0.0f;
      const uint32_t row = row_at(tile_k(chunk & 1) + panel * kPanel, r);
#pragma unroll 1
      for (int x = 0; x < 8 * kVecs; ++x) {
        uint16_t y;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(y) : "r"(vec_of(row, x >> 3) + 2u * (x & 7)) : "memory");
        if ((y & 0x7c00u) != 0x7c00u) top = fmaxf(top, fabsf(__half2float(__ushort_as_half(y))));
      }
    }
    const float wide = warp_max(top != 0.0f ? fabsf(wt) : 0.0f);
    if constexpr (!kState) sh.key[set][r] = static_cast<uint8_t>((__float_as_uint(top) + 0x7fffffu) >> 23);
    const float most = kState ? 0.0f : warp_max(top);
    const float least =
        kState ? 0.0f : __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(in ? top : 65504.0f)));
    top = warp_max(top * fabsf(wt));
    if (lane == 0) {
      const int at = (r >> 5) + 4 * panel;
      sh.red_k[set][at] = top;
      sh.red_w[set][at] = wide;
      if constexpr (!kState) {
        sh.top_k[set][at] = most;
        sh.low_k[set][at] = least;
      }
    }
    if (!named_bar_and(id, kState ? 2 * kGroup : kGroup, ok)) return false;
    const int e = min(up_to_half(max_of(sh.red_k[set])), up_to_half(max_of(sh.red_w[set])));
    if (r == 0 && panel == 0) sh.exp_k[chunk & 3] = e;
    *f = wt * pow2(e);
    return true;
  };
  auto decay_k = [&](int chunk, int r, int panel, float f) {
    const uint32_t row = row_at(tile_k(chunk & 1) + panel * kPanel, r);
    const uint32_t row2 = row_at(tile_lo(chunk & 1) + panel * kPanel, r);
    const bool in = (back ? kC - 1 - r : r) < tokens(chunk);
    const __half2 wh = lin_half2_finite(f, f);
    const float rest = f - __low2float(wh);
    const __half2 wl = lin_half2_finite(rest, rest);
#pragma unroll
    for (int x0 = 0; x0 < kVecs; x0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = lds128(vec_of(row, x0 + x));
      if (!in)
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        uint4 hi, lo;
        const __half2* k2 = reinterpret_cast<const __half2*>(&v[x]);
        __half2* h2 = reinterpret_cast<__half2*>(&hi);
        __half2* l2 = reinterpret_cast<__half2*>(&lo);
#pragma unroll
        for (int i = 0; i < 4; ++i) h2[i] = __hmul2(k2[i], wh);
        sts128(vec_of(row, x0 + x), hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) l2[i] = __hfma2(k2[i], wl, __hfma2(k2[i], wh, __hneg2(h2[i])));
        sts128(vec_of(row2, x0 + x), lo);
      }
    }
    fence_proxy_async_smem();
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------------------------- TMA
      const uint64_t pol = l2_policy_evict_normal();
      auto col = [&](int64_t stride) { return static_cast<int32_t>(h * stride); };
      int issued = 0, q_issued = 0;
      for (int ch = 0; ch < chunks; ++ch) {
        const int s = ch & 1;
        if (ch >= 2 && !wait_bounded(smem_u32(&sh.bars.empty[s]), ((ch >> 1) - 1) & 1, abort_flag,
                                     c.status))
          break;
        const uint32_t bar = smem_u32(&sh.bars.full[s]);
        mbar_arrive_expect_tx(bar, 2 * kTile);
        const int32_t y = static_cast<int32_t>(row0(ch));
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          tma_load_2d(tile_k(s) + p * kPanel, mk, bar, col(w.k_h) + 64 * p, y, pol);
          tma_load_2d(tile_v(s) + p * kPanel, mv, bar, col(w.v_h) + 64 * p, y, pol);
        }
        issued = ch + 1;
        if constexpr (!kState) {
          // Q has one place: the products and the row warps are done with the chunk before
          if (ch > 0 && (!wait_bounded(smem_u32(&sh.bars.qk), (ch - 1) & 1, abort_flag, c.status) ||
                         !wait_bounded(smem_u32(&sh.bars.q_read), (ch - 1) & 1, abort_flag, c.status)))
            break;
          const uint32_t qbar = smem_u32(&sh.bars.q_full[s]);
          mbar_arrive_expect_tx(qbar, kTile);
#pragma unroll
          for (int p = 0; p < 2; ++p)
            tma_load_2d(tile_q + p * kPanel, mq, qbar, col(w.q_h) + 64 * p, y, pol);
          q_issued = ch + 1;
        }
      }
      for (int ch = issued > 2 ? issued - 2 : 0; ch < issued; ++ch)   // all land before the block ends
        mbar_wait_bounded(smem_u32(&sh.bars.full[ch & 1]), (ch >> 1) & 1, kDrainNs, nullptr, c.status);
      if (q_issued > 0)
        mbar_wait_bounded(smem_u32(&sh.bars.q_full[(q_issued - 1) & 1]), ((q_issued - 1) >> 1) & 1,
                          kDrainNs, nullptr, c.status);
    }
    if (warp == 1) {
      // ---------------------------------------------------------------------------- MMA
      auto commit = [&](uint64_t& bar) { tc_commit_warp(smem_u32(&bar)); };
      bool ok = true;
      for (int ch = 0; ok && ch < chunks; ++ch) {
        const int s = ch & 1, ph = (ch >> 1) & 1;
        if constexpr (kState) {
          // K' and V are ready, and the update before is read
          ok = wait(sh.bars.v[s], ph) && wait(sh.bars.k[s], ph) &&
               (ch == 0 || wait(sh.bars.state[s ^ 1], ((ch - 1) >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          product_mn(t_upd, tile_v(s), tile_k(s), 0);
          product_mn(t_upd, tile_v(s), tile_lo(s), 1);
          commit(sh.bars.upd);
        } else {
          // scores, in P's place: the product that read it last has completed
          ok = wait(sh.bars.full[s], ph) && wait(sh.bars.q_full[s], ph) &&
               (ch == 0 || wait(sh.bars.out[s ^ 1], ((ch - 1) >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          product_kk(t_p, tile_q, tile_k(s));
          commit(sh.bars.scores[s]);
          // Q S: the state is in shared memory, and the outputs before are read
          ok = wait(sh.bars.state[s], ph) &&
               (ch == 0 || wait(sh.bars.drained[s ^ 1], ((ch - 1) >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          product_kk(t_qs, tile_q, tile_s);
          commit(sh.bars.qk);
          ok = wait(sh.bars.v[s], ph) && wait(sh.bars.k[s], ph);
          if (!ok) break;
          tc_fence_after();
          product_mn(t_upd, tile_v(s), tile_k(s), 0);
          product_mn(t_upd, tile_v(s), tile_lo(s), 1);
          commit(sh.bars.upd);
          ok = wait(sh.bars.p[s], ph);
          if (!ok) break;
          tc_fence_after();
          product_tm(t_pv, t_p, tile_v(s));
          commit(sh.bars.out[s]);
        }
        commit(sh.bars.empty[s]);
    }
      commit(sh.bars.drain);
      mbar_wait_bounded(smem_u32(&sh.bars.drain), 0, kDrainNs, nullptr, c.status);
      __syncwarp();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------------------ state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
    const int q = warp & 3, r = 32 * q + lane;     // TMEM lane: row of S^T
    const uint32_t lane_addr = static_cast<uint32_t>(32 * q) << 16;
    const size_t state0 = (static_cast<size_t>(g.seq) * c.H + h) * kD * kD;
    float* seg = w.seg ? w.seg + (static_cast<size_t>(blockIdx.x) * c.H + h) * kD * kD : nullptr;
    uint64_t S[kD / 2];                            // pairs of values
    {
      const float* from = nullptr;
      size_t sk = kD, sv = 1;
      if (!kState && c.split && !whole) {
        from = seg;
      } else if (!kState && w.s0) {
        from = w.s0 + state0;
        sk = static_cast<size_t>(w.s_key);
        sv = static_cast<size_t>(w.s_val);
      }
#pragma unroll
      for (int i = 0; i < kD / 2; ++i) {
        const float x = from ? from[2 * i * sk + r * sv] : 0.0f;
        const float y = from ? from[(2 * i + 1) * sk + r * sv] : 0.0f;
        S[i] = chunks > 0 ? pair(lin_nan_if_inf(x), lin_nan_if_inf(y)) : pair(x, y);
      }
    }
    float top[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (!kState) {
#pragma unroll
      for (int i = 0; i < kD / 2; ++i) {
        const float2 x = unpair(S[i]);
        top[i & 3] = max3_abs(top[i & 3], x.x, x.y);
      }
    }
    // the state for chunk ch: scaled, rounded and written as the B operand of Q S
    auto publish = [&](int ch, bool ok) {
      const float m = warp_max(max_of(top));
      if (lane == 0) sh.red_s[q] = m;
      if (!named_bar_and(1, kGroup, ok)) return false;
      const int e = up_to_half(max_of(sh.red_s));
      if (r == 0) sh.exp_s[ch & 1] = e;
      const uint64_t f2 = pair(pow2(e), pow2(e));
      const uint32_t s_row = row_at(tile_s, r);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = unpair(mul2(S[4 * x + i], f2));
          u[i] = pack2(y.x, y.y);
        }
        sts128(vec_of(s_row, x), make_uint4(u[0], u[1], u[2], u[3]));
      }
      fence_proxy_async_smem();
      arrive(sh.bars.state[ch & 1]);
      return true;
    };
    bool ok = true;
    if constexpr (!kState) ok = publish(0, true);
    for (int ch = 0; ok && ch < chunks; ++ch) {
      const bool w2 = wait(sh.bars.upd, ch & 1);
      if (w2) {
        tc_fence_after();
        const float decay = tokens(ch) < kC ? sh.decay.last : sh.decay.of(ch);
        const float f = pow2(-sh.exp_k[ch & 3]);
        const uint64_t decay2 = pair(decay, decay), f2 = pair(f, f);
        top[0] = top[1] = top[2] = top[3] = 0.0f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t d[32];
          tc_ld_32x32b_x32(t_upd + lane_addr + 32u * b, d);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint64_t& x = S[16 * b + i];
            x = fma2(decay2, x, mul2(pair(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), f2));
            if constexpr (!kState) {
              const float2 y = unpair(x);
              top[i & 3] = max3_abs(top[i & 3], y.x, y.y);
            }
          }
        }
        tc_fence_before();
      }
      if constexpr (kState) {
        ok = w2;
        if (ok) arrive(sh.bars.state[ch & 1]);
      } else {
        ok = publish(ch + 1, w2);
      }
    }
    ok = named_bar_and(1, kGroup, ok);
    const bool mine = kState || (whole && w.sT != nullptr);
    if (ok && mine) {
      float* to = kState ? seg : w.sT + state0;
      const size_t sk = kState ? kD : static_cast<size_t>(w.s_key);
      const size_t sv = kState ? 1 : static_cast<size_t>(w.s_val);
      const bool bad = *reinterpret_cast<volatile int*>(&sh.any_bad) && sh.bad_at[r] != 0x7fffffff;
#pragma unroll
      for (int i = 0; i < kD / 2; ++i) {
        const float2 x = unpair(S[i]);
        to[2 * i * sk + r * sv] = bad ? __int_as_float(0x7fffffff) : x.x;
        to[(2 * i + 1) * sk + r * sv] = bad ? __int_as_float(0x7fffffff) : x.y;
      }
    }
  } else if (warp < 12) {
    // --------------------------------------------------------------------------- K to K'
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecay));
    const int r = 32 * (warp & 3) + lane;
    // The group meets at barriers without a time limit, so its warps give up together: what a warp's
    // wait said goes into the next barrier (here or in find_exp), and all leave there.  (Carried into
    // the next chunk's find_exp instead of a barrier of its own, backward 4 x 2048 took 146 us, so 143.)
    for (int ch = 0; ch < chunks; ++ch) {
      const int s = ch & 1, ph = (ch >> 1) & 1;
      const bool ok = wait(sh.bars.full[s], ph);
      if (ok) clean_v(ch, r);
      if constexpr (kState) {
        if (!ok) break;
        arrive(sh.bars.v[s]);
      } else {
        float f;
        if (!find_exp(ch, r, 0, 2, ok, &f)) break;
        arrive(sh.bars.v[s]);
        // K is no longer read as such, nor the second part of the K' before
        const bool go = wait(sh.bars.scores[s], ph) && (ch == 0 || wait(sh.bars.upd, (ch - 1) & 1));
        if (!named_bar_and(2, kGroup, go)) break;
        decay_k(ch, r, 0, f);
        arrive(sh.bars.k[s]);
      }
    }
  } else {
    // ----------------------------------------------------------------------------- tokens
    const int q = warp & 3, r = 32 * q + lane;     // TMEM lane: token row
    const int turn = warp < 16 ? 0 : 1;
    if constexpr (kState) {
      for (int ch = 0; ch < chunks; ++ch) {
        const bool ok = wait(sh.bars.full[ch & 1], (ch >> 1) & 1);
        float f;
        if (!find_exp(ch, r, turn, 3, ok, &f)) break;
        decay_k(ch, r, turn, f);
        arrive(sh.bars.k[ch & 1]);
      }
    } else {
      const uint32_t lane_addr = static_cast<uint32_t>(32 * q) << 16;
      const int i = back ? kC - 1 - r : r;         // place in the chunk
      __half* op = static_cast<__half*>(w.o) + h * w.o_h;
      const bool wide = ((reinterpret_cast<uintptr_t>(op) | static_cast<uintptr_t>(2 * w.o_t)) & 31) == 0;
      // blocks of 32 columns with tokens up to the warp's rows
      const int b0 = back ? q : 0, b1 = back ? 3 : q;
      // gamma^(i-j) a of a block but for the column's part: before the warp's rows a row's factor
      // times a column's, both at most 1; across them, from the table
      auto row_factor = [&](int b) {
        return b == q ? w.a : w.a * sh.pow[back ? 32 * b - r : r - 32 * b - 31];
      };
      for (int ch = turn; ch < chunks; ch += 2) {
        const int ph = (ch >> 1) & 1;
        // The row's power of two, from a bound on its scores, 128 max|q_i| max|k|: a few bits more than
        // they have, of the 29 between fp16's largest and smallest normal values.  Where the chunk's
        // keys differ by more than 2^kKeyBits, a later one, or one that has decayed away, would cost too
        // many: there over the tokens up to the row's own and decayed, max gamma^(i-j) |k_j| (for all chunks
        // it takes 3 % longer).
        if (!wait(sh.bars.q_full[turn], ph)) break;
        const float top_q = row_top(row_at(tile_q, r));
        arrive(sh.bars.q_read);
        if (!wait(sh.bars.v[turn], ph)) break;
        float most = max_of(sh.top_k[turn]);
        if (min_of(sh.low_k[turn]) * static_cast<float>(1 << kKeyBits) < most) {
          auto key = [&](int row) { return __uint_as_float(static_cast<uint32_t>(sh.key[turn][row]) << 23); };
          // up to each row's token: of the warp's rows (scanned; a lane without a neighbour that far gets
          // the outermost one's, which does no harm), then of the blocks before them
          most = key(r);
#pragma unroll 1
          for (int o = 1; o < 32; o <<= 1)
            most = fmaxf(most, __shfl_sync(0xffffffffu, most, max(0, min(31, back ? lane + o : lane - o))) * sh.pow[o]);
          float before = 0.0f;
#pragma unroll 1
          for (int b = b0; b <= b1; ++b)
            if (b != q)
              before = fmaxf(before, key(32 * b + lane) * sh.pow[back ? 32 * (b - q) + lane - 31 : 32 * (q - b) - lane]);
          most = fmaxf(most, warp_max(before) * sh.pow[back ? 31 - lane : lane]);
        }
        const int e = up_to_half(top_q * most * (128.0f * fabsf(w.a)));
        const bool bad = *reinterpret_cast<volatile int*>(&sh.any_bad) != 0;
        const bool bad_k = bad || tokens(ch) < kC;   // rows past the end may hold anything
        if (!wait(sh.bars.scores[turn], ph)) break;
        tc_fence_after();
        // ascending blocks: the packed columns of a block lie on blocks that are done with
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          uint32_t u[16];
          if (b >= b0 && b <= b1) {
            uint32_t d[32];
            tc_ld_32x32b_x32(t_p + lane_addr + 32u * b, d);
            tc_wait_ld();
            const float f = row_factor(b) * pow2(e);
            if (b != q) {
              const uint64_t f2 = pair(f, f);
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const ulonglong2 c4 = *reinterpret_cast<const ulonglong2*>(&sh.diag[(back ? 32 : 4) + j]);
                const float2 x = unpair(mul2(pair(__uint_as_float(d[j]), __uint_as_float(d[j + 1])),
                                             mul2(c4.x, f2)));
                const float2 y = unpair(mul2(pair(__uint_as_float(d[j + 2]), __uint_as_float(d[j + 3])),
                                             mul2(c4.y, f2)));
                u[j / 2] = pack2(x.x, x.y);
                u[j / 2 + 1] = pack2(y.x, y.y);
              }
            } else {
              if (bad_k) {
                // not a product with 0: the score of a later token may be anything
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (back ? j < lane : j > lane) d[j] = 0u;
              }
              const float* pw = sh.diag + (back ? 32 : 35) - lane;
#pragma unroll
              for (int j = 0; j < 32; j += 2)
                u[j / 2] = pack2(__uint_as_float(d[j]) * (pw[j] * f), __uint_as_float(d[j + 1]) * (pw[j + 1] * f));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) u[j] = 0u;
          }
          st_x16(t_p + lane_addr + 16u * b, u);
        }
        tc_wait_st();
        tc_fence_before();
        if (!wait(sh.bars.state[turn], ph)) break;   // its exponent is read below
        arrive(sh.bars.p[turn]);
        if (!wait(sh.bars.out[turn], ph)) break;
        tc_fence_after();
        const float fi = w.b * sh.pow[i + 1 - lag] * pow2(-sh.exp_s[ch & 1]);
        const float fa = w.b * pow2(-e);
        const uint64_t fi2 = pair(fi, fi), fa2 = pair(fa, fa);
        const bool in = i < tokens(ch);
        __half* row = op + (row0(ch) + r) * w.o_t;
#pragma unroll 1
        for (int b = 0; b < 8; ++b) {
          uint32_t x[32], y[32];   // sixteen of each
          tc_ld_32x32b_x16(t_qs + lane_addr + 16u * b, x);
          tc_ld_32x32b_x16(t_pv + lane_addr + 16u * b, y);
          tc_wait_ld();
          if (b == 7) {
            tc_fence_before();
            arrive(sh.bars.drained[turn]);
          }
          uint32_t u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 o = unpair(
                fma2(pair(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), fi2,
                     mul2(pair(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1])), fa2)));
            u[j] = pack2(o.x, o.y);
          }
          if (bad) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (ch * kC + i >= sh.bad_at[16 * b + j]) u[j / 2] |= (j & 1) ? 0x7fff0000u : 0x7fffu;
          }
          if (in) {
            __half* p = row + 16 * b;
            if (wide) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
                           "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
              *reinterpret_cast<uint4*>(p + 8) = make_uint4(u[4], u[5], u[6], u[7]);
            }
          }
        }
      }
    }
  }

  // Every MMA has completed (the MMA warp drained them) and every TMEM read is done.
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

template <bool kState>
cudaError_t launch(const LinCall& c, const LinMaps& maps, cudaStream_t s) {
  using L = Lay<kState>;
  static std::once_flag once[kMaxDevices];
  static cudaError_t attr[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    attr[dev] = cudaFuncSetAttribute(lin_tc_kernel<kState>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  });
  if (attr[dev] != cudaSuccess) return attr[dev];
  const dim3 grid(static_cast<unsigned>(c.n_items), static_cast<unsigned>(c.H),
                  static_cast<unsigned>(c.n_sweeps));
  lin_tc_kernel<kState><<<grid, kThreads, L::kSmem, s>>>(c, maps);
  return cudaGetLastError();
}

// A matrix of heads as rows of tokens: head h begins at column h * head_stride of every row (the
// rows may overlap in memory, which only loads ever see).
bool map_heads(CUtensorMap* m, const void* p, int64_t T, int H, int64_t t_stride, int64_t h_stride) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p,
                      static_cast<uint64_t>((H - 1) * h_stride + kD), static_cast<uint64_t>(T),
                      static_cast<uint64_t>(t_stride) * 2, 64, kC, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t launch_lin_tc(const LinCall& c, cudaStream_t s) {
  LinMaps maps;
  for (int i = 0; i < c.n_sweeps; ++i) {
    const LinSweep& w = c.sw[i];
    if (!map_heads(&maps.m[3 * i], w.k, c.T, c.H, w.k_t, w.k_h) ||
        !map_heads(&maps.m[3 * i + 1], w.v, c.T, c.H, w.v_t, w.v_h) ||
        !map_heads(&maps.m[3 * i + 2], w.q, c.T, c.H, w.q_t, w.q_h))
      return cudaErrorInvalidValue;
  }
  if (c.split) {
    cudaError_t e = launch<true>(c, maps, s);
    if (e == cudaSuccess) e = launch_lin_join(c, s);
    if (e != cudaSuccess) return e;
  }
  return launch<false>(c, maps, s);
}

}  // namespace mmf
