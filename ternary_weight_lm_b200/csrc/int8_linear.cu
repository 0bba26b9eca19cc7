// The 8-bit projection: weights held as int8 codes with one scale for each output channel, for
// layers that are not ternarised (an output head, odd layers), on the activation codes that the
// library's pre-pass writes.
//
//   s_n  = max_k |W_nk| / 127,  c_nk = clamp(round_half_even(W_nk / s_n), -127, 127)
//   y_tn = (sum_k q_tk c_nk) * (gamma_t / 127 * s_n)          (the sum exact in int32)
//
// The contraction keeps the orientation of the ternary one: the MMA's M side is 128 weight rows,
// its N side BN tokens, so that a single token costs one narrow MMA.  The codes are int8 already,
// so both operands go from TMA to shared memory to tcgen05.mma (kind::i8) untouched, and the
// only other work is the epilogue.  Few tokens: bound by the weight stream (N K bytes once).  Measured
// back to back: one token, 2048 -> 32000, 9.0 us (65.5 MB, part of it from L2); 64 tokens, 2048 ->
// 11264, 9.9 us; many tokens on the CTA pairs, 8192 x 2048 -> 11264, 127 us, 91 % of twice the bf16
// rate.
#include <cuda_fp16.h>

#include <mutex>

#include "int8_linear.cuh"
#include "ptx.cuh"

namespace mmf {
namespace {

// ------------------------------------------------------------------------------- weights
// A block takes kHeld / V rows at a time, a thread V vectors of eight values of each, held in
// registers between the maximum and the encoding: 32 to 64 KB in flight whatever the row's length.
// Rows of more than 4096 values are taken one at a time, beyond kHeld vectors read again (from L2).
// Bound by the stream in fp32: 32000 x 2048 take 54 to 59 us, 85 to 93 % of a copy's rate (72 us with one
// row a block and a division for every value).  In fp16, half the bytes, 56 us, 54 % of it: there the
// instructions for a value (conversion, maximum, encoding) are what counts.
constexpr int kQThreads = 128;
constexpr int kHeld = 8;

struct Vec8 {
  float v[8];
};

template <typename TW>
__device__ __forceinline__ Vec8 load8(const TW* p);
template <>
__device__ __forceinline__ Vec8 load8<float>(const float* p) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
template <>
__device__ __forceinline__ Vec8 load8<__half>(const __half* p) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
  const __half2* h = reinterpret_cast<const __half2*>(&a);
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    r.v[2 * i] = f.x;
    r.v[2 * i + 1] = f.y;
  }
  return r;
}

// round(x / s).  The product with 1 / s is off by less than 2^-15 (three roundings of up to 2^-24 of
// at most 127), so unless it lies that close to a half it rounds to the same code; next to a half
// (a band of 2^-13 for each of eight values: about one vector in a thousand) the division itself decides.
__device__ __forceinline__ uint2 encode8(const Vec8& x, float s, float inv) {
  int c[8];
  bool sure = inv <= 3.0e38f;   // not of a scale of zero, or one whose reciprocal overflows
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = x.v[i] * inv;
    c[i] = __float2int_rn(y);
    sure &= fabsf(fabsf(y - static_cast<float>(c[i])) - 0.5f) > 0x1p-14f;   // false for a NaN
  }
  if (!sure) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s > 0.0f ? __float2int_rn(__fdiv_rn(x.v[i], s)) : 0;
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i >> 2] |= (static_cast<uint32_t>(max(-127, min(127, c[i]))) & 0xFFu) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

template <typename TW, int V>
__global__ void __launch_bounds__(kQThreads) quantize_rows_i8_kernel(const TW* __restrict__ W,
                                                                     int64_t N, int K,
                                                                     int8_t* __restrict__ W8,
                                                                     float* __restrict__ wscale) {
  constexpr int R = kHeld / V;
  __shared__ float s_max[R][kQThreads / 32];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * R;
  const int nvec = K / 8;
  Vec8 held[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = threadIdx.x + j * kQThreads;
      held[r][j] = i < nvec && row0 + r < N ? load8<TW>(W + (row0 + r) * K + static_cast<int64_t>(i) * 8)
                                            : Vec8{};
    }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(held[r][j].v[e]));
    if constexpr (R == 1) {
      for (int i = threadIdx.x + V * kQThreads; i < nvec; i += kQThreads) {
        const Vec8 x = load8<TW>(W + row0 * K + static_cast<int64_t>(i) * 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x.v[e]));
      }
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if ((threadIdx.x & 31) == 0) s_max[r][threadIdx.x >> 5] = m;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (row0 + r >= N) break;
    const float m = fmaxf(fmaxf(s_max[r][0], s_max[r][1]), fmaxf(s_max[r][2], s_max[r][3]));
    const float s = __fdiv_rn(m, 127.0f), inv = __fdiv_rn(1.0f, s);
    if (threadIdx.x == 0) wscale[row0 + r] = s;
    uint2* out = reinterpret_cast<uint2*>(W8 + (row0 + r) * K);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = threadIdx.x + j * kQThreads;
      if (i < nvec) out[i] = encode8(held[r][j], s, inv);
    }
    if constexpr (R == 1)
      for (int i = threadIdx.x + V * kQThreads; i < nvec; i += kQThreads)
        out[i] = encode8(load8<TW>(W + row0 * K + static_cast<int64_t>(i) * 8), s, inv);
  }
}

template <typename TW>
cudaError_t quantize_rows(const TW* W, int64_t N, int K, int8_t* W8, float* wscale, cudaStream_t s) {
  const int per = (K / 8 + kQThreads - 1) / kQThreads;   // vectors a thread has of a row
  auto blocks = [&](int rows) { return static_cast<unsigned>((N + rows - 1) / rows); };
  if (per <= 1)
    quantize_rows_i8_kernel<TW, 1><<<blocks(8), kQThreads, 0, s>>>(W, N, K, W8, wscale);
  else if (per <= 2)
    quantize_rows_i8_kernel<TW, 2><<<blocks(4), kQThreads, 0, s>>>(W, N, K, W8, wscale);
  else if (per <= 4)
    quantize_rows_i8_kernel<TW, 4><<<blocks(2), kQThreads, 0, s>>>(W, N, K, W8, wscale);
  else
    quantize_rows_i8_kernel<TW, 8><<<blocks(1), kQThreads, 0, s>>>(W, N, K, W8, wscale);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------- contraction
constexpr int kKB = 128;                    // K bytes per stage and operand row
constexpr int kRows = 128;                  // weight rows per tile
constexpr int kWStage = kRows * kKB;        // 16 KB
constexpr int kThreads = 192;               // warps: 0 TMA, 1 TMEM + MMA, 2-5 epilogue
constexpr int kEpiThreads = 128;
constexpr uint64_t kDrainNs = 2000000000ull;
// Two blocks share an SM (148 of them), so that one block's start and end overlap the other's
// stream and 149 to 296 tiles still run at once.
constexpr int kSlots = 296;

template <int BN>
struct Cfg {
  static constexpr int kActStage = BN * kKB;
  static constexpr int kStage = kActStage + kWStage;
  static constexpr int kBudget = 110 * 1024;
  static constexpr int kStages = kBudget / kStage;
  static constexpr int kTmemCols = BN < 32 ? 32 : BN;
  static constexpr int kChunk = BN < 32 ? BN : 32;   // token columns per epilogue pass
  static constexpr int kBarBytes = 8 * (2 * kStages + 1);
  static constexpr int kSmem = 1024 + kStages * kStage + ((kBarBytes + 15) / 16) * 16 + 4 * BN;
  static_assert(kStages >= 3, "pipeline depth");
  static_assert(kSmem <= 113 * 1024, "two blocks per SM");
  static_assert(BN * kRows * 4 <= kStages * kStage, "partial sums must fit the stages");
};

struct Params {
  int64_t T;
  int nkb;
  int N;
  int out_f16;
  const float* gamma;
  const float* wscale;
  void* y;
  unsigned* status;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ void tc_mma_i8_ss_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                  uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__host__ __device__ constexpr uint32_t idesc_i8_s8s8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void put(const Params& p, int64_t t, int n, int32_t acc, float sc) {
  const float f = static_cast<float>(acc) * sc;
  const int64_t off = t * p.N + n;
  if (p.out_f16)
    reinterpret_cast<__half*>(p.y)[off] = __float2half_rn(f);
  else
    reinterpret_cast<float*>(p.y)[off] = f;
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 2)
int8_linear_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                   const Params p) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* s_w = smem;
  uint8_t* s_act = smem + C::kStages * kWStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_act + C::kStages * C::kActStage);
  float* s_gam = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) +
                                          ((C::kBarBytes + 15) / 16) * 16);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the gridDim.z blocks of a cluster share a tile, each with a range of k-blocks
  const int csize = static_cast<int>(gridDim.z);
  const int kb0 = static_cast<int>(blockIdx.z) * p.nkb / csize;
  const int nkb = (static_cast<int>(blockIdx.z) + 1) * p.nkb / csize - kb0;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * BN;
  const int n0 = static_cast<int>(blockIdx.x) * kRows;

  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + C::kStages + s); };
  const uint32_t accfull = smem_u32(bars + 2 * C::kStages);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(accfull, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_a);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      // one token tile: every weight byte is used once; several: the tiles share the weights
      const uint64_t pol_w = gridDim.y > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
      const uint64_t pol_a = l2_policy_evict_last();
      int issued = 0;
      for (int kb = 0; kb < nkb; ++kb) {
        const int s = kb % C::kStages;
        if (kb >= C::kStages && !mbar_wait_bounded(empty(s), ((kb / C::kStages) - 1) & 1,
                                                   p.wait_limit_ns, abort_flag, p.status))
          break;
        mbar_arrive_expect_tx(full(s), C::kStage);
        const int kx = (kb0 + kb) * kKB;   // columns at or beyond K arrive as zeros
        tma_load_2d(smem_u32(s_w + s * kWStage), &tm_w, full(s), kx, n0, pol_w);
        tma_load_2d(smem_u32(s_act + s * C::kActStage), &tm_a, full(s), kx,
                    static_cast<int32_t>(t0), pol_a);
        issued = kb + 1;
      }
      // every copy this thread started lands before the block may exit
      for (int kb = issued > C::kStages ? issued - C::kStages : 0; kb < issued; ++kb)
        mbar_wait_bounded(full(kb % C::kStages), (kb / C::kStages) & 1, kDrainNs, nullptr, p.status);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_i8_s8s8(kRows, BN);
    const uint64_t adesc0 = smem_desc_kmajor_sw128(smem_u32(s_w));
    const uint64_t bdesc0 = smem_desc_kmajor_sw128(smem_u32(s_act));
    for (int kb = 0; kb < nkb; ++kb) {
      const int s = kb % C::kStages;
      const bool w = mbar_wait_bounded(full(s), (kb / C::kStages) & 1, p.wait_limit_ns, abort_flag,
                                       p.status);
      if (!__all_sync(0xFFFFFFFFu, w)) break;
      tc_fence_after();
      // start addresses in 16-byte units; a 32-deep k step is 32 bytes inside the swizzled rows
      const uint64_t ad = adesc0 + static_cast<uint64_t>((s * kWStage) >> 4);
      const uint64_t bd = bdesc0 + static_cast<uint64_t>((s * C::kActStage) >> 4);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        tc_mma_i8_ss_warp(tmem, ad + 2 * j, bd + 2 * j, idesc, (kb > 0 || j > 0) ? 1u : 0u);
      tc_commit_warp(empty(s));
    }
    tc_commit_warp(accfull);
    mbar_wait_bounded(accfull, 0, kDrainNs, nullptr, p.status);
    __syncwarp();
  } else {
    // epilogue: thread = weight row = TMEM lane; token scales staged while the stream runs
    const int q = warp & 3, r = q * 32 + lane;
    const int et = static_cast<int>(threadIdx.x) - 64;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    for (int i = et; i < BN; i += kEpiThreads)
      s_gam[i] = t0 + i < p.T ? __fdiv_rn(p.gamma[t0 + i], 127.0f) : 0.0f;
    const int n = n0 + r;
    const float ws = n < p.N ? p.wscale[n] : 0.0f;
    const bool w = mbar_wait_bounded(accfull, 0, p.wait_limit_ns, abort_flag, p.status);
    // the barrier also publishes s_gam
    const bool ok = named_bar_and(1, kEpiThreads, __all_sync(0xFFFFFFFFu, w));
    if (ok) {
      tc_fence_after();
      int32_t* part = reinterpret_cast<int32_t*>(smem);   // all copies landed, all MMAs done
      for (int c0 = 0; c0 < BN; c0 += C::kChunk) {
        if (t0 + c0 >= p.T) break;                        // same for every thread
        uint32_t acc[32];
        if constexpr (C::kChunk == 32)
          tc_ld_32x32b_x32(tmem + lane_addr + c0, acc);
        else
          tc_ld_32x32b_x16(tmem + lane_addr + c0, acc);
        tc_wait_ld();
        if (csize > 1) {
#pragma unroll
          for (int j = 0; j < C::kChunk; ++j)
            part[(c0 + j) * kRows + r] = static_cast<int32_t>(acc[j]);
        } else if (n < p.N) {
#pragma unroll
          for (int j = 0; j < C::kChunk; ++j)
            if (t0 + c0 + j < p.T)
              put(p, t0 + c0 + j, n, static_cast<int32_t>(acc[j]), s_gam[c0 + j] * ws);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (csize > 1) {
    // every thread of every block of the cluster reaches both barriers on every path
    cluster_sync_all();
    if (warp >= 2 && !s_abort) {
      const int r = (warp & 3) * 32 + lane;
      const int n = n0 + r;
      const uint32_t part0 = smem_u32(smem);
      const float ws = n < p.N ? p.wscale[n] : 0.0f;
      // eight tokens at a time, so that their loads from the other blocks overlap
      constexpr int kAtOnce = 8;
      const int live = static_cast<int>(min(static_cast<int64_t>(BN), p.T - t0));
      for (int j0 = static_cast<int>(cluster_ctarank()); j0 < live; j0 += csize * kAtOnce) {
        int32_t v[kAtOnce];   // exact, so the order of the blocks does not matter
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) v[u] = 0;
        for (int c = 0; c < csize; ++c) {
          const uint32_t from = map_peer(part0 + 4u * static_cast<uint32_t>(j0 * kRows + r), c);
          int32_t x[kAtOnce];
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u)
            x[u] = j0 + u * csize < live ? ld_cluster_s32(from + 4u * static_cast<uint32_t>(u * csize * kRows)) : 0;
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) v[u] += x[u];
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int j = j0 + u * csize;
          if (j < live && n < p.N) put(p, t0 + j, n, v[u], s_gam[j] * ws);
        }
      }
    }
    cluster_sync_all();   // the partial sums stay readable until everyone is done
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int BN>
cudaError_t launch_bn(const Int8Call& c, cudaStream_t s) {
  using Cf = Cfg<BN>;
  static std::once_flag once[kMaxDevices];
  static cudaError_t attr[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    attr[dev] = cudaFuncSetAttribute(int8_linear_kernel<BN>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::kSmem);
  });
  if (attr[dev] != cudaSuccess) return attr[dev];

  CUtensorMap tm_w, tm_a;
  const uint64_t K = static_cast<uint64_t>(c.K);
  if (!make_tmap_2d_u8(&tm_w, c.W8, K, static_cast<uint64_t>(c.N), K, kKB, kRows,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d_u8(&tm_a, c.A, K, static_cast<uint64_t>(c.T), K, kKB, BN,
                       CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;

  Params p;
  p.T = c.T;
  p.nkb = (c.K + kKB - 1) / kKB;
  p.N = c.N;
  p.out_f16 = c.out_mode == kOutF16;
  p.gamma = c.gamma;
  p.wscale = c.wscale;
  p.y = c.y;
  p.status = c.status;
  p.wait_limit_ns = c.wait_limit_ns;

  const unsigned ntiles = static_cast<unsigned>((c.N + kRows - 1) / kRows);
  const int64_t ttiles = (c.T + BN - 1) / BN;
  if (ttiles > 65535) return cudaErrorInvalidConfiguration;
  const int64_t tiles = ntiles * ttiles;
  int csize = 1;
  while (csize * 2 <= 8 && csize * 2 <= p.nkb && tiles * csize * 2 <= kSlots) csize *= 2;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ntiles, static_cast<unsigned>(ttiles), static_cast<unsigned>(csize));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cf::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = 1;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = static_cast<unsigned>(csize);
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, int8_linear_kernel<BN>, tm_w, tm_a, p);
}

}  // namespace

cudaError_t launch_quantize_weights_i8(const void* W, int wdt, int64_t N, int K, int8_t* W8,
                                       float* wscale, cudaStream_t s) {
  if (wdt == kInF16) return quantize_rows(static_cast<const __half*>(W), N, K, W8, wscale, s);
  return quantize_rows(static_cast<const float*>(W), N, K, W8, wscale, s);
}

// Which contraction.  The CTA-pair pipeline takes 256 x 256 tiles over the whole of K (about 5 us
// plus 0.27 us for each k-block of 128 and round of 74 tiles); this file's splits K over a cluster
// when its 128-row tiles are few.  Measured (us, here / pairs): T 129, K 5632, N 2048 12.1 / 17.1;
// T 512, K 8192, N 1024 14.1 / 22.7; T 256, K 4096, N 4096 12.9 / 14.3; but T 512, K 4096, N 4096
// 16.6 / 14.9; T 256, K 2048, N 2048 11.2 / 9.6; T 128, K 2048, N 11264 13.0 / 11.1; T 64, K 2048,
// N 11264 9.9 / 11.2.  So: up to 64 tokens here; beyond, here only for a deep K that at least four
// blocks can share.
cudaError_t launch_int8_linear(const Int8Call& c, cudaStream_t s) {
  const int64_t tiles = ((c.N + kRows - 1) / kRows) * ((c.T + 127) / 128);
  const int nkb = (c.K + kKB - 1) / kKB;
  if (c.T > 64 && !(nkb >= 28 && 4 * tiles <= kSlots)) return launch_int8_pairs(c, s);
  if (c.T <= 16) return launch_bn<16>(c, s);
  if (c.T <= 32) return launch_bn<32>(c, s);
  if (c.T <= 64) return launch_bn<64>(c, s);
  return launch_bn<128>(c, s);
}

}  // namespace mmf
