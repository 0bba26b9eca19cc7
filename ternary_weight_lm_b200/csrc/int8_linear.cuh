// Host-side launchers of the 8-bit projection (one scale for each output channel).  Internal to
// libmmf.so.
#pragma once

#include "kernels.cuh"

namespace mmf {

// W [N x K] -> codes W8 [N x K] and scales wscale [N].
cudaError_t launch_quantize_weights_i8(const void* W, int wdt, int64_t N, int K, int8_t* W8,
                                       float* wscale, cudaStream_t s);

// y [T x N] from activation codes A [T x K] with scales gamma [T].
struct Int8Call {
  const int8_t* A;
  const float* gamma;
  const int8_t* W8;
  const float* wscale;
  int64_t T;
  int K;                  // % 16 == 0
  int N;                  // % 8 == 0
  void* y;
  int out_mode;           // kOutF32 or kOutF16
  unsigned* status;
  uint64_t wait_limit_ns;
};
cudaError_t launch_int8_linear(const Int8Call& c, cudaStream_t s);

// The same on the CTA-pair pipeline of the ternary prefill contraction (any T; whole 256 x 256
// tiles of work).
cudaError_t launch_int8_pairs(const Int8Call& c, cudaStream_t s);

}  // namespace mmf
