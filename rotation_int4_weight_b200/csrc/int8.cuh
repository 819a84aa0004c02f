// The 8-bit path (int8_codes.cu, w8a8.cu): int8 codes with a scale for each
// row, and the int8 x int8 linears on them.
#pragma once

#include <atomic>

#include "paro_internal.cuh"

namespace paro {

// Allows a kernel up to `bytes` of dynamic shared memory on the current device,
// once for each device (`done` has a bit for each, and is the kernel's own).
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done);

// ---- int8_codes.cu ---------------------------------------------------------------
// Row codes of 16-bit activations [M][d], any d >= 1: with `norm` the RMS norm
// (h = x + residual stored to hidden when residual is given, gain may be null)
// first.  All pointers 16-byte aligned (sx 4).  bf16 or fp16 by `f16`.
cudaError_t launch_int8_codes(const uint16_t* x, const uint16_t* residual, const uint16_t* gain, uint16_t* hidden,
                              int8_t* q, float* sx, int M, int d, bool f16, bool norm, float eps,
                              cudaStream_t stream);
// Row codes of fp32 weights [rows][d].
cudaError_t launch_int8_pack(const float* W, int8_t* q, float* s, int rows, int d, cudaStream_t stream);

// ---- w8a8.cu -----------------------------------------------------------------------
// One int8 linear: y[m][n] = sx[m] sw[n] sum_k q[m][k] w[n][k] (+ bias[n]), or,
// with w2, y = silu(that) * (the same product on w2, sw2).  16-bit bias and y.
struct W8a8Args {
  const int8_t* q;       // [M][d_in]
  const float* sx;       // [M]
  const int8_t* w;       // [d_out][d_in]
  const float* sw;       // [d_out]
  const int8_t* w2;      // [d_out][d_in] or null
  const float* sw2;      // [d_out] with w2
  const uint16_t* bias;  // [d_out] or null
  uint16_t* y;           // [M][d_out]
  int M, d_in, d_out;
  bool f16;              // y and bias: fp16, else bf16
};
cudaError_t launch_w8a8(const W8a8Args& a, int* status, cudaStream_t stream);
// How that call is cut: tokens and channels of a tile (256 tokens: w8a8_many.cu,
// else w8a8_few.cu) and the shares of d_in.
struct W8a8Form {
  int tokens, channels, shares;
};
W8a8Form w8a8_form(int M, int d_in, int d_out, bool gated);

}  // namespace paro
