// What follows an int8 product's 32-bit sums: scales, gate, rounding.
#pragma once

#include <cuda.h>

#include "int8.cuh"

namespace paro {

// How the kernel for few tokens cuts a call: tiles of 128 channels, mtiles of
// `tokens` tokens, and each tile's d_in into `split` shares.  An estimate of
// LLONG_MAX: it does not take the call.
struct W8a8Few {
  int tokens, tiles, mtiles, split;
  long long ns;  // estimate of the call's time
};
W8a8Few w8a8_few_shape(const W8a8Args& a);

// What paro_set_test_hooks changes of a launch: the SM clocks after which a role's
// wait on an mbarrier gives up, and the CTA of every cluster whose copies stop when
// its ring is full (-1: none; looked at from there on only, as 0.07 us of a short
// call went into looking before the first copy).
struct W8a8Hooks {
  long long wait;
  int rank;
};
W8a8Hooks w8a8_hooks(int cluster);

// The two kernels of launch_w8a8.
cudaError_t launch_w8a8_few(const W8a8Args& a, const W8a8Few& f, int* status, cudaStream_t stream);
cudaError_t launch_w8a8_many(const W8a8Args& a, int* status, cudaStream_t stream);

// Tensor map of int8 [rows][d_in]: boxes of 128 columns x box_rows, 128-byte
// swizzle, zeros outside.
bool w8_map(CUtensorMap* map, const int8_t* p, int rows, int d_in, int box_rows);
// Tensor map of 16-bit y [rows][d_out], d_out a multiple of 8: boxes of 32 x 32, 64-byte swizzle.
bool w8_out_map(CUtensorMap* map, const uint16_t* y, int rows, int d_out);

// A token's scale.  A sum (below 2^31) times a scale above 2^97 may pass fp32's
// range although the channel's scale brings the product back; such a scale is
// taken 2^-40 of its size and the product 2^40.  Powers of two, so no digit
// changes; what is smaller by 2^40 on the way is still above 2^50 times the
// channel's scale.
struct __align__(8) TokenScale {
  float s, back;
};
__device__ __forceinline__ TokenScale token_scale(float sx) {
  const bool large = fabsf(sx) > 0x1p+90f;
  return {large ? sx * 0x1p-40f : sx, large ? 0x1p+40f : 1.0f};
}

__device__ __forceinline__ float w8a8_scaled(int acc, float s, float sw) {
  return __fmul_rn(__fmul_rn(__int2float_rn(acc), s), sw);
}

// silu(g) * u.  Fast exp and divide are within 2e-5 of g / (1 + exp(-g)), far inside
// half a step of the 16-bit result (bf16 2^-9, fp16 2^-12), for g above -87.3.  Below,
// the divisor passes 2^126, for which the fast quotient is -0: silu(g) is then taken
// as 0, at most 1.1e-36 off.  (Both sides a quarter of their size keep the divisor
// below 2^126, which brings values down to 2.7e-37 back, and cost 3% of a gated call of
// 128-1024 tokens 1536 -> 8960: 12.06 us for 11.73.)
__device__ __forceinline__ float w8a8_gate(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

template <bool F16>
__device__ __forceinline__ float from_16(uint16_t v) {
  return F16 ? __half2float(__ushort_as_half(v)) : __bfloat162float(__ushort_as_bfloat16(v));
}
template <bool F16>
__device__ __forceinline__ uint16_t to_16(float v) {
  return F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

}  // namespace paro
