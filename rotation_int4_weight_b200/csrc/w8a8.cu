// int8 x int8 linears with scales for each token and channel:
//   y[m][n] = sx[m] sw[n] sum_k q[m][k] w[n][k] (+ bias[n]),
// and the gated pair y = silu(gate) * up of two such products.  The inner sums
// are exact 32-bit integers (|sum| <= 49152 * 2^14 < 2^31), so they do not
// depend on any order; what follows is fp32 and one rounding to y's type.
#include "int8.cuh"
#include "w8a8.cuh"

namespace paro {
namespace {

constexpr int kTile = 64, kStep = 64;

// A 64 x 64 tile of y, the columns in steps of 64 through shared memory.
template <bool GATED, bool F16>
__global__ void __launch_bounds__(256) w8a8_tile_kernel(const W8a8Args A) {
  __shared__ int xs[kTile][kStep / 4 + 1], ws[1 + GATED][kTile][kStep / 4 + 1];
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[1 + GATED][4][4] = {};
  for (int k0 = 0; k0 < A.d_in; k0 += kStep) {
    const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;  // 16 bytes of a row
    auto fetch = [&](const int8_t* p, int row, int rows, int* dst) {
      int4 v = make_int4(0, 0, 0, 0);
      if (row < rows && k0 + c < A.d_in) v = *reinterpret_cast<const int4*>(p + (size_t)row * A.d_in + k0 + c);
      dst[0] = v.x, dst[1] = v.y, dst[2] = v.z, dst[3] = v.w;
    };
    __syncthreads();
    fetch(A.q, m0 + r, A.M, &xs[r][c / 4]);
    fetch(A.w, n0 + r, A.d_out, &ws[0][r][c / 4]);
    if constexpr (GATED) fetch(A.w2, n0 + r, A.d_out, &ws[1][r][c / 4]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep / 4; ++k)
#pragma unroll
      for (int g = 0; g < 1 + GATED; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[g][i][j] = __dp4a(xs[ty + 16 * i][k], ws[g][tx + 16 * j][k], acc[g][i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= A.M || n >= A.d_out) continue;
      float v = w8a8_scaled(acc[0][i][j], A.sx[m], A.sw[n]);
      if constexpr (GATED) v = w8a8_gate(v, w8a8_scaled(acc[1][i][j], A.sx[m], A.sw2[n]));
      else if (A.bias) v += from_16<F16>(A.bias[n]);
      A.y[(size_t)m * A.d_out + n] = to_16<F16>(v);
    }
}

}  // namespace

cudaError_t launch_w8a8(const W8a8Args& a, int* status, cudaStream_t stream) {
  (void)status;
  const dim3 grid((a.d_out + kTile - 1) / kTile, (a.M + kTile - 1) / kTile);
  if (a.w2) {
    if (a.f16) w8a8_tile_kernel<true, true><<<grid, 256, 0, stream>>>(a);
    else w8a8_tile_kernel<true, false><<<grid, 256, 0, stream>>>(a);
  } else {
    if (a.f16) w8a8_tile_kernel<false, true><<<grid, 256, 0, stream>>>(a);
    else w8a8_tile_kernel<false, false><<<grid, 256, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace paro
