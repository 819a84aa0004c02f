// int8 x int8 linears with scales for each token and channel:
//   y[m][n] = sx[m] sw[n] sum_k q[m][k] w[n][k] (+ bias[n]),
// and the gated pair y = silu(gate) * up of two such products: the choice
// between the two kernels, and what both need from the host.  The inner sums are
// exact 32-bit integers (|sum| <= 49152 * 2^14 < 2^31), so they do not depend on
// any order; what follows is fp32 and one rounding to y's type.
#include <atomic>

#include "int8.cuh"
#include "w4_stream.cuh"  // device_sm_count
#include "w8a8.cuh"

namespace paro {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static std::atomic<EncodeTiled> known{nullptr};
  EncodeTiled fn = known.load(std::memory_order_acquire);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<EncodeTiled>(p);
      known.store(fn, std::memory_order_release);
    }
  }
  return fn;
}

}  // namespace

bool w8_map(CUtensorMap* map, const int8_t* p, int rows, int d_in, int box_rows) {
  const EncodeTiled enc = encode_fn();
  const cuuint64_t dims[2] = {(cuuint64_t)d_in, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)d_in};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, elem[2] = {1, 1};
  return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, elem,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool w8_out_map(CUtensorMap* map, const uint16_t* y, int rows, int d_out) {
  const EncodeTiled enc = encode_fn();
  const cuuint64_t dims[2] = {(cuuint64_t)d_out, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)d_out * 2};
  const cuuint32_t box[2] = {32, 32}, elem[2] = {1, 1};
  return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<uint16_t*>(y), dims, strides, box, elem,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

W8a8Hooks w8a8_hooks(int cluster) {
  const int skip = hook_skip_ready_flags();
  return {hook_flag_wait(), skip == 0 ? -1 : skip == 2 ? 0 : cluster - 1};
}

// The kernel with the smaller estimate, both fits to measured times (bf16, GPU time
// of calls in a row, weights from HBM).  The kernel for many tokens takes 0.35 us
// per 128 columns and round of tiles (256 x 256 on a pair of SMs) and 5.6 us around
// it, 4 more where rows of y are not whole 16 bytes, which no TMA store can write.
// Measured, few / many, us:
//   4096 -> 4096:  M 256: 12.9 / 17, M 512: 17.0 / 17, M 768: 26 / 17.5;
//   4096 -> 14336: M 100: 19.2 / 18.5, M 129: 27 / 18.5, M 512: 53 / 29.6;
//   1552 -> 1100:  M 203: 6.5 / 12;
//   gated 1536 -> 8960: M 33: 11 / 14, M 129: 21 / 11.9;
//   gated 14336 -> 4096: M 128: 33.8 / 45, M 129: 52 / 45.
static bool takes_few(const W8a8Args& a, const W8a8Few& f) {
  const long long blocks = (a.d_in + 127) / 128, pairs = device_sm_count() / 2;
  const int nc = a.w2 ? 128 : 256;
  const long long tiles = ((a.M + 255LL) / 256) * ((a.d_out + nc - 1) / nc);
  const long long many = 5600 + (a.d_out % 8 ? 4000 : 0) + (tiles + pairs - 1) / pairs * blocks * 350;
  return a.M <= 32 || f.ns <= many;
}

cudaError_t launch_w8a8(const W8a8Args& a, int* status, cudaStream_t stream) {
  const W8a8Few f = w8a8_few_shape(a);
  return takes_few(a, f) ? launch_w8a8_few(a, f, status, stream) : launch_w8a8_many(a, status, stream);
}

W8a8Form w8a8_form(int M, int d_in, int d_out, bool gated) {
  W8a8Args a{};
  const int8_t some = 0;
  a.w2 = gated ? &some : nullptr;
  a.M = M, a.d_in = d_in, a.d_out = d_out;
  const W8a8Few f = w8a8_few_shape(a);
  if (takes_few(a, f)) return {f.tokens, 128, f.split};
  return {256, gated ? 128 : 256, 1};
}

}  // namespace paro
