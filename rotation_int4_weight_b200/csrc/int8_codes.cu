// int8 codes with one scale for each row: of activations, of RMS-normalised
// activations with the residual's sum, and of weights.
//
//   row v with a = max_c |v_c|:  q_c = the whole number nearest to 127 v_c / a
//   (ties to the even one), scale a / 127; an all-zero row has scale 1.
//   RMS norm:  h = x + residual, rounded to the activations' type (the hidden
//   state that the next layer adds to), v_c = h_c g_c r with
//   r = 1 / sqrt(mean_c h_c^2 + eps).  r > 0 is common to the row and cancels
//   in 127 v / a, so the codes are those of h g and r enters the scale alone:
//   one reduction (the largest |h g| and the sum of h^2 together) and no second
//   look at the row's statistics.
//
// Codes are exact.  h g of two bf16 (16 bits) or fp16 (22 bits) values is exact
// in fp32 (unless it underflows), and so is an fp32 weight.  t = v * (127 / a)
// in fp32 is within 127 * 2^-22 = 3.1e-5 of 127 v / a; only where t lies within
// 2^-13 of a border k + 1/2 (about one value in 4000) does the comparison
// 254 |v| against (2k + 1) a decide, in fp64, where both products are exact (32
// bits at most).  So the codes do not depend on the order of any sum.
//
// A row is read once, kept in registers as 8-value chunks, and its codes are
// written from there: 3 bytes a value, 7 with a residual.  Bound by HBM for
// many rows, by one row's latency (load, reduction, store) for few.  Chunks are
// cut at multiples of 8 of the flat index, not of the column, so that rows of
// an odd width still move as 16-byte loads and 8-byte stores; the first and
// last chunk of such a row go value by value, and its gain comes from two
// aligned 16-byte loads shifted by the row's phase.
#include "int8.cuh"
#include "tc_ptx.cuh"

namespace paro {
namespace {

struct CodeArgs {
  const void* x;
  const void* residual;
  const void* gain;
  void* hidden;
  int8_t* q;
  float* sx;
  long long M;
  int d;
  float eps;
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(float f, __nv_bfloat16& o) { o = __float2bfloat16_rn(f); }
__device__ __forceinline__ void from_f32(float f, __half& o) { o = __float2half_rn(f); }
__device__ __forceinline__ void from_f32(float f, float& o) { o = f; }

// Eight consecutive values of one row.
template <typename T>
struct __align__(16) Chunk {
  T v[8];
};

template <typename T>
__device__ __forceinline__ Chunk<T> load_vec(const T* p) {
  Chunk<T> c;
  const uint4* s = reinterpret_cast<const uint4*>(p);
  uint4* o = reinterpret_cast<uint4*>(&c);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Chunk<T>) / 16); ++i) o[i] = s[i];
  return c;
}

// Values lo .. hi - 1 of the chunk at p (the others zero), one by one.
template <typename T>
__device__ __forceinline__ Chunk<T> load_part(const T* p, int lo, int hi) {
  Chunk<T> c;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    from_f32(0.0f, c.v[e]);
    if (e >= lo && e < hi) c.v[e] = p[e];
  }
  return c;
}

// gain[c .. c + 7], columns outside 0 .. d - 1 zero.  c & 7 is the same for
// all chunks of a row.
template <typename T>
__device__ __forceinline__ Chunk<T> load_gain(const T* g, int c, int d) {
  const int a = c & ~7, sh = c & 7;
  if (a < 0 || a + (sh ? 16 : 8) > d) return load_part(g + c, -c, d - c);
  const Chunk<T> A = load_vec(g + a);
  if (sh == 0) return A;
  const Chunk<T> B = load_vec(g + a + 8);
  uint32_t w[8];
  const uint32_t* pa = reinterpret_cast<const uint32_t*>(&A);
  const uint32_t* pb = reinterpret_cast<const uint32_t*>(&B);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pa[i];
    w[4 + i] = pb[i];
  }
  if (sh & 4) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (sh & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (sh & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  Chunk<T> o;
  uint32_t* po = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
  for (int i = 0; i < 4; ++i) po[i] = w[i];
  return o;
}

// The code of v where t = v * (127 / a) lies next to a border between two codes.
__device__ __noinline__ int border_code(float v, float a, float t) {
  const int k = (int)fabsf(t);  // t is near k + 1/2: the whole part is certain
  const double lhs = 254.0 * (double)fabsf(v), rhs = (double)(2 * k + 1) * (double)a;
  const int m = lhs > rhs ? k + 1 : (lhs < rhs ? k : k + (k & 1));
  return v < 0.0f ? -m : m;
}

// Codes of eight values; `up` scales v and a alike (a power of two) so that
// 127 / a stays finite for rows of the smallest magnitudes.
__device__ __forceinline__ uint2 code8(const float (&v)[8], float a, float inv, float up) {
  int q[8];
  bool near = false;
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t[e] = __fmul_rn(__fmul_rn(v[e], up), inv);
    const float k = rintf(t[e]);
    near |= fabsf(__fsub_rn(t[e], k)) > 0.5f - 0x1p-13f;
    q[e] = (int)k;
  }
  if (near) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (fabsf(__fsub_rn(t[e], rintf(t[e]))) > 0.5f - 0x1p-13f) q[e] = border_code(__fmul_rn(v[e], up), a, t[e]);
  }
  uint2 o;
  o.x = (q[0] & 0xFF) | ((q[1] & 0xFF) << 8) | ((q[2] & 0xFF) << 16) | ((uint32_t)q[3] << 24);
  o.y = (q[4] & 0xFF) | ((q[5] & 0xFF) << 8) | ((q[6] & 0xFF) << 16) | ((uint32_t)q[7] << 24);
  return o;
}

// threadIdx.x runs over a row's chunks (NC of them a thread, blockDim.x apart),
// threadIdx.y over the rows of the CTA (more than one only at 32 threads a row).
// EVEN: d is a multiple of 8, every chunk is whole and starts at a column
// multiple of 8.
template <typename T, int NC, bool NORM, bool EVEN>
__global__ void __launch_bounds__(1024)
codes_kernel(const CodeArgs A) {
  __shared__ uint32_t red_a[32];
  __shared__ float red_s[32];
  ptx::grid_trigger();
  ptx::grid_wait();  // launched over the end of the kernel before; nothing is read or written until that is done
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= A.M) return;  // whole warps: a CTA of several rows has one warp for each and no barrier
  const int d = A.d, T1 = blockDim.x;
  const long long base = row * d, first = base & ~7LL;  // flat index of the row, of its first chunk
  const int head = (int)(base - first);
  const int chunks = (head + d + 7) >> 3;
  const T* x = static_cast<const T*>(A.x) + first;
  const T* res = static_cast<const T*>(A.residual) + (A.residual ? first : 0);
  const T* gain = static_cast<const T*>(A.gain);
  T* hid = static_cast<T*>(A.hidden) + (A.hidden ? first : 0);
  int8_t* q = A.q + first;

  Chunk<T> h[NC];
  // the loads of all chunks first, so that they are in flight together
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int j = threadIdx.x + i * T1, c = j * 8 - head;
    if (j < chunks) {
      if (EVEN || (c >= 0 && c + 8 <= d)) h[i] = load_vec(x + j * 8);
      else h[i] = load_part(x + j * 8, -c, d - c);
    }
  }
  uint32_t amax = 0u;  // bits of the largest |v|: inf and NaN order above every number
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int j = threadIdx.x + i * T1, c = j * 8 - head;
    if (j < chunks) {
      const bool whole = EVEN || (c >= 0 && c + 8 <= d);
      if (NORM && A.residual) {
        const Chunk<T> r = whole ? load_vec(res + j * 8) : load_part(res + j * 8, -c, d - c);
#pragma unroll
        for (int e = 0; e < 8; ++e) from_f32(__fadd_rn(to_f32(h[i].v[e]), to_f32(r.v[e])), h[i].v[e]);
        if (whole) {
#pragma unroll
          for (int w = 0; w < (int)(sizeof(Chunk<T>) / 16); ++w)
            reinterpret_cast<uint4*>(hid + j * 8)[w] = reinterpret_cast<const uint4*>(&h[i])[w];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e >= 0 && c + e < d) hid[j * 8 + e] = h[i].v[e];
        }
      }
      if (NORM && A.gain) {
        const Chunk<T> g = EVEN ? load_vec(gain + j * 8) : load_gain(gain, c, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = to_f32(h[i].v[e]);
          ss = fmaf(f, f, ss);
          amax = max(amax, __float_as_uint(fabsf(__fmul_rn(f, to_f32(g.v[e])))));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = to_f32(h[i].v[e]);
          if (NORM) ss = fmaf(f, f, ss);
          amax = max(amax, __float_as_uint(fabsf(f)));
        }
      }
    }
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T1 >> 5;
  auto row_sum = [&](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps > 1) {
      if (lane == 0) red_s[warp] = v;
      __syncthreads();
      v = lane < warps ? red_s[lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
  };
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (warps > 1 && lane == 0) red_a[warp] = amax;
  if (NORM) ss = row_sum(ss);
  else if (warps > 1) __syncthreads();
  if (warps > 1) amax = __reduce_max_sync(0xffffffffu, lane < warps ? red_a[lane] : 0u);

  const bool finite = amax < 0x7F800000u;
  // sums of squares beyond fp32's range, or so small that they lost digits,
  // once more on h scaled by a power of two (uniform over the row)
  float hs = 1.0f;
  if (NORM && finite && amax != 0u && (!(ss <= 3.0e38f) || ss < 0x1p-90f)) {
    hs = ss < 1.0f ? 0x1p+80f : 0x1p-80f;
    float s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if ((int)threadIdx.x + i * T1 < chunks) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = to_f32(h[i].v[e]) * hs;
          s2 = fmaf(f, f, s2);
        }
      }
    if (warps > 1) __syncthreads();  // red_s is read above
    ss = row_sum(s2);
  }

  const float up = __uint_as_float(amax) < 0x1p-100f ? 0x1p+100f : 1.0f;
  const float a = __uint_as_float(amax) * up;
  const float inv = finite && amax != 0u ? __fdiv_rn(127.0f, a) : 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int j = threadIdx.x + i * T1, c = j * 8 - head;
    if (j < chunks) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = to_f32(h[i].v[e]);
      if (NORM && A.gain) {
        const Chunk<T> g = EVEN ? load_vec(gain + j * 8) : load_gain(gain, c, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], to_f32(g.v[e]));
      }
      if (!finite) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
      }
      const uint2 o = code8(v, a, inv, up);
      if (EVEN || (c >= 0 && c + 8 <= d)) {
        *reinterpret_cast<uint2*>(q + j * 8) = o;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e >= 0 && c + e < d) q[j * 8 + e] = (int8_t)((e < 4 ? o.x : o.y) >> (8 * (e & 3)));
      }
    }
  }
  if (threadIdx.x == 0) {
    // one thread, after the codes: r in fp64 (a product that leaves fp32's range
    // on the way cannot spoil the scale)
    double s = 1.0;
    if (!finite) {
      s = __longlong_as_double(0x7FF8000000000000LL);
    } else if (amax != 0u) {
      s = (double)__uint_as_float(amax) / 127.0;
      if (NORM) s /= sqrt((double)ss / ((double)hs * hs) / d + (double)A.eps);
    }
    A.sx[row] = (float)s;
  }
}

template <typename T, bool NORM, bool EVEN>
cudaError_t launch_nc(const CodeArgs& A, int nc, int threads, cudaStream_t s) {
  const int rows = threads == 32 ? 4 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((A.M + rows - 1) / rows));
  cfg.blockDim = dim3(threads, rows);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (nc <= 1) return cudaLaunchKernelEx(&cfg, codes_kernel<T, 1, NORM, EVEN>, A);
  if (nc <= 2) return cudaLaunchKernelEx(&cfg, codes_kernel<T, 2, NORM, EVEN>, A);
  if (nc <= 4) return cudaLaunchKernelEx(&cfg, codes_kernel<T, 4, NORM, EVEN>, A);
  return cudaLaunchKernelEx(&cfg, codes_kernel<T, 8, NORM, EVEN>, A);
}

template <typename T, bool NORM>
cudaError_t launch_rows(const CodeArgs& A, cudaStream_t s) {
  const int chunks = A.d % 8 ? A.d / 8 + 2 : A.d / 8;
  const int nc = A.M <= 296 ? 1 : 4;
  int threads = (chunks + nc - 1) / nc;
  threads = (threads + 31) / 32 * 32;
  if (threads > 1024) threads = 1024;
  const int need = (chunks + threads - 1) / threads;
  if (need > 8) return cudaErrorInvalidValue;
  return A.d % 8 == 0 ? launch_nc<T, NORM, true>(A, need, threads, s) : launch_nc<T, NORM, false>(A, need, threads, s);
}

}  // namespace

cudaError_t launch_int8_codes(const uint16_t* x, const uint16_t* residual, const uint16_t* gain, uint16_t* hidden,
                              int8_t* q, float* sx, int M, int d, bool f16, bool norm, float eps,
                              cudaStream_t stream) {
  const CodeArgs A{x, residual, gain, hidden, q, sx, M, d, eps};
  if (norm) return f16 ? launch_rows<__half, true>(A, stream) : launch_rows<__nv_bfloat16, true>(A, stream);
  return f16 ? launch_rows<__half, false>(A, stream) : launch_rows<__nv_bfloat16, false>(A, stream);
}

cudaError_t launch_int8_pack(const float* W, int8_t* q, float* s, int rows, int d, cudaStream_t stream) {
  if (d % 8) return cudaErrorInvalidValue;
  const CodeArgs A{W, nullptr, nullptr, nullptr, q, s, rows, d, 0.0f};
  const int chunks = d / 8, nc = rows <= 296 ? 1 : 4;
  int threads = (chunks + nc - 1) / nc;
  threads = (threads + 31) / 32 * 32;
  if (threads > 1024) threads = 1024;
  const int need = (chunks + threads - 1) / threads;
  if (need > 8) return cudaErrorInvalidValue;
  return launch_nc<float, false, true>(A, need, threads, stream);
}

}  // namespace paro
