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
// in fp32 (unless it underflows), and so is an fp32 weight.  v * (127 / a) with
// the quotient rounded to fp32 is within 127 * 2^-24 = 7.6e-6 of 127 v / a; only
// where it lies within 2^-16 of a border k + 1/2 (about one value in 30000) does
// the comparison of 254 |v| with (2k + 1) a decide, in fp64, where both products
// are exact (32 bits at most).  So the codes do not depend on any sum's order.
//
// A row is read once, kept in registers as 16-value chunks, and its codes are
// written from there: 3 bytes a value, 7 with a residual.  Chunks are cut at
// multiples of 16 of the flat index, not of the column, so that rows of an odd
// width still move as 16-byte loads and stores; the first and last chunk of such
// a row go value by value, and its gain comes from aligned 16-byte loads shifted
// by the row's phase.  For many rows HBM bounds it: added rows come at its rate
// (norm with a residual, 4096 wide: 4096 more rows in 18.8 us, 6.2 TB/s; codes, 14336
// wide: 2048 more in 13.5 us, 6.5 TB/s), and the instructions, about 14 a value, fill
// 37% of the issue slots.  A call has 4 us (norm) to 8 us (codes) around that, for the
// launch, the first rows' loads with nothing to compute yet, and the last rows: 2048 x
// 4096 with a residual in 13.7 us (4.3 TB/s), 4096 x 8192 in 43.7 us (5.4 TB/s), packing
// 14336 x 4096 fp32 in 44-45 us (6.6 TB/s).  One row's latency is 2.5 us.
#include "int8.cuh"
#include "tc_ptx.cuh"
#include "w4_stream.cuh"  // device_sm_count

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

constexpr int kW = 16;  // values of a chunk

// kW consecutive values of one row, as they lie in memory.
template <typename T>
struct __align__(16) Chunk {
  uint32_t w[kW * sizeof(T) / 4];
};

__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float value(__half v) { return __half2float(v); }
__device__ __forceinline__ float value(float v) { return v; }

__device__ __forceinline__ void values(const Chunk<__nv_bfloat16>& c, float (&v)[kW]) {
#pragma unroll
  for (int i = 0; i < kW / 2; ++i) {
    v[2 * i] = __uint_as_float(c.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(c.w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void values(const Chunk<__half>& c, float (&v)[kW]) {
#pragma unroll
  for (int i = 0; i < kW / 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c.w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void values(const Chunk<float>& c, float (&v)[kW]) {
#pragma unroll
  for (int i = 0; i < kW; ++i) v[i] = __uint_as_float(c.w[i]);
}

// a + b, rounded to T.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  const __half2 b = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <typename T>
__device__ __forceinline__ void add_to(Chunk<T>& a, const Chunk<T>& b) {
  float x[kW], y[kW];
  values(a, x);
  values(b, y);
#pragma unroll
  for (int i = 0; i < kW / 2; ++i)
    a.w[i] = pack2(__fadd_rn(x[2 * i], y[2 * i]), __fadd_rn(x[2 * i + 1], y[2 * i + 1]), T());
}
template <typename T>
__device__ __forceinline__ void times(float (&v)[kW], const Chunk<T>& g) {
  float f[kW];
  values(g, f);
#pragma unroll
  for (int e = 0; e < kW; ++e) v[e] = __fmul_rn(v[e], f[e]);
}

template <typename T>
__device__ __forceinline__ Chunk<T> load_vec(const T* p) {
  Chunk<T> c;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(c) / 16); ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    c.w[4 * i] = u.x, c.w[4 * i + 1] = u.y, c.w[4 * i + 2] = u.z, c.w[4 * i + 3] = u.w;
  }
  return c;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Chunk<T>& c) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(c) / 16); ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(c.w[4 * i], c.w[4 * i + 1], c.w[4 * i + 2], c.w[4 * i + 3]);
}

// Values lo .. hi - 1 of the chunk at p (the others zero), one by one.
__device__ __forceinline__ uint32_t bits(const __nv_bfloat16* p) { return *reinterpret_cast<const uint16_t*>(p); }
__device__ __forceinline__ uint32_t bits(const __half* p) { return *reinterpret_cast<const uint16_t*>(p); }
template <typename T>
__device__ __forceinline__ Chunk<T> load_part(const T* p, int lo, int hi) {
  Chunk<T> c = {};
#pragma unroll
  for (int e = 0; e < kW; ++e)
    if (e >= lo && e < hi) c.w[e / 2] |= bits(p + e) << (16 * (e & 1));
  return c;
}
template <typename T>
__device__ __forceinline__ void store_part(T* p, const Chunk<T>& c, int lo, int hi) {
#pragma unroll
  for (int e = 0; e < kW; ++e)
    if (e >= lo && e < hi) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(c.w[e / 2] >> (16 * (e & 1)));
}

// The chunk at p, columns c .. c + kW - 1 of a row of d, cut to the row: STEP as
// the kernel's.
template <typename T, int STEP>
__device__ __forceinline__ Chunk<T> load_chunk(const T* p, int c, int d) {
  if constexpr (STEP == 16) return load_vec(p);
  if (c >= 0 && c + kW <= d) return load_vec(p);
  if constexpr (STEP == 1) return load_part(p, -c, d - c);
  Chunk<T> o = {};
#pragma unroll
  for (int i = 0; i < (int)(sizeof(o) / 32); ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    o.w[4 * i] = u.x, o.w[4 * i + 1] = u.y, o.w[4 * i + 2] = u.z, o.w[4 * i + 3] = u.w;
  }
  return o;
}
template <typename T, int STEP>
__device__ __forceinline__ void store_chunk(T* p, const Chunk<T>& v, int c, int d) {
  if (STEP == 16 || (c >= 0 && c + kW <= d)) store_vec(p, v);
  else if (STEP == 1) store_part(p, v, -c, d - c);
  else *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

// gain[c .. c + kW - 1], columns outside 0 .. d - 1 zero.  c & 7 is the same for
// all chunks of a row.
template <typename T>
__device__ __forceinline__ Chunk<T> load_gain(const T* g, int c, int d) {
  const int a = c & ~7, sh = c & 7;
  if (a < 0 || a + kW + 8 > d) return load_part(g + c, -c, d - c);
  uint32_t w[kW / 2 + 4];
#pragma unroll
  for (int i = 0; i < (kW + 8) / 8; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(g + a)[i];
    w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
  }
  if (sh & 4) {
#pragma unroll
    for (int i = 0; i < kW / 2 + 2; ++i) w[i] = w[i + 2];
  }
  if (sh & 2) {
#pragma unroll
    for (int i = 0; i < kW / 2 + 1; ++i) w[i] = w[i + 1];
  }
  if (sh & 1) {
#pragma unroll
    for (int i = 0; i < kW / 2; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  Chunk<T> o;
#pragma unroll
  for (int i = 0; i < kW / 2; ++i) o.w[i] = w[i];
  return o;
}

// The largest magnitude met so far, as bits: of two 16-bit values side by side, or
// of one fp32.  Magnitudes order as unsigned numbers, infinity and NaN last.
template <typename T>
__device__ __forceinline__ uint32_t widest(uint32_t m, const Chunk<T>& c) {
  constexpr uint32_t kMask = sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
#pragma unroll
  for (int i = 0; i < (int)(kW * sizeof(T) / 4); i += 2) {
    if constexpr (sizeof(T) == 2) m = __vimax3_u16x2(m, c.w[i] & kMask, c.w[i + 1] & kMask);
    else m = __vimax3_u32(m, c.w[i] & kMask, c.w[i + 1] & kMask);
  }
  return m;
}
// The wider of the two halves as fp32 bits.
__device__ __forceinline__ uint32_t widest_bits(uint32_t m, __nv_bfloat16) { return max(m & 0xFFFFu, m >> 16) << 16; }
__device__ __forceinline__ uint32_t widest_bits(uint32_t m, __half) {
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)max(m & 0xFFFFu, m >> 16))));
}
__device__ __forceinline__ uint32_t widest_bits(uint32_t m, float) { return m; }

// The code of v where 127 v / a lies next to a border between two codes.
__device__ __noinline__ float border_code(float v, float a, float inv) {
  const int k = (int)fabsf(__fmul_rn(v, inv));  // near k + 1/2: the whole part is certain
  const double lhs = 254.0 * (double)fabsf(v), rhs = (double)(2 * k + 1) * (double)a;
  const int m = lhs > rhs ? k + 1 : (lhs < rhs ? k : k + (k & 1));
  return v < 0.0f ? -(float)m : (float)m;
}

// Codes of a chunk's values.  Adding 1.5 * 2^23 rounds to a whole number, ties to
// even, and leaves it in the sum's low bits.
__device__ __forceinline__ uint4 codes_of(const float (&v)[kW], float a, float inv) {
  constexpr float kWhole = 12582912.0f, kNear = 0.5f - 0x1p-16f;
  uint32_t o[kW / 4];
#pragma unroll
  for (int i = 0; i < kW; i += 4) {
    float m[4], off[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e] = __fmaf_rn(v[i + e], inv, kWhole);
      off[e] = __fmaf_rn(v[i + e], inv, -__fsub_rn(m[e], kWhole));
    }
    // three-input minima and maxima
    const float lo = fminf(fminf(fminf(off[0], off[1]), off[2]), off[3]);
    const float hi = fmaxf(fmaxf(fmaxf(off[0], off[1]), off[2]), off[3]);
    if (fmaxf(hi, -lo) > kNear) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (fabsf(off[e]) > kNear) m[e] = __fadd_rn(border_code(v[i + e], a, inv), kWhole);
    }
    o[i / 4] = __byte_perm(__byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0040),
                           __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0040), 0x5410);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A row's scale, in fp64: a product that leaves fp32's range on the way cannot
// spoil it.  ss: the sum of (hs h)^2.
template <bool NORM>
__device__ __forceinline__ float row_scale(float amax, bool finite, float ss, float hs, int d, float eps) {
  if (!finite) return __int_as_float(0x7FC00000);
  if (amax == 0.0f) return 1.0f;
  const double s = (double)amax / 127.0;
  return (float)(NORM ? s / sqrt((double)ss / ((double)hs * hs) / d + (double)eps) : s);
}

// True where fp32 sums of squares overflowed, or lost digits to underflow.
__device__ __forceinline__ bool out_of_range(float ss) { return !(ss <= 3.0e38f) || ss < 0x1p-90f; }

// threadIdx.x runs over a row's chunks (NC of them a thread, blockDim.x apart),
// threadIdx.y over the rows of the CTA (more than one only at 32 threads a row).
// STEP: 16 or 8 where d is a multiple of it, every chunk starts at a column
// multiple of kW, and with 8 the last may be half and codes are stored by 8 bytes;
// else 1.
template <typename T, int NC, bool NORM, int STEP>
__global__ void __launch_bounds__(1024)
codes_kernel(const CodeArgs A) {
  constexpr bool EVEN = STEP > 1;
  __shared__ uint32_t red_a[32];
  __shared__ float red_s[32];
  ptx::grid_trigger();
  ptx::grid_wait();  // launched over the end of the kernel before; nothing is read or written until that is done
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= A.M) return;  // whole warps: a CTA of several rows has one warp for each and no barrier
  const int d = A.d, T1 = blockDim.x;
  const long long base = row * d, first = EVEN ? base : base & ~(long long)(kW - 1);  // flat index of the row, of its first chunk
  const int head = EVEN ? 0 : (int)(base - first);
  const int chunks = (head + d + kW - 1) / kW;
  const bool with_res = NORM && A.residual != nullptr, with_gain = NORM && A.gain != nullptr;
  const T* x = static_cast<const T*>(A.x) + first;
  const T* res = static_cast<const T*>(A.residual) + (with_res ? first : 0);
  const T* gain = static_cast<const T*>(A.gain);
  T* hid = static_cast<T*>(A.hidden) + (with_res ? first : 0);
  int8_t* q = A.q + first;

  // All loads of a thread come before its first store (hidden may be x or the
  // residual, so the compiler would keep their order), to be in flight together.
  // Values stay packed and are multiplied by their gains twice: registers decide
  // how many rows an SM has in flight.
  Chunk<T> h[NC];
  {
    [[maybe_unused]] Chunk<T> r[NORM ? NC : 1];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int j = threadIdx.x + i * T1, c = j * kW - head;
      if (j < chunks) {
        h[i] = load_chunk<T, STEP>(x + j * kW, c, d);
        if constexpr (NORM)
          if (with_res) r[i] = load_chunk<T, STEP>(res + j * kW, c, d);
      }
    }
    if constexpr (NORM)
      if (with_res) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int j = threadIdx.x + i * T1, c = j * kW - head;
          if (j < chunks) {
            add_to(h[i], r[i]);
            store_chunk<T, STEP>(hid + j * kW, h[i], c, d);
          }
        }
      }
  }
  // the values of a chunk whose codes are wanted
  auto row_values = [&](int i, int j, float (&v)[kW]) {
    values(h[i], v);
    if constexpr (NORM)
      if (with_gain) times(v, EVEN ? load_chunk<T, STEP>(gain + j * kW, j * kW, d) : load_gain(gain, j * kW - head, d));
  };
  uint32_t wide = 0u;  // bits of the largest |v|
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int j = threadIdx.x + i * T1;
    if (j < chunks) {
      if constexpr (NORM) {
        float v[kW];
        values(h[i], v);
#pragma unroll
        for (int e = 0; e < kW; ++e) ss = fmaf(v[e], v[e], ss);
        if (with_gain) times(v, EVEN ? load_chunk<T, STEP>(gain + j * kW, j * kW, d) : load_gain(gain, j * kW - head, d));
        Chunk<float> c;
#pragma unroll
        for (int e = 0; e < kW; ++e) c.w[e] = __float_as_uint(v[e]);
        wide = widest(wide, c);
      } else {
        wide = widest(wide, h[i]);
      }
    }
  }
  if constexpr (!NORM) wide = widest_bits(wide, T());

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T1 >> 5;
  // both reductions at once
  auto reduce = [&]() {
    wide = __reduce_max_sync(0xffffffffu, wide);
    if (NORM) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (warps > 1) {
      if (lane == 0) {
        red_a[warp] = wide;
        if (NORM) red_s[warp] = ss;
      }
      __syncthreads();
      wide = __reduce_max_sync(0xffffffffu, lane < warps ? red_a[lane] : 0u);
      if (NORM) {
        ss = lane < warps ? red_s[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      }
    }
  };
  reduce();
  const float amax = __uint_as_float(wide);
  const bool finite = wide < 0x7F800000u;
  // sums of squares beyond fp32's range, or so small that they lost digits,
  // once more on h scaled by a power of two (uniform over the row, and rare)
  float hs = 1.0f;
  if (NORM && finite && amax != 0.0f && out_of_range(ss)) {
    hs = ss < 1.0f ? 0x1p+80f : 0x1p-80f;
    ss = 0.0f;
    const T* hp = with_res ? hid : x;
    for (int j = threadIdx.x; j < chunks; j += T1)
      for (int e = 0; e < kW; ++e) {
        const int c = j * kW - head + e;
        const float f = c >= 0 && c < d ? value(hp[j * kW + e]) * hs : 0.0f;
        ss = fmaf(f, f, ss);
      }
    if (warps > 1) __syncthreads();  // the first sums have been read
    reduce();
  }

  // rows that are not finite get codes 0; for the smallest magnitudes v and a are
  // taken a power of two larger, so that 127 / a stays in fp32's range
  const float up = amax < 0x1p-100f ? 0x1p+100f : 1.0f;
  const float a = amax * up, inv = finite && amax != 0.0f ? __fdiv_rn(127.0f, a) : 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int j = threadIdx.x + i * T1, c = j * kW - head;
    if (j < chunks) {
      float v[kW];
      row_values(i, j, v);
      if (!finite || up != 1.0f) {
#pragma unroll
        for (int e = 0; e < kW; ++e) v[e] = finite ? v[e] * up : 0.0f;
      }
      const uint4 o = codes_of(v, a, inv);
      if (STEP == 8) {
        *reinterpret_cast<uint2*>(q + j * kW) = make_uint2(o.x, o.y);
        if (c + kW <= d) *reinterpret_cast<uint2*>(q + j * kW + 8) = make_uint2(o.z, o.w);
      } else if (EVEN || (c >= 0 && c + kW <= d)) {
        *reinterpret_cast<uint4*>(q + j * kW) = o;
      } else {
        const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < kW; ++e)
          if (c + e >= 0 && c + e < d) q[j * kW + e] = (int8_t)(w[e / 4] >> (8 * (e & 3)));
      }
    }
  }
  if (threadIdx.x == 0) A.sx[row] = row_scale<NORM>(amax, finite, ss, hs, d, A.eps);
}

template <typename T, bool NORM, int STEP>
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
  if (nc <= 1) return cudaLaunchKernelEx(&cfg, codes_kernel<T, 1, NORM, STEP>, A);
  if (nc <= 2) return cudaLaunchKernelEx(&cfg, codes_kernel<T, 2, NORM, STEP>, A);
  return cudaLaunchKernelEx(&cfg, codes_kernel<T, 4, NORM, STEP>, A);
}

template <typename T, bool NORM>
cudaError_t launch_rows(const CodeArgs& A, cudaStream_t s) {
  // Chunks a thread takes.  Each row costs its threads the same instructions for
  // addresses, reduction and scale, so fewer threads with more chunks gain, as long
  // as enough of them are in flight and registers last (a norm's do for two chunks).
  // Measured, us, with 1, 2, 4 chunks (bf16): norm 300 x 8960: 8.0, 7.0, 10.6; 2048
  // x 4096: 15.6, 13.7, 18.1; 4096 x 8192: 54.7, 43.7, 54.0; codes 300 x 8960: 4.7,
  // 6.1, 8.8; 2048 x 1536: 4.7, 6.9, 8.5; 4096 x 8192: 25.2, 23.9, 23.2; 2048 x
  // 14336: 32.8, 23.9, 21.5; fp32 14336 x 4096: 45.0, 44.4, 62.1.
  const int chunks = A.d % 8 ? A.d / kW + 2 : (A.d + kW - 1) / kW;
  const long long per_sm = A.M * chunks / device_sm_count();
  const int want = NORM ? (per_sm >= 1024 ? 2 : 1) : sizeof(T) == 2 && per_sm >= 8192 ? 4 : per_sm >= 2048 ? 2 : 1;
  int threads = ((chunks + want - 1) / want + 31) / 32 * 32;
  if (threads > 1024) threads = 1024;
  const int need = (chunks + threads - 1) / threads;
  if (need > 4) return cudaErrorInvalidValue;
  if (A.d % 16 == 0) return launch_nc<T, NORM, 16>(A, need, threads, s);
  if constexpr (sizeof(T) == 4) return cudaErrorInvalidValue;  // weights' rows are whole chunks
  else return A.d % 8 == 0 ? launch_nc<T, NORM, 8>(A, need, threads, s) : launch_nc<T, NORM, 1>(A, need, threads, s);
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
  const CodeArgs A{W, nullptr, nullptr, nullptr, q, s, rows, d, 0.0f};
  return launch_rows<float, false>(A, stream);
}

}  // namespace paro
