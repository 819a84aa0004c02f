// int8 linears for many tokens: pairs of CTAs on 256 x 256 tiles of the 5th-
// generation tensor cores (tcgen05 kind::i8, cta_group::2).
//
// A pair (one CTA on each of two SMs) walks tiles of 256 tokens x 256 weight
// rows; with a gate the rows are 128 of each weight matrix, so that a token's
// gate and up sums meet in one thread.  Each CTA holds half of either operand:
// 128 tokens and 128 weight rows (the gate's in one CTA, up's in the other), 128
// columns of d_in a stage, and the sums of its 128 tokens in tensor memory:
//   warp 0    TMA: its halves of a stage, completing on the first CTA's barrier;
//   warp 1    MMA (first CTA only): four tcgen05.mma 256 x 256 x 32 a stage on
//             both SMs, then a commit that frees the stage in both CTAs;
//   warps 2-9 epilogue: thread = token, half of the tile's channels, 32 at a
//             time; scales, gate or bias, rounding, then through shared memory
//             (64-byte swizzle) and a TMA store, which writes whole sectors and
//             leaves out what lies outside y.
// A 256 x 256 tile on a pair reads each operand once for both SMs' tensor cores, 32
// KB an SM for 512 clocks of MMAs; a 128 x 256 tile on one SM would read 48.
// Bound by the tensor cores under the power cap, and by the last round of tiles:
// 2048 tokens 14336 -> 4096 in 85 us (2.83 PFLOP/s; 98 us when it runs for
// seconds), gated 4096 -> 14336 in 166 us (2.90).
// Two sets of sums (2 x 256 columns of tensor memory) let the next tile's MMAs
// run under a tile's epilogue.  Every wait on an mbarrier is bounded; when one runs
// out, the roles of both CTAs end, their copies and MMAs in flight are waited for,
// and the call reports PARO_ERR_TIMEOUT.
#include "int8.cuh"
#include "tc_ptx.cuh"
#include "w4_stream.cuh"  // device_sm_count
#include "w8a8.cuh"

namespace paro {
namespace {

using namespace ptx;

constexpr int kTile = 256, kHalf = 128, kK = 128, kStages = 5;
constexpr int kEpiWarps = 8, kThreads = 64 + 32 * kEpiWarps;
constexpr int kOutBytes = 32 * 64;  // a warp's 32 tokens x 32 channels on their way out; two of them a warp
constexpr int kHalfBytes = kHalf * kK, kStageBytes = 2 * kHalfBytes;
constexpr int kUsed = kStages * kStageBytes + 2 * kEpiWarps * kOutBytes + 1024;
// The CTA takes all of tensor memory, so it asks for more shared memory than it
// uses: none that wants tensor memory beside it may fit the same SM (w8a8_few.cu).
constexpr int kSmem = 216 * 1024;
static_assert(kUsed <= kSmem && kSmem >= (228 - 16) * 1024, "shared memory of a CTA");

struct ManyArgs {
  CUtensorMap q, w, w2, out;  // out: y in boxes of 32 x 32, where its rows are a multiple of 16 bytes
  const float* sx;
  const float* sw;
  const float* sw2;
  const uint16_t* bias;
  uint16_t* y;
  int M, d_out, blocks;  // blocks: of 128 columns of d_in
  int mtiles, tiles;
  W8a8Hooks hooks;
};

template <bool GATED, bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
w8a8_many_kernel(const __grid_constant__ ManyArgs A, int* status) {
  constexpr int NC = GATED ? kHalf : kTile;  // output channels of a tile
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, s_issued, s_committed;
  // a tile's channel scales, with the up scales behind the gate's, and its bias
  __shared__ __align__(16) float s_sw[2][kTile], s_bias[2][GATED ? 4 : kTile];

  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t ring = smem_u32(smem);
  const uint32_t b_full = smem_u32(&bars[0]), b_empty = smem_u32(&bars[kStages]);
  const uint32_t b_acc_full = smem_u32(&bars[2 * kStages]), b_acc_empty = smem_u32(&bars[2 * kStages + 2]);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    prefetch_map(&A.q);
    prefetch_map(GATED && rank ? &A.w2 : &A.w);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(b_full + 8 * s, 1);   // (first CTA) its own arrival and both CTAs' bytes
      mbar_init(b_empty + 8 * s, 1);  // the commit of the MMAs that read the stage
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(b_acc_full + 8 * s, 1);
      mbar_init(b_acc_empty + 8 * s, 2 * kEpiWarps);  // (first CTA) the epilogue warps of both CTAs
    }
    abort_flag = 0;
    s_issued = 0;
    s_committed = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(&tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // the other CTA's barriers and tensor memory are ready
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  grid_trigger();
  grid_wait();  // the kernel before is done: what follows reads and writes

  auto fail = [&]() {
    report_status(status, kStatusTimeout);
    atomicExch(&abort_flag, 1);
  };
  // a wait that also ends, false, when another role gave up
  auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait_unless(bar, parity, &abort_flag, A.hooks.wait); };

  // One thread's step (wait, barrier, copies or MMAs) has to stay below the 512
  // clocks that a stage's MMAs take: stages and parities are counted, and the abort
  // flag is looked at only while waiting.
  if (warp == 0) {
    if (lane == 0) {
      const CUtensorMap* wmap = GATED && rank ? &A.w2 : &A.w;
      const uint32_t first = mapa(b_full, 0);  // the first CTA's barriers
      int it = 0, s = 0;
      uint32_t phase = 1;
      bool ok = true;
#pragma unroll 1
      for (int t = pair; ok && t < A.tiles; t += pairs) {
        const int m0 = (t % A.mtiles) * kTile + rank * kHalf;
        const int n0 = (t / A.mtiles) * NC + (GATED ? 0 : rank * kHalf);
#pragma unroll 1
        for (int x = 0; x < A.blocks * kK; x += kK, ++it) {
          if (it >= kStages) {
            if (rank == A.hooks.rank) { ok = false; break; }
            if (!wait(b_empty + 8 * s, phase)) { fail(); ok = false; break; }
          }
          const uint32_t bar = first + 8 * s, dst = ring + s * kStageBytes;
          if (rank == 0) mbar_expect_tx(b_full + 8 * s, 2 * kStageBytes);
          tma_load_pair(dst, &A.q, x, m0, bar);
          tma_load_pair(dst + kHalfBytes, wmap, x, n0, bar);
          if (++s == kStages) s = 0, phase ^= 1;
        }
      }
      s_issued = it;
      // the last stages' commits have arrived before this CTA, and its barriers with it, may go
      if (it < kStages) s = 0, phase = 0;
      for (int n = it < kStages ? it : kStages; ok && n > 0; --n) {
        if (!wait(b_empty + 8 * s, phase)) { fail(); ok = false; }
        if (++s == kStages) s = 0, phase ^= 1;
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = idesc_s8(kTile, kTile);
      int it = 0, j = 0, s = 0;
      uint32_t phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int t = pair; ok && t < A.tiles; t += pairs, ++j) {
        const uint32_t acc = tmem + (j & 1) * kTile;
        if (j >= 2 && !wait(b_acc_empty + 8 * (j & 1), ((j >> 1) - 1) & 1)) { fail(); break; }
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < A.blocks; ++k, ++it) {
          if (!wait(b_full + 8 * s, phase)) { fail(); ok = false; break; }
          tc_fence_after();
          const uint64_t a = desc_sw128(ring + s * kStageBytes), b = desc_sw128(ring + s * kStageBytes + kHalfBytes);
#pragma unroll
          for (int kk = 0; kk < kK / 32; ++kk) mma_s8<2>(acc, a + kk * 2, b + kk * 2, idesc, (k > 0 || kk > 0) ? 1u : 0u);
          commit_pair(b_empty + 8 * s);
          if (++s == kStages) s = 0, phase ^= 1;
        }
        if (ok) commit_pair(b_acc_full + 8 * (j & 1));
      }
      s_committed = it;
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    unsigned char* out = smem + kStages * kStageBytes + (warp - 2) * 2 * kOutBytes;
    const bool by_tma = (A.d_out & 7) == 0;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    int j = 0, turn = 0;
    bool ok = true;  // the same in all lanes; a warp that gave up still meets the others at their barriers
#pragma unroll 1
    for (int t = pair; t < A.tiles; t += pairs, ++j) {
      const int acc = j & 1;
      const int m_warp = (t % A.mtiles) * kTile + rank * kHalf + quarter * 32, m = m_warp + lane, n0 = (t / A.mtiles) * NC;
      const TokenScale sx = token_scale(m < A.M ? A.sx[m] : 0.0f);
      const bool any_large = __any_sync(0xffffffffu, sx.back != 1.0f);
      // the tile's channel values, while its MMAs run; two sets, so that a warp
      // may be one tile ahead of another
      for (int c = threadIdx.x - 64; c < kTile; c += 32 * kEpiWarps) {
        const bool up = GATED && c >= kHalf;
        const int n = n0 + (up ? c - kHalf : c);
        s_sw[acc][c] = n < A.d_out ? (up ? A.sw2 : A.sw)[n] : 0.0f;
        if constexpr (!GATED) s_bias[acc][c] = A.bias && n < A.d_out ? from_16<F16>(A.bias[n]) : 0.0f;
      }
      asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kEpiWarps) : "memory");
      if (!ok) continue;
      ok = __all_sync(0xffffffffu, wait(b_acc_full + 8 * acc, (j >> 1) & 1));
      if (!ok) { fail(); continue; }
      tc_fence_after();
      // (none where all of the warp's tokens lie behind the last one: every use of a
      // box below commits one store, which the wait two uses later counts on)
      const int c_end = m_warp < A.M ? min((half + 1) * (NC / 2), A.d_out - n0) : 0;
#pragma unroll 1
      for (int c0 = half * (NC / 2); c0 < c_end; c0 += 32) {
        int v[32], u[GATED ? 32 : 1];
        tmem_ld(lanes + acc * kTile + c0, v);
        if constexpr (GATED) tmem_ld(lanes + acc * kTile + kHalf + c0, u);
        tmem_ld_wait();
        const int n = n0 + c0;
        uint32_t o[16];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&s_sw[acc][c0 + c]);
          float f[4] = {w8a8_scaled(v[c], sx.s, w.x), w8a8_scaled(v[c + 1], sx.s, w.y), w8a8_scaled(v[c + 2], sx.s, w.z),
                        w8a8_scaled(v[c + 3], sx.s, w.w)};
          if constexpr (GATED) {
            const float4 w2 = *reinterpret_cast<const float4*>(&s_sw[acc][kHalf + c0 + c]);
            f[0] = w8a8_gate(f[0], w8a8_scaled(u[c], sx.s, w2.x));
            f[1] = w8a8_gate(f[1], w8a8_scaled(u[c + 1], sx.s, w2.y));
            f[2] = w8a8_gate(f[2], w8a8_scaled(u[c + 2], sx.s, w2.z));
            f[3] = w8a8_gate(f[3], w8a8_scaled(u[c + 3], sx.s, w2.w));
          } else {
            const float4 b = *reinterpret_cast<const float4*>(&s_bias[acc][c0 + c]);
            f[0] = __fmaf_rn(f[0], sx.back, b.x), f[1] = __fmaf_rn(f[1], sx.back, b.y);
            f[2] = __fmaf_rn(f[2], sx.back, b.z), f[3] = __fmaf_rn(f[3], sx.back, b.w);
          }
          o[c / 2] = to_16<F16>(f[0]) | ((uint32_t)to_16<F16>(f[1]) << 16);
          o[c / 2 + 1] = to_16<F16>(f[2]) | ((uint32_t)to_16<F16>(f[3]) << 16);
        }
        // row = token, 64 bytes, its 16-byte parts swapped by bits 1-2 of the row
        unsigned char* box = out + turn * kOutBytes;
        turn ^= 1;
        bulk_read_wait<1>();  // the box before the last has left its place
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(box + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        if (GATED && any_large) {
          // tokens of large scales once more, with the factor that a gate cannot take
          // later (two multiplications for every output would cost 3% of a short call)
#pragma unroll 1
          for (int c = 0; c < 32; ++c) {
            int g1, u1;
            tmem_ld(lanes + acc * kTile + c0 + c, g1);
            tmem_ld(lanes + acc * kTile + kHalf + c0 + c, u1);
            tmem_ld_wait();
            const float f = w8a8_gate(w8a8_scaled(g1, sx.s, s_sw[acc][c0 + c]) * sx.back,
                                      w8a8_scaled(u1, sx.s, s_sw[acc][kHalf + c0 + c]) * sx.back);
            *reinterpret_cast<uint16_t*>(box + lane * 64 + (((c >> 3) ^ ((lane >> 1) & 3)) << 4) + (c & 7) * 2) = to_16<F16>(f);
          }
        }
        if (by_tma) {
          async_fence();
          __syncwarp();
          if (lane == 0) {
            tma_store(&A.out, smem_u32(box), n, m_warp);
            bulk_commit();
          }
        } else {
          // rows of y at any even address: 32 or, where rows start on 4 bytes, 2 x 16 lanes side by side
          __syncwarp();
          const int wide = (A.d_out & 1) == 0, c = wide ? 2 * (lane & 15) : lane;
#pragma unroll 8
          for (int r = wide ? lane >> 4 : 0; r < 32; r += 1 + wide) {
            const unsigned char* from = box + r * 64 + (((c >> 3) ^ ((r >> 1) & 3)) << 4) + (c & 7) * 2;
            uint16_t* to = A.y + (size_t)(m_warp + r) * A.d_out + n + c;
            if (m_warp + r < A.M && n + c < A.d_out) {
              if (wide) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
              else *to = *reinterpret_cast<const uint16_t*>(from);
            }
          }
        }
      }
      __syncwarp();
      tc_fence_before();
      if (lane == 0) mbar_arrive_cluster(mapa(b_acc_empty + 8 * acc, 0));
    }
    bulk_wait();
  }

  // ---- teardown ----------------------------------------------------------------------
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // both CTAs are done with the other's barriers and shared memory, unless a wait gave up:
  cluster_wait();
  bool any = abort_flag != 0;
  any |= ld_cluster(mapa(smem_u32(&abort_flag), rank ^ 1)) != 0;
  if (any) {
    // then copies and MMAs in flight end before the memory goes away.  The two
    // CTAs may have issued different numbers of stages: a slot's last phase is
    // made whole by what the one that stopped first did not send
    if (rank == 0 && threadIdx.x == 0) {
      const int mine = s_issued, theirs = ld_cluster(mapa(smem_u32(&s_issued), 1));
      auto last_of = [](int cnt, int slot) { return cnt > slot ? slot + ((cnt - 1 - slot) / kStages) * kStages : -1; };
      bool done = true;
      for (int s = 0; s < kStages; ++s) {
        const int a = last_of(mine, s), b = last_of(theirs, s), jm = last_of(s_committed, s);
        if (a > b) mbar_complete_tx(b_full + 8 * s, kStageBytes);
        if (b > a) mbar_expect_tx(b_full + 8 * s, kStageBytes);
        const int last = a > b ? a : b;
        if (last >= 0) done = mbar_wait(b_full + 8 * s, (last / kStages) & 1) && done;
        if (jm >= 0) done = mbar_wait(b_empty + 8 * s, (jm / kStages) & 1) && done;
      }
      if (!done) report_status(status, kStatusTimeout);
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem, 512);
  }
  cluster_arrive();  // neither CTA ends while the other may still read it
  cluster_wait();
}

template <bool GATED, bool F16>
cudaError_t launch_many(const ManyArgs& A, int* status, cudaStream_t s) {
  auto kernel = w8a8_many_kernel<GATED, F16>;
  static std::atomic<uint64_t> limit{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kSmem, limit);
  if (e != cudaSuccess) return e;
  const int pairs = device_sm_count() / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (A.tiles < pairs ? A.tiles : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, A, status);
}

}  // namespace

cudaError_t launch_w8a8_many(const W8a8Args& a, int* status, cudaStream_t stream) {
  ManyArgs A;
  if (!w8_map(&A.q, a.q, a.M, a.d_in, kHalf) || !w8_map(&A.w, a.w, a.d_out, a.d_in, kHalf) ||
      (a.w2 && !w8_map(&A.w2, a.w2, a.d_out, a.d_in, kHalf)))
    return cudaErrorInvalidValue;
  if (a.d_out % 8 == 0 && !w8_out_map(&A.out, a.y, a.M, a.d_out)) return cudaErrorInvalidValue;
  A.sx = a.sx;
  A.sw = a.sw;
  A.sw2 = a.sw2;
  A.bias = a.bias;
  A.y = a.y;
  A.M = a.M;
  A.d_out = a.d_out;
  A.blocks = (a.d_in + kK - 1) / kK;
  A.hooks = w8a8_hooks(2);
  A.mtiles = (a.M + kTile - 1) / kTile;
  const int nc = a.w2 ? kHalf : kTile;
  A.tiles = A.mtiles * ((a.d_out + nc - 1) / nc);
  if (a.w2) return a.f16 ? launch_many<true, true>(A, status, stream) : launch_many<true, false>(A, status, stream);
  return a.f16 ? launch_many<false, true>(A, status, stream) : launch_many<false, false>(A, status, stream);
}

}  // namespace paro
