// int8 linears for few tokens: weights are the tensor core's 128 rows, tokens its
// columns, and the weights stream from HBM once.
//
// One CTA takes 128 output channels (with a gate, the same 128 of both weight
// matrices), TN tokens and a share of d_in; the CTAs of a cluster hold the
// shares of one tile:
//   warp 0    TMA: per 128 columns of d_in the weights' 128 x 128 bytes and the
//             tokens' TN x 128 bytes (128-byte swizzle) into a ring of stages;
//   warp 1    MMA: four tcgen05.mma kind::i8 (128 x TN x 32) a stage, into 32-bit
//             sums in tensor memory;
//   warps 2-5 epilogue: thread = channel.  Token t of a tile belongs to CTA t mod
//             the cluster's size, which adds up all shares' sums for it and
//             writes y (a warp takes a token, a lane four channels).  Up to 32
//             tokens, every CTA stores its sums into the owners' shared memory,
//             beside their rings, and ends; more stay in the CTA's own, where the
//             ring was, for the owners to read between two cluster barriers.
//             Measured, stored / read, us: 16 tokens gated 1536 -> 8960 9.3 /
//             10.2, 1 token 1536 -> 1536 3.7 / 4.2; 64 tokens 4096 -> 4096 11.0 /
//             9.6, 128 tokens 14.0 / 11.8.
// Whole sums: the order of the shares does not matter, there is no workspace and
// nothing to reset between calls.
//
// Bound by the weights from HBM and about 3 us of set-up, first loads and shares'
// sums around them: one token 4096 -> 14336 in 13.5 us (58.7 MB, 4.3 TB/s), 14336 ->
// 4096 in 13.2-13.6 us, gated 4096 -> 14336 in 22.6 us (5.2 TB/s), 1536 -> 1536 in 3.4
// us; between 4096 -> 4096 and 14336 -> 4096 the added bytes come at 5.9 TB/s.
//
// The launch overlaps the kernel before it: until that one is done a CTA sets up
// its barriers and asks for its weights in L2 only, which is right whoever wrote
// them last; every read and write of its own comes after the wait.
//
// Every wait on an mbarrier is bounded: when one runs out, the CTA's roles end, its
// copies and MMAs in flight are waited for, no CTA writes what it has no sums of, and
// the call reports PARO_ERR_TIMEOUT.
#include <climits>

#include "int8.cuh"
#include "tc_ptx.cuh"
#include "w4_stream.cuh"  // device_sm_count
#include "w8a8.cuh"

namespace paro {
namespace {

using namespace ptx;

constexpr int kRows = 128, kK = 128, kThreads = 192;
constexpr int kMaxSmem = 105 * 1024;  // a CTA's ring, or its sums
constexpr int kMaxStages = 8, kMaxSplit = 8;  // 8: the portable size of a cluster
// Stages asked for in L2 before the kernel before is done.  With 0, 2, 4, 16: one
// token 4096 -> 4096 7.3, 6.6, 6.6, 6.6 us, 14336 -> 4096 13.7, 13.7, 13.3, 13.8,
// gated 16 tokens 1536 -> 8960 9.4, 8.7, 9.1, 9.1, 203 tokens 1552 -> 1100 6.0, 6.2,
// 6.5, 6.5, gated 4096 -> 14336 23.9, 23.3, 23.5, 28.0.
constexpr int kAhead = 2;

struct FewArgs {
  CUtensorMap w, w2, q;
  // in front: what the first copies wait for is in one line of the constant cache
  W8a8Hooks hooks;
  int M, d_out, blocks;      // blocks: of 128 columns of d_in
  int split, stages, xrows;  // xrows: tokens a copy brings, at most TN
  const float* sx;
  const float* sw;
  const float* sw2;
  const uint16_t* bias;
  uint16_t* y;
};

template <int TN, bool GATED>
struct FewGeo {
  static constexpr int NW = GATED ? 2 : 1;
  static constexpr int STAGE = NW * kRows * kK + TN * kK;
  static constexpr int SUMS = TN * NW * kRows * 4;  // the sums that a CTA holds
  static constexpr bool STORED = TN <= 32;          // ... of its own tokens, beside the ring
  static constexpr int COLS = NW * TN < 32 ? 32 : NW * TN;
};

template <int TN, bool GATED, bool F16>
__global__ void __launch_bounds__(kThreads)
w8a8_few_kernel(const __grid_constant__ FewArgs A, int* status) {
  using Geo = FewGeo<TN, GATED>;
  constexpr int NW = Geo::NW;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, s_issued, s_committed;
  __shared__ TokenScale s_sx[TN];

  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t ring = smem_u32(smem);
  const uint32_t b_full = smem_u32(&bars[0]), b_empty = smem_u32(&bars[kMaxStages]);
  const uint32_t b_acc = smem_u32(&bars[2 * kMaxStages]), b_sums = smem_u32(&bars[2 * kMaxStages + 1]);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = A.split, stages = A.stages;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int n0 = (blockIdx.x / split) * kRows, m0 = blockIdx.y * TN;
  const int k0 = (int)((long long)rank * A.blocks / split), k1 = (int)((long long)(rank + 1) * A.blocks / split);
  const int nk = k1 - k0;

  if (warp == 0 && lane == 0) {
    prefetch_map(&A.w);
    prefetch_map(&A.q);
    if constexpr (GATED) prefetch_map(&A.w2);
    for (int s = 0; s < stages; ++s) {
      mbar_init(b_full + 8 * s, 1);
      mbar_init(b_empty + 8 * s, 1);
    }
    mbar_init(b_acc, 1);
    mbar_init(b_sums, 4 * split);  // the epilogue warps of all shares
    abort_flag = 0;
    s_issued = 0;
    s_committed = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(&tmem_slot), Geo::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  cluster_arrive();  // (the wait comes before the first store to another CTA)
  grid_trigger();
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < nk && i < kAhead; ++i) {
      tma_prefetch(&A.w, (k0 + i) * kK, n0);
      if constexpr (GATED) tma_prefetch(&A.w2, (k0 + i) * kK, n0);
    }
  }
  grid_wait();

  auto fail = [&]() {
    report_status(status, kStatusTimeout);
    atomicExch(&abort_flag, 1);
  };
  // a wait that also ends, false, when another role gave up
  auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait_unless(bar, parity, &abort_flag, A.hooks.wait); };

  // The two loops below set the pace: each step of one thread costs 280 clocks and
  // up (waits, barrier, copies), so stages and parities are counted, not divided,
  // and the abort flag is looked at only while waiting.  With divisions a step took
  // 800 clocks, which held every SM to 40 GB/s.
  if (warp == 0) {
    if (lane == 0) {
      int i = 0, s = 0, x = k0 * kK;
      uint32_t phase = 1, dst = ring, bar = b_full;
      bool ok = true;
#pragma unroll 1
      for (; i < nk; ++i, x += kK) {
        // (phase starts at 1: the first wait, a round later, is for parity 0)
        if (i >= stages) {
          if (rank == A.hooks.rank) { ok = false; break; }
          if (!wait(bar + (b_empty - b_full), phase)) { fail(); ok = false; break; }
        }
        mbar_expect_tx(bar, (NW * kRows + A.xrows) * kK);
        tma_load(dst, &A.w, x, n0, bar);
        if constexpr (GATED) tma_load(dst + kRows * kK, &A.w2, x, n0, bar);
        tma_load(dst + NW * kRows * kK, &A.q, x, m0, bar);
        if (++s == stages) s = 0, phase ^= 1, dst = ring, bar = b_full;
        else dst += Geo::STAGE, bar += 8;
      }
      s_issued = i;
      // the last stages' commits have arrived before the CTA, and the barriers with it, may go
      if (i < stages) s = 0, phase = 0;
      for (int n = i < stages ? i : stages; ok && n > 0; --n) {
        if (!wait(b_empty + 8 * s, phase)) { fail(); ok = false; }
        if (++s == stages) s = 0, phase ^= 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_s8(kRows, TN);
      int i = 0, s = 0;
      uint32_t phase = 0, w = ring, bar = b_full;
      bool ok = true;
#pragma unroll 1
      for (; i < nk; ++i) {
        if (!wait(bar, phase)) { fail(); ok = false; break; }
        tc_fence_after();
        const uint64_t dw = desc_sw128(w), dx = desc_sw128(w + NW * kRows * kK);
#pragma unroll
        for (int kk = 0; kk < kK / 32; ++kk)
#pragma unroll
          for (int g = 0; g < NW; ++g)
            mma_s8<1>(tmem + g * TN, dw + (g * kRows * kK + kk * 32) / 16, dx + kk * 2, idesc, (i > 0 || kk > 0) ? 1u : 0u);
        commit(bar + (b_empty - b_full));
        if (++s == stages) s = 0, phase ^= 1, w = ring, bar = b_full;
        else w += Geo::STAGE, bar += 8;
      }
      if (ok) commit(b_acc);
      s_committed = i;
    }
  }
  __syncwarp();

  // ---- epilogue ----------------------------------------------------------------------
  const int tokens = min(TN, A.M - m0);
  const int n = n0 + 4 * lane;  // this lane's channels n .. n + 3, of warp - 2, warp + 2, ...'s tokens
  float sw[NW][4], bias[4];
  if (warp >= 2) {
    for (int t = threadIdx.x - 64; t < tokens; t += kRows) s_sx[t] = token_scale(A.sx[m0 + t]);
    asm volatile("bar.sync 1, 128;\n" ::: "memory");
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = n + e < A.d_out;
      sw[0][e] = in ? A.sw[n + e] : 0.0f;
      if constexpr (GATED) sw[NW - 1][e] = in ? A.sw2[n + e] : 0.0f;
      bias[e] = !GATED && A.bias && in ? from_16<F16>(A.bias[n + e]) : 0.0f;
    }
  }
  const int quarter = warp & 3, ch = quarter * 32 + lane;  // the tensor memory lanes this warp may read
  const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
  // put(t, g, sum) of this thread's channel for every token and weight matrix
  auto drain = [&](auto put) {
    tc_fence_after();
#pragma unroll 1
    for (int c0 = 0; c0 < tokens; c0 += 16) {
      int v[NW][16];
#pragma unroll
      for (int g = 0; g < NW; ++g) tmem_ld(lanes + g * TN + c0, v[g]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (c0 + c < tokens)
#pragma unroll
          for (int g = 0; g < NW; ++g) put(c0 + c, g, v[g][c]);
    }
  };
  // y of token t for this lane's four channels from get(share, g)
  auto finish = [&](int t, auto get) {
    int4 part[NW][kMaxSplit];
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r)
      if (r < split)
#pragma unroll
        for (int g = 0; g < NW; ++g) part[g][r] = get(r, g);
    int sum[NW][4] = {};
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r)
      if (r < split)
#pragma unroll
        for (int g = 0; g < NW; ++g) {
          sum[g][0] += part[g][r].x;
          sum[g][1] += part[g][r].y;
          sum[g][2] += part[g][r].z;
          sum[g][3] += part[g][r].w;
        }
    const TokenScale sx = s_sx[t];
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = w8a8_scaled(sum[0][e], sx.s, sw[0][e]);
      if constexpr (GATED) v = w8a8_gate(v * sx.back, w8a8_scaled(sum[NW - 1][e], sx.s, sw[NW - 1][e]) * sx.back);
      else v = __fmaf_rn(v, sx.back, bias[e]);
      o[e] = to_16<F16>(v);
    }
    uint16_t* dst = A.y + (size_t)(m0 + t) * A.d_out + n;
    if ((A.d_out & 3) == 0) {
      if (n < A.d_out) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < A.d_out) dst[e] = (uint16_t)o[e];
    }
  };

  if constexpr (Geo::STORED) {
    cluster_wait();  // all barriers of the cluster are there
    if (warp >= 2) {
      // [share][its slot of the owner's tokens][NW][128]
      const uint32_t sums = ring + stages * Geo::STAGE;
      const int shift = 31 - __clz(split), slots = (tokens + split - 1) >> shift;  // split: a power of two
      const bool good = __all_sync(0xffffffffu, mbar_wait(b_acc, 0, A.hooks.wait));
      if (good) {
        drain([&](int t, int g, int v) {
          const int slot = t >> shift, owner = t & (split - 1);
          st_cluster(mapa(sums + (((rank * slots + slot) * NW + g) * kRows + ch) * 4, owner), v);
        });
        __syncwarp();
        if (lane < split && lane < tokens) mbar_arrive_cluster(mapa(b_sums, lane));
      } else {
        fail();
      }
      if (rank < tokens) {
        if (good && mbar_wait(b_sums, 0, A.hooks.wait)) {
          const int4* from = reinterpret_cast<const int4*>(smem + stages * Geo::STAGE) + lane;
#pragma unroll 2
          for (int t = rank + split * (warp - 2); t < tokens; t += split * 4)
            finish(t, [&](int r, int g) { return from[((r * slots + (t >> shift)) * NW + g) * (kRows / 4)]; });
        } else {
          fail();
        }
      }
    }
    __syncwarp();
  } else {
    if (warp >= 2) {
      int* sums = reinterpret_cast<int*>(smem);  // [token][NW][128]
      if (__all_sync(0xffffffffu, mbar_wait(b_acc, 0, A.hooks.wait))) drain([&](int t, int g, int v) { sums[(t * NW + g) * kRows + ch] = v; });
      else fail();
    }
    // a CTA whose wait gave up has no sums: nobody of its cluster writes then
    __syncwarp();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
    if (warp >= 2) {
      const uint32_t flag = smem_u32(&abort_flag);
      if (__all_sync(0xffffffffu, lane >= split || ld_cluster(mapa(flag, lane)) == 0)) {
        const uint32_t mine = ring + lane * 16;
#pragma unroll 2
        for (int t = rank + split * (warp - 2); t < tokens; t += split * 4)
          finish(t, [&](int r, int g) { return ld_cluster4(mapa(mine + (t * NW + g) * (kRows * 4), r)); });
      }
    }
    __syncwarp();
    cluster_arrive();  // the others' sums are read: their CTAs may end
    cluster_wait();
  }

  tc_fence_before();
  __syncthreads();
  if (abort_flag && threadIdx.x == 0) {
    // copies and MMAs in flight end before the memory goes away
    auto last_of = [&](int cnt, int slot) { return cnt > slot ? slot + ((cnt - 1 - slot) / stages) * stages : -1; };
    for (int s = 0; s < stages; ++s) {
      const int jt = last_of(s_issued, s), jm = last_of(s_committed, s);
      bool done = true;
      if (jt >= 0) done = mbar_wait(b_full + 8 * s, (jt / stages) & 1);
      if (jm >= 0) done = mbar_wait(b_empty + 8 * s, (jm / stages) & 1) && done;
      if (!done) report_status(status, kStatusTimeout);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, Geo::COLS);
  }
  if (abort_flag) {  // a CTA that gave up outlives what others may still store to it (or they have ended)
    cluster_arrive();
    cluster_wait();
  }
}

// tcgen05.alloc waits for columns to come free, and a CTA waits for its cluster's:
// two launches at once must never wait for each other.  They cannot, because the
// CTAs that an SM's shared memory lets in never want more than its 512 columns,
// and one that takes all 512 (w8a8_many, w4_tc) leaves no shared memory for another.
// Other libraries' kernels on pairs of SMs wait for columns too.  They fill shared
// memory; a CTA here asks for 72 KB at least, so that none with more than 155 KB fits
// beside it (28 KB, where a share is one step, left room for one of 199).
constexpr int kLeastSmem = 72 * 1024;
template <int TN, bool GATED>
constexpr int least_smem() {
  using Geo = FewGeo<TN, GATED>;
  const int used = 1024 + (Geo::STORED ? Geo::STAGE + Geo::SUMS : Geo::STAGE > Geo::SUMS ? Geo::STAGE : Geo::SUMS);
  return used > kLeastSmem ? used : kLeastSmem;
}

template <int TN, bool GATED, bool F16>
cudaError_t launch_few(FewArgs& A, const W8a8Few& f, int* status, cudaStream_t stream) {
  using Geo = FewGeo<TN, GATED>;
  constexpr int kSmSmem = 228 * 1024;
  static_assert(kSmSmem / least_smem<TN, GATED>() * Geo::COLS <= 512, "tensor memory of the CTAs that fit an SM");
  const int per = (A.blocks + f.split - 1) / f.split;
  A.split = f.split;
  constexpr int kBudget = 104 * 1024;  // of 228 KB, for two CTAs
  int stages = (kBudget - (Geo::STORED ? Geo::SUMS : 0)) / Geo::STAGE;
  if (stages < 2) stages = 2;
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages > per) stages = per;
  int bytes = stages * Geo::STAGE;
  if (Geo::STORED) bytes += Geo::SUMS;
  else if (bytes < Geo::SUMS) bytes = Geo::SUMS;
  A.stages = stages;
  A.hooks = w8a8_hooks(f.split);
  bytes += 1024;
  if (bytes < kLeastSmem) bytes = kLeastSmem;
  auto kernel = w8a8_few_kernel<TN, GATED, F16>;
  static std::atomic<uint64_t> limit{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kMaxSmem, limit);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(f.tiles * f.split, f.mtiles);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = f.split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, A, status);
}

template <int TN>
cudaError_t launch_tn(const W8a8Args& a, FewArgs& A, const W8a8Few& f, int* status, cudaStream_t s) {
  // rows of the last tile's box behind the last token are zeros; where M < TN the
  // columns behind it multiply what lies there, unread
  A.xrows = a.M < TN ? a.M : TN;
  if (!w8_map(&A.q, a.q, a.M, a.d_in, A.xrows)) return cudaErrorInvalidValue;
  if constexpr (TN <= 64)
    if (a.w2) return a.f16 ? launch_few<TN, true, true>(A, f, status, s) : launch_few<TN, true, false>(A, f, status, s);
  return a.f16 ? launch_few<TN, false, true>(A, f, status, s) : launch_few<TN, false, false>(A, f, status, s);
}

}  // namespace

W8a8Few w8a8_few_shape(const W8a8Args& a) {
  // Token tiles with what a call costs, in ns, fitted to measured times: `base` for
  // the set-up and the epilogue of a full tile (`alone` where no SM has two CTAs),
  // down to the smallest tile's for an empty one, and `block` for every 128 columns
  // of a share.  No call takes less than its weights take from HBM.  Measured with
  // tiles of 16, 32, 64, 128 tokens, us:
  //   1536 -> 1536:  M 128: 6.5 5.6 8.9 7.5;     M 256: 9.5 7.1 7.4 10.0
  //   4096 -> 4096:  M 64: 11.8 9.0 10.0 10.1;   M 203: 34.6 18.7 14.5 12.5
  //   14336 -> 4096: M 32: 17.6 14.4 15.4 15.4;  M 128: 51.3 29.2 20.4 19.0
  //   512 -> 512:    M 100: 3.5 3.6 5.2 6.0
  // and a gated pair with 16, 32, 64 (128 tokens' sums would leave room for one CTA
  // on an SM):
  //   1536 -> 1536:  M 40: 5.8 6.6 8.0;          M 203: 12.4 9.8 10.6
  //   4096 -> 4096:  M 32: 12.4 11.4 13.0;       M 128: 26.7 18.8 16.6
  struct Cost {
    int tokens, base, alone, block;
  };
  static constexpr Cost kPlain[] = {{16, 3200, 3200, 450}, {32, 3600, 3600, 450}, {64, 7800, 5600, 450}, {128, 9500, 6800, 470}};
  static constexpr Cost kGated[] = {{16, 4000, 4000, 620}, {32, 5200, 5200, 700}, {64, 9500, 8500, 750}};
  const Cost* costs = a.w2 ? kGated : kPlain;
  const int sms = device_sm_count(), blocks = (a.d_in + kK - 1) / kK;
  const long long hbm = 4000 + (long long)a.d_in * a.d_out * (a.w2 ? 2 : 1) / 5200;
  W8a8Few best;
  best.ns = LLONG_MAX;
  for (int i = 0; i < (a.w2 ? 3 : 4); ++i) {
    const Cost& c = costs[i];
    if (i && a.M <= costs[i - 1].tokens) break;
    W8a8Few f;
    f.tokens = c.tokens;
    f.tiles = (a.d_out + kRows - 1) / kRows;
    f.mtiles = (a.M + f.tokens - 1) / f.tokens;
    if (f.mtiles > 65535) continue;  // grid.y
    // As many shares of d_in as still leave every CTA resident at once, two on an
    // SM: clusters of 4 and 8 do not fill every GPC (284 and 264 of 296 places).
    // One CTA draws at most about 60 GB/s from HBM, so more of them pay up to there:
    // with 1, 2, 4, 8 shares 14336 -> 4096 at one token takes 34.1, 19.6, 13.9, 13.3
    // us, 4096 -> 14336 14.3, 13.6, 15.6, 20.5, gated 1536 -> 8960 at 16 tokens 13.5,
    // 9.5, 9.1, 15.8.  Tiles of fewer rows that even out the SMs' bytes won 4% at
    // most, and lost it elsewhere.
    const long long places = 2 * sms, tiles = (long long)f.tiles * f.mtiles;
    auto fits = [&](int n) { return tiles * n <= (n == 8 ? places * 8 / 9 : n == 4 ? places * 19 / 20 : places); };
    f.split = 1;
    while (f.split < kMaxSplit && fits(2 * f.split) && 2 * f.split <= blocks) f.split *= 2;
    const long long ctas = tiles * f.split, rounds = (ctas + places - 1) / places;
    const long long rows = (long long)f.mtiles * f.tokens, full = (ctas <= sms ? c.alone : c.base) - costs[0].base;
    f.ns = costs[0].base + full * a.M / rows + (blocks + f.split - 1) / f.split * rounds * c.block;
    f.ns = (f.ns > hbm ? f.ns : hbm) + f.ns / 16;  // among equals of HBM, the one with less to do
    if (f.ns < best.ns) best = f;
  }
  return best;
}

cudaError_t launch_w8a8_few(const W8a8Args& a, const W8a8Few& f, int* status, cudaStream_t stream) {
  FewArgs A;
  if (!w8_map(&A.w, a.w, a.d_out, a.d_in, kRows) || (a.w2 && !w8_map(&A.w2, a.w2, a.d_out, a.d_in, kRows)))
    return cudaErrorInvalidValue;
  A.sx = a.sx;
  A.sw = a.sw;
  A.sw2 = a.sw2;
  A.bias = a.bias;
  A.y = a.y;
  A.M = a.M;
  A.d_out = a.d_out;
  A.blocks = (a.d_in + kK - 1) / kK;
  switch (f.tokens) {
    case 16: return launch_tn<16>(a, A, f, status, stream);
    case 32: return launch_tn<32>(a, A, f, status, stream);
    case 64: return launch_tn<64>(a, A, f, status, stream);
    default: return launch_tn<128>(a, A, f, status, stream);
  }
}

}  // namespace paro
