// int8_gemm.cu -- the product of two 8-bit row matrices on the 5th-generation
// tensor cores (tcgen05 kind::i8, INT32 accumulation):
//
//   acc[t, n] = sum_k Xq[t, k] Wq[n, k]           exact for K <= 131072
//   Y[t, n]   = BF16_RNE(RN32(RN32(float(acc) * sx[t]) * sw[n]))
//
// One CTA owns 128 weight rows (the MMA's M) against nt tokens (its N, 16 to
// 128: tokens past T arrive as zeros) over a range of the contraction; the
// weights stream through TMA once per token tile.  The ranges of a tile are
// the CTAs of one cluster: each leaves its INT32 tile in its own shared memory
// (the drained ring), token by token, and after a cluster barrier every CTA
// sums its share over the cluster through distributed shared memory.  Integer
// sums do not depend on their order, so neither does the result.
//
// With a few tokens the weights' bytes are the cost, so they load before the
// dependency wait when only the activations come from the kernel before.
// For a few tokens the weights' stream bounds it, between a start and a sum that
// are fixed, over SMs that hold two or three CTAs each.  From 64 to 512 no rate
// does: 101 tokens on 4096 x 14336 use 38 % of DRAM, 27 % of L2, 22 % of the
// tensor pipe; about half the time is the start of two CTAs an SM and the
// cluster's sum (7.0 us in int8_gemm_geom's estimate of 14.6).  With the
// quantizing launch and without: 16 tokens on 14336 x 4096 14.6 and 13.5 us
// (4.0 TB/s; 9.1 of it the stream at the copy rate), 101 on 4096 x 14336 18.8
// and 17.4 us.
//
// Warps: 0 TMA producer, 1 tensor-memory allocation + MMA issue, 2-5 epilogue.

#include "common.cuh"
#include "gemm_common.cuh"
#include "int8_common.cuh"
#include "kernels.h"
#include "ring.cuh"

namespace qlora {

using namespace gemm;
using int8::kPitch;

namespace {

constexpr int WM = 128;                       // weight rows per CTA
constexpr int KB = 128;                       // contraction bytes per stage
constexpr int W_BYTES = WM * KB;              // 16 KiB
constexpr int kMaxStages = 8;
constexpr int kThreads = 192;
constexpr int kBarBytes = 8 * (2 * kMaxStages + 1) + 8;
constexpr int kFixed = kBarBytes + 1024;      // + alignment slack for the swizzle atoms
constexpr int kMaxSmem = 220 * 1024;   // three of the narrow tiles' 74 KiB rings share an SM
constexpr int kMaxSplits = 8;

}  // namespace

template <int NT>
__global__ void __launch_bounds__(kThreads)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const Int8GemmArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr uint32_t X_BYTES = NT * KB;
  constexpr uint32_t STAGE = W_BYTES + X_BYTES;
  constexpr uint32_t TMEM_COLS = NT < 32 ? 32u : static_cast<uint32_t>(NT);
  constexpr int CW = NT < 32 ? 16 : 32;
  const int NS = a.stages;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = base + static_cast<uint32_t>(NS) * STAGE;
  auto stage_w = [&](int s) { return base + static_cast<uint32_t>(s) * STAGE; };
  auto stage_x = [&](int s) { return base + static_cast<uint32_t>(s) * STAGE + W_BYTES; };
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  const uint32_t acc_bar = bar0 + 8u * (2 * kMaxStages);
  const uint32_t tmem_slot = acc_bar + 8;
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const int splits = static_cast<int>(gridDim.y), split = static_cast<int>(blockIdx.y);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * WM;
  const int64_t t0 = static_cast<int64_t>(blockIdx.z) * NT;
  const int kb_all = static_cast<int>((a.K + KB - 1) / KB);
  const int kb0 = split * a.kb_per_split;
  const int nst = min(a.kb_per_split, kb_all - kb0);   // >= 1: splits = ceil(kb_all / kb_per_split)

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(tmem_slot);

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (elect_one()) {
      if (!a.early) grid_dep_wait();
      const int lead = min(NS, nst);
      for (int st = 0; st < lead; ++st) {   // the ring's first round: nothing to wait for
        mbar_arrive_expect_tx(full(st), STAGE);
        tma_load_2d(stage_w(st), &tm_w, full(st), (kb0 + st) * KB, static_cast<int32_t>(n0));
      }
      if (a.early) grid_dep_wait();
      grid_dep_launch();
      for (int st = 0; st < lead; ++st)
        tma_load_2d(stage_x(st), &tm_x, full(st), (kb0 + st) * KB, static_cast<int32_t>(t0));
      feed_ring(
          lead, nst, NS,
          [&](int s, uint32_t ph) {
            if (!s_abort && mbar_wait_spin(empty(s), ph, a.status)) return true;
            s_abort = 1;
            return false;
          },
          [&](int s, int st) {
            mbar_arrive_expect_tx(full(s), STAGE);
            tma_load_2d(stage_w(s), &tm_w, full(s), (kb0 + st) * KB, static_cast<int32_t>(n0));
            tma_load_2d(stage_x(s), &tm_x, full(s), (kb0 + st) * KB, static_cast<int32_t>(t0));
          },
          [&](int s, uint32_t ph) { return mbar_wait(full(s), ph, a.status); });
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issue ----------------
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_i8_s32(WM, NT);
      // one thread issues everything: the ring position, its barriers and the
      // descriptors' low words advance by additions
      const uint64_t w0 = smem_desc_sw128(stage_w(0), 16, 1024), x0 = smem_desc_sw128(stage_x(0), 16, 1024);
      const uint32_t hi = static_cast<uint32_t>(w0 >> 32);   // the same for both operands
      const uint32_t w_lo0 = static_cast<uint32_t>(w0), x_lo0 = static_cast<uint32_t>(x0);
      uint32_t off = 0, ph = 0, fb = full(0), eb = empty(0), acc = 0;
      int s = 0;
      bool ok = true;
      for (int st = 0; st < nst; ++st) {
        if (!mbar_wait_spin(fb, ph, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          tc_mma_ss_i8_lo(tmem, w_lo0 + off + 2 * kk, hi, x_lo0 + off + 2 * kk, hi, idesc, acc);
          acc = 1;
        }
        tc_commit(eb);
        off += STAGE >> 4;
        fb += 8;
        eb += 8;
        if (++s == NS) {
          s = 0;
          ph ^= 1u;
          off = 0;
          fb = full(0);
          eb = empty(0);
        }
      }
      if (!ok) s_abort = 1;
      tc_commit(acc_bar);   // also drains: arrives once everything issued has completed
    }
    __syncwarp();
  }
  // the scales of a caller's kernel, or of the quantizer before this launch
  // (and no CTA completes before the kernel preceding its launch)
  if (warp != 0) grid_dep_wait();
  const int tv = static_cast<int>(min(static_cast<int64_t>(NT), a.T - t0));   // tokens of this tile
  if (warp >= 2) {
    // ---------------- the INT32 tile to shared memory, token-major ----------------
    const int q = warp & 3;
    const int row = q * 32 + static_cast<int>(lane);
    const bool fail = !mbar_wait(acc_bar, 0, a.status) || s_abort;
    const bool have = __all_sync(0xffffffffu, !fail);   // tcgen05.ld is warp-collective
    tc_fence_after();
    const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
    int8::tile_to_smem<CW>(trow, base, row, tv, have);
  }
  tc_fence_before();
  __syncwarp();
  if (splits > 1) cluster_arrive_wait();
  else __syncthreads();

  // this CTA's share of the tile
  const float *sx = a.sx + t0;
  int8::join_splits<kThreads / 32>(base, splits, split, tv, t0, n0, a.N, [=](int t) { return __ldcg(sx + t); }, a.sw, a.y);
  __syncwarp();
  // no CTA leaves (and frees its shared memory) while another still reads it
  if (splits > 1) cluster_arrive_wait_relaxed();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// The variant and its geometry.  Measured (microseconds, weights from HBM, 18
// token counts on each of seven weight shapes):
//   up to 32 tokens, one tile of 16 or 32: bound by the weights' bytes.  Split
//   until every SM has a CTA (1 token on 1024 x 4096, 8 tiles: 3.4 with eight
//   ranges, 3.7 with six), and on, up to three CTAs an SM, while a range keeps
//   eight blocks (14336 x 4096, 112 tiles: 14.4 with two ranges, 13.5 with
//   three; 4096 x 4096, 32 tiles: 6.9 with four, 7.9 with eight of four blocks;
//   22016 x 1040, 172 tiles: 7.8 with one, 9.0 with two of five).
//   More tokens: the least of these estimates, S = the contraction blocks of
//   the SM with the most work:
//     64-token tiles 4.2 + 0.27 S with one CTA an SM, 5.5 + 0.165 S with two,
//     7.5 + 0.165 S with more; 128-token tiles 5.2 + 0.35 S and 7 + 0.27 S;
//     pairs 4.2 + 0.185 S for half tiles, 6 + 0.31 S with full ones;
//     none less than 4 + the weights' bytes at 6 TB/s.
//   (256 tokens: 4096 x 4096 10.8 split against 10.9 on pairs, 4096 x 14336
//   21.9 against 27.8, 14336 x 4096 25.8 against 17.9.)
//   Ranges come in powers of two there: with one CTA an SM, clusters of three
//   leave SMs of a GPU partition idle (1024 x 4096, 768 tokens, 48 tiles: 15.4
//   with three ranges, 10.9 with two).
Int8GemmGeom int8_gemm_geom(int64_t T, int64_t N, int64_t K, int num_sms) {
  Int8GemmGeom g;
  const int64_t rows = (N + WM - 1) / WM, kb = (K + KB - 1) / KB;
  auto set = [&](int nt, int stages, int64_t splits) {
    g.nt = nt;
    g.stages = stages;
    g.smem = stages * (W_BYTES + nt * KB) + kFixed;
    g.kb_per_split = static_cast<int>((kb + splits - 1) / splits);
    g.splits = static_cast<int>((kb + g.kb_per_split - 1) / g.kb_per_split);
  };
  g.pair = false;
  if (T <= 32) {
    int64_t s = 1;
    while (s < kMaxSplits && s < kb &&
           (rows * (s + 1) <= num_sms || (kb / (s + 1) >= 8 && rows * (s + 1) <= 3 * static_cast<int64_t>(num_sms))))
      ++s;
    const int nt = T <= 16 ? 16 : 32;
    // three 32-token rings of four stages do not share an SM
    set(nt, nt == 32 && rows * s > 2 * static_cast<int64_t>(num_sms) ? 3 : 4, s);
    return g;
  }
  double best = 0.0;
  for (int nt = 64; nt <= 128; nt *= 2) {
    if (nt / 2 >= T) break;
    const int64_t tiles = rows * ((T + nt - 1) / nt);
    for (int64_t s = 1; s <= kMaxSplits && s <= kb; s *= 2) {
      const int64_t ctas = tiles * s, waves = (ctas + num_sms - 1) / num_sms, per = (kb + s - 1) / s;
      if (s > 1 && waves > (nt == 64 ? 3 : 2)) break;
      const double work = static_cast<double>(waves * per);
      const double t = nt == 64 ? (waves == 1 ? 4.2 + 0.27 * work : (waves == 2 ? 5.5 : 7.5) + 0.165 * work)
                                : (waves == 1 ? 5.2 + 0.35 * work : 7.0 + 0.27 * work);
      if (best == 0.0 || t < best) {
        best = t;
        set(nt, waves == 1 || (nt == 64 && waves == 2) ? 4 : 3, s);
      }
    }
  }
  const double weights = 4.0 + static_cast<double>(N) * static_cast<double>(K) / 6e6;
  const Int8PairUnits w = int8_pair_units(T, N, num_sms);
  double pair = (w.rounds_full > 0 ? 6.0 : 4.2) +
                static_cast<double>(kb) * (0.31 * w.rounds_full + 0.185 * w.rounds_half);
  best = best > weights ? best : weights;
  pair = pair > weights ? pair : weights;
  // (the one-CTA grid holds 65535 token tiles)
  g.pair = pair <= best || (T + g.nt - 1) / g.nt > 65535;
  return g;
}

namespace {
template <int NT>
cudaError_t launch_nt(const Int8GemmArgs &a, const Int8GemmGeom &g, const CUtensorMap &tm_w, const CUtensorMap &tm_x,
                      cudaStream_t st, bool pdl) {
  const int stage = W_BYTES + NT * KB;
  // the INT32 tile takes the place of the drained ring
  if (g.stages < 1 || g.stages > kMaxStages || g.stages * stage < NT * kPitch * 4 ||
      g.smem != g.stages * stage + kFixed || g.smem > kMaxSmem)
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_optin(reinterpret_cast<const void *>(int8_gemm_kernel<NT>), kMaxSmem);
  if (e != cudaSuccess) return e;
  const int64_t tt = (a.T + NT - 1) / NT;
  if (tt > 65535) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + WM - 1) / WM), static_cast<unsigned>(g.splits),
                     static_cast<unsigned>(tt));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(g.smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (g.splits > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 1;
    attr[na].val.clusterDim.y = static_cast<unsigned>(g.splits);
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, int8_gemm_kernel<NT>, tm_w, tm_x, a);
}
}  // namespace

cudaError_t launch_int8_gemm(const Int8GemmArgs &a, const Int8GemmGeom &g, const CUtensorMap &tm_w,
                             const CUtensorMap &tm_x, cudaStream_t st, bool pdl) {
  if (a.T <= 0 || a.N <= 0 || a.K <= 0 || a.N % 8 != 0 || g.splits < 1 || g.splits > kMaxSplits)
    return cudaErrorInvalidValue;
  const int64_t kb = (a.K + KB - 1) / KB;
  if (g.splits != (kb + g.kb_per_split - 1) / g.kb_per_split || a.kb_per_split != g.kb_per_split ||
      a.stages != g.stages)
    return cudaErrorInvalidValue;
  switch (g.nt) {
    case 16: return launch_nt<16>(a, g, tm_w, tm_x, st, pdl);
    case 32: return launch_nt<32>(a, g, tm_w, tm_x, st, pdl);
    case 64: return launch_nt<64>(a, g, tm_w, tm_x, st, pdl);
    case 128: return launch_nt<128>(a, g, tm_w, tm_x, st, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qlora
