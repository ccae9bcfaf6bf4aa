// int8_decode.cu -- the int8 product for one to four tokens, with their
// quantization in the same launch:
//
//   x[T, K] BF16 -> codes and scales per token (the format of int8.cu), then
//   Y[t, n] = BF16_RNE(RN32(RN32(float(sum_k Xq[t, k] Wq[n, k]) * sx[t]) * sw[n]))
//
// A CTA owns 128 weight rows and a range of the contraction, the ranges of a
// tile are the CTAs of one cluster, as in int8_gemm.cu.  While its weights are
// on their way (TMA, from HBM), warps read the CTA's range of the tokens, take
// each token's maximum over it, exchange the maxima through the cluster's
// shared memory, and write the codes of the range into the swizzled tiles the
// MMA reads.
//
// Against a quantizing launch and the product (whose weights load during the
// former), in a graph, us: 1 token on 1024 x 4096 5.3 and 5.3, on 4096 x 4096
// 7.9 and 8.3, 4 tokens on 1024 x 4096 5.5 and 5.7; but 16 tokens there 6.9 and
// 5.8 (every row tile quantizes them again), and 1 token on 14336 x 4096 15.2
// and 14.7 (the stream of weights starts later).  Launched one by one the host
// is what bounds short calls, and one launch less with no scratch to allocate
// takes them from 12.6 to 7.7 us.  So the variant is taken up to four tokens
// and 32 MiB of weights.
//
// Warps: 0 TMA producer, 1 tensor-memory allocation + MMA issue, 2-5
// quantization, then the accumulator's drain.

#include "common.cuh"
#include "gemm_common.cuh"
#include "int8_common.cuh"
#include "kernels.h"
#include "ring.cuh"

namespace qlora {

using namespace gemm;
using namespace int8;

namespace {

constexpr int WM = 128;                       // weight rows per CTA
constexpr int KB = 128;                       // contraction bytes per stage
constexpr int NT = 16;                        // the MMA's N
constexpr int kMaxTokens = 4;
constexpr int64_t kMaxWeights = 32ll << 20;
constexpr int W_BYTES = WM * KB;              // 16 KiB
constexpr int X_BYTES = NT * KB;              // 2 KiB of codes per block
constexpr int kMaxStages = 4;
constexpr int kMaxBlocks = 32;                // blocks of a range: 64 KiB of codes
constexpr int kMaxSplits = 8;
constexpr int kQuantWarps = 4;                // a token each
static_assert(kMaxTokens <= kQuantWarps, "a token per warp");
constexpr int kThreads = 64 + 32 * kQuantWarps;
// full, empty, accumulator, codes, tensor-memory slot; then the maxima and the scales
constexpr int kBarBytes = 8 * (2 * kMaxStages + 2) + 8;
constexpr int kFixed = kBarBytes + 2 * NT * 4 + 1024;   // + alignment slack for the swizzle atoms
constexpr int kSmSmem = 227 * 1024;
constexpr int kReserved = 2 * 1024;           // per CTA: the system's KiB and the static variables'

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 3)
    int8_decode_kernel(const __grid_constant__ CUtensorMap tm_w, const Int8DecodeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int NS = a.stages;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t x0 = base + static_cast<uint32_t>(NS) * W_BYTES;
  const uint32_t bar0 = x0 + static_cast<uint32_t>(a.kb_per_split) * X_BYTES;
  auto stage_w = [&](int s) { return base + static_cast<uint32_t>(s) * W_BYTES; };
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  const uint32_t acc_bar = bar0 + 8u * (2 * kMaxStages);
  const uint32_t x_bar = acc_bar + 8;
  const uint32_t tmem_slot = x_bar + 8;
  const uint32_t s_max = tmem_slot + 8;         // [NT] this range's maxima, |bits|
  const uint32_t s_scale = s_max + NT * 4;      // [NT] the tokens' scales
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const int splits = static_cast<int>(gridDim.y), split = static_cast<int>(blockIdx.y);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * WM;
  const int kb_all = static_cast<int>((a.K + KB - 1) / KB);
  const int kb0 = split * a.kb_per_split;
  const int nst = min(a.kb_per_split, kb_all - kb0);   // >= 1: splits = ceil(kb_all / kb_per_split)
  const int lead = min(NS, nst);
  const int64_t c0 = static_cast<int64_t>(kb0) * KB;                                      // first column
  const int units = static_cast<int>((min(a.K, c0 + static_cast<int64_t>(nst) * KB) - c0) / 16);   // of 16 columns

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_bar, 1);
    mbar_init(x_bar, kQuantWarps);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 32);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tm_w);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(tmem_slot);
  grid_dep_wait();
  grid_dep_launch();

  if (warp == 0) {
    if (elect_one()) {
      for (int st = 0; st < lead; ++st) {   // the ring's first round: nothing to wait for
        mbar_arrive_expect_tx(full(st), W_BYTES);
        tma_load_2d(stage_w(st), &tm_w, full(st), (kb0 + st) * KB, static_cast<int32_t>(n0));
      }
    }
    __syncwarp();
  } else if (warp >= 2) {
    // each token's maximum over this range
    const int t = warp - 2;
    if (t < a.T) {
      const uint4 *src = reinterpret_cast<const uint4 *>(a.x + static_cast<int64_t>(t) * a.K + c0);
      uint32_t m = 0;
#pragma unroll 4
      for (int i = static_cast<int>(lane); i < 2 * units; i += 32) m = __vmaxu2(m, abs_max8(src[i]));
      m = __reduce_max_sync(0xffffffffu, fold_u16x2(m));
      if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(s_max + 4u * t), "r"(m) : "memory");
    }
    __syncwarp();
  }
  // every range's maxima
  if (splits > 1) cluster_arrive_wait();
  else __syncthreads();

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (elect_one()) {
      feed_ring(
          lead, nst, NS,
          [&](int s, uint32_t ph) {
            if (!s_abort && mbar_wait_spin(empty(s), ph, a.status)) return true;
            s_abort = 1;
            return false;
          },
          [&](int s, int st) {
            mbar_arrive_expect_tx(full(s), W_BYTES);
            tma_load_2d(stage_w(s), &tm_w, full(s), (kb0 + st) * KB, static_cast<int32_t>(n0));
          },
          [&](int s, uint32_t ph) { return mbar_wait(full(s), ph, a.status); });
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issue ----------------
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_i8_s32(WM, NT);
      const uint64_t w0 = smem_desc_sw128(stage_w(0), 16, 1024), xd = smem_desc_sw128(x0, 16, 1024);
      const uint32_t hi = static_cast<uint32_t>(w0 >> 32);   // the same for both operands
      const uint32_t w_lo0 = static_cast<uint32_t>(w0);
      uint32_t off = 0, x_lo = static_cast<uint32_t>(xd), ph = 0, fb = full(0), eb = empty(0), acc = 0;
      int s = 0;
      bool ok = mbar_wait_spin(x_bar, 0, a.status);
      for (int st = 0; st < nst && ok; ++st) {
        if (!mbar_wait_spin(fb, ph, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          tc_mma_ss_i8_lo(tmem, w_lo0 + off + 2 * kk, hi, x_lo + 2 * kk, hi, idesc, acc);
          acc = 1;
        }
        tc_commit(eb);
        off += W_BYTES >> 4;
        x_lo += X_BYTES >> 4;
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
  } else {
    // ---------------- quantization of this range ----------------
    // (rows past T and columns past K are left as they are: the former are
    // columns of the accumulator that nothing reads, the latter meet weights
    // that TMA filled with zeros)
    const int t = warp - 2;
    if (t < a.T) {
      uint32_t m = 0;
      if (static_cast<int>(lane) < splits) m = ld_dsmem_u32(mapa_shared(s_max + 4u * t, lane));
      const RowScale r = row_scale(__reduce_max_sync(0xffffffffu, m));
      if (lane == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(s_scale + 4u * t), "f"(r.scale) : "memory");
      const uint4 *src = reinterpret_cast<const uint4 *>(a.x + static_cast<int64_t>(t) * a.K + c0);
      const uint32_t row = x0 + static_cast<uint32_t>(t) * 128u, sw = static_cast<uint32_t>(t) & 7u;
#pragma unroll 2
      for (int i = static_cast<int>(lane); i < units; i += 32) {
        const uint2 lo = codes8(src[2 * i], r), up = codes8(src[2 * i + 1], r);
        st_shared_v4(row + static_cast<uint32_t>(i >> 3) * X_BYTES + ((static_cast<uint32_t>(i & 7) ^ sw) << 4), lo.x,
                     lo.y, up.x, up.y);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(x_bar);
    // ---------------- the INT32 tile to shared memory, token-major ----------------
    const int q = warp & 3;
    const bool fail = !mbar_wait(acc_bar, 0, a.status) || s_abort;
    const bool have = __all_sync(0xffffffffu, !fail);   // tcgen05.ld is warp-collective
    tc_fence_after();
    tile_to_smem<16>(tmem + (static_cast<uint32_t>(q * 32) << 16), base, q * 32 + static_cast<int>(lane), a.T, have);
  }
  tc_fence_before();
  __syncwarp();
  if (splits > 1) cluster_arrive_wait();
  else __syncthreads();
  // this CTA's share of the tile
  join_splits<kThreads / 32>(base, splits, split, a.T, 0, n0, a.N,
                             [=](int t) { return __uint_as_float(ld_shared_u32(s_scale + 4u * t)); }, a.sw, a.y);
  __syncwarp();
  // no CTA leaves (and frees its shared memory) while another still reads it
  if (splits > 1) cluster_arrive_wait_relaxed();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 32);
  }
}

bool int8_decode_geom(int64_t T, int64_t N, int64_t K, int num_sms, Int8DecodeGeom &g) {
  if (T < 1 || T > kMaxTokens || N * K > kMaxWeights) return false;
  // the ranges of int8_gemm.cu
  const Int8GemmGeom s = int8_gemm_geom(T, N, K, num_sms);
  if (s.pair || s.nt != NT || s.kb_per_split > kMaxBlocks) return false;
  g.splits = s.splits;
  g.kb_per_split = s.kb_per_split;
  // as many stages as let the CTAs of one wave share the SMs
  const int64_t ctas = (N + WM - 1) / WM * s.splits;
  int64_t per_sm = (ctas + num_sms - 1) / num_sms;
  if (per_sm > 3) per_sm = 3;
  const int64_t room = kSmSmem / per_sm - kReserved - kFixed - static_cast<int64_t>(s.kb_per_split) * X_BYTES;
  const int64_t stages = room / W_BYTES;
  if (stages < 2) return false;
  g.stages = static_cast<int>(stages < kMaxStages ? stages : kMaxStages);
  g.smem = g.stages * W_BYTES + g.kb_per_split * X_BYTES + kFixed;
  return true;
}

cudaError_t launch_int8_decode(const Int8DecodeArgs &a, const Int8DecodeGeom &g, const CUtensorMap &tm_w,
                               cudaStream_t st, bool pdl) {
  const int64_t kb = (a.K + KB - 1) / KB;
  if (a.T < 1 || a.T > kMaxTokens || a.N <= 0 || a.N % 8 != 0 || a.K <= 0 || a.K % 16 != 0 || g.splits < 1 ||
      g.splits > kMaxSplits || g.kb_per_split < 1 || g.kb_per_split > kMaxBlocks || g.stages < 1 ||
      g.stages > kMaxStages || g.splits != (kb + g.kb_per_split - 1) / g.kb_per_split ||
      a.kb_per_split != g.kb_per_split || a.stages != g.stages ||
      g.smem != g.stages * W_BYTES + g.kb_per_split * X_BYTES + kFixed || g.smem > kSmSmem - kReserved)
    return cudaErrorInvalidValue;
  static_assert(NT * kPitch * 4 <= W_BYTES, "the INT32 tile takes the place of the drained ring");
  cudaError_t e = ensure_smem_optin(reinterpret_cast<const void *>(int8_decode_kernel), kSmSmem - kReserved);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + WM - 1) / WM), static_cast<unsigned>(g.splits), 1);
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
  return cudaLaunchKernelEx(&cfg, int8_decode_kernel, tm_w, a);
}

}  // namespace qlora
