// int8_gemm.cu -- the product of two 8-bit row matrices on the 5th-generation
// tensor cores (tcgen05 kind::i8, INT32 accumulation):
//
//   acc[t, n] = sum_k Xq[t, k] Wq[n, k]           exact for K <= 131072
//   Y[t, n]   = BF16_RNE(RN32(RN32(float(acc) * sx[t]) * sw[n]))
//
// One CTA owns 128 weight rows (the MMA's M) against nt tokens (its N, 16 to
// 256: tokens past T arrive as zeros) over a range of the contraction; the
// weights stream through TMA once per token tile.  The ranges of a tile are
// the CTAs of one cluster: each leaves its INT32 tile in its own shared memory
// (the drained ring), token by token, and after a cluster barrier every CTA
// sums its share over the cluster through distributed shared memory.  Integer
// sums do not depend on their order, so neither does the result.
//
// With a few tokens the weights' bytes are the cost, so they load before the
// dependency wait when only the activations come from the kernel before.
//
// Warps: 0 TMA producer, 1 tensor-memory allocation + MMA issue, 2-5 epilogue.

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace qlora {

using namespace gemm;

namespace {

constexpr int WM = 128;                       // weight rows per CTA
constexpr int KB = 128;                       // contraction bytes per stage
constexpr int W_BYTES = WM * KB;              // 16 KiB
constexpr int kMaxStages = 8;
constexpr int kThreads = 192;
constexpr int kBarBytes = 8 * (2 * kMaxStages + 1) + 8;
constexpr int kFixed = kBarBytes + 1024;      // + alignment slack for the swizzle atoms
constexpr int kPitch = WM + 4;                // INT32 per token row of the partial tile
constexpr int kMaxSmem = 220 * 1024;
constexpr int kMaxSplits = 8;

__device__ __forceinline__ int4 ld_dsmem_i4(uint32_t cluster_addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

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
    if (lane == 0) {
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
      int issued = lead;
      for (int st = lead; st < nst; ++st) {
        const int s = st % NS;
        if (s_abort || !mbar_wait(empty(s), ((st / NS) & 1) ^ 1, a.status)) {
          s_abort = 1;
          break;
        }
        mbar_arrive_expect_tx(full(s), STAGE);
        tma_load_2d(stage_w(s), &tm_w, full(s), (kb0 + st) * KB, static_cast<int32_t>(n0));
        tma_load_2d(stage_x(s), &tm_x, full(s), (kb0 + st) * KB, static_cast<int32_t>(t0));
        issued = st + 1;
      }
      if (s_abort) {
        // every copy in flight lands before the CTA can exit
        for (int st = max(0, issued - NS); st < issued; ++st) mbar_wait(full(st % NS), (st / NS) & 1, a.status);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issue ----------------
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_i8_s32(WM, NT);
      bool ok = true;
      for (int st = 0; st < nst; ++st) {
        const int s = st % NS;
        if (!mbar_wait(full(s), (st / NS) & 1, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_ss_i8(tmem, smem_desc_sw128(stage_w(s) + kk * 32, 16, 1024),
                       smem_desc_sw128(stage_x(s) + kk * 32, 16, 1024), idesc, (st > 0 || kk > 0) ? 1u : 0u);
        tc_commit(empty(s));
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
#pragma unroll 1
    for (int c0 = 0; c0 < tv; c0 += CW) {
      uint32_t v[CW];
      if (have) {
        if constexpr (CW == 16) tmem_ld_32x32b_x16(trow + c0, v);
        else tmem_ld_32x32b_x32(trow + c0, v);
        tc_wait_ld();
      } else {
#pragma unroll
        for (int j = 0; j < CW; ++j) v[j] = 0u;
      }
#pragma unroll
      for (int j = 0; j < CW; ++j)
        if (c0 + j < tv)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + static_cast<uint32_t>((c0 + j) * kPitch + row) * 4u),
                       "r"(v[j])
                       : "memory");
    }
  }
  tc_fence_before();
  __syncwarp();
  if (splits > 1) cluster_arrive_wait();
  else __syncthreads();

  // this CTA's share of the tile: groups of four features of a token, dealt to
  // the cluster's threads in turn
  const int items = tv * (WM / 4);
  for (int i = split * kThreads + static_cast<int>(threadIdx.x); i < items; i += splits * kThreads) {
    const int t = i >> 5, f = (i & 31) * 4;
    const uint32_t local = base + static_cast<uint32_t>(t * kPitch + f) * 4u;
    int4 s = make_int4(0, 0, 0, 0);
    for (int k = 0; k < splits; ++k) {
      const int4 p = ld_dsmem_i4(mapa_shared(local, static_cast<uint32_t>(k)));
      s.x += p.x;
      s.y += p.y;
      s.z += p.z;
      s.w += p.w;
    }
    if (n0 + f < a.N) {   // N % 8 == 0: four features are inside or outside together
      const float sx = __ldcg(a.sx + t0 + t);
      const float4 sw = __ldcg(reinterpret_cast<const float4 *>(a.sw + n0 + f));
      const uint32_t y0 = pack_bf16x2(__fmul_rn(__fmul_rn(static_cast<float>(s.x), sx), sw.x),
                                      __fmul_rn(__fmul_rn(static_cast<float>(s.y), sx), sw.y));
      const uint32_t y1 = pack_bf16x2(__fmul_rn(__fmul_rn(static_cast<float>(s.z), sx), sw.z),
                                      __fmul_rn(__fmul_rn(static_cast<float>(s.w), sx), sw.w));
      *reinterpret_cast<uint2 *>(a.y + (t0 + t) * a.N + n0 + f) = make_uint2(y0, y1);
    }
  }
  __syncwarp();
  // no CTA leaves (and frees its shared memory) while another still reads it
  if (splits > 1) cluster_arrive_wait();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

Int8GemmGeom int8_gemm_geom(int64_t T, int64_t N, int64_t K) {
  Int8GemmGeom g;
  g.pair = T > 256;
  g.nt = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
  const int stage = W_BYTES + g.nt * KB;
  g.stages = g.nt <= 32 ? 4 : g.nt <= 128 ? 3 : 4;
  g.smem = g.stages * stage + kFixed;
  const int per_sm = kMaxSmem / g.smem < 1 ? 1 : kMaxSmem / g.smem;
  const int64_t tiles = (N + WM - 1) / WM * ((T + g.nt - 1) / g.nt);
  const int64_t kb = (K + KB - 1) / KB;
  // one wave of CTAs; at least two contraction blocks each
  int64_t s = static_cast<int64_t>(per_sm) * 148 / tiles;
  if (s > kMaxSplits) s = kMaxSplits;
  if (s > (kb + 1) / 2) s = (kb + 1) / 2;
  if (s < 1) s = 1;
  g.kb_per_split = static_cast<int>((kb + s - 1) / s);
  g.splits = static_cast<int>((kb + g.kb_per_split - 1) / g.kb_per_split);
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
    case 256: return launch_nt<256>(a, g, tm_w, tm_x, st, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qlora
