// int8_gemm_2sm.cu -- the int8 product of int8_gemm.cu for token counts that
// fill the GPU with 256 x 256 tiles, on CTA pairs:
//
//   Y[t, n] = BF16_RNE(RN32(RN32(float(sum_k Xq[t, k] Wq[n, k]) * sx[t]) * sw[n]))
//
// A cluster of two CTAs on two SMs owns 256 weight rows x 256 tokens; the even
// CTA issues tcgen05.mma.cta_group::2.kind::i8 (M = 256, N = 256, K = 32).  Per
// 128-byte contraction stage each CTA loads its 128 weight rows and 128 tokens
// by TMA (32 KiB), so an operand byte feeds 256 products; six stages are in
// flight.  Two 256-column INT32 accumulators in tensor memory let the epilogue
// of one tile run under the next tile's MMAs: tcgen05.ld, conversion and the
// two scales, BF16 pairs into a swizzled 64-token staging chunk, TMA store; two
// groups of four warps with a staging chunk each.
//
// Bound by the tensor cores; the tiles run in blocks of eight weight tiles by
// all token tiles, so that the pairs running at one time share operands in L2.
// 4096 tokens on 14336 x 4096: 145.8 us, 3.30 Pop/s, tensor pipe active 92 to
// 93 % of the cycles in which an SM is (86 % of all) at 1.62 GHz; in a long run
// the power cap lowers the clock further and it takes 180.
//
// Warps: 0-7 epilogue, 8 TMA, 9 paired tensor-memory allocation and, on the
// even CTA, the MMA issue.

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace qlora {

using namespace gemm;

namespace {

constexpr int PM = 128;                        // weight rows per CTA (256 per pair)
constexpr int PN = 256;                        // tokens per tile
constexpr int HN = 128;                        // tokens loaded by each CTA
constexpr int KB = 128;                        // contraction bytes per stage
constexpr int STAGES = 6;
constexpr int A_BYTES = PM * KB;               // 16 KiB
constexpr int B_BYTES = HN * KB;               // 16 KiB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int CHUNK_T = 64;                    // tokens per staging chunk
constexpr int BOX_BYTES = CHUNK_T * 128;       // 64 tokens x 64 features, BF16
constexpr int CHUNK_BYTES = 2 * BOX_BYTES;
constexpr int kThreads = 320;
constexpr int kTmemCols = 512;
constexpr int kGroupM = 8;                     // weight tiles per block of tiles
constexpr int kEpiWarps = 8;                   // two groups of four

constexpr int OFF_OUT = STAGES * STAGE_BYTES;
constexpr int OFF_SX = OFF_OUT + 2 * CHUNK_BYTES;
constexpr int OFF_BAR = OFF_SX + PN * 4;
// full[S], empty[S], acc_full[2], acc_empty[2], drain
constexpr int NUM_BARS = 2 * STAGES + 5;
constexpr int OFF_ABORT = OFF_BAR + 8 * NUM_BARS + 8;   // after the tensor-memory slot
constexpr int SMEM_BYTES = OFF_ABORT + 8;
constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");

struct Tile {
  int m, tok0, ntok;
};

// Full tiles run in blocks of kGroupM weight tiles by all token tiles.
__device__ __forceinline__ Tile tile_of(const Int8PairUnits &w, int u) {
  Tile r;
  r.ntok = u < w.full ? PN : HN;
  int t = u, half = 0;
  if (u >= w.full) {
    const int h = u - w.full;
    t = w.full + (h >> 1);
    half = h & 1;
    const int all = w.m_tiles * w.n_full;
    if (t >= all) {   // the half tiles of the last token tile
      r.m = h - 2 * (all - w.full);
      r.tok0 = w.n_full * PN;
      return r;
    }
  }
  const int per = kGroupM * w.n_full;
  const int g = t / per, i = t - g * per;
  const int gm = min(kGroupM, w.m_tiles - g * kGroupM);
  r.m = g * kGroupM + i % gm;
  r.tok0 = (i / gm) * PN + half * HN;
  return r;
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    int8_gemm_2sm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ CUtensorMap tm_xh, const __grid_constant__ CUtensorMap tm_y,
                         const Int8PairArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto sm_a = [&](int s) { return base + static_cast<uint32_t>(s) * STAGE_BYTES; };
  auto sm_b = [&](int s) { return base + static_cast<uint32_t>(s) * STAGE_BYTES + A_BYTES; };
  auto full = [&](int s) { return base + OFF_BAR + 8u * s; };
  auto empty = [&](int s) { return base + OFF_BAR + 8u * (STAGES + s); };
  auto acc_full = [&](int b) { return base + OFF_BAR + 8u * (2 * STAGES + b); };
  auto acc_empty = [&](int b) { return base + OFF_BAR + 8u * (2 * STAGES + 2 + b); };
  const uint32_t drain = base + OFF_BAR + 8u * (2 * STAGES + 4);
  const uint32_t tmem_slot = base + OFF_BAR + 8u * NUM_BARS;
  // (not a static variable: it would be padded to the alignment of the ring)
  volatile int &s_abort = *reinterpret_cast<volatile int *>(smem_raw + (base - smem_u32(smem_raw)) + OFF_ABORT);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;
  const int n_units = p.units.full + p.units.halves;
  auto lead = [&](uint32_t local_addr) { return mapa_shared(local_addr, 0); };

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 2 * kEpiWarps);   // both CTAs'
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_xh);
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tm_y);
  if (warp == 9) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive_wait();   // the leader's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(tmem_slot);

  if (warp == 9) {
    // ---------------- MMA issue (even CTA) ----------------
    if (leader && elect_one()) {
      constexpr uint32_t idesc_full = idesc_i8_s32(2 * PM, PN), idesc_half = idesc_i8_s32(2 * PM, HN);
      const uint64_t a0 = smem_desc_sw128(sm_a(0), 16, 1024), b0 = smem_desc_sw128(sm_b(0), 16, 1024);
      const uint32_t a_lo0 = static_cast<uint32_t>(a0), b_lo0 = static_cast<uint32_t>(b0);
      const uint32_t hi = static_cast<uint32_t>(a0 >> 32);   // the same for both operands
      int s = 0, tc = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = cluster_id; u < n_units && ok; u += num_clusters, ++tc) {
        const uint32_t idesc = tile_of(p.units, u).ntok == PN ? idesc_full : idesc_half;
        const uint32_t d = tmem + static_cast<uint32_t>((tc & 1) * PN);
        if (!mbar_wait(acc_empty(tc & 1), ((tc >> 1) & 1) ^ 1, p.status)) { ok = false; break; }
        tc_fence_after();
        for (int ks = 0; ks < p.ksteps; ++ks) {
          if (!mbar_wait_spin(full(s), ph, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t off = static_cast<uint32_t>(s) * (STAGE_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_ss_pair_i8_lo(d, a_lo0 + off + 2 * kk, hi, b_lo0 + off + 2 * kk, hi, idesc,
                                 (ks > 0 || kk > 0) ? 1u : 0u);
          tc_commit_pair_mc(empty(s), 0x3);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair_mc(acc_full(tc & 1), 0x3);
      }
      if (!ok) s_abort = 1;
      tc_commit_pair_mc(drain, 0x1);   // every MMA issued so far has completed
      mbar_wait(drain, 0, p.status);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---------------- TMA producer: this CTA's weight rows and token half ----------------
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true, dep_done = false;
      for (int u = cluster_id; u < n_units && ok; u += num_clusters) {
        const Tile w = tile_of(p.units, u);
        const bool half = w.ntok != PN;
        const int m0 = w.m * 2 * PM + static_cast<int>(rank) * PM;
        const int t0 = w.tok0 + static_cast<int>(rank) * (w.ntok / 2);
        const CUtensorMap *mx = half ? &tm_xh : &tm_x;
        const uint32_t bytes = 2u * static_cast<uint32_t>(A_BYTES + (half ? B_BYTES / 2 : B_BYTES));
        int ks = 0;
        if (!dep_done) {
          // the ring's first round: the weights load while the kernel before
          // still quantizes the activations
          const int n = min(STAGES, p.ksteps);
          if (!p.early) grid_dep_wait();
          for (int i = 0; i < n; ++i) {
            if (leader) mbar_arrive_expect_tx(full(i), bytes);
            tma_load_2d_pair(sm_a(i), &tm_w, lead(full(i)), i * KB, m0);
          }
          if (p.early) grid_dep_wait();
          grid_dep_launch();
          dep_done = true;
          for (int i = 0; i < n; ++i) tma_load_2d_pair(sm_b(i), mx, lead(full(i)), i * KB, t0);
          ks = n;
          s = n == STAGES ? 0 : n;
          ph = n == STAGES ? 1u : 0u;
        }
        for (; ks < p.ksteps; ++ks) {
          if (s_abort || !mbar_wait_spin(empty(s), ph ^ 1, p.status)) { ok = false; break; }
          const uint32_t fb = lead(full(s));
          if (leader) mbar_arrive_expect_tx(full(s), bytes);
          tma_load_2d_pair(sm_a(s), &tm_w, fb, ks * KB, m0);
          tma_load_2d_pair(sm_b(s), mx, fb, ks * KB, t0);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!dep_done) {
        grid_dep_wait();
        grid_dep_launch();
      }
      if (!ok) s_abort = 1;
    }
    __syncwarp();
  } else {
    // ---------------- epilogue (warps 0-7) ----------------
    // Two groups of four warps; group e takes the 64-token chunks c with c % 2
    // == e, each through its own staging chunk.  Lane l of warp q (of a group)
    // holds feature m = 32 q + l; features 0-63 go to box 0 of the staging
    // chunk, 64-127 to box 1, each [64 tokens][64 features] with the 128-byte
    // swizzle.  Lanes 2i and 2i + 1 swap one value so that each writes a BF16
    // pair of adjacent features: the even lane for token j, the odd lane for
    // token j + 4 (j & 4 == 0), whose rows fall in complementary bank halves.
    grid_dep_wait();   // sx may be the preceding kernel's output
    const int q = warp & 3, grp = warp >> 2;
    const int et = static_cast<int>(threadIdx.x) & 127;   // thread of the group
    const int bar = 1 + grp;
    const bool odd = (lane & 1) != 0;
    const int fm = 32 * (q & 1) + static_cast<int>(lane & ~1u);
    const uint32_t chunk = static_cast<uint32_t>(fm >> 3);
    const uint32_t stage = base + OFF_OUT + static_cast<uint32_t>(grp) * CHUNK_BYTES;
    const uint32_t out = stage + static_cast<uint32_t>(q >> 1) * BOX_BYTES + (odd ? 4u * 128u : 0u) +
                         static_cast<uint32_t>((fm & 7) >> 1) * 4u;
    uint32_t xo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xo[i] = (chunk ^ static_cast<uint32_t>(i + (odd ? 4 : 0))) << 4;
    int tc = 0;
    bool ok = true;
    for (int u = cluster_id; u < n_units && ok; u += num_clusters, ++tc) {
      const Tile w = tile_of(p.units, u);
      const int feat0 = w.m * 2 * PM + static_cast<int>(rank) * PM;
      const int64_t n = static_cast<int64_t>(feat0) + et;
      const float sw = n < p.N ? __ldcg(p.sw + n) : 0.f;
      // the scales of this group's chunks (those of the tile before were last
      // read before its last barrier)
      const int tok = (2 * (et >> 6) + grp) * CHUNK_T + (et & 63);
      const float sxv = tok < w.ntok && static_cast<int64_t>(w.tok0) + tok < p.T ? __ldcg(p.sx + w.tok0 + tok) : 0.f;
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + OFF_SX + 4u * tok), "f"(sxv) : "memory");
      const bool fail = s_abort || !mbar_wait(acc_full(tc & 1), (tc >> 1) & 1, p.status);
      if (named_bar_any(bar, 128, fail)) { ok = false; break; }
      tc_fence_after();
      const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>((tc & 1) * PN);
      const int nch = w.ntok / CHUNK_T;
#pragma unroll 1
      for (int c = grp; c < nch; c += 2) {
        uint32_t ra[32], rb[32];
        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(c * CHUNK_T), ra);
        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(c * CHUNK_T + 32), rb);
        // the store of this group's chunk before has finished reading it
        if (et == 0) tma_store_wait_read<0>();
        tc_wait_ld();
        reg_fence(ra);
        reg_fence(rb);
        if (c + 2 >= nch) {
          // this warp's accumulator columns are all in registers: release them
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(lead(acc_empty(tc & 1)));
        }
        named_bar_sync(bar, 128);
        const uint32_t sxa = base + OFF_SX + 4u * static_cast<uint32_t>(c * CHUNK_T);
        auto emit = [&](const uint32_t (&r)[32], int j0) {
#pragma unroll
          for (int jj = 0; jj < 32; jj += 8) {
            float sx[8];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(sx[0]), "=f"(sx[1]), "=f"(sx[2]), "=f"(sx[3])
                         : "r"(sxa + 4u * (j0 + jj)));
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(sx[4]), "=f"(sx[5]), "=f"(sx[6]), "=f"(sx[7])
                         : "r"(sxa + 4u * (j0 + jj + 4)));
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = __fmul_rn(__fmul_rn(static_cast<float>(static_cast<int32_t>(r[jj + i])), sx[i]), sw);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float recv = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 4], 1);
              const uint32_t w2 = odd ? pack_bf16x2(recv, v[i + 4]) : pack_bf16x2(v[i], recv);
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(out + static_cast<uint32_t>(j0 + jj + i) * 128u + xo[i]),
                           "r"(w2)
                           : "memory");
            }
          }
        };
        emit(ra, 0);
        emit(rb, 32);
        fence_proxy_async_smem();
        named_bar_sync(bar, 128);
        if (et == 0) {
          for (int b = 0; b < 2; ++b)
            tma_store_2d(&tm_y, stage + b * BOX_BYTES, feat0 + 64 * b, w.tok0 + c * CHUNK_T);
          tma_store_commit();
        }
      }
    }
    if (et == 0) tma_store_wait_all<0>();
    if (!ok) s_abort = 1;
  }

  tc_fence_before();
  __syncthreads();
  settle_loads(s_abort != 0);
  cluster_arrive_wait();   // both CTAs are done with the pair's tensor memory
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// A half tile takes 0.6 of a full one's time (its weight rows load all the
// same).  The tiles of a last round that is not full run as halves when that
// ends sooner; a last token tile of at most 128 tokens is one half.
Int8PairUnits int8_pair_units(int64_t T, int64_t N, int num_sms) {
  const int pairs = num_sms / 2;
  const int64_t cols = (T + HN - 1) / HN;
  Int8PairUnits best;
  double best_t = 0.0;
  for (int split = 0; split < 2; ++split) {
    Int8PairUnits w;
    w.m_tiles = static_cast<int>((N + 2 * PM - 1) / (2 * PM));
    w.n_full = static_cast<int>(cols / 2);
    const int64_t tiles = static_cast<int64_t>(w.m_tiles) * w.n_full;
    const int64_t last = split ? tiles % pairs : 0;
    w.full = static_cast<int>(tiles - last);
    w.halves = static_cast<int>(2 * last + (cols % 2) * w.m_tiles);
    // unit u runs on pair u % pairs: the pairs before `full % pairs` have one
    // full tile more than the others, who take the first halves
    const int base = w.full / pairs, extra = w.full % pairs, total = w.full + w.halves;
    double t = 0.0;
    for (int c = 0; c < 2; ++c) {   // a pair with the extra full tile, and one without
      const int pair = c == 0 ? (extra > 0 ? 0 : -1) : (extra < pairs ? extra : -1);
      if (pair < 0 || pair >= total) continue;
      const int f = base + (pair < extra ? 1 : 0), h = (total - pair + pairs - 1) / pairs - f;
      if (f + 0.6 * h > t) {
        t = f + 0.6 * h;
        w.rounds_full = f;
        w.rounds_half = h;
      }
    }
    if (split == 0 || t < best_t) {
      best = w;
      best_t = t;
    }
  }
  return best;
}

cudaError_t launch_int8_gemm_2sm(const Int8PairArgs &args, const CUtensorMap &tm_w, const CUtensorMap &tm_x,
                                 const CUtensorMap &tm_xh, const CUtensorMap &tm_y, int num_sms, cudaStream_t st,
                                 bool pdl) {
  Int8PairArgs p = args;
  if (p.T <= 0 || p.N <= 0 || p.K <= 0 || p.N % 8 != 0) return cudaErrorInvalidValue;
  p.ksteps = static_cast<int>((p.K + KB - 1) / KB);
  if ((p.N + 2 * PM - 1) / (2 * PM) * ((p.T + HN - 1) / HN) > 0x3fffffff) return cudaErrorInvalidValue;   // int units
  p.units = int8_pair_units(p.T, p.N, num_sms);
  const int64_t units = p.units.full + static_cast<int64_t>(p.units.halves), pairs = num_sms / 2;
  const int64_t clusters = units < pairs ? units : pairs;
  cudaError_t e = ensure_smem_optin(reinterpret_cast<const void *>(int8_gemm_2sm_kernel), SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = SMEM_ALLOC;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, int8_gemm_2sm_kernel, tm_w, tm_x, tm_xh, tm_y, p);
}

}  // namespace qlora
