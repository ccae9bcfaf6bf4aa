// da_int8.cu -- the adapter gradient dA from an activation kept in 8 bits
// ("QLoRA: Efficient Fine-Tuning", Step 4 eq. 5, x "cached from the forward
// pass", here as signed codes with FP32 scales):
//
//   dA[j, k] = sum_t dU[t, j] scale[t, g(k)] code[t, k]
//
// g(k) = k / 128 (one scale per 128 features of a token) or 0 (one per token).
// A CTA owns 128 features, so it sees one scale per token either way, and the
// scale moves to the small operand: dU'[t, j] = dU[t, j] scale[t], while the
// codes, integers of at most 7 bits and a sign, are exact in BF16.  The product
// then runs on tcgen05.mma kind::f16 with nothing of the activation rounded.
// dU arrives as its hi and lo planes; (hi + lo) scale is split again into a hi
// and a lo plane (about 16 significant bits), stacked into one N = 2 nb operand
// whose two accumulator halves are added when they are drained.
//
// Per 64-token stage: TMA brings the codes [64 t][128 k] and the dU^T planes
// [nb j][64 t], one warp the 64 scales; eight warps turn the codes into the
// MN-major, 128-byte swizzled BF16 tile the MMA reads (two boxes of 64
// features) and the planes into the scaled planes; one thread issues the MMAs.
// The tokens are split over the CTAs of a cluster, which sum their FP32 tiles
// in split order through distributed shared memory.
//
// Bound by latency per stage (load, convert, MMA), not by a rate: the codes are
// half of what the BF16 kernel reads.  4096 x 4096, r = 16, alone: 11.6 us
// against 13.5 from BF16; the whole backward 134.7 against 138.6.
//
// Launched after the dX GEMM as a programmatic dependent whose inputs were all
// complete before that GEMM started: it runs on the SMs the GEMM's last round
// leaves idle and waits for it only before it exits.  (In front of the GEMM it
// took 2 us longer at 4096^3, and no less with the codes brought to L2 during
// the launch before.)
//
// Warps: 0 TMA producer, 1 tensor-memory allocation + MMA issue, 2-9
// conversion (2-5 also the epilogue), 10 the scales.

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "ring.cuh"

namespace qlora {

using namespace gemm;

namespace {

constexpr int AM = 128;                       // features per CTA (MMA M)
constexpr int AT = 64;                        // tokens per stage
constexpr int RAW_X = AT * AM;                // 8 KiB of codes
constexpr int CONV_X = AT * AM * 2;           // 16 KiB: two boxes [64 t][64 k]
constexpr int kConvStages = 2;
constexpr int kMaxRaw = 6;
constexpr int kConvWarps = 8;
constexpr int kConvThreads = 32 * kConvWarps;
constexpr int kThreads = 64 + kConvThreads + 32;
// raw full/empty, conv full/empty, accumulator, tensor-memory slot
constexpr int kBarBytes = 8 * (2 * kMaxRaw + 2 * kConvStages + 1) + 8;
constexpr int kFixed = kBarBytes + 1024;
constexpr int kPitch = AM + 4;
constexpr int kMaxSmem = 224 * 1024;
constexpr int kMaxSplits = 8;

constexpr int SC_BYTES = AT * 4;              // one stage's scales

int raw_stage_bytes(int nb) { return RAW_X + 2 * nb * AT * 2 + SC_BYTES; }
int conv_stage_bytes(int nb) { return CONV_X + 2 * nb * AT * 2; }

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// Two signed bytes of `w` -> two BF16, exact.  0x4300 | b reads as 128 + b for
// b < 128 and as 256 + 2 (b - 128) above; with its bit 7 moved to a second
// operand, code = (128 + (b & 127)) - (128 or 256), one packed subtraction.
__device__ __forceinline__ uint32_t bytes_to_bf16x2(uint32_t w, uint32_t sel) {
  const uint32_t v = prmt(w, 0x43434343u, sel);
  const uint32_t p = v & 0xFF7FFF7Fu, m = v & 0xFF80FF80u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&p),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&m));
  return *reinterpret_cast<const uint32_t *>(&d);
}

}  // namespace

template <int NB>
__global__ void __launch_bounds__(kThreads, 1)
    da_int8_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_hi,
                   const __grid_constant__ CUtensorMap tm_lo, const DaInt8Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr uint32_t Q_BYTES = NB * AT * 2;                  // one plane [NB j][64 t]
  constexpr uint32_t RAW = RAW_X + 2 * Q_BYTES, CONV = CONV_X + 2 * Q_BYTES;
  constexpr uint32_t TMEM_COLS = 2 * NB;
  constexpr int CW = NB < 32 ? 16 : 32;
  constexpr int Q_ITEMS = NB * 8;                            // (j, 8-token chunk) pairs of a stage
  constexpr int Q_ITER = (Q_ITEMS + kConvThreads - 1) / kConvThreads;
  const int NR = a.raw_stages;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t raw0 = base + kConvStages * CONV;
  const uint32_t sc0 = raw0 + static_cast<uint32_t>(NR) * RAW;
  const uint32_t bar0 = sc0 + static_cast<uint32_t>(NR) * SC_BYTES;
  // the swizzled planes of a stage come first: whole 1 KiB atoms
  auto raw_q = [&](int s) { return raw0 + static_cast<uint32_t>(s) * RAW; };
  auto raw_x = [&](int s) { return raw0 + static_cast<uint32_t>(s) * RAW + 2 * Q_BYTES; };
  auto raw_sc = [&](int s) { return sc0 + static_cast<uint32_t>(s) * SC_BYTES; };
  auto conv_x = [&](int s) { return base + static_cast<uint32_t>(s) * CONV; };
  auto conv_q = [&](int s) { return base + static_cast<uint32_t>(s) * CONV + CONV_X; };
  auto rfull = [&](int s) { return bar0 + 8u * s; };
  auto rempty = [&](int s) { return bar0 + 8u * (kMaxRaw + s); };
  auto cfull = [&](int s) { return bar0 + 8u * (2 * kMaxRaw + s); };
  auto cempty = [&](int s) { return bar0 + 8u * (2 * kMaxRaw + kConvStages + s); };
  const uint32_t acc_bar = bar0 + 8u * (2 * kMaxRaw + 2 * kConvStages);
  const uint32_t tmem_slot = acc_bar + 8;
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const int splits = static_cast<int>(gridDim.y), split = static_cast<int>(blockIdx.y);
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * AM;
  const int64_t tbeg = static_cast<int64_t>(split) * a.t_per_split;
  const int64_t tend = min(a.T, tbeg + a.t_per_split);
  const int nst = static_cast<int>((tend - tbeg + AT - 1) / AT);

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < NR; ++s) {
      mbar_init(rfull(s), 2);   // the TMA producer and the scales' warp
      mbar_init(rempty(s), kConvWarps);
    }
    for (int s = 0; s < kConvStages; ++s) {
      mbar_init(cfull(s), kConvWarps);
      mbar_init(cempty(s), 1);
    }
    mbar_init(acc_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_hi);
    tma_prefetch_desc(&tm_lo);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(tmem_slot);
  grid_dep_launch();

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (elect_one()) {
      feed_ring(
          0, nst, NR,
          [&](int s, uint32_t ph) {
            if (!s_abort && mbar_wait_spin(rempty(s), ph, a.status)) return true;
            s_abort = 1;
            return false;
          },
          [&](int s, int st) {
            const int32_t t = static_cast<int32_t>(tbeg + static_cast<int64_t>(st) * AT);
            mbar_arrive_expect_tx(rfull(s), RAW);
            tma_load_2d(raw_x(s), &tm_x, rfull(s), static_cast<int32_t>(k0), t);   // [64 t][128 k]
            tma_load_2d(raw_q(s), &tm_hi, rfull(s), t, 0);                         // [NB j][64 t]
            tma_load_2d(raw_q(s) + Q_BYTES, &tm_lo, rfull(s), t, 0);
          },
          [&](int s, uint32_t ph) { return mbar_wait(rfull(s), ph, a.status); });
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issue ----------------
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_bf16_f32(AM, 2 * NB, true, false);
      bool ok = true;
      for (int st = 0; st < nst; ++st) {
        const int s = st % kConvStages;
        if (!mbar_wait_spin(cfull(s), (st / kConvStages) & 1, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_ss(tmem, smem_desc_sw128(conv_x(s) + kk * 2048, CONV_X / 2, 1024),
                    smem_desc_sw128(conv_q(s) + kk * 32, 16, 1024), idesc, (st > 0 || kk > 0) ? 1u : 0u);
        tc_commit(cempty(s));
      }
      if (!ok) s_abort = 1;
      tc_commit(acc_bar);   // also drains: arrives once everything issued has completed
    }
    __syncwarp();
  } else if (warp == 2 + kConvWarps) {
    // ---------------- the scales, loaded four stages ahead ----------------
    const float *sg = a.scales + (a.grouped ? static_cast<int64_t>(blockIdx.x) * a.T : 0);
    float2 r[4];
    auto load = [&](int st, float2 &v) {
      const int64_t t = tbeg + static_cast<int64_t>(st) * AT + lane;
      v.x = st < nst && t < tend ? __ldg(sg + t) : 0.f;
      v.y = st < nst && t + 32 < tend ? __ldg(sg + t + 32) : 0.f;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) load(i, r[i]);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int st0 = 0; st0 < nst && ok; st0 += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (ok && st0 + i < nst) {
          ok = __all_sync(0xffffffffu, !s_abort && mbar_wait(rempty(s), ph, a.status));
          if (ok) {
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(raw_sc(s) + 4u * lane), "f"(r[i].x) : "memory");
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(raw_sc(s) + 4u * lane + 128u), "f"(r[i].y) : "memory");
            load(st0 + i + 4, r[i]);
            __syncwarp();
            if (lane == 0) mbar_arrive(rfull(s));
            if (++s == NR) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
      }
    }
    if (!ok) s_abort = 1;
  } else {
    // ---------------- conversion ----------------
    const int ct = static_cast<int>(threadIdx.x) - 64;
    // The codes: 16 features of one token per item, two items a thread.  A
    // warp takes eight tokens; eight lanes (a quarter of a shared-memory
    // access) take four 16-feature chunks of one box for two tokens whose
    // numbers differ by 5 in exclusive or: with both swizzles, their reads and
    // their writes then fall in different 16-byte bank groups.
    uint32_t xr[2], xw0[2], xw1[2];   // offsets: the item read, its two 16-byte halves written
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t c = lane & 3u, h = (lane >> 3) & 1u, p = 2u * i + (lane >> 4);
      const uint32_t x = (lane & 4u) ? p ^ 5u : p;               // token of the warp's eight
      const uint32_t row = static_cast<uint32_t>(warp - 2) * 1024u + x * 128u;
      xr[i] = row + (((4u * h + c) ^ x) << 4);
      xw0[i] = h * (CONV_X / 2) + row + (((2u * c) ^ x) << 4);
      xw1[i] = h * (CONV_X / 2) + row + (((2u * c + 1u) ^ x) << 4);
    }
    const uint32_t ch = ct & 7u;   // this thread's 8-token chunk of the planes
    int rs = 0, cs = 0;
    uint32_t rph = 0, cph = 1;
    for (int st = 0; st < nst; ++st) {
      bool ok = !s_abort && mbar_wait(rfull(rs), rph, a.status);
      ok = ok && mbar_wait(cempty(cs), cph, a.status);
      if (!__all_sync(0xffffffffu, ok)) {
        s_abort = 1;
        break;
      }
      const uint32_t src = raw_x(rs), dst = conv_x(cs);
      uint4 q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) q[i] = ld_shared_v4(src + xr[i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        st_shared_v4(dst + xw0[i], bytes_to_bf16x2(q[i].x, 0x4140u), bytes_to_bf16x2(q[i].x, 0x4342u),
                     bytes_to_bf16x2(q[i].y, 0x4140u), bytes_to_bf16x2(q[i].y, 0x4342u));
        st_shared_v4(dst + xw1[i], bytes_to_bf16x2(q[i].z, 0x4140u), bytes_to_bf16x2(q[i].z, 0x4342u),
                     bytes_to_bf16x2(q[i].w, 0x4140u), bytes_to_bf16x2(q[i].w, 0x4342u));
      }
      // the planes: eight tokens of one column j per item
      if (ct < Q_ITEMS) {
        const uint4 s0 = ld_shared_v4(raw_sc(rs) + ch * 32u), s1 = ld_shared_v4(raw_sc(rs) + ch * 32u + 16u);
        const uint32_t sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int i = 0; i < Q_ITER; ++i) {
          const uint32_t j = static_cast<uint32_t>(ct >> 3) + i * (kConvThreads / 8);
          const uint32_t off = j * 128u + ((ch ^ (j & 7u)) << 4);
          const uint4 hv = ld_shared_v4(raw_q(rs) + off), lv = ld_shared_v4(raw_q(rs) + Q_BYTES + off);
          const uint32_t hw[4] = {hv.x, hv.y, hv.z, hv.w}, lw[4] = {lv.x, lv.y, lv.z, lv.w};
          uint32_t oh[4], ol[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v0 = (__uint_as_float(hw[e] << 16) + __uint_as_float(lw[e] << 16)) * __uint_as_float(sc[2 * e]);
            const float v1 = (__uint_as_float(hw[e] & 0xFFFF0000u) + __uint_as_float(lw[e] & 0xFFFF0000u)) *
                             __uint_as_float(sc[2 * e + 1]);
            oh[e] = pack_bf16x2(v0, v1);
            ol[e] = pack_bf16x2(v0 - __uint_as_float(oh[e] << 16), v1 - __uint_as_float(oh[e] & 0xFFFF0000u));
          }
          st_shared_v4(conv_q(cs) + off, oh[0], oh[1], oh[2], oh[3]);
          st_shared_v4(conv_q(cs) + Q_BYTES + off, ol[0], ol[1], ol[2], ol[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(rempty(rs));
        mbar_arrive(cfull(cs));
      }
      if (++rs == NR) {
        rs = 0;
        rph ^= 1u;
      }
      if (++cs == kConvStages) {
        cs = 0;
        cph ^= 1u;
      }
    }
    if (warp < 6) {
      // ---------------- the FP32 tile to shared memory, column j by column j ----------------
      const int q = warp & 3;
      const int row = q * 32 + static_cast<int>(lane);
      const bool fail = !mbar_wait(acc_bar, 0, a.status) || s_abort;
      const bool have = __all_sync(0xffffffffu, !fail);   // tcgen05.ld is warp-collective
      tc_fence_after();
      // (the accumulator is complete only after the last conversion: no warp
      // reads or writes the rings any more)
      const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < a.R; c0 += CW) {
        uint32_t v[CW], w[CW];
        if (have) {
          if constexpr (CW == 16) {
            tmem_ld_32x32b_x16(trow + c0, v);
            tmem_ld_32x32b_x16(trow + NB + c0, w);
          } else {
            tmem_ld_32x32b_x32(trow + c0, v);
            tmem_ld_32x32b_x32(trow + NB + c0, w);
          }
          tc_wait_ld();
          reg_fence(v);
          reg_fence(w);
        } else {
#pragma unroll
          for (int j = 0; j < CW; ++j) v[j] = w[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < CW; ++j)
          if (c0 + j < a.R)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + static_cast<uint32_t>((c0 + j) * kPitch + row) * 4u),
                         "f"(__uint_as_float(v[j]) + __uint_as_float(w[j]))
                         : "memory");
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if (splits > 1) cluster_arrive_wait();
  else __syncthreads();
  const int items = a.R * (AM / 4);
  for (int i = split * kThreads + static_cast<int>(threadIdx.x); i < items; i += splits * kThreads) {
    const int j = i >> 5, f = (i & 31) * 4;
    const uint32_t local = base + static_cast<uint32_t>(j * kPitch + f) * 4u;
    float4 part[kMaxSplits];   // the cluster's loads all in flight
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k)
      if (k < splits) part[k] = ld_dsmem_f4(mapa_shared(local, static_cast<uint32_t>(k)));
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k) {   // split order: the sum does not depend on timing
      if (k < splits) {
        s.x += part[k].x;
        s.y += part[k].y;
        s.z += part[k].z;
        s.w += part[k].w;
      }
    }
    if (k0 + f < a.K)   // K % 64 == 0
      *reinterpret_cast<uint2 *>(a.dA + static_cast<int64_t>(j) * a.K + k0 + f) =
          make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
  __syncwarp();
  // no CTA leaves (and frees its shared memory) while another still reads it
  if (splits > 1) cluster_arrive_wait_relaxed();
  else __syncthreads();
  grid_dep_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

DaInt8Geom da_int8_geom(int64_t T, int64_t K, int r, int num_sms) {
  DaInt8Geom g;
  g.nb = r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128;
  const int conv = kConvStages * conv_stage_bytes(g.nb) + kFixed;
  int per_sm = 2;
  g.raw_stages = (kMaxSmem / 2 - conv) / raw_stage_bytes(g.nb);
  if (g.raw_stages < 3) {
    per_sm = 1;
    g.raw_stages = (kMaxSmem - conv) / raw_stage_bytes(g.nb);
  }
  if (g.raw_stages > kMaxRaw) g.raw_stages = kMaxRaw;
  g.smem = conv + g.raw_stages * raw_stage_bytes(g.nb);
  // one wave of CTAs, at least four stages a split; a power of two, so that
  // clusters fill the GPU's partitions
  const int64_t tiles = (K + AM - 1) / AM, steps = (T + AT - 1) / AT;
  int64_t s = 1;
  while (2 * s <= kMaxSplits && 2 * s * tiles <= per_sm * static_cast<int64_t>(num_sms) && steps >= 8 * s) s *= 2;
  g.t_per_split = (steps + s - 1) / s * AT;
  g.splits = static_cast<int>((T + g.t_per_split - 1) / g.t_per_split);
  return g;
}

namespace {
template <int NB>
cudaError_t launch_nb(const DaInt8Args &a, const DaInt8Geom &g, const CUtensorMap &tm_x, const CUtensorMap &tm_hi,
                      const CUtensorMap &tm_lo, cudaStream_t st, bool pdl) {
  const int ring = kConvStages * conv_stage_bytes(NB) + g.raw_stages * raw_stage_bytes(NB);
  if (g.smem != ring + kFixed || g.smem > kMaxSmem || ring < a.R * kPitch * 4 || a.R > NB) return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_optin(reinterpret_cast<const void *>(da_int8_kernel<NB>), kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.K + AM - 1) / AM), static_cast<unsigned>(g.splits), 1);
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
  return cudaLaunchKernelEx(&cfg, da_int8_kernel<NB>, tm_x, tm_hi, tm_lo, a);
}
}  // namespace

cudaError_t launch_da_int8(const DaInt8Args &a, const DaInt8Geom &g, const CUtensorMap &tm_x,
                           const CUtensorMap &tm_du_hi, const CUtensorMap &tm_du_lo, cudaStream_t st, bool pdl) {
  if (a.T <= 0 || a.K <= 0 || a.K % 64 != 0 || a.R < 1 || g.raw_stages < 1 || g.raw_stages > kMaxRaw ||
      g.splits < 1 || g.splits > kMaxSplits)
    return cudaErrorInvalidValue;
  if (a.raw_stages != g.raw_stages || a.t_per_split != g.t_per_split || g.t_per_split % AT != 0 ||
      g.splits != (a.T + g.t_per_split - 1) / g.t_per_split)
    return cudaErrorInvalidValue;
  switch (g.nb) {
    case 16: return launch_nb<16>(a, g, tm_x, tm_du_hi, tm_du_lo, st, pdl);
    case 32: return launch_nb<32>(a, g, tm_x, tm_du_hi, tm_du_lo, st, pdl);
    case 64: return launch_nb<64>(a, g, tm_x, tm_du_hi, tm_du_lo, st, pdl);
    case 128: return launch_nb<128>(a, g, tm_x, tm_du_hi, tm_du_lo, st, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qlora
