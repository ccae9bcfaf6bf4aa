// int8_common.cuh -- the joined epilogue of the split int8 products: a tile of
// INT32 sums, token-major in the shared memory of each CTA that holds a part of
// the contraction, summed over those CTAs, scaled and stored.
#pragma once

#include "common.cuh"
#include "gemm_common.cuh"

namespace qlora {
namespace int8 {

constexpr int kFeat = 128;           // features of a CTA's tile (tensor-memory lanes)
constexpr int kPitch = kFeat + 4;    // INT32 per token row: 16-byte rows, banks spread
constexpr int kWarps = 6;            // warps of a CTA, all of which join

__device__ __forceinline__ int4 ld_dsmem_i4(uint32_t cluster_addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// Tokens 0 .. tv - 1 of this thread's feature (tensor-memory lane `row`) to
// shared memory; the next columns load while these are stored.  Warp-collective.
template <int CW>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[CW]) {
  if constexpr (CW == 16) tmem_ld_32x32b_x16(taddr, v);
  else tmem_ld_32x32b_x32(taddr, v);
}

template <int CW>
__device__ __forceinline__ void put_cols(uint32_t dst, int n, const uint32_t (&v)[CW]) {
#pragma unroll
  for (int j = 0; j < CW; ++j)
    if (j < n) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + static_cast<uint32_t>(j * kPitch) * 4u), "r"(v[j]) : "memory");
}

template <int CW>
__device__ __forceinline__ void tile_to_smem(uint32_t trow, uint32_t base, int row, int tv, bool have) {
  const uint32_t dst = base + static_cast<uint32_t>(row) * 4u;
  if (!have) {   // a wait ran out: zeros, and the status word says so
    for (int c = 0; c < tv; ++c)
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + static_cast<uint32_t>(c * kPitch) * 4u), "r"(0) : "memory");
    return;
  }
  uint32_t a[CW], b[CW];
  tmem_ld_cols<CW>(trow, a);
  tc_wait_ld();
  reg_fence(a);
#pragma unroll 1
  for (int c = 0; c < tv; c += 2 * CW) {
    if (c + CW < tv) tmem_ld_cols<CW>(trow + static_cast<uint32_t>(c + CW), b);
    put_cols<CW>(dst + static_cast<uint32_t>(c * kPitch) * 4u, tv - c, a);
    tc_wait_ld();
    reg_fence(b);
    if (c + CW >= tv) break;
    if (c + 2 * CW < tv) tmem_ld_cols<CW>(trow + static_cast<uint32_t>(c + 2 * CW), a);
    put_cols<CW>(dst + static_cast<uint32_t>((c + CW) * kPitch) * 4u, tv - c - CW, b);
    tc_wait_ld();
    reg_fence(a);
  }
}

// Y rows t0 .. t0 + tv - 1, features n0 .. n0 + 127, summed over `splits` CTAs
// whose cluster ranks are stride * k + first.  A warp takes a token (a lane four
// of its features), the tokens are dealt to the warps of the CTAs in turn, and
// a lane keeps S * U = 8 remote loads in flight: one takes most of a
// microsecond, so a loop that waited for each cost more than the product.
template <int S>
__device__ __forceinline__ void join_and_store(uint32_t base, int splits, int split, uint32_t stride, uint32_t first,
                                               int tv, int64_t t0, int64_t n0, int64_t N, const float *sx,
                                               const float *sw, uint16_t *y) {
  constexpr int U = 8 / S;
  const int warp = static_cast<int>(threadIdx.x >> 5), f = static_cast<int>(threadIdx.x & 31) * 4;
  const int step = kWarps * splits;
  const bool in = n0 + f < N;   // N % 8 == 0: four features are inside or outside together
  const float4 w = in ? __ldcg(reinterpret_cast<const float4 *>(sw + n0 + f)) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int tb = split * kWarps + warp; tb < tv; tb += U * step) {
    int4 part[U][S];
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * step;
      x[u] = t < tv ? __ldcg(sx + t0 + t) : 0.f;
#pragma unroll
      for (int k = 0; k < S; ++k)
        if (t < tv && k < splits)
          part[u][k] = ld_dsmem_i4(mapa_shared(base + static_cast<uint32_t>(t * kPitch + f) * 4u,
                                               stride * static_cast<uint32_t>(k) + first));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * step;
      if (t < tv) {
        int4 s = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < S; ++k) {
          if (k < splits) {
            s.x += part[u][k].x;
            s.y += part[u][k].y;
            s.z += part[u][k].z;
            s.w += part[u][k].w;
          }
        }
        const uint32_t y0 = pack_bf16x2(__fmul_rn(__fmul_rn(static_cast<float>(s.x), x[u]), w.x),
                                        __fmul_rn(__fmul_rn(static_cast<float>(s.y), x[u]), w.y));
        const uint32_t y1 = pack_bf16x2(__fmul_rn(__fmul_rn(static_cast<float>(s.z), x[u]), w.z),
                                        __fmul_rn(__fmul_rn(static_cast<float>(s.w), x[u]), w.w));
        if (in) *reinterpret_cast<uint2 *>(y + (t0 + t) * N + n0 + f) = make_uint2(y0, y1);
      }
    }
  }
}

__device__ __forceinline__ void join_splits(uint32_t base, int splits, int split, uint32_t stride, uint32_t first,
                                            int tv, int64_t t0, int64_t n0, int64_t N, const float *sx, const float *sw,
                                            uint16_t *y) {
  if (splits == 1) join_and_store<1>(base, splits, split, stride, first, tv, t0, n0, N, sx, sw, y);
  else if (splits == 2) join_and_store<2>(base, splits, split, stride, first, tv, t0, n0, N, sx, sw, y);
  else if (splits <= 4) join_and_store<4>(base, splits, split, stride, first, tv, t0, n0, N, sx, sw, y);
  else join_and_store<8>(base, splits, split, stride, first, tv, t0, n0, N, sx, sw, y);
}

}  // namespace int8
}  // namespace qlora
