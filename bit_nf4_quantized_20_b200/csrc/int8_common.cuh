// int8_common.cuh -- shared by the int8 kernels: the arithmetic of the 8-bit
// format, and the joined epilogue of the split products: a tile of INT32 sums,
// token-major in the shared memory of each CTA that holds a part of the
// contraction, summed over those CTAs, scaled and stored.
#pragma once

#include "common.cuh"
#include "gemm_common.cuh"

namespace qlora {
namespace int8 {

// ---------------------------------------------------------------------------
// The 8-bit format (int8.cu states it)
// ---------------------------------------------------------------------------
constexpr float kRoundMagic = 12582912.0f;   // 1.5 * 2^23
constexpr float kMinScale = 0x1p-126f;

// elementwise max over |bits| of eight BF16 values (BF16 order = magnitude order), as u16x2
__device__ __forceinline__ uint32_t abs_max8(const uint4 &v) {
  return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}

__device__ __forceinline__ uint32_t fold_u16x2(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

struct RowScale {
  float scale, inv;
  bool bad;
};

__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale r;
  r.bad = amax_bits >= 0x7F80u;
  const float s = fmaxf(__fdiv_rn(__uint_as_float(amax_bits << 16), 127.0f), kMinScale);
  r.scale = r.bad ? __uint_as_float(0x7FC00000u) : s;
  r.inv = __frcp_rn(s);
  return r;
}

// two BF16 values of a word -> the sums whose low bytes are their codes
__device__ __forceinline__ uint32_t code_lo(uint32_t w, float inv) {
  return __float_as_uint(__fmaf_rn(__uint_as_float(w << 16), inv, kRoundMagic));
}
__device__ __forceinline__ uint32_t code_hi(uint32_t w, float inv) {
  return __float_as_uint(__fmaf_rn(__uint_as_float(w & 0xFFFF0000u), inv, kRoundMagic));
}

__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
  const uint32_t a = prmt(code_lo(w0, inv), code_hi(w0, inv), 0x0040);
  const uint32_t b = prmt(code_lo(w1, inv), code_hi(w1, inv), 0x0040);
  return prmt(a, b, 0x5410);
}

__device__ __forceinline__ uint2 codes8(const uint4 &v, const RowScale &r) {
  if (r.bad) return make_uint2(0u, 0u);
  return make_uint2(codes4(v.x, v.y, r.inv), codes4(v.z, v.w, r.inv));
}

// ---------------------------------------------------------------------------
// The joined epilogue of the split products
// ---------------------------------------------------------------------------

constexpr int kFeat = 128;           // features of a CTA's tile (tensor-memory lanes)
constexpr int kPitch = kFeat + 4;    // INT32 per token row: 16-byte rows, banks spread

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
  if (!have) {   // a wait ran out, copies may still land here: no result, as the status word says
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

// Y rows t0 .. t0 + tv - 1, features n0 .. n0 + 127, summed over the `splits`
// CTAs of a cluster (this is CTA `split`).  A warp takes a token (a lane four
// of its features), the tokens are dealt to the warps of the CTAs in turn, and
// a lane keeps S * U = 8 remote loads in flight: one takes most of a
// microsecond (waiting for each: 512 tokens on 4096 x 4096 in 15.8 us, not 13.9).
// WARPS: those of a CTA, all of which join.  sx(t): the scale of the tile's token t.
template <int S, int WARPS, class Scale>
__device__ __forceinline__ void join_and_store(uint32_t base, int splits, int split, int tv, int64_t t0, int64_t n0,
                                               int64_t N, const Scale &sx, const float *sw, uint16_t *y) {
  constexpr int U = 8 / S;
  const int warp = static_cast<int>(threadIdx.x >> 5), f = static_cast<int>(threadIdx.x & 31) * 4;
  const int step = WARPS * splits;
  const bool in = n0 + f < N;   // N % 8 == 0: four features are inside or outside together
  const float4 w = in ? __ldcg(reinterpret_cast<const float4 *>(sw + n0 + f)) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int tb = split * WARPS + warp; tb < tv; tb += U * step) {
    int4 part[U][S];
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * step;
      x[u] = t < tv ? sx(t) : 0.f;
#pragma unroll
      for (int k = 0; k < S; ++k)
        if (t < tv && k < splits)
          part[u][k] = ld_dsmem_i4(
              mapa_shared(base + static_cast<uint32_t>(t * kPitch + f) * 4u, static_cast<uint32_t>(k)));
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

template <int WARPS, class Scale>
__device__ __forceinline__ void join_splits(uint32_t base, int splits, int split, int tv, int64_t t0, int64_t n0,
                                            int64_t N, const Scale &sx, const float *sw, uint16_t *y) {
  if (splits == 1) join_and_store<1, WARPS>(base, splits, split, tv, t0, n0, N, sx, sw, y);
  else if (splits == 2) join_and_store<2, WARPS>(base, splits, split, tv, t0, n0, N, sx, sw, y);
  else if (splits <= 4) join_and_store<4, WARPS>(base, splits, split, tv, t0, n0, N, sx, sw, y);
  else join_and_store<8, WARPS>(base, splits, split, tv, t0, n0, N, sx, sw, y);
}

}  // namespace int8
}  // namespace qlora
