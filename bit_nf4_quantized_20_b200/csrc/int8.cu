// int8.cu -- the 8-bit row format: quantization of a BF16 matrix to signed
// 8-bit codes with one FP32 scale per row or per 128 consecutive columns of a
// row, and its dequantization.
//
//   amax  = max |x| over the group
//   scale = max(RN32(amax / 127), 2^-126),  inv = RN32(1 / scale)
//   code  = RNE_int(x inv), the exact product rounded once
//   value = code * scale
//
// The exact product needs no second rounding: fma(x, inv, 1.5 * 2^23) rounds
// x inv + 1.5 * 2^23 to an integer (ulp 1 there), ties to even, and leaves the
// code as the two's complement low byte of the sum.  |x| inv <= 127 (1 + 2^-23),
// so no code leaves [-127, 127].  The floor of 2^-126 keeps inv finite for rows
// of subnormals and zeros.  A group that holds an infinity or a NaN gets scale
// NaN and codes 0: whatever is computed from it is NaN, never a wrong number.
//
// Inputs are read with coherent loads after griddepcontrol.wait: the kernel
// before may still have been writing them when this one started.
//
// Both kernels move each byte once (2 + 1 bytes an element in, 1 + 2 out):
// bound by HBM for large matrices, by launch latency for a few rows.  A row
// stays in registers between its maximum and its codes, so nothing is read
// twice (but for rows longer than 32768 columns).  4096 x 4096, floor 7.7 us
// each way: 8.8 us by row (5.7 TB/s), 9.8 in groups, 10.1 to 10.5 back; there
// and back 17.6, the codes read from L2.  16 x 512 there and back: 4.0 us.
#include "common.cuh"
#include "int8_common.cuh"
#include "kernels.h"

namespace qlora {

using namespace int8;

namespace {

// One scale a row.  A row is held in registers by THREADS threads, VPT 16-byte
// loads each, so it is read once; the maximum crosses the warps of the row
// through shared memory.  ROWS rows share a CTA when a row is one warp.
template <int THREADS, int VPT, int ROWS>
__global__ void __launch_bounds__(THREADS *ROWS) quantize_rows_kernel(const uint4 *__restrict__ x, int64_t rows,
                                                                      int vecs, uint2 *__restrict__ codes,
                                                                      float *__restrict__ scales) {
  static_assert(ROWS == 1 || THREADS == 32, "rows share a CTA only one warp each");
  grid_dep_wait();
  grid_dep_launch();
  const int tid = ROWS == 1 ? threadIdx.x : threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (ROWS == 1 ? 0 : threadIdx.x >> 5);
  if (row >= rows) return;   // (whole warps: ROWS > 1 only)
  const uint4 *src = x + row * vecs;
  uint4 v[VPT];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * THREADS + tid;
    v[i] = c < vecs ? __ldcg(src + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) m = __vmaxu2(m, abs_max8(v[i]));
  uint32_t a = __reduce_max_sync(0xffffffffu, fold_u16x2(m));
  if constexpr (THREADS > 32) {
    __shared__ uint32_t s_max[THREADS / 32];
    if ((tid & 31) == 0) s_max[tid >> 5] = a;
    __syncthreads();
    a = (tid & 31) < THREADS / 32 ? s_max[tid & 31] : 0u;
    a = __reduce_max_sync(0xffffffffu, a);
  }
  const RowScale r = row_scale(a);
  if (tid == 0) scales[row] = r.scale;
  uint2 *dst = codes + row * vecs;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * THREADS + tid;
    if (c < vecs) dst[c] = codes8(v[i], r);
  }
}

// Rows longer than the registers of a CTA: the row is read twice (the second
// read hits L2).
__global__ void __launch_bounds__(1024) quantize_long_rows_kernel(const uint4 *__restrict__ x, int64_t vecs,
                                                                  uint2 *__restrict__ codes,
                                                                  float *__restrict__ scales) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t s_max[32];
  const int64_t row = blockIdx.x;
  const uint4 *src = x + row * vecs;
  uint32_t m = 0;
  for (int64_t c = threadIdx.x; c < vecs; c += 1024) m = __vmaxu2(m, abs_max8(__ldcg(src + c)));
  uint32_t a = __reduce_max_sync(0xffffffffu, fold_u16x2(m));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = a;
  __syncthreads();
  a = __reduce_max_sync(0xffffffffu, s_max[threadIdx.x & 31]);
  const RowScale r = row_scale(a);
  if (threadIdx.x == 0) scales[row] = r.scale;
  uint2 *dst = codes + row * vecs;
  for (int64_t c = threadIdx.x; c < vecs; c += 1024) dst[c] = codes8(__ldcg(src + c), r);
}

// One scale per 128 columns of a row: 16 lanes hold a group (8 values each), a
// warp two neighbouring groups of kGroupRows rows, whose loads are in flight
// together.  Scales are stored group by group, [groups][rows], so that the
// kGroupRows scales of a group are one 32-byte sector.
constexpr int kGroupRows = 8;
constexpr int kGroupWarps = 4;

__global__ void __launch_bounds__(32 * kGroupWarps)
    quantize_groups_kernel(const uint4 *__restrict__ x, int64_t rows, int vecs, int groups, int pairs,
                           uint2 *__restrict__ codes, float *__restrict__ scales) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGroupWarps + (threadIdx.x >> 5);
  const int64_t slab = unit / pairs;
  const int64_t row0 = slab * kGroupRows;
  if (row0 >= rows) return;
  const int pair = static_cast<int>(unit - slab * pairs);
  const int c = pair * 32 + lane;
  const bool in = c < vecs;
  const int n = static_cast<int>(min(static_cast<int64_t>(kGroupRows), rows - row0));
  uint4 v[kGroupRows];
#pragma unroll
  for (int i = 0; i < kGroupRows; ++i)
    v[i] = in && i < n ? __ldcg(x + (row0 + i) * vecs + c) : make_uint4(0, 0, 0, 0);
  // the maxima of two rows at a time, as u16x2, over the 16 lanes of a group
  uint32_t m = 0;   // this lane's row: row (lane & 15) of the slab
#pragma unroll
  for (int i = 0; i < kGroupRows; i += 2) {
    const uint32_t a = abs_max8(v[i]), b = abs_max8(v[i + 1]);
    uint32_t ab = __vmaxu2(prmt(a, b, 0x5410), prmt(a, b, 0x7632));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ab = __vmaxu2(ab, __shfl_xor_sync(0xffffffffu, ab, o));
    if ((lane & 15) == i) m = ab & 0xFFFFu;
    if ((lane & 15) == i + 1) m = ab >> 16;
  }
  // one division and one reciprocal a lane, for its row; the others take them
  const RowScale mine = row_scale(m);
  const float inv = mine.bad ? -1.0f : mine.inv;
#pragma unroll
  for (int i = 0; i < kGroupRows; ++i) {
    RowScale r;
    r.inv = __shfl_sync(0xffffffffu, inv, i, 16);
    r.bad = r.inv < 0.f;
    if (in && i < n) codes[(row0 + i) * vecs + c] = codes8(v[i], r);
  }
  const int g = pair * 2 + (lane >> 4);
  if (g < groups && (lane & 15) < n) scales[static_cast<int64_t>(g) * rows + row0 + (lane & 15)] = mine.scale;
}

__device__ __forceinline__ uint32_t value2(uint32_t w, int byte, float s) {
  const float lo = static_cast<float>(static_cast<int8_t>(w >> (8 * byte)));
  const float hi = static_cast<float>(static_cast<int8_t>(w >> (8 * byte + 8)));
  return pack_bf16x2(__fmul_rn(lo, s), __fmul_rn(hi, s));
}

// BF16_RNE(RN32(code * scale)).  A thread takes the same 8 codes (one 8-byte
// load, one 16-byte store) of kDeqRows rows, all loads in flight together.
constexpr int kDeqRows = 4;

__global__ void __launch_bounds__(256) dequantize_int8_kernel(const uint2 *codes, const float *scales, int64_t rows,
                                                              int units, int group_units, uint4 *__restrict__ out) {
  grid_dep_wait();
  grid_dep_launch();
  const int u = static_cast<int>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (u >= units) return;
  const float *sg = scales + (group_units ? static_cast<int64_t>(u / group_units) * rows : 0);
  const int64_t slab = static_cast<int64_t>(blockDim.y) * kDeqRows;
  for (int64_t row0 = blockIdx.y * slab + threadIdx.y; row0 < rows; row0 += gridDim.y * slab) {
    uint2 q[kDeqRows];
    float s[kDeqRows];
#pragma unroll
    for (int i = 0; i < kDeqRows; ++i) {
      const int64_t row = row0 + i * blockDim.y;
      if (row < rows) {
        q[i] = __ldcg(codes + row * units + u);
        s[i] = __ldca(sg + row);
      }
    }
#pragma unroll
    for (int i = 0; i < kDeqRows; ++i) {
      const int64_t row = row0 + i * blockDim.y;
      if (row < rows)
        out[row * units + u] =
            make_uint4(value2(q[i].x, 0, s[i]), value2(q[i].x, 2, s[i]), value2(q[i].y, 0, s[i]), value2(q[i].y, 2, s[i]));
    }
  }
}

cudaLaunchConfig_t make_cfg(dim3 grid, dim3 block, cudaStream_t st, bool pdl, cudaLaunchAttribute *attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cfg;
}

}  // namespace

cudaError_t launch_quantize_int8(const uint16_t *x, int64_t rows, int64_t cols, int group, int8_t *codes,
                                 float *scales, cudaStream_t st, bool pdl) {
  if (rows <= 0) return cudaSuccess;
  const uint4 *src = reinterpret_cast<const uint4 *>(x);
  uint2 *dst = reinterpret_cast<uint2 *>(codes);
  const int64_t vecs = cols / 8;
  cudaLaunchAttribute attr[1];
  if (group != 0) {
    const int groups = static_cast<int>((cols + kInt8Group - 1) / kInt8Group);
    const int pairs = (groups + 1) / 2;
    const int64_t units = (rows + kGroupRows - 1) / kGroupRows * pairs;
    const int64_t blocks = (units + kGroupWarps - 1) / kGroupWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const cudaLaunchConfig_t cfg = make_cfg(dim3(static_cast<unsigned>(blocks)), dim3(32 * kGroupWarps), st, pdl, attr);
    return cudaLaunchKernelEx(&cfg, quantize_groups_kernel, src, rows, static_cast<int>(vecs), groups, pairs, dst,
                              scales);
  }
  if (rows > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned n = static_cast<unsigned>(rows);
  const int nv = static_cast<int>(vecs);
  if (vecs <= 32 * 4) {
    const cudaLaunchConfig_t cfg = make_cfg(dim3((n + 3) / 4), dim3(128), st, pdl, attr);
    return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<32, 4, 4>, src, rows, nv, dst, scales);
  }
  if (vecs <= 32 * 8 && rows >= 1024) {   // many short rows: fewer CTAs (16384 x 1040: 18.1 -> 9.5 us)
    const cudaLaunchConfig_t cfg = make_cfg(dim3((n + 3) / 4), dim3(128), st, pdl, attr);
    return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<32, 8, 4>, src, rows, nv, dst, scales);
  }
  if (vecs <= 128 * 4) {
    const cudaLaunchConfig_t cfg = make_cfg(dim3(n), dim3(128), st, pdl, attr);
    return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<128, 4, 1>, src, rows, nv, dst, scales);
  }
  if (vecs <= 512 * 4) {
    const cudaLaunchConfig_t cfg = make_cfg(dim3(n), dim3(512), st, pdl, attr);
    return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<512, 4, 1>, src, rows, nv, dst, scales);
  }
  if (vecs <= 1024 * 4) {
    const cudaLaunchConfig_t cfg = make_cfg(dim3(n), dim3(1024), st, pdl, attr);
    return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<1024, 4, 1>, src, rows, nv, dst, scales);
  }
  const cudaLaunchConfig_t cfg = make_cfg(dim3(n), dim3(1024), st, pdl, attr);
  return cudaLaunchKernelEx(&cfg, quantize_long_rows_kernel, src, vecs, dst, scales);
}

cudaError_t launch_dequantize_int8(const int8_t *codes, const float *scales, int64_t rows, int64_t cols, int group,
                                   uint16_t *out, cudaStream_t st, bool pdl) {
  if (rows <= 0) return cudaSuccess;
  const int64_t units = cols / 8;
  int bx = 1;
  while (bx < 256 && bx < units) bx *= 2;
  const int by = 256 / bx;
  const int64_t gy = (rows + by * kDeqRows - 1) / (by * kDeqRows);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      make_cfg(dim3(static_cast<unsigned>((units + bx - 1) / bx), static_cast<unsigned>(gy < 65535 ? gy : 65535)),
               dim3(static_cast<unsigned>(bx), static_cast<unsigned>(by)), st, pdl, attr);
  return cudaLaunchKernelEx(&cfg, dequantize_int8_kernel, reinterpret_cast<const uint2 *>(codes), scales, rows,
                            static_cast<int>(units), group / 8, reinterpret_cast<uint4 *>(out));
}

}  // namespace qlora
