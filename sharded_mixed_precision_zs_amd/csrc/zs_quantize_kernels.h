/*
 * zs_quantize_kernels.h -- microscaled copies of a matrix, along its rows or
 * along its columns (gfx950). Bound by HBM: 4 or 2 bytes in, 17/32 or 33/32
 * out per element, and 2 more where the rounded values are asked for.
 */
#ifndef ZS_QUANTIZE_KERNELS_H
#define ZS_QUANTIZE_KERNELS_H

#include "zs_mx.h"

namespace zs {

struct QuantArgs {
  const void *src;
  uint64_t rows, cols, ld;
  uint8_t *codes, *scales;
  uint16_t *values;      /* [rows][cols], optional */
  uint64_t padded;       /* the blocked dimension rounded up to whole groups */
  uint64_t vecs;         /* rows variant: vectors of eight in all */
};


/* Along the rows: eight elements per thread, a block per quad of lanes. */
template <int DT, bool AL, int FMT, int VDT>
__global__ __launch_bounds__(kBlock) void quant_rows_kernel(QuantArgs a) {
  const uint32_t id = blockIdx.x * kBlock + threadIdx.x;   /* a launch has below 2^32 */
  if (id >= a.vecs) return;   /* whole quads: a row has a multiple of 16 vectors */
  const uint32_t vpr = (uint32_t)(a.padded / 8);
  const uint64_t row = id / vpr, v = id % vpr;
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  float x[8];
  load8<DT, AL>(static_cast<const char *>(a.src) + row * a.ld * esz, v * 8, a.cols, x);
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = umax(top, mag_bits(x[j]));
  const uint32_t byte = mx_scale_byte<FMT>(quad_max(top));
  uint32_t code[2];
  mx_encode<FMT>(x, byte, code);
  uint8_t *out = a.codes + row * mx_bytes<FMT>(a.padded) + mx_bytes<FMT>(v * 8);
  if constexpr (FMT == ZS_MX_E2M1) *reinterpret_cast<uint32_t *>(out) = code[0];
  else *reinterpret_cast<u32x2 *>(out) = u32x2{code[0], code[1]};
  if ((v & 3) == 0) a.scales[row * (a.padded / kMxBlock) + v / 4] = (uint8_t)byte;
  if (a.values) {
    mx_decode<FMT>(code, byte, x);
    store8<VDT, AL>(a.values + row * a.cols, v * 8, a.cols, x);
  }
}

/* Along the columns: a block takes 128 rows (one group) of 64 columns
 * through LDS, as float; then each thread holds one column's block of 32, the
 * four blocks of a column in neighbouring lanes, which write whole lines
 * together. A row stride of 65 floats and 16 more for every 32 rows keep both
 * ways of walking the tile off each other's banks. */
constexpr uint32_t kColTileR = 128, kColTileC = 64;

__device__ __forceinline__ uint32_t col_row(uint32_t r) { return r * (kColTileC + 1) + r / 32 * 16; }

template <int DT, bool AL, int FMT, int VDT>
__global__ __launch_bounds__(kBlock) void quant_cols_kernel(QuantArgs a) {
  __shared__ float tile[kColTileR * (kColTileC + 1) + 48];
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  const uint64_t r0 = (uint64_t)blockIdx.y * kColTileR, c0 = (uint64_t)blockIdx.x * kColTileC;
  const uint32_t t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lr = i * 32 + t / 8, lc = (t % 8) * 8;
    float x[8];
    if (r0 + lr < a.rows) {
      load8<DT, AL>(static_cast<const char *>(a.src) + (r0 + lr) * a.ld * esz, c0 + lc, a.cols, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[col_row(lr) + lc + j] = x[j];
  }
  __syncthreads();
  const uint32_t lc = t / 4, blk = t % 4;   /* a column and its block of 32 rows */
  if (c0 + lc < a.cols) {
    constexpr uint32_t kColStride = kColTileC + 1;
    float *col = tile + col_row(blk * 32) + lc;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) top = umax(top, mag_bits(col[j * kColStride]));
    const uint32_t byte = mx_scale_byte<FMT>(top);
    uint32_t words[8];
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      float x[8];
      uint32_t code[2];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = col[(o * 8 + j) * kColStride];
      mx_encode<FMT>(x, byte, code);
      if constexpr (FMT == ZS_MX_E2M1) {
        words[o] = code[0];
      } else {
        words[2 * o] = code[0];
        words[2 * o + 1] = code[1];
      }
      if (a.values) {
        mx_decode<FMT>(code, byte, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) col[(o * 8 + j) * kColStride] = x[j];
      }
    }
    const uint64_t orow = c0 + lc, k = r0 + blk * 32;
    u32x4 *out = reinterpret_cast<u32x4 *>(a.codes + orow * mx_bytes<FMT>(a.padded) +
                                           mx_bytes<FMT>(k));
    out[0] = u32x4{words[0], words[1], words[2], words[3]};
    if constexpr (FMT == ZS_MX_E4M3) out[1] = u32x4{words[4], words[5], words[6], words[7]};
    a.scales[orow * (a.padded / kMxBlock) + k / kMxBlock] = (uint8_t)byte;
  }
  if (!a.values) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lr = i * 32 + t / 8, vc = (t % 8) * 8;
    if (r0 + lr >= a.rows) break;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = tile[col_row(lr) + vc + j];
    store8<VDT, AL>(a.values + (r0 + lr) * a.cols, c0 + vc, a.cols, x);
  }
}

}  // namespace zs
#endif  // ZS_QUANTIZE_KERNELS_H
