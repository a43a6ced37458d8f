/*
 * zs_quantize_kernels.h -- microscaled copies of a matrix, along its rows or
 * along its columns (gfx950). Bound by HBM: 4 or 2 bytes in, 17/32 or 33/32
 * out per element, and 2 more where the rounded values are asked for. The
 * codes stay in the caches for the product; the values, which go into a
 * buffer of a later time, are stored non-temporally (bf16 8191 x 4096 along
 * the columns: 33.3 us plain, 32.2).
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
  uint32_t tiles_r, tiles_c;   /* columns variant: tiles down and across */
};

/* Along the rows: eight elements per thread, a block of 32 per quad of lanes,
 * whose maximum two lane moves join: no LDS and one pass. fp32 50257 x 768 to
 * E2M1: 26 us (6.8 TB/s), with values 43 (5.8 TB/s). */
template <int DT, bool AL, int FMT, int VDT>
__global__ __launch_bounds__(kBlock) void quant_rows_kernel(QuantArgs a) {
  const uint32_t id = blockIdx.x * kBlock + threadIdx.x;   /* a launch has below 2^32 */
  if (id >= a.vecs) return;   /* whole quads: a row has a multiple of 16 vectors */
  const uint32_t vpr = (uint32_t)(a.padded / 8);
  const uint64_t row = id / vpr, v = id % vpr;
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  float x[8];
  load8<DT, AL, true>(static_cast<const char *>(a.src) + row * a.ld * esz, v * 8, a.cols, x);
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
    store8<VDT, AL, true>(a.values + row * a.cols, v * 8, a.cols, x);
  }
}

/* Along the columns: a block takes 128 rows (one group) of 64 words, one
 * column of fp32 or two of 16 bits each, through LDS; then each thread holds
 * a word's column or columns of 32 rows, the four blocks of a column in
 * neighbouring lanes, which write whole lines together. A row stride of 65
 * words and 16 more for every 32 rows keep both ways of walking the tile off
 * each other's banks. bf16 8191 x 4096 to E4M3 with values: 32 us, 5.2 TB/s
 * (one 16-bit column to a word, blocks in the grid's order and plain loads:
 * 40 us). Bound by HBM, where a tile's 256-byte rows come and its columns'
 * 128 bytes go; finding the maxima in half the instructions changed nothing. */
constexpr uint32_t kColTileR = 128, kColTileW = 64, kColBand = 4;

template <int DT>
constexpr uint32_t kColsPerWord = DT == ZS_FP32 ? 1 : 2;

__device__ __forceinline__ uint32_t col_row(uint32_t r) { return r * (kColTileW + 1) + r / 32 * 16; }

template <int DT, bool AL, int FMT, int VDT>
__global__ __launch_bounds__(kBlock) void quant_cols_kernel(QuantArgs a) {
  __shared__ uint32_t tile[kColTileR * (kColTileW + 1) + 48];
  constexpr uint64_t esz = DT == ZS_FP32 ? 4 : 2;
  /* P columns per word; W words to a thread's eight columns, kAcross threads
   * to a row and kDown rows at a time */
  constexpr uint32_t P = kColsPerWord<DT>, W = 8 / P, kAcross = kColTileW / W;
  constexpr uint32_t kDown = kBlock / kAcross, kPasses = kColTileR / kDown;
  /* Blocks go round the eight XCDs; each XCD takes a run of tiles, and runs
   * walk down bands of kColBand tiles across: what the groups of a column
   * write next to each other, its scales above all, then meets in one L2. */
  const uint32_t total = a.tiles_r * a.tiles_c, per = total / 8, extra = total % 8;
  const uint32_t xcd = blockIdx.x % 8;
  const uint32_t id = xcd * per + (xcd < extra ? xcd : extra) + blockIdx.x / 8;
  const uint32_t band = id / (kColBand * a.tiles_r), in_band = id % (kColBand * a.tiles_r);
  const uint32_t rest = a.tiles_c - band * kColBand, wide = rest < kColBand ? rest : kColBand;
  const uint64_t r0 = (uint64_t)(in_band / wide) * kColTileR;
  const uint64_t c0 = (uint64_t)(band * kColBand + in_band % wide) * kColTileW * P;
  const uint32_t t = threadIdx.x, tr = t / kAcross, tw = t % kAcross * W;
  uint32_t raw[kPasses][W];   /* all of a thread's loads are under way together */
#pragma unroll
  for (uint32_t i = 0; i < kPasses; ++i) {
    const uint64_t row = r0 + i * kDown + tr;
    const char *src = static_cast<const char *>(a.src) + row * a.ld * esz;
    const uint64_t cols = row < a.rows ? a.cols : 0;   /* past the last row: zeros */
    if constexpr (P == 1) {
      float x[8];
      load8<DT, AL, true>(src, c0 + tw, cols, x);
#pragma unroll
      for (uint32_t j = 0; j < W; ++j) raw[i][j] = __float_as_uint(x[j]);
    } else {
      const Raw16<8> x = load8_raw<AL, true>(src, c0 + tw * P, cols);
#pragma unroll
      for (uint32_t j = 0; j < W; ++j) raw[i][j] = x.w[j];
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < kPasses; ++i)
#pragma unroll
    for (uint32_t j = 0; j < W; ++j) tile[col_row(i * kDown + tr) + tw + j] = raw[i][j];
  __syncthreads();
  const uint32_t lw = t / 4, blk = t % 4;   /* a word and its block of 32 rows */
  constexpr uint32_t kStride = kColTileW + 1, kWords = FMT == ZS_MX_E2M1 ? 4 : 8;
  uint32_t *col = tile + col_row(blk * 32) + lw;
  if (c0 + lw * P < a.cols) {
    uint32_t w[32], code[P][kWords], byte[P];
#pragma unroll
    for (uint32_t j = 0; j < 32; ++j) w[j] = col[j * kStride];
    auto value = [&](uint32_t j, uint32_t p) {
      if constexpr (P == 1) return __uint_as_float(w[j]);
      else return p ? up_hi<DT>(w[j]) : up_lo<DT>(w[j]);
    };
#pragma unroll
    for (uint32_t p = 0; p < P; ++p) {
      uint32_t top = 0;
#pragma unroll
      for (uint32_t j = 0; j < 32; ++j) top = umax(top, mag_bits(value(j, p)));
      byte[p] = mx_scale_byte<FMT>(top);
#pragma unroll
      for (uint32_t o = 0; o < 4; ++o) {
        float x[8];
        uint32_t c[2];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) x[j] = value(o * 8 + j, p);
        mx_encode<FMT>(x, byte[p], c);
        if constexpr (FMT == ZS_MX_E2M1) {
          code[p][o] = c[0];
        } else {
          code[p][2 * o] = c[0];
          code[p][2 * o + 1] = c[1];
        }
      }
      const uint64_t orow = c0 + lw * P + p, k = r0 + blk * 32;
      if (orow < a.cols) {
        u32x4 *out = reinterpret_cast<u32x4 *>(a.codes + orow * mx_bytes<FMT>(a.padded) +
                                               mx_bytes<FMT>(k));
#pragma unroll
        for (uint32_t q = 0; q < kWords / 4; ++q)
          out[q] = u32x4{code[p][4 * q], code[p][4 * q + 1], code[p][4 * q + 2],
                         code[p][4 * q + 3]};
        a.scales[orow * (a.padded / kMxBlock) + k / kMxBlock] = (uint8_t)byte[p];
      }
    }
    if (a.values) {   /* they take the source's place in the tile */
#pragma unroll
      for (uint32_t o = 0; o < 4; ++o) {
        float x[P][8];
#pragma unroll
        for (uint32_t p = 0; p < P; ++p) {
          uint32_t c[2] = {code[p][FMT == ZS_MX_E2M1 ? o : 2 * o], 0};
          if constexpr (FMT == ZS_MX_E4M3) c[1] = code[p][2 * o + 1];
          mx_decode<FMT>(c, byte[p], x[p]);
        }
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
          uint32_t v;
          if constexpr (P == 1) v = __float_as_uint(x[0][j]);
          else v = pack2<VDT>(x[0][j], x[1][j]);
          col[(o * 8 + j) * kStride] = v;
        }
      }
    }
  }
  if (!a.values) return;
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < kPasses; ++i) {
    const uint64_t row = r0 + i * kDown + tr;
    if (row >= a.rows) break;
    const uint32_t *from = tile + col_row(i * kDown + tr) + tw;
    uint16_t *to = a.values + row * a.cols;
    if constexpr (P == 1) {
      float x[8];
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) x[j] = __uint_as_float(from[j]);
      store8<VDT, AL, true>(to, c0 + tw, a.cols, x);
    } else {
      store8_raw<AL, true>(to, c0 + tw * P, a.cols, u32x4{from[0], from[1], from[2], from[3]});
    }
  }
}

}  // namespace zs
#endif  // ZS_QUANTIZE_KERNELS_H
