/*
 * zs_matmul_kernels.h -- C = A B^T of microscaled operands on the matrix
 * cores (gfx950): A in E4M3 or E2M1, B in E2M1, fp32 sums.
 *
 * v_mfma_scale_f32_32x32x64_f8f6f4 takes 64 elements of K of 32 rows a side;
 * lane l holds row l % 32. With g = l / 32, E2M1 rows come as elements
 * 32g .. 32g+31 (16 bytes), E4M3 rows as 16g .. 16g+15 and 32+16g .. (two
 * times 16 bytes), and the lane's scale byte is that of block g. B is the
 * instruction's first operand, so that a lane's four consecutive results lie
 * along a row of C: result i of lane l is row l % 32 of A against row
 * 8*(i/4) + 4g + i%4 of B.
 */
#ifndef ZS_MATMUL_KERNELS_H
#define ZS_MATMUL_KERNELS_H

#include "zs_mx.h"

namespace zs {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct MatmulArgs {
  const uint8_t *a, *as, *b, *bs;
  void *c;
  uint64_t ldc;
  uint32_t m, n, padded;   /* padded: K rounded up to whole groups */
};

/* The matrix instruction's name for an element format. */
template <int FMT>
constexpr int kMfmaFormat = FMT == ZS_MX_E2M1 ? 4 : 0;

template <int CDT>
__device__ __forceinline__ void store_c4(void *c, uint64_t at, uint32_t col, uint32_t cols,
                                         const float (&x)[4], bool vec) {
  if (col >= cols) return;
  if constexpr (CDT == ZS_FP32) {
    float *p = static_cast<float *>(c) + at + col;
    if (vec && col + 4 <= cols) {
      *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
      for (uint32_t j = 0; j < 4 && col + j < cols; ++j) p[j] = x[j];
    }
  } else {
    uint16_t *p = static_cast<uint16_t *>(c) + at + col;
    if (vec && col + 4 <= cols) {
      *reinterpret_cast<u32x2 *>(p) = u32x2{pack2<CDT>(x[0], x[1]), pack2<CDT>(x[2], x[3])};
    } else {
      for (uint32_t j = 0; j < 4 && col + j < cols; ++j) p[j] = pack1<CDT>(x[j]);
    }
  }
}

/* One 32 x 32 tile of C per wave, operands straight from global memory. */
template <int AF, int CDT>
__global__ __launch_bounds__(kBlock) void matmul_kernel(MatmulArgs p, int vec) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t r = lane & 31, g = lane >> 5;
  const uint32_t m0 = blockIdx.y * 64 + (wave >> 1) * 32, n0 = blockIdx.x * 64 + (wave & 1) * 32;
  const uint64_t ra = m0 + r < p.m ? m0 + r : p.m - 1, rb = n0 + r < p.n ? n0 + r : p.n - 1;
  const uint8_t *a = p.a + ra * mx_bytes<AF>(p.padded), *b = p.b + rb * (p.padded / 2);
  const uint8_t *as = p.as + ra * (p.padded / 32), *bs = p.bs + rb * (p.padded / 32);
  f32x16 acc = {};
  for (uint32_t k = 0; k < p.padded; k += 64) {
    i32x8 fa = {}, fb = {};
    const u32x4 wb = *reinterpret_cast<const u32x4 *>(b + k / 2 + g * 16);
    fb[0] = wb.x; fb[1] = wb.y; fb[2] = wb.z; fb[3] = wb.w;
    const u32x4 wa = *reinterpret_cast<const u32x4 *>(a + mx_bytes<AF>(k) + g * 16);
    fa[0] = wa.x; fa[1] = wa.y; fa[2] = wa.z; fa[3] = wa.w;
    if constexpr (AF == ZS_MX_E4M3) {
      const u32x4 wh = *reinterpret_cast<const u32x4 *>(a + k + 32 + g * 16);
      fa[4] = wh.x; fa[5] = wh.y; fa[6] = wh.z; fa[7] = wh.w;
    }
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb, fa, acc, 4, kMfmaFormat<AF>, 0,
                                                          bs[k / 32 + g], 0, as[k / 32 + g]);
  }
  if (m0 + r >= p.m) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float x[4] = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    store_c4<CDT>(p.c, (uint64_t)(m0 + r) * p.ldc, n0 + q * 8 + g * 4, p.n, x, vec);
  }
}

}  // namespace zs
#endif  // ZS_MATMUL_KERNELS_H
